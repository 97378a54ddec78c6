"""The calls of the 8-bit cache refuse bad arguments on the host (CPU only:
nothing dereferences these addresses, and every call fails its checks)."""
import ctypes

import pytest
import torch

BATCH, WIDTH, PAGES, TOKENS = 3, 128, 64, 9
# arguments of one call: places far apart, and the bytes that a call reads or writes there
NAMES = ["q", "off", "pool", "scales", "bt", "lens", "out", "ws", "err", "k", "v", "pos", "slots",
         "q_out", "starts"]
PLACE = {n: (i + 1) << 32 for i, n in enumerate(NAMES)}
Q_ROW, KV_ROW = 32 * 64 * 2, 8 * 64 * 2
SIZE = {"off": 4 * (BATCH + 1), "pool": PAGES * 16384, "scales": PAGES * 16,
        "bt": 4 * BATCH * WIDTH, "lens": 4 * BATCH, "err": 4, "pos": 4 * BATCH, "slots": 4 * BATCH,
        "starts": 4 * BATCH}


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_04_gb300 import build
    build.build()
    from paged_kv_decode_04_gb300 import binding
    return binding


def call(name, args):
    """A call of every argument in order; `p` names take the places above."""
    def run(B, **kw):
        bad = set(kw) - {n for n, _ in args}
        assert not bad, bad
        a = [kw.get(n, ctypes.c_void_p(PLACE[n]) if v is None else v) for n, v in args]
        a = [ctypes.c_void_p(x) if n in PLACE and isinstance(x, int) else x
             for (n, _), x in zip(args, a)]
        return getattr(B.lib(), name)(*a)
    run.__name__ = name[4:]
    return run


CACHE = [("pool", None), ("scales", None), ("fmt", 0), ("pages", PAGES)]
TABLE = [("bt", None), ("mb", WIDTH)]
DIMS = [("hkv", 8), ("d", 64), ("ps", 16)]
MASKS = [("window", 0), ("sinks", 0), ("scale", 0.125)]
END = [("err", None), ("stream", ctypes.c_void_p(0))]
PARTS = [("ws", None), ("wsb", 0), ("splits", 2)]

append = call("pkv_kv8_append", [("k", None), ("v", None), *CACHE, *TABLE, ("pos", None),
                                 ("slots", None), ("batch", BATCH), *DIMS, ("theta", 5e5),
                                 ("q", None), ("q_out", None), ("hq", 32), *END])
write = call("pkv_kv8_write_prefill", [("k", None), ("v", None), ("n", TOKENS), ("off", None),
                                       ("starts", None), *CACHE, *TABLE, ("batch", BATCH), *DIMS,
                                       ("theta", 5e5), *END])
read = call("pkv_kv8_read", [*CACHE, *TABLE, ("off", None), ("starts", None), ("n", TOKENS),
                             ("batch", BATCH), *DIMS, ("k", None), ("v", None), *END])
decode = call("pkv_paged8_decode_attention", [
    ("q", None), *CACHE, *TABLE, ("lens", None), ("batch", BATCH), ("hq", 32), *DIMS, *MASKS,
    ("out", None), *PARTS, *END])
chunk = call("pkv_paged8_chunk_attention", [
    ("q", None), ("n", TOKENS), ("off", None), *CACHE, *TABLE, ("lens", None), ("batch", BATCH),
    ("hq", 32), *DIMS, *MASKS, ("out", None), *PARTS, *END])
# each call's outputs, and what else it names
CALLS = {
    append: (["pool", "scales", "q_out", "err"], ["k", "v", "bt", "pos", "slots", "q"]),
    write: (["pool", "scales", "err"], ["k", "v", "off", "starts", "bt"]),
    read: (["k", "v", "err"], ["pool", "scales", "bt", "off", "starts"]),
    decode: (["out", "err"], ["q", "pool", "scales", "bt", "lens"]),
    chunk: (["out", "err"], ["q", "off", "pool", "scales", "bt", "lens"]),
}
ATTEND = [decode, chunk]


def ids(c):
    return c.__name__ if callable(c) else None


NULL = ctypes.c_void_p(0)
NEEDED = [(c, n) for c, (outs, ins) in CALLS.items() for n in outs + ins
          if n not in ("err", "slots", "q_out") and (c, n) != (append, "q")]


@pytest.mark.parametrize("call,name", NEEDED, ids=ids)
def test_null(B, call, name):
    assert call(B, **{name: NULL}) == B.PKV_EINVAL


@pytest.mark.parametrize("call", CALLS, ids=ids)
@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=65536), dict(pages=0),
                                 dict(pages=2 ** 31), dict(mb=0), dict(mb=2 ** 28)])
def test_sizes(B, call, bad):
    assert call(B, **bad) == B.PKV_EINVAL


@pytest.mark.parametrize("call,bad", [
    *[(c, dict(theta=t)) for c in (append, write)
      for t in (0.0, -1.0, float("inf"), float("nan"))],
    *[(c, dict(n=-1)) for c in (write, read, chunk)],
    (append, dict(q=NULL)), (append, dict(q_out=NULL)),
    *[(c, {k: -1}) for c in ATTEND for k in ("window", "sinks", "splits")],
    *[(c, dict(scale=s)) for c in ATTEND for s in (0.0, -0.5, float("inf"), float("nan"))],
])
def test_values(B, call, bad):
    assert call(B, **bad) == B.PKV_EINVAL


@pytest.mark.parametrize("call", CALLS, ids=ids)
@pytest.mark.parametrize("bad", [dict(hkv=4), dict(hkv=32), dict(d=128), dict(ps=32), dict(hq=16),
                                 dict(fmt=2), dict(fmt=-1)])
def test_unsupported(B, call, bad):
    if "hq" in bad and call in (write, read):
        return
    assert call(B, **bad) == B.PKV_EUNSUPPORTED


ALIGN = {"pool": 16, "scales": 16, "q": 16, "out": 16, "ws": 16, "k": 16, "v": 16}
ALIGNED = [(c, n, 2 if c is append and n in ("k", "q", "q_out") else
            4 if (c, n) in ((append, "v"), (decode, "out")) else ALIGN.get(n, 4))
           for c, (outs, ins) in CALLS.items()
           for n in outs + ins + (["ws"] if c in ATTEND else [])]


@pytest.mark.parametrize("call,name,need", ALIGNED, ids=ids)
def test_alignment(B, call, name, need):
    assert call(B, **{name: PLACE[name] + need // 2}) == B.PKV_EALIGN
    if call in ATTEND and name != "ws":
        assert call(B, **{name: PLACE[name] + need}) == B.PKV_EWORKSPACE


@pytest.mark.parametrize("call", CALLS, ids=ids)
def test_nothing_to_do(B, call):
    assert call(B, batch=0) == B.PKV_OK
    if call in (write, read, chunk):
        assert call(B, n=0) == B.PKV_OK


def sizes(call):
    rows = BATCH if call in (append, decode) else TOKENS
    return dict(SIZE, q=rows * Q_ROW, out=rows * Q_ROW, q_out=rows * Q_ROW, k=rows * KV_ROW,
                v=rows * KV_ROW)


PAIRS = [(c, o, other) for c, (outs, ins) in CALLS.items()
         for i, o in enumerate(outs) for other in ins + outs[:i]]


@pytest.mark.parametrize("call,out,other", PAIRS,
                         ids=[f"{c.__name__}-{o}-{x}" for c, o, x in PAIRS])
def test_outputs_that_overlap(B, call, out, other):
    size = sizes(call)
    for at in (0, (size[other] - 1) & ~15, -((size[out] - 1) & ~15)):  # start, last, first bytes
        assert call(B, **{out: PLACE[other] + at}) == B.PKV_EINVAL, at


@pytest.mark.parametrize("call", ATTEND, ids=ids)
def test_outputs_that_touch(B, call):
    """Right behind, or right in front of, every other argument: no overlap, so
    the calls go on to miss their workspace."""
    size = sizes(call)
    outs, others = CALLS[call]
    for out in outs:
        for other in others:
            for at in (-(-size[other] // 16) * 16, -(-size[out] // 16) * -16):
                assert call(B, **{out: PLACE[other] + at}) == B.PKV_EWORKSPACE, (out, other, at)


def need_of(B, call):
    return (B.decode8_workspace_bytes(BATCH, WIDTH, 2) if call is decode else
            B.chunk8_workspace_bytes(TOKENS, BATCH, WIDTH, 2))


@pytest.mark.parametrize("call", ATTEND, ids=ids)
def test_workspaces(B, call):
    size, need = sizes(call), need_of(B, call)
    assert need > 0
    assert call(B, wsb=need - 1) == call(B, ws=NULL, wsb=need) == B.PKV_EWORKSPACE
    outs, others = CALLS[call]
    for other in outs + others:
        for at in (0, (size[other] - 1) & ~15, -((need - 1) & ~15)):
            assert call(B, ws=PLACE[other] + at, wsb=need) == B.PKV_EINVAL, (other, at)


def test_workspace_sizes(B):
    for f in (lambda: B.decode8_workspace_bytes(1, 8, -1),
              lambda: B.decode8_workspace_bytes(1, 8, 1, window=-1),
              lambda: B.decode8_workspace_bytes(1, 8, 1, sinks=-1),
              lambda: B.chunk8_workspace_bytes(4, -1, 8),
              lambda: B.chunk8_workspace_bytes(-1, 1, 8)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: B.decode8_workspace_bytes(65536, 8, 1),
              lambda: B.decode8_workspace_bytes(1, 0, 1),
              lambda: B.chunk8_workspace_bytes(4, 1, 0, 1)):
        with pytest.raises(B.PkvError):
            f()
    assert B.decode8_workspace_bytes(0, 8) == B.chunk8_workspace_bytes(0, 4, 8) == 0
    assert B.decode8_workspace_bytes(5, 64, 1) == B.chunk8_workspace_bytes(4, 1, 64, 1) == 0
    # long chunks: their pages as bf16, of every chunk that the tokens can be
    page = 2 * 16 * 8 * 64 * 2
    assert 10 * page <= B.chunk8_workspace_bytes(5, 1, 10, 1) < 11 * page
    assert 20 * page <= B.chunk8_workspace_bytes(14, 9, 10, 1) < 21 * page
    # ... and 2 GiB of them at a time where the tables name more
    assert B.chunk8_workspace_bytes(2 ** 20, 1000, 2048, 1) < 2 ** 31 + 2 ** 26


def pool_of(dtype=torch.int8):
    return torch.zeros((2, 2, 8, 16, 64), dtype=dtype), torch.zeros((2, 2, 8), dtype=torch.uint8)


def python_calls(B, pool, scales):
    q = torch.zeros((1, 32, 64), dtype=torch.bfloat16)
    kv = torch.zeros((1, 8, 64), dtype=torch.bfloat16)
    bt, n = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    off = torch.tensor([0, 1], dtype=torch.int32)
    return [lambda: B.kv8_append(kv, kv, pool, scales, bt, n),
            lambda: B.kv8_write_prefill(kv, kv, off, n, pool, scales, bt),
            lambda: B.kv8_read(off, n, pool, scales, bt, kv, kv.clone()),
            lambda: B.paged8_decode_attention(q, pool, scales, bt, n),
            lambda: B.paged8_chunk_attention(q, off, pool, scales, bt, n)]


def test_binding_wants_cuda_tensors(B):
    for f in python_calls(B, *pool_of()):
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.mark.parametrize("make,error,text", [
    (lambda p: p.to(torch.bfloat16), TypeError, "int8"),
    (lambda p: p.to(torch.uint8), TypeError, "int8"), (lambda p: None, TypeError, "int8"),
    (lambda p: p[..., :32], ValueError, "codes"), (lambda p: p[0], ValueError, "codes"),
    (lambda p: p.transpose(2, 3), ValueError, "codes"),
    (lambda p: torch.zeros((2, 2, 8, 64, 16), dtype=p.dtype).transpose(3, 4), ValueError,
     "contiguous"),
])
def test_binding_refuses_other_pools(B, make, error, text):
    pool, scales = pool_of()
    for f in python_calls(B, make(pool), scales):
        with pytest.raises(error, match=text):
            f()
