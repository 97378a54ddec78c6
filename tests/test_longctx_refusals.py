"""The long-context entry points refuse bad arguments on the host (CPU only)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_04_gb300 import build
    build.build()
    from paged_kv_decode_04_gb300 import binding
    return binding


# addresses far apart that nothing dereferences: every call fails its checks
A1, A2, A3, A4, A5, A6, A7, A8, A9 = (ctypes.c_void_p(0x10000000 * i) for i in range(1, 10))
ODD = ctypes.c_void_p(0x10000002)


def chunk(B, **kw):
    a = dict(q=A1, n=8, off=A2, pool=A3, pages=64, bt=A4, mb=128, lens=A5, batch=2, hq=32, hkv=8,
             d=64, ps=16, window=0, sinks=0, scale=0.125, out=A6, ws=None, wsb=0, splits=1,
             err=None, stream=None)
    a.update(kw)
    return B.lib().pkv_paged_chunk_attention(*a.values())


def window(B, **kw):
    a = dict(q=A1, pool=A3, pages=64, bt=A4, mb=128, lens=A5, batch=2, hq=32, hkv=8, d=64, ps=16,
             window=64, sinks=0, scale=0.125, out=A6, ws=None, wsb=0, splits=1, err=None,
             stream=None)
    a.update(kw)
    return B.lib().pkv_paged_window_attention(*a.values())


def scored(B, **kw):
    a = dict(q=A1, pool=A3, pages=64, bt=A4, mb=128, lens=A5, batch=2, hq=32, hkv=8, d=64, ps=16,
             scale=0.125, out=A6, mass=A7, stride=2048, ws=None, wsb=0, splits=1, err=None,
             stream=None)
    a.update(kw)
    return B.lib().pkv_paged_scored_attention(*a.values())


def evict(B, **kw):
    a = dict(mass=A1, stride=2048, pool=A2, pages=64, bt=A3, mb=128, lens=A4, batch=2, hkv=8, d=64,
             ps=16, budget=64, sinks=4, recent=16, dst=A5, dmb=4, new_lens=A6, new_mass=A7,
             new_stride=64, kept=A8, err=None, stream=None)
    a.update(kw)
    return B.lib().pkv_kv_evict(*a.values())


def append(B, **kw):
    a = dict(k=A1, v=A2, pool=A3, pages=64, bt=A4, mb=128, pos=A5, slots=A6, batch=2, hkv=8, d=64,
             ps=16, theta=500000.0, q_in=None, q_out=None, hq=0, err=None, stream=None)
    a.update(kw)
    return B.lib().pkv_kv_append_at(*a.values())


@pytest.mark.parametrize("call,bad", [
    (chunk, dict(q=None)), (chunk, dict(off=None)), (chunk, dict(out=None)),
    (chunk, dict(n=-1)), (chunk, dict(batch=-1)), (chunk, dict(batch=65536)),
    (chunk, dict(window=-1)), (chunk, dict(sinks=-1)), (chunk, dict(splits=-1)),
    (chunk, dict(scale=0.0)), (chunk, dict(scale=float("inf"))), (chunk, dict(pages=0)),
    (chunk, dict(mb=0)), (chunk, dict(mb=2 ** 28)), (chunk, dict(out=A1)),
    (window, dict(window=0)), (window, dict(sinks=-3)), (window, dict(lens=None)),
    (window, dict(scale=float("nan"))), (window, dict(out=A1)), (window, dict(mb=2 ** 28)),
    (scored, dict(mass=None)), (scored, dict(stride=2047)), (scored, dict(splits=-2)),
    (scored, dict(out=A1)), (scored, dict(scale=-1.0)),
    (scored, dict(mb=2 ** 27 - 1, stride=2 ** 31)),
    (evict, dict(budget=0)), (evict, dict(sinks=-1)), (evict, dict(recent=-1)),
    (evict, dict(sinks=40, recent=25)), (evict, dict(sinks=65)), (evict, dict(dmb=3)),
    (evict, dict(stride=2047)), (evict, dict(new_stride=63)), (evict, dict(new_mass=A1)),
    (evict, dict(new_lens=A4)), (evict, dict(kept=A7)), (evict, dict(dst=None)),
    (evict, dict(kept=None)), (evict, dict(recent=2 ** 31 - 1)),
    (evict, dict(mb=2 ** 27 - 1, stride=2 ** 31)), (evict, dict(dmb=2 ** 27 - 1)),
    (append, dict(slots=None)), (append, dict(theta=0.0)), (append, dict(q_in=A7)),
    (append, dict(q_in=A7, q_out=A7, hq=32)), (append, dict(mb=2 ** 28)),
])
def test_invalid(B, call, bad):
    assert call(B, **bad) == B.PKV_EINVAL


@pytest.mark.parametrize("call", [chunk, window, scored])
@pytest.mark.parametrize("bad", [dict(hq=16), dict(hkv=4), dict(d=128), dict(ps=32)])
def test_unsupported(B, call, bad):
    assert call(B, **bad) == B.PKV_EUNSUPPORTED


def test_unsupported_cache(B):
    assert evict(B, hkv=4) == evict(B, d=32) == evict(B, ps=8) == B.PKV_EUNSUPPORTED
    assert append(B, hkv=4) == append(B, q_in=A7, q_out=A8, hq=16) == B.PKV_EUNSUPPORTED


@pytest.mark.parametrize("call,bad", [
    (chunk, dict(q=ODD)), (chunk, dict(pool=ODD)), (chunk, dict(out=ODD)), (chunk, dict(off=ODD)),
    (window, dict(lens=ODD)), (window, dict(ws=ODD)), (scored, dict(mass=ODD)),
    (evict, dict(kept=ODD)), (evict, dict(pool=ODD)), (append, dict(slots=ODD)),
])
def test_misaligned(B, call, bad):
    assert call(B, **bad) == B.PKV_EALIGN


def test_nothing_to_do(B):
    assert chunk(B, n=0) == chunk(B, batch=0) == B.PKV_OK
    assert window(B, batch=0) == scored(B, batch=0) == evict(B, batch=0) == B.PKV_OK
    assert append(B, batch=0) == B.PKV_OK


def test_workspace_sizes(B):
    for f in (lambda: B.chunk_workspace_bytes(4, -1, 8),
              lambda: B.window_workspace_bytes(1, 8, 0),
              lambda: B.scored_workspace_bytes(1, 8, -1)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: B.chunk_workspace_bytes(4, 1, 0),
              lambda: B.window_workspace_bytes(1, 0, 4),
              lambda: B.scored_workspace_bytes(65536, 8, 1)):
        with pytest.raises(B.PkvError):
            f()
    assert B.chunk_workspace_bytes(64, 1, 64, 1) == 0
    assert B.window_workspace_bytes(1, 64, 512, 1) == 0


def test_binding_wants_cuda_tensors(B):
    pool = torch.zeros((2, 2, 16, 8, 64), dtype=torch.bfloat16)
    q = torch.zeros((1, 32, 64), dtype=torch.bfloat16)
    bt, n = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    mass = torch.zeros((1, 8, 16))
    off = torch.tensor([0, 1], dtype=torch.int32)
    kv = torch.zeros((1, 8, 64), dtype=torch.bfloat16)
    for f in (lambda: B.paged_chunk_attention(q, off, pool, bt, n),
              lambda: B.paged_window_attention(q, pool, bt, n, 4),
              lambda: B.paged_scored_attention(q, pool, bt, n, mass),
              lambda: B.kv_evict(mass, pool, bt, n, bt, budget=4),
              lambda: B.kv_append_at(kv, kv, pool, bt, n, n)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
