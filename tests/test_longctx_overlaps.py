"""The long-context entry points refuse outputs and workspaces that share memory
with another argument (CPU only: nothing dereferences these addresses, and
every call is refused, for the overlap or for the workspace that is missing)."""
import ctypes

import pytest

# arguments of one call: places far apart
PLACE = {n: (i + 1) << 32 for i, n in enumerate(
    ["q", "off", "pool", "bt", "lens", "out", "mass", "ws", "err", "k", "v", "pos", "slots",
     "q_out", "dst", "new_lens", "new_mass", "kept"])}
BATCH, WIDTH, PAGES, TOKENS, BUDGET = 3, 128, 64, 9, 64
Q_ROW, KV_ROW = 32 * 64 * 2, 8 * 64 * 2
MASS_STRIDE = WIDTH * 16 + 8
# bytes that a call reads or writes at each place
SIZE = {"off": 4 * (BATCH + 1), "pool": PAGES * 2 * 16 * 8 * 64 * 2, "bt": 4 * BATCH * WIDTH,
        "lens": 4 * BATCH, "mass": 4 * ((BATCH * 8 - 1) * MASS_STRIDE + WIDTH * 16), "err": 4,
        "k": BATCH * KV_ROW, "v": BATCH * KV_ROW, "pos": 4 * BATCH, "slots": 4 * BATCH,
        "q_out": BATCH * Q_ROW, "dst": 4 * BATCH * 4, "new_lens": 4 * BATCH,
        "new_mass": 4 * BATCH * 8 * BUDGET, "kept": 4 * BATCH * 8 * BUDGET}


@pytest.fixture(scope="module")
def B():
    from paged_kv_decode_04_gb300 import build
    build.build()
    from paged_kv_decode_04_gb300 import binding
    return binding


def p(a, name):
    return ctypes.c_void_p(a[name])


def chunk(B, a, ws_bytes):
    return B.lib().pkv_paged_chunk_attention(
        p(a, "q"), TOKENS, p(a, "off"), p(a, "pool"), PAGES, p(a, "bt"), WIDTH, p(a, "lens"),
        BATCH, 32, 8, 64, 16, 0, 0, 0.125, p(a, "out"), p(a, "ws"), ws_bytes, 2, p(a, "err"), None)


def window(B, a, ws_bytes):
    return B.lib().pkv_paged_window_attention(
        p(a, "q"), p(a, "pool"), PAGES, p(a, "bt"), WIDTH, p(a, "lens"), BATCH, 32, 8, 64, 16,
        1000, 0, 0.125, p(a, "out"), p(a, "ws"), ws_bytes, 2, p(a, "err"), None)


def scored(B, a, ws_bytes):
    return B.lib().pkv_paged_scored_attention(
        p(a, "q"), p(a, "pool"), PAGES, p(a, "bt"), WIDTH, p(a, "lens"), BATCH, 32, 8, 64, 16,
        0.125, p(a, "out"), p(a, "mass"), MASS_STRIDE, p(a, "ws"), ws_bytes, 2, p(a, "err"), None)


def evict(B, a, _):
    return B.lib().pkv_kv_evict(
        p(a, "mass"), MASS_STRIDE, p(a, "pool"), PAGES, p(a, "bt"), WIDTH, p(a, "lens"), BATCH, 8,
        64, 16, BUDGET, 4, 16, p(a, "dst"), 4, p(a, "new_lens"), p(a, "new_mass"), BUDGET,
        p(a, "kept"), p(a, "err"), None)


def append(B, a, _):
    return B.lib().pkv_kv_append_at(
        p(a, "k"), p(a, "v"), p(a, "pool"), PAGES, p(a, "bt"), WIDTH, p(a, "pos"), p(a, "slots"),
        BATCH, 8, 64, 16, 5e5, p(a, "q"), p(a, "q_out"), 32, p(a, "err"), None)


def sizes(call):
    rows = TOKENS if call is chunk else BATCH
    return dict(SIZE, q=rows * Q_ROW, out=rows * Q_ROW)


# (call, its outputs, what else it names)
CALLS = [
    (chunk, ["out", "err"], ["q", "off", "pool", "bt", "lens"]),
    (window, ["out", "err"], ["q", "pool", "bt", "lens"]),
    (scored, ["out", "mass", "err"], ["q", "pool", "bt", "lens"]),
    (evict, ["new_lens", "new_mass", "kept", "err"], ["mass", "pool", "bt", "lens", "dst"]),
    (append, ["q_out", "err"], ["q", "k", "v", "pool", "bt", "pos", "slots"]),
]
PAIRS = [(call, o, other) for call, outs, ins in CALLS
         for i, o in enumerate(outs) for other in ins + outs[:i]]


@pytest.mark.parametrize("call,out,other", PAIRS,
                         ids=[f"{c.__name__}-{o}-{x}" for c, o, x in PAIRS])
def test_outputs_that_overlap(B, call, out, other):
    size = sizes(call)
    for at in (0, size[other] - 16, 16 - size[out]):      # same start, last bytes, first bytes
        a = dict(PLACE)
        a[out] = PLACE[other] + (at & ~15 if at > 0 else -(-at & ~15))
        assert call(B, a, 0) == B.PKV_EINVAL, (at, hex(a[out]))


@pytest.mark.parametrize("call", [chunk, window, scored])
def test_outputs_that_touch(B, call):
    """Right behind, or right in front of, every other argument: no overlap, so
    the calls go on to miss their workspace."""
    size = sizes(call)
    outs, others = next((o, i) for c, o, i in CALLS if c is call)
    for out in outs:
        for other in others:
            for at in (-(-size[other] // 16) * 16, -(-size[out] // 16) * -16):
                a = dict(PLACE)
                a[out] = PLACE[other] + at
                assert call(B, a, 0) == B.PKV_EWORKSPACE, (out, other, at)


@pytest.mark.parametrize("call", [chunk, window, scored])
def test_workspaces_that_overlap(B, call):
    size = sizes(call)
    outs, others = next((o, i) for c, o, i in CALLS if c is call)
    need = {chunk: lambda: B.chunk_workspace_bytes(TOKENS, BATCH, WIDTH, 2),
            window: lambda: B.window_workspace_bytes(BATCH, WIDTH, 1000, 2),
            scored: lambda: B.scored_workspace_bytes(BATCH, WIDTH, 2)}[call]()
    assert need > 0
    for other in outs + others:
        for at in (0, (size[other] - 1) & ~15, -((need - 1) & ~15)):
            a = dict(PLACE, ws=PLACE[other] + at)
            assert call(B, a, need) == B.PKV_EINVAL, (other, at)
