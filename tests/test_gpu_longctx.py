"""The long-context operators against plain 64-bit implementations (GPU)."""
import numpy as np
import pytest
import torch

import oracle
from _gpu_util import binding, cuda_or_skip
from _longctx_util import (G, HKV, HQ, P, attend, check, chunk_reference, make_cache, normal,
                           offsets, visible)

pytestmark = pytest.mark.gpu

DEVERR_PAGE, DEVERR_SEQLEN, DEVERR_POSITION, DEVERR_OFFSETS = 1, 2, 4, 16


def dev_err(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def lens_t(lens):
    return torch.tensor(lens, dtype=torch.int32)


# ------------------------------------------------------------------- chunks --

def run_chunk(lens, counts, window=0, sinks=0, *, splits=0, seed=1, pad=0, cache=None, scale=None,
              q_scale=1.0, **kw):
    dev, b = cuda_or_skip(), binding()
    pool, bt = cache or make_cache(lens, seed=seed)
    off = offsets(counts)
    rows = int(off[-1]) + pad
    q = normal((rows, HQ, 64), seed + 1) * q_scale
    out0 = torch.full((rows, HQ, 64), 7.0, dtype=torch.bfloat16)
    err = dev_err(dev)
    out = out0.to(dev)
    b.paged_chunk_attention(q.to(dev), off.to(dev), pool.to(dev), bt.to(dev), lens_t(lens).to(dev),
                            out, window=window, sinks=sinks, num_splits=splits, dev_err=err,
                            scale=scale, **kw)
    want, tol = chunk_reference(q, off, pool, bt, lens, window, sinks, out0,
                                **({} if scale is None else {"scale": scale}))
    check(out, want, tol, f"{lens} {counts} window {window} sinks {sinks} splits {splits}")
    return int(err.item())


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("lens,counts", [
    ([1], [1]), ([17], [17]), ([16], [1]), ([129], [128]), ([515], [5]), ([300], [300]),
    ([40, 3, 131], [5, 3, 1]), ([33, 7, 64, 5], [0, 7, 0, 1]), ([700, 64, 200], [130, 64, 33]),
    ([1100], [1]), ([257, 256, 255, 1], [9, 65, 31, 1]), ([4], [4]), ([5], [5]),
    ([500, 499, 17, 1300], [2, 3, 4, 1]),
])
def test_chunk_causal(lens, counts, splits):
    assert run_chunk(lens, counts, splits=splits, pad=2) == 0


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("window,sinks", [
    (1, 0), (1, 1), (16, 3), (100, 200), (128, 16), (130, 0), (64, 129), (2 ** 31 - 1, 5),
    (700, 4),
])
def test_chunk_window(window, sinks, splits):
    assert run_chunk([700, 90, 33], [140, 90, 2], window, sinks, splits=splits) == 0


@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("lens,counts,window", [
    # several items for each CTA: of one kv tile, of none, of both row tiles
    ([100] * 70, [2] * 70, 0), ([1 + i for i in range(64)], [1] * 64, 0),
    ([90 + 20 * i for i in range(40)], [1 + (i * 29) % 80 for i in range(40)], 0),
    ([200 + 7 * (i % 5) for i in range(45)], [(0, 1, 33, 64, 70)[i % 5] for i in range(45)], 60),
    ([8 + (i * 61) % 300 for i in range(90)], [1 + i % 4 if i % 9 else 5 for i in range(90)], 40),
])
def test_chunk_many_items(lens, counts, window, splits):
    assert run_chunk(lens, counts, window, 3 if window else 0, splits=splits) == 0


@pytest.mark.parametrize("counts", [[70], [4]])
def test_chunk_scales(counts):
    # flat weights, and weights that all fall on a few tokens
    run_chunk([400], counts, scale=2.0 ** -20)
    run_chunk([400], counts, scale=2.0)


@pytest.mark.parametrize("counts,splits", [([90], 1), ([90], 2), ([20], 1), ([3], 1), ([3], 3)])
@pytest.mark.parametrize("shape", ["rising", "falling", "steps"])
def test_chunk_scores_that_ramp(counts, splits, shape):
    """Scores that rise or fall by hundreds over the cache: the reference
    maximum moves in every tile, or never after the first."""
    lens = [700]
    pool, bt = make_cache(lens, seed=25)
    t = np.arange(700)
    ramp = {"rising": t / 2.0, "falling": -t / 2.0, "steps": (t // 150) * 90.0 % 270}[shape]
    for tok in range(700):
        # dim 0 of the keys, against queries of 1 there
        pool[int(bt[0, tok // P]), 0, tok % P, :, 0] = float(ramp[tok])
    off = offsets(counts)
    q = normal((counts[0], HQ, 64), 26)
    q[..., 0] = 1.0
    dev, b = cuda_or_skip(), binding()
    out = b.paged_chunk_attention(q.to(dev), off.to(dev), pool.to(dev), bt.to(dev),
                                  lens_t(lens).to(dev), scale=0.5, num_splits=splits)
    want, tol = chunk_reference(q, off, pool, bt, lens, 0, 0, torch.zeros_like(q), 0.5)
    check(out, want, tol, shape)


@pytest.mark.parametrize("splits", [1, 4])
def test_chunk_masked_places_do_not_matter(splits):
    """NaN and infinities in K and V of tokens that a query does not see."""
    dev, b = cuda_or_skip(), binding()
    lens, counts, window, sinks = [330, 150], [70, 20], 90, 5
    pool, bt = make_cache(lens, seed=5)
    off = offsets(counts)
    q = normal((int(off[-1]), HQ, 64), 6)
    bad = {0: [290, 300, 329, 180, 8], 1: [149, 45]}
    for s, toks in bad.items():
        for i, t in enumerate(toks):
            pid = int(bt[s, t // P])
            val = [float("nan"), float("inf"), float("-inf")][i % 3]
            pool[pid, 1, t % P, :, i::7] = val
            pool[pid, 0, t % P, ::2, 0] = float("nan")
    err = dev_err(dev)
    out = b.paged_chunk_attention(q.to(dev), off.to(dev), pool.to(dev), bt.to(dev),
                                  lens_t(lens).to(dev), window=window, sinks=sinks,
                                  num_splits=splits, dev_err=err).cpu()
    assert int(err.item()) == 0
    seen = unseen = 0
    for s in range(2):
        for i in range(counts[s]):
            pos, r = lens[s] - counts[s] + i, int(off[s]) + i
            vis = visible(pos, window, sinks)
            hit = [t for t in bad[s] if t in vis]
            got = out[r].float().reshape(HKV, G, 64)
            if not hit:
                unseen += 1
                want, tol, _, _ = attend(q[r], pool, bt[s], vis)
                check(out[r], want, tol, f"row {r}")
            else:
                # a NaN key makes its head's rows NaN; other heads stay finite
                # but for the dims that hold a non-finite value
                seen += 1
                assert torch.isnan(got[::2]).all()
                dims = np.zeros(64, bool)
                for t in hit:
                    dims[bad[s].index(t)::7] = True
                assert not torch.isfinite(got[1::2][..., torch.from_numpy(dims)]).any()
                assert torch.isfinite(got[1::2][..., torch.from_numpy(~dims)]).all()
    assert seen > 5 and unseen > 20


def test_chunk_longer_than_its_sequence():
    assert run_chunk([3, 20], [8, 2]) == DEVERR_POSITION
    assert run_chunk([0, 20], [4, 2]) == DEVERR_POSITION
    assert run_chunk([0, 20], [0, 2]) == 0


@pytest.mark.parametrize("splits", [1, 2])
def test_chunk_bad_pages_are_skipped(splits):
    lens, counts = [200, 180], [40, 3]
    pool, bt = make_cache(lens, seed=9)
    bt[0, 2], bt[0, 11], bt[1, 0] = -5, pool.shape[0], 2 ** 30
    assert run_chunk(lens, counts, splits=splits, cache=(pool, bt)) == DEVERR_PAGE


def test_chunk_pages_outside_the_window_are_not_read():
    lens, counts = [2000], [30]
    pool, bt = make_cache(lens, seed=10)
    bt[0, 1:110] = -1            # sinks in page 0; the window starts at 1970 - 199 = 1771
    assert run_chunk(lens, counts, 200, 9, cache=(pool, bt)) == 0


def test_chunk_bad_lengths_and_offsets():
    dev, b = cuda_or_skip(), binding()
    pool, bt = make_cache([40, 40], seed=11)
    q = normal((12, HQ, 64), 12).to(dev)
    for lens, off, bit in (([41 + 100, 40], [0, 4, 12], DEVERR_SEQLEN),
                           ([-1, 40], [0, 3, 12], DEVERR_SEQLEN),
                           ([40, 40], [0, 9, 5], DEVERR_OFFSETS),
                           ([40, 40], [-3, 4, 12], DEVERR_OFFSETS),
                           ([40, 40], [0, 4, 13], DEVERR_OFFSETS),
                           ([40, 40], [0, 2 ** 31 - 1, -2 ** 31], DEVERR_OFFSETS)):
        err = dev_err(dev)
        b.paged_chunk_attention(q, torch.tensor(off, dtype=torch.int32, device=dev), pool.to(dev),
                                bt.to(dev), lens_t(lens).to(dev), dev_err=err)
        assert int(err.item()) & bit, (lens, off, int(err.item()))


def test_chunk_long_cache():
    """More pages than one CTA's page list, and a table wider than needed."""
    lens, counts = [20000], [3]
    cache = make_cache(lens, seed=13, width=1400)
    assert run_chunk(lens, counts, cache=cache) == 0
    assert run_chunk(lens, counts, 3001, 40, cache=cache) == 0


def test_chunk_repeats_bit_for_bit_and_replays():
    dev, b = cuda_or_skip(), binding()
    lens, counts = [900, 77, 300], [60, 1, 200]
    pool, bt = make_cache(lens, seed=14)
    off = offsets(counts)
    q = normal((int(off[-1]), HQ, 64), 15).to(dev)
    args = (off.to(dev), pool.to(dev), bt.to(dev), lens_t(lens).to(dev))
    ws = torch.empty(max(16, b.chunk_workspace_bytes(q.shape[0], 3, bt.shape[1], 3)),
                     dtype=torch.uint8, device=dev)
    first = b.paged_chunk_attention(q, *args, num_splits=3, workspace=ws)
    for _ in range(3):
        assert torch.equal(first, b.paged_chunk_attention(q, *args, num_splits=3, workspace=ws))
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.paged_chunk_attention(q, *args, out, num_splits=3, workspace=ws)
    q2 = normal(q.shape, 16).to(dev)
    q.copy_(q2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, b.paged_chunk_attention(q2, *args, num_splits=3, workspace=ws))


def test_waits_that_run_out():
    """With a wait limit of 0 every kernel gives up at its first look at a copy
    that has not landed, reports it, and leaves the stream and the next calls as
    they should be.  (The pages come from memory, what a kernel reads before
    that look from L2, so such a copy is certain.)"""
    dev, b = cuda_or_skip(), binding()
    lens, counts = [900, 70, 1500, 333], [3, 70, 200, 1]
    pool, bt = (x.to(dev) for x in make_cache(lens, seed=19))
    off, ln = offsets(counts).to(dev), lens_t(lens).to(dev)
    q = normal((sum(counts), HQ, 64), 20).to(dev)
    mass = torch.zeros((4, HKV, bt.shape[1] * P), device=dev)
    calls = [lambda e: b.paged_chunk_attention(q, off, pool, bt, ln, dev_err=e),
             lambda e: b.paged_chunk_attention(q, off, pool, bt, ln, num_splits=3, dev_err=e),
             lambda e: b.paged_window_attention(q[:4], pool, bt, ln, 500, dev_err=e),
             lambda e: b.paged_scored_attention(q[:4], pool, bt, ln, mass.zero_(), dev_err=e)]
    for call in calls:
        want = call(None)
        old = b.set_wait_limit_ns(0)
        err = dev_err(dev)
        torch.empty(1 << 28, dtype=torch.uint8, device=dev).zero_()
        for x in (q, off, bt, ln):
            x.clone()
        try:
            call(err)
        finally:
            b.set_wait_limit_ns(old)
        torch.cuda.synchronize()
        assert int(err.item()) & 8
        assert not torch.isnan(mass).any()
        err = dev_err(dev)
        assert torch.equal(want, call(err)) and int(err.item()) == 0


def test_calls_on_another_stream():
    dev, b = cuda_or_skip(), binding()
    lens, counts = [333, 40], [50, 7]
    pool, bt = (x.to(dev) for x in make_cache(lens, seed=17))
    off, ln = offsets(counts).to(dev), lens_t(lens).to(dev)
    q = normal((57, HQ, 64), 18).to(dev)
    want = b.paged_chunk_attention(q, off, pool, bt, ln, num_splits=2)
    w1 = b.paged_window_attention(q[:2], pool, bt, ln, 50, sinks=2, num_splits=2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        got = b.paged_chunk_attention(q, off, pool, bt, ln, num_splits=2, stream=s)
        g1 = b.paged_window_attention(q[:2], pool, bt, ln, 50, sinks=2, num_splits=2, stream=s)
        torch.empty(1 << 20, dtype=torch.uint8, device=dev).fill_(0xFF)
        s.synchronize()
        assert torch.equal(want, got) and torch.equal(w1, g1)


def test_results_of_a_side_stream_keep_clear_of_the_current_one():
    """A call on another stream makes its result of memory that the current
    stream's work, still running, is about to write."""
    dev, b = cuda_or_skip(), binding()
    lens = [333, 40]
    pool, bt = (x.to(dev) for x in make_cache(lens, seed=17))
    ln, q = lens_t(lens).to(dev), normal((2, HQ, 64), 18).to(dev)
    off = offsets([1, 1]).to(dev)
    calls = (lambda **kw: b.paged_window_attention(q, pool, bt, ln, 50, num_splits=2, **kw),
             lambda **kw: b.paged_chunk_attention(q, off, pool, bt, ln, num_splits=2, **kw))
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        freed = torch.empty_like(q)
        torch.cuda._sleep(20_000_000)
        freed.fill_(9)
        del freed
        got = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("counts", [[5], [3]])
def test_largest_table(counts):
    """Positions up to the last one a table can name."""
    dev, b = cuda_or_skip(), binding()
    blocks, window, sinks, n = 2 ** 27 - 1, 200, 3, counts[0]
    L = blocks * 16 - 2
    last = 16                                   # the table's pages that exist: 0 and the last 16
    pool = normal((last + 1, 2, 16, HKV, 64), 40)
    q = normal((n, HQ, 64), 41)
    bt = torch.full((1, blocks), -1, dtype=torch.int32, device=dev)
    bt[0, 0] = last
    bt[0, blocks - last:] = torch.arange(last, dtype=torch.int32, device=dev)
    near = np.concatenate([[last], np.arange(last)]).astype(np.int32)
    want, tol = np.zeros((n, HQ, 64)), np.zeros((n, HQ, 64))
    for i in range(n):
        p = L - n + i
        t = np.concatenate([np.arange(sinks), 16 + np.arange(p - window + 1, p + 1) -
                            16 * (blocks - last)])
        want[i], tol[i], _, _ = attend(q[i], pool, near, t)
    args = pool.to(dev), bt, torch.tensor([L], dtype=torch.int32, device=dev)
    err = dev_err(dev)
    out = b.paged_chunk_attention(q.to(dev), offsets(counts).to(dev), *args, window=window,
                                  sinks=sinks, dev_err=err)
    check(out, want, tol, "chunk")
    out = b.paged_window_attention(q[-1:].to(dev), *args, window, sinks=sinks, dev_err=err)
    check(out, want[-1:], tol[-1:], "window")
    assert int(err.item()) == 0


# ------------------------------------------------- one token under a window --

def run_window(lens, window, sinks, *, splits=0, seed=21, cache=None):
    dev, b = cuda_or_skip(), binding()
    pool, bt = cache or make_cache(lens, seed=seed)
    q = normal((len(lens), HQ, 64), seed + 1)
    err = dev_err(dev)
    out = b.paged_window_attention(q.to(dev), pool.to(dev), bt.to(dev), lens_t(lens).to(dev),
                                   window, sinks=sinks, num_splits=splits, dev_err=err)
    got = [attend(q[i], pool, bt[i], visible(n - 1, window, sinks) if n else [])
           for i, n in enumerate(lens)]
    check(out, np.stack([x[0] for x in got]), np.stack([x[1] for x in got]),
          f"{lens} window {window} sinks {sinks} splits {splits}")
    return int(err.item())


@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 17), (16, 16), (33, 4), (100, 150),
                                          (1000, 5), (2 ** 31 - 1, 2 ** 31 - 1), (640, 1)])
def test_window(window, sinks, splits):
    lens = [1, 2, 16, 17, 33, 50, 0, 117, 640, 641, 1500]
    assert run_window(lens, window, sinks, splits=splits) == 0


@pytest.mark.parametrize("batch", [1, 200])
def test_window_batches(batch):
    lens = [1 + (i * 97) % 700 for i in range(batch)]
    lens[0] = 700
    assert run_window(lens, 257, 4) == 0


def test_window_masked_places_do_not_matter():
    lens, window, sinks = [500, 37], 100, 5
    pool, bt = make_cache(lens, seed=23)
    for t in (5, 6, 15, 16, 200, 399):        # 400..499 and 0..4 are seen
        pool[int(bt[0, t // P]), :, t % P] = float("nan")
    assert run_window(lens, window, sinks, cache=(pool, bt)) == 0
    bt[0, 2:24] = -1                          # and pages between need not exist
    assert run_window(lens, window, sinks, cache=(pool, bt)) == 0
    bt[0, 28] = pool.shape[0]
    assert run_window(lens, window, sinks, cache=(pool, bt)) == DEVERR_PAGE


# ------------------------------------------------------ weights and eviction --

def mass_reference(q, pool, bt, lens, mass):
    out, tol, m, mt = [], [], mass.double().numpy().copy(), np.zeros(mass.shape)
    for i, n in enumerate(lens):
        o, a, (t, w), rel = attend(q[i], pool, bt[i], np.arange(n))
        out.append(o)
        tol.append(a)
        ws = w.reshape(len(t), HKV, G).sum(-1)
        m[i][:, t] += ws.T
        # the four weights' relative errors, their sum's and the addition's roundings
        mt[i][:, t] = (ws * (rel + 2.0 ** -22)).T + 2.0 ** -24 * np.abs(m[i][:, t]) * 1.01
    return np.stack(out), np.stack(tol), m, mt + 1e-38


@pytest.mark.parametrize("splits", [0, 1, 2, 6])
@pytest.mark.parametrize("lens", [[1], [16, 17, 0, 300], [700], [1, 1500, 64, 65, 31],
                                  [4200, 40]])
def test_scored(lens, splits):
    dev, b = cuda_or_skip(), binding()
    pool, bt = make_cache(lens, seed=31)
    q = normal((len(lens), HQ, 64), 32)
    mass = torch.from_numpy(np.random.default_rng(33).random(
        (len(lens), HKV, bt.shape[1] * P + 5)).astype(np.float32))
    got, err = mass.to(dev), dev_err(dev)
    out = b.paged_scored_attention(q.to(dev), pool.to(dev), bt.to(dev), lens_t(lens).to(dev), got,
                                   num_splits=splits, dev_err=err)
    o, ot, m, mt = mass_reference(q, pool, bt, lens, mass)
    check(out, o, ot, "out")
    check(got, m, mt, "mass")
    assert int(err.item()) == 0
    again = mass.to(dev)
    assert torch.equal(out, b.paged_scored_attention(
        q.to(dev), pool.to(dev), bt.to(dev), lens_t(lens).to(dev), again, num_splits=splits))
    assert torch.equal(got, again)


@pytest.mark.parametrize("splits", [1, 2])
def test_scored_bad_pages(splits):
    dev, b = cuda_or_skip(), binding()
    lens = [200, 90]
    pool, bt = make_cache(lens, seed=34)
    bt[0, 3], bt[1, 5] = -1, pool.shape[0] + 4
    q = normal((2, HQ, 64), 35)
    mass = torch.zeros((2, HKV, bt.shape[1] * P))
    got, err = mass.to(dev), dev_err(dev)
    out = b.paged_scored_attention(q.to(dev), pool.to(dev), bt.to(dev), lens_t(lens).to(dev), got,
                                   num_splits=splits, dev_err=err)
    o, ot, m, mt = mass_reference(q, pool, bt, lens, mass)
    check(out, o, ot, "out")
    check(got, m, mt, "mass")
    assert int(err.item()) == DEVERR_PAGE


def evict_reference(mass, n, budget, sinks, recent):
    """Kept tokens per kv head of one sequence."""
    if n <= budget:
        return [np.arange(n)] * HKV
    kept = []
    for h in range(HKV):
        m = mass[h, :n].double().numpy().copy()
        m[np.isnan(m)] = np.inf                       # as heavy as can be ...
        key = np.stack([np.isnan(mass[h, :n].numpy()).astype(float), m])
        free = np.arange(sinks, n - recent)
        order = free[np.lexsort((free, -key[1][free], -key[0][free]))]
        kept.append(np.sort(np.concatenate([np.arange(sinks), order[:budget - sinks - recent],
                                            np.arange(n - recent, n)])))
    return kept


def run_evict(lens, budget, sinks, recent, mass=None, seed=41, extra=1, width=None):
    dev, b = cuda_or_skip(), binding()
    B = len(lens)
    wide = -(-budget // P) + extra
    pool, bt = make_cache(lens, seed=seed, spare=B * wide + 2, width=width)
    free = sorted(set(range(pool.shape[0])) - set(bt[bt >= 0].tolist()))
    dst = torch.tensor(np.random.default_rng(seed).permutation(free)[:B * wide].reshape(B, wide),
                       dtype=torch.int32)
    rng = np.random.default_rng(seed + 1)
    if mass is None:
        mass = np.round(rng.exponential(4.0, (B, HKV, bt.shape[1] * P + 3)) * 8) / 8  # many ties
    mass = torch.from_numpy(np.asarray(mass, np.float32))
    gp, err = pool.to(dev), dev_err(dev)
    new_lens, new_mass, kept = b.kv_evict(mass.to(dev), gp, bt.to(dev), lens_t(lens).to(dev),
                                          dst.to(dev), budget=budget, sinks=sinks, recent=recent,
                                          dev_err=err)
    assert int(err.item()) == 0
    want_pool = pool.clone()
    for i, n in enumerate(lens):
        k = min(n, budget)
        assert int(new_lens[i]) == k
        for h, keep in enumerate(evict_reference(mass[i], n, budget, sinks, recent)):
            assert kept[i, h].tolist() == keep.tolist() + [-1] * (budget - k)
            assert torch.equal(new_mass[i, h].cpu().view(torch.int32),
                               torch.cat([mass[i, h, keep], torch.zeros(new_mass.shape[2] - k)]
                                         ).view(torch.int32))
            at = torch.arange(k)
            src = torch.from_numpy(keep)
            want_pool[dst[i, at // P].long(), :, at % P, h] = \
                pool[bt[i, src // P].long(), :, src % P, h]
    # every byte of the pool: old pages and slots past the end as they were
    assert torch.equal(gp.cpu().view(torch.int16), want_pool.view(torch.int16))
    return new_lens, new_mass, dst, gp


@pytest.mark.parametrize("budget,sinks,recent", [
    (1, 0, 0), (1, 1, 0), (1, 0, 1), (16, 0, 0), (17, 2, 5), (64, 4, 16), (64, 64, 0),
    (64, 0, 64), (100, 30, 70), (255, 4, 100), (600, 4, 16)])
def test_evict(budget, sinks, recent):
    run_evict([700, 1, 16, 64, 65, 0, 300, 101], budget, sinks, recent)


def test_evict_long():
    run_evict([20011, 5000], 1000, 4, 200)


@pytest.mark.parametrize("width", [512, 513, 3100, 4000])
def test_evict_wide_tables(width):
    # tables of 8192 and of 49152 tokens and more select with other kernels
    run_evict([700, 1, 300, 64], 100, 4, 16, width=width)


def test_evict_wide_tables_of_a_large_batch():
    # more (sequence, head) pairs than SMs, tables of more than 8192 tokens
    run_evict([700, 1, 300, 9600] + [64, 0, 129, 500] * 4, 100, 4, 16, width=600)


def test_evict_values_at_their_limits():
    """NaN, infinities, zeros of both signs, subnormals, negative values."""
    n, B = 300, 1
    vals = np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, -3.0, 2.5],
                    np.float32)
    for budget in (20, 60, 100, 130, 160, 200, 290):
        mass = np.zeros((B, HKV, 304), np.float32)
        for h in range(HKV):
            mass[0, h] = np.random.default_rng(h).choice(vals, 304)
        run_evict([n], budget, 1, 3, mass)
        run_evict([n], budget, 0, 0, np.full((B, HKV, 304), np.float32(0.25)))


def test_evict_bad_pages_and_lengths():
    dev, b = cuda_or_skip(), binding()
    pool, bt = make_cache([64, 64], seed=43, spare=12)
    free = sorted(set(range(pool.shape[0])) - set(bt[bt >= 0].tolist()))
    dst = torch.tensor(free[:4], dtype=torch.int32).reshape(2, 2)
    mass = torch.zeros((2, HKV, 64))
    good = None
    for case in ("good", "src", "dst", "len"):
        t, d, ln, err = bt.clone(), dst.clone(), lens_t([64, 64]), dev_err(dev)
        if case == "src":
            t[0, 0] = -1
        if case == "dst":
            d[1, 0] = pool.shape[0]
        if case == "len":
            ln[1] = 65
        gp = pool.to(dev)
        nl, nm, kept = b.kv_evict(mass.to(dev), gp, t.to(dev), ln.to(dev), d.to(dev), budget=32,
                                  sinks=16, recent=16, dev_err=err)
        bits = gp.cpu().view(torch.int16)
        want = {"good": 0, "src": DEVERR_PAGE, "dst": DEVERR_PAGE, "len": DEVERR_SEQLEN}[case]
        assert int(err.item()) == want
        assert nl.tolist() == [32, 32]
        if case == "good":
            good = bits
        elif case == "src":      # sequence 0's first 16 rows stay unwritten
            ref = good.clone()
            ref[int(dst[0, 0])] = pool.view(torch.int16)[int(dst[0, 0])]
            assert torch.equal(bits, ref)
        elif case == "dst":
            ref = good.clone()
            ref[int(dst[1, 0])] = pool.view(torch.int16)[int(dst[1, 0])]
            assert torch.equal(bits, ref)
        else:
            assert torch.equal(bits, good)


# ----------------------------------------------------- append at another slot --

@pytest.mark.parametrize("batch", [1, 3, 300])
def test_append_at(batch):
    dev, b = cuda_or_skip(), binding()
    rng = np.random.default_rng(batch)
    lens = [1 + (i * 37) % 90 for i in range(batch)]
    pool, bt = make_cache(lens, seed=51)
    pos = rng.integers(0, 2 ** 20, batch).astype(np.int32)
    pos[0] = 2 ** 31 - 1 if batch > 1 else 2047
    slots = np.array(lens, np.int32) - 1
    k, v, q = (normal((batch, n, 64), 52 + n) for n in (HKV, HKV, HQ))
    v = -v
    gp, err, qo = pool.to(dev), dev_err(dev), torch.zeros_like(q).to(dev)
    b.kv_append_at(k.to(dev), v.to(dev), gp, bt.to(dev), torch.from_numpy(pos).to(dev),
                   torch.from_numpy(slots).to(dev), q_in=q.to(dev), q_out=qo, dev_err=err)
    assert int(err.item()) == 0
    want = pool.clone().view(torch.int16)
    qi, ki = (x.view(torch.int16).numpy().view(np.uint16) for x in (q, k))
    for i in range(batch):
        pid, s = int(bt[i, slots[i] // P]), int(slots[i]) % P
        for h in range(HKV):
            want[pid, 0, s, h] = torch.from_numpy(
                oracle.rope_rotate(ki[i, h], int(pos[i]), 500000.0).view(np.int16))
        want[pid, 1, s] = v.view(torch.int16)[i]
        for j in range(0, HQ, 7):
            assert np.array_equal(qo[i, j].cpu().view(torch.int16).numpy().view(np.uint16),
                                  oracle.rope_rotate(qi[i, j], int(pos[i]), 500000.0))
    assert torch.equal(gp.cpu().view(torch.int16), want)


def test_append_at_positions_is_append():
    dev, b = cuda_or_skip(), binding()
    lens = [5, 40, 33]
    pool, bt = make_cache(lens, seed=53)
    k, v = normal((3, HKV, 64), 54).to(dev), normal((3, HKV, 64), 55).to(dev)
    at = (lens_t(lens) - 1).to(dev)
    p1, p2 = pool.to(dev), pool.to(dev)
    b.kv_append(k, v, p1, bt.to(dev), at)
    b.kv_append_at(k, v, p2, bt.to(dev), at, at)
    assert torch.equal(p1.view(torch.int16), p2.view(torch.int16))


def test_append_at_bad_slots():
    dev, b = cuda_or_skip(), binding()
    pool, bt = make_cache([20], seed=56)
    k = normal((1, HKV, 64), 57).to(dev)
    for pos, slot, page, bit in ((-1, 3, None, DEVERR_POSITION), (3, -1, None, DEVERR_POSITION),
                                 (3, 32, None, DEVERR_POSITION), (3, 17, -1, DEVERR_PAGE),
                                 (3, 2 ** 31 - 1, None, DEVERR_POSITION)):
        t, gp, err = bt.clone(), pool.to(dev), dev_err(dev)
        if page is not None:
            t[0, 1] = page
        b.kv_append_at(k, k, gp, t.to(dev), lens_t([pos]).to(dev), lens_t([slot]).to(dev),
                       dev_err=err)
        assert int(err.item()) == bit
        assert torch.equal(gp.cpu().view(torch.int16), pool.view(torch.int16))


# ------------------------------------------------------------------ together --

def test_a_long_conversation():
    """A prompt prefilled in chunks, decode steps whose weights are tracked, an
    eviction, further steps on the smaller cache, and one windowed step: every
    output against the 64-bit attention over the cache as it stands."""
    dev, b = cuda_or_skip(), binding()
    prompt, chunk, budget, sinks, recent = 150, 64, 48, 4, 8
    pages = 40
    pool = torch.full((pages, 2, P, HKV, 64), float("nan"), dtype=torch.bfloat16, device=dev)
    order = np.random.default_rng(61).permutation(pages).astype(np.int32)
    bt = torch.from_numpy(order[:12][None]).contiguous().to(dev)
    mass = torch.zeros((1, HKV, 12 * P), device=dev)
    err = dev_err(dev)
    ws = None
    for at in range(0, prompt, chunk):
        n = min(chunk, prompt - at)
        k, v, q = (normal((n, h, 64), 62 + at + h).to(dev) for h in (HKV, HKV, HQ))
        off = offsets([n]).to(dev)
        b.kv_write_prefill(k, v, off, lens_t([at]).to(dev), pool, bt, dev_err=err)
        out = b.paged_chunk_attention(q, off, pool, bt, lens_t([at + n]).to(dev), dev_err=err)
        want, tol = chunk_reference(q.cpu(), off.cpu(), pool.cpu(), bt.cpu(), [at + n], 0, 0,
                                    torch.zeros_like(q).cpu())
        check(out, want, tol, f"chunk at {at}")
    cached, pos = prompt, prompt

    def step(window=None):
        nonlocal cached, pos
        k, v, q = (normal((1, h, 64), 900 + pos + h).to(dev) for h in (HKV, HKV, HQ))
        qr = torch.empty_like(q)
        b.kv_append_at(k, v, pool, bt, lens_t([pos]).to(dev), lens_t([cached]).to(dev), q_in=q,
                       q_out=qr, dev_err=err)
        cached, pos = cached + 1, pos + 1
        ln = lens_t([cached]).to(dev)
        if window:
            out = b.paged_window_attention(qr, pool, bt, ln, window, sinks=sinks, dev_err=err)
            vis = visible(cached - 1, window, sinks)
        else:
            before = mass.cpu()
            out = b.paged_scored_attention(qr, pool, bt, ln, mass, dev_err=err)
            vis = np.arange(cached)
            _, _, m, mt = mass_reference(qr.cpu(), pool.cpu(), bt.cpu(), [cached], before)
            check(mass, m, mt, f"mass at {pos}")
        want, tol, _, _ = attend(qr[0].cpu(), pool.cpu(), bt[0].cpu(), vis)
        check(out[0], want, tol, f"step at {pos}")

    for _ in range(5):
        step()
    dst = torch.from_numpy(order[12:24][None]).contiguous().to(dev)
    n, mass, kept = b.kv_evict(mass, pool, bt, lens_t([cached]).to(dev), dst, budget=budget,
                               sinks=sinks, recent=recent, dev_err=err)
    assert kept[0, 0, :sinks].tolist() == list(range(sinks))
    assert kept[0, :, -recent:].tolist() == [list(range(cached - recent, cached))] * HKV
    cached, bt = int(n[0]), dst
    assert cached == budget
    for _ in range(4):
        step()
    step(window=20)
    assert int(err.item()) == 0
