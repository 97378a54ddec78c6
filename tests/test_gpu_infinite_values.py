"""Seen V values that are not finite (GPU): weights are positive, so a dim of a
row is the sum of what it sees there that is not finite, +inf, -inf or NaN,
and the other dims and the rows that do not see such a token are as without."""
import numpy as np
import pytest
import torch

from _gpu_util import binding, cuda_or_skip
from _longctx_util import HQ, P, attend, check, make_cache, normal, offsets, visible

pytestmark = pytest.mark.gpu

INF = float("inf")
LENS = [700, 90, 17]
# (sequence, token, dim, value): in pages that every row sees, in the last page,
# at both ends of windows, among the sinks, two values of one dim
VALUES = [(0, 3, 1, INF), (0, 5, 63, -INF), (0, 200, 2, INF), (0, 333, 3, -INF),
          (0, 334, 4, float("nan")), (0, 400, 5, INF), (0, 401, 5, -INF), (0, 500, 6, INF),
          (0, 650, 6, INF), (0, 651, 7, -INF), (0, 699, 8, INF), (0, 640, 9, -INF),
          (1, 10, 1, -INF), (1, 40, 2, INF), (1, 89, 3, -INF), (1, 80, 4, INF), (2, 16, 10, INF),
          (2, 0, 11, -INF)]


def cache(seed):
    """(pool, the pool with zeros for those values, tables)."""
    pool, bt = make_cache(LENS, seed=seed)
    clean = pool.clone()
    for s, t, d, x in VALUES:
        pool[int(bt[s, t // P]), 1, t % P, :, d] = x
        clean[int(bt[s, t // P]), 1, t % P, :, d] = 0.0
    return pool, clean, bt


def check_row(got, q, clean, bt, s, tokens, what):
    """got [32][64] of the query q of sequence s that sees `tokens`."""
    want, tol, _, _ = attend(q, clean, bt[s], tokens)
    special = np.zeros(64)
    seen = set(np.asarray(tokens).tolist())
    for b, t, d, x in VALUES:
        if b == s and t in seen:
            special[d] += x
    odd = special != 0
    got = got.double().numpy()
    assert np.array_equal(got[:, odd], np.broadcast_to(special[odd], (HQ, int(odd.sum()))),
                          equal_nan=True), (what, special[odd], got[0, odd])
    check(torch.from_numpy(got[:, ~odd]), want[:, ~odd], tol[:, ~odd], what)


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (300, 4), (60, 20)])
def test_window(window, sinks, splits):
    dev, b = cuda_or_skip(), binding()
    pool, clean, bt = cache(131)
    q = normal((len(LENS), HQ, 64), 132)
    out = b.paged_window_attention(q.to(dev), pool.to(dev), bt.to(dev),
                                   torch.tensor(LENS, dtype=torch.int32, device=dev), window,
                                   sinks=sinks, num_splits=splits).cpu()
    for s, n in enumerate(LENS):
        check_row(out[s], q[s], clean, bt, s, visible(n - 1, window, sinks), f"sequence {s}")


@pytest.mark.parametrize("splits", [0, 1, 3])
def test_scored(splits):
    dev, b = cuda_or_skip(), binding()
    pool, clean, bt = cache(133)
    q = normal((len(LENS), HQ, 64), 134)
    mass = torch.zeros((len(LENS), 8, bt.shape[1] * P), device=dev)
    out = b.paged_scored_attention(q.to(dev), pool.to(dev), bt.to(dev),
                                   torch.tensor(LENS, dtype=torch.int32, device=dev), mass,
                                   num_splits=splits).cpu()
    assert torch.isfinite(mass).all()
    for s, n in enumerate(LENS):
        check_row(out[s], q[s], clean, bt, s, np.arange(n), f"sequence {s}")


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 4), (60, 20)])
@pytest.mark.parametrize("counts", [[1, 2, 4], [4, 3, 1], [70, 80, 17], [20, 4, 9]])
def test_chunk(counts, window, sinks, splits):
    dev, b = cuda_or_skip(), binding()
    pool, clean, bt = cache(135)
    off = offsets(counts)
    q = normal((int(off[-1]), HQ, 64), 136)
    out = b.paged_chunk_attention(q.to(dev), off.to(dev), pool.to(dev), bt.to(dev),
                                  torch.tensor(LENS, dtype=torch.int32, device=dev),
                                  window=window, sinks=sinks, num_splits=splits).cpu()
    for s, n in enumerate(LENS):
        for i in range(counts[s]):
            r = int(off[s]) + i
            check_row(out[r], q[r], clean, bt, s, visible(n - counts[s] + i, window, sinks),
                      f"row {i} of sequence {s}")
