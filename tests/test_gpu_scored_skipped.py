"""The mass of cached tokens that a scored call cannot read (a page id that is
not of the pool), next to keys whose scores make a row NaN (GPU): those
entries, and the ones past the sequence's end, keep every bit."""
import numpy as np
import pytest
import torch

from _gpu_util import binding, cuda_or_skip
from _longctx_util import G, HKV, HQ, P, attend, check, make_cache, normal

pytestmark = pytest.mark.gpu

DEVERR_PAGE = 1


@pytest.mark.parametrize("splits", [0, 1, 2, 6])
@pytest.mark.parametrize("value", ["nan", "inf", "finite"])
@pytest.mark.parametrize("lens", [[200, 90], [700], [4200, 40]])
def test_mass_of_skipped_pages_stands(lens, value, splits):
    dev, b = cuda_or_skip(), binding()
    pool, bt = make_cache(lens, seed=71)
    skipped = {0: [3, 7, (lens[0] - 1) // P], len(lens) - 1: [0, 2]}
    # kv heads 0, 2, 4 and 6 see a key that makes their rows' sums NaN
    if value != "finite":
        for s in range(len(lens)):
            pool[int(bt[s, 1]), 0, 5, ::2, :] = float(value)
    for s, pages in skipped.items():
        for i, page in enumerate(pages):
            bt[s, page] = [-1, pool.shape[0] + 4, 2 ** 31 - 1][i]
    q = normal((len(lens), HQ, 64), 72).abs()
    before = np.random.default_rng(73).random((len(lens), HKV, bt.shape[1] * P + 5))
    before = before.astype(np.float32)
    before[:, :, ::7] = -0.0
    before[:, :, 3::11] = np.inf
    mass = torch.from_numpy(before).to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = b.paged_scored_attention(q.to(dev), pool.to(dev), bt.to(dev),
                                   torch.tensor(lens, dtype=torch.int32, device=dev), mass,
                                   num_splits=splits, dev_err=err)
    assert int(err.item()) == DEVERR_PAGE
    got = mass.cpu().numpy()
    heads = np.arange(HKV)
    clean = heads if value == "finite" else heads[1::2]
    for s, n in enumerate(lens):
        t = np.arange(before.shape[2])
        read = (t < n) & ~np.isin(t // P, skipped.get(s, []))
        assert np.array_equal(got[s][:, ~read].view(np.int32), before[s][:, ~read].view(np.int32))
        if value != "finite":
            assert np.isnan(got[s][::2][:, read]).all()
            pool[int(bt[s, 1]), 0, 5, ::2, :] = 0.0       # so that the other heads' is finite
        want, tol, (tt, w), rel = attend(q[s], pool, bt[s], np.arange(n))
        rows = np.repeat(np.isin(heads, clean), G)
        check(out[s].cpu()[torch.from_numpy(rows)], want[rows], tol[rows], f"out {s}")
        ws = w.reshape(len(tt), HKV, G).sum(-1).T
        m = before[s].astype(np.float64)
        m[:, tt] += ws
        # the weights' relative errors, their sum's and the addition's roundings
        mt = np.zeros_like(m)
        mt[:, tt] = ws * (rel + 2.0 ** -22) + 2.0 ** -24 * 1.01 * np.where(
            np.isinf(m[:, tt]), 0.0, m[:, tt])
        fin = np.isfinite(m) & np.isin(heads, clean)[:, None]
        assert (np.abs(got[s][fin] - m[fin]) <= mt[fin] + 1e-38).all()
