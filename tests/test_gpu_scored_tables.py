"""Scored attention around the width of table where the scores move from
shared memory to the workspace: the limit leaves room for two CTAs an SM, and
the place makes no difference to the bits (GPU)."""
import numpy as np
import pytest
import torch

from _gpu_util import binding, cuda_or_skip
from _longctx_util import G, HKV, HQ, P, attend, check, make_cache, normal

LIMIT = 191        # pages: (228 KiB / 2 - 1 KiB - rings of 64 KiB and their slack) / 256 bytes


def test_where_scores_are_kept():
    b = binding()
    assert b.scored_workspace_bytes(3, LIMIT, 1) == 0
    assert b.scored_workspace_bytes(3, LIMIT + 2, 1) == 3 * HKV * (LIMIT + 2) * P * G * 4


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[LIMIT * P, 17, 1], [2000, LIMIT * P - 3]])
def test_the_place_makes_no_difference(lens):
    dev, b = cuda_or_skip(), binding()
    pool, bt = make_cache(lens, width=LIMIT, seed=101)
    q = normal((len(lens), HQ, 64), 102)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    start = torch.from_numpy(np.random.default_rng(103).random(
        (len(lens), HKV, LIMIT * P)).astype(np.float32))
    results = []
    for width in (LIMIT, LIMIT + 2, LIMIT + 70):
        t = torch.full((len(lens), width), -1, dtype=torch.int32)
        t[:, :LIMIT] = bt
        mass = torch.zeros((len(lens), HKV, width * P))
        mass[..., :LIMIT * P] = start
        got = mass.to(dev)
        out = b.paged_scored_attention(q.to(dev), pool.to(dev), t.to(dev), ln, got, num_splits=1)
        assert not got[..., LIMIT * P:].any()
        results.append((out.cpu(), got[..., :LIMIT * P].cpu()))
    for out, got in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(got, results[0][1])
    ref = [attend(q[i], pool, bt[i], np.arange(n)) for i, n in enumerate(lens)]
    check(results[0][0], np.stack([r[0] for r in ref]), np.stack([r[1] for r in ref]), "out")
