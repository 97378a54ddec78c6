"""Appends with more rope_theta values than the library keeps tables for, near
and far, in every order of the first calls (GPU): the stored bits are those of
the FP64 rotation.  (Run after the tests that build tables: it fills them all.)"""
import numpy as np
import pytest
import torch

import oracle
from _gpu_util import binding, cuda_or_skip
from _longctx_util import HKV, HQ, P, make_cache, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [1, 40])
def test_many_thetas(batch):
    dev, b = cuda_or_skip(), binding()
    lens = [1 + (i * 37) % 90 for i in range(batch)]
    pool, bt = make_cache(lens, seed=121)
    slots = torch.tensor(lens, dtype=torch.int32) - 1
    k, q = normal((batch, HKV, 64), 122), normal((batch, HQ, 64), 123)
    ki, qi = (x.view(torch.int16).numpy().view(np.uint16) for x in (k, q))
    rng = np.random.default_rng(124)
    for i, theta in enumerate((500000.0, 1e4, 2.0, 1e6, 77.5, 1234.5, 500000.0, 9e8)):
        pos = rng.integers(0, 2000 if i % 2 else 2 ** 22, batch).astype(np.int32)
        gp, qo = pool.to(dev), torch.zeros_like(q).to(dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        b.kv_append_at(k.to(dev), k.to(dev), gp, bt.to(dev), torch.from_numpy(pos).to(dev),
                       slots.to(dev), rope_theta=theta, q_in=q.to(dev), q_out=qo, dev_err=err)
        assert int(err.item()) == 0
        got, qg = gp.cpu().view(torch.int16).numpy().view(np.uint16), qo.cpu().view(torch.int16)
        for s in range(0, batch, 3):
            pid, at = int(bt[s, int(slots[s]) // P]), int(slots[s]) % P
            for h in range(HKV):
                assert np.array_equal(got[pid, 0, at, h],
                                      oracle.rope_rotate(ki[s, h], int(pos[s]), theta))
            for j in range(0, HQ, 9):
                assert np.array_equal(qg[s, j].numpy().view(np.uint16),
                                      oracle.rope_rotate(qi[s, j], int(pos[s]), theta))
