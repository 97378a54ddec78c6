"""Calls with long chunks and many single tokens, one right after the other on
a stream: the two kernels of a call run beside each other, and what follows
sees both (GPU)."""
import pytest
import torch

from _gpu_util import binding, cuda_or_skip
from _longctx_util import HQ, make_cache, normal, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("long_chunks,singles,cached", [
    ([200], 60, 300), ([5], 250, 200), ([700, 64], 150, 250), ([2000], 3, 100), ([6] * 20, 200, 90),
])
def test_a_chain_of_calls(long_chunks, singles, cached):
    """Each call's queries are the rows that the last one wrote, over one
    workspace: the same bits whether or not each call is waited for."""
    dev, b = cuda_or_skip(), binding()
    counts = long_chunks + [1] * singles
    lens = [n + 50 for n in long_chunks] + [cached + i % 40 for i in range(singles)]
    pool, bt = (x.to(dev) for x in make_cache(lens, seed=91))
    off = offsets(counts).to(dev)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    q = normal((sum(counts), HQ, 64), 92).to(dev)
    for splits in (0, 2):
        ws = torch.empty(max(16, b.chunk_workspace_bytes(q.shape[0], len(lens), bt.shape[1],
                                                         splits)), dtype=torch.uint8, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)

        def chain(wait):
            rows = [q] + [torch.zeros_like(q) for _ in range(6)]
            for i in range(6):
                b.paged_chunk_attention(rows[i], off, pool, bt, ln, rows[i + 1], workspace=ws,
                                        num_splits=splits, dev_err=err)
                if wait:
                    torch.cuda.synchronize()
            return rows[1:]

        want = chain(True)
        assert torch.isfinite(want[-1]).all() and want[-1].any()
        for _ in range(8):
            for x, y in zip(chain(False), want):
                assert torch.equal(x, y)
        assert int(err.item()) == 0
