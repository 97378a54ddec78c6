"""One sequence's few new tokens in a q of more rows than that (a q of a fixed
size, as a captured graph needs), over a long cache (GPU)."""
import pytest
import torch

from _gpu_util import binding, cuda_or_skip
from _longctx_util import HQ, check, chunk_reference, make_cache, normal, offsets

pytestmark = pytest.mark.gpu


def test_padding_takes_no_range_away():
    """The cache is read in ranges however many rows q has: with tables of 100
    pages a long chunk needs no partials, so the workspace is the ranges'."""
    cuda_or_skip()
    b = binding()
    assert b.chunk_workspace_bytes(4, 1, 100) > 0
    for rows in (5, 8, 64):
        assert b.chunk_workspace_bytes(rows, 1, 100) >= b.chunk_workspace_bytes(4, 1, 100)


@pytest.mark.parametrize("window,sinks", [(0, 0), (2000, 20)])
@pytest.mark.parametrize("rows", [5, 8, 70, 600])
@pytest.mark.parametrize("n", [1, 3, 4, 5])
def test_padded_sequence(n, rows, window, sinks):
    dev, b = cuda_or_skip(), binding()
    lens = [5003]
    pool, bt = make_cache(lens, seed=81)
    off = offsets([n])
    q = normal((rows, HQ, 64), 82)
    q[n:] = float("nan")
    kept = torch.full((rows, HQ, 64), 3.0, dtype=torch.bfloat16)
    out, err = kept.to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    b.paged_chunk_attention(q.to(dev), off.to(dev), pool.to(dev), bt.to(dev),
                            torch.tensor(lens, dtype=torch.int32, device=dev), out,
                            window=window, sinks=sinks, dev_err=err)
    want, tol = chunk_reference(q, off, pool, bt, lens, window, sinks, kept)
    check(out, want, tol, f"{n} of {rows}")
    assert int(err.item()) == 0
