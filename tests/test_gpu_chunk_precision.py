"""Chunks of up to four tokens weigh V with 16 significant bits, as the
one-token calls do: results near zero that large values cancel to (GPU)."""
import numpy as np
import pytest
import torch

from _gpu_util import binding, cuda_or_skip
from _longctx_util import G, HQ, P, attend, check, make_cache, normal, offsets, rows_of

pytestmark = pytest.mark.gpu


def sharp(q, pool, bt_row, tokens):
    """attend's result and its tolerance with weights off by 2^-16: the first
    term is off by half a step, 2^-8 of the weight, the second, of what the
    first leaves (exact in FP32), by 2^-8 of that."""
    out, _, (t, w), rel = attend(q, pool, bt_row, tokens)
    _, v, _ = rows_of(pool, bt_row, tokens)
    a = np.einsum("tj,tjd->jd", w, np.abs(np.repeat(v, G, 1)))
    tol = 2.0 ** -8 * np.abs(out) + a * (2.0 ** -16 + rel + len(t) * 2.0 ** -23)
    return out, tol * (1 + 2.0 ** -7) + 2.0 ** -126


@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("beside", [0, 70])
@pytest.mark.parametrize("counts,lens", [([1, 1, 1], [2, 17, 40]), ([4, 2, 3], [4, 20, 33]),
                                         ([1, 3], [300, 129])])
def test_cancelling_values(counts, lens, beside, splits):
    dev, b = cuda_or_skip(), binding()
    counts, lens = counts + [beside] * (beside > 0), lens + [beside + 9] * (beside > 0)
    pool, bt = make_cache(lens, seed=111)
    for s, n in enumerate(lens):          # values of alternating sign around 64
        for t in range(n):
            pool[int(bt[s, t // P]), 1, t % P] += 64.0 * (-1) ** t
    off = offsets(counts)
    q = normal((int(off[-1]), HQ, 64), 112) * 0.25
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    out = b.paged_chunk_attention(q.to(dev), off.to(dev), pool.to(dev), bt.to(dev), ln,
                                  num_splits=splits).cpu()
    last = []
    for s, n in enumerate(counts):
        for i in range(n if n <= 4 else 0):
            r = int(off[s]) + i
            want, tol = sharp(q[r], pool, bt[s], np.arange(lens[s] - n + i + 1))
            check(out[r], want, tol, f"row {i} of sequence {s}")
        last.append(int(off[s + 1]) - 1)
    # the newest tokens by the one-token calls, within the same tolerance
    for call in (lambda x: b.paged_decode_attention(x, pool.to(dev), bt.to(dev), ln),
                 lambda x: b.paged_window_attention(x, pool.to(dev), bt.to(dev), ln, 2 ** 20)):
        one = call(q[last].to(dev)).cpu()
        for s, n in enumerate(lens):
            want, tol = sharp(q[last[s]], pool, bt[s], np.arange(n))
            check(one[s], want, tol, f"sequence {s} by a one-token call")
