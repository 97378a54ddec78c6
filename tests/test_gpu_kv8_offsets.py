"""Prompt writes into the 8-bit cache and reads from it with offsets that do not fall but
are bad at their ends: the sequences whose own offsets are good are written and read, the
others' pages and rows stay (GPU)."""
import numpy as np
import pytest
import torch

import oracle
from _gpu_util import binding, cuda_or_skip
from _kv8_util import D, FORMATS, as_pool, bits, decode, put_block, rotated, values
from _longctx_util import HKV, P
from test_gpu_kv8 import OFFSETS, bf16, err_of, i32, oracle_bits, random_cache, same

pytestmark = pytest.mark.gpu

ROWS, WIDTH, THETA = 70, 6, 1e4
OFF = [[3, 10, 20, 70], [0, 10, 20, 39], [-1, 10, 20, 70], [0, 10, 20, 71], [-40, -3, 33, 70],
       [0, 33, 71, 90], [0, 64, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 0, 17, 70], [5, 5, 5, 5],
       [0, 0, 50, 50], [40, 50, 60, 69]]


def good(off):
    """The sequences, with their rows, whose offsets lie within the rows."""
    return [(i, a, z) for i, (a, z) in enumerate(zip(off, off[1:])) if 0 <= a < z <= ROWS]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("starts", [[0, 0, 0], [5, 16, 23]], ids=str)
@pytest.mark.parametrize("off", OFF, ids=str)
def test_write_and_read_of_the_good_sequences(fmt, starts, off):
    dev, b = cuda_or_skip(), binding()
    rng = np.random.default_rng(11)
    k, v = (oracle_bits(rng.standard_normal((ROWS, HKV, D)).astype(np.float32)) for _ in range(2))
    codes, scales = random_cache(rng, 3 * WIDTH + 2, fmt)
    bt = rng.permutation(3 * WIDTH).reshape(3, WIDTH).astype(np.int32)
    pool, sc, err = as_pool(codes, fmt).to(dev), torch.from_numpy(scales).to(dev), err_of(dev)
    where = (i32(off, dev), i32(starts, dev))
    b.kv8_write_prefill(bf16(k, dev), bf16(v, dev), *where, pool, sc, i32(bt, dev),
                        rope_theta=THETA, dev_err=err)
    assert int(err.item()) == OFFSETS
    for i, a, z in good(off):
        f, n = starts[i], z - a
        both = rotated(k[a:z], range(f, f + n), THETA), oracle.bf16_to_f64(v[a:z])
        for page0 in range(f // P * P, f + n, P):
            lo, hi = max(f, page0), min(f + n, page0 + P)
            page = bt[i, page0 // P]
            for kv, x in enumerate(both):
                for h in range(HKV):
                    codes[page, kv, h], scales[page, kv, h] = put_block(
                        codes[page, kv, h], scales[page, kv, h], lo - page0,
                        x[lo - f:hi - f, h], fmt)
    same(bits(sc), scales, "scales")
    same(decode(bits(pool), fmt), decode(codes, fmt), "codes")

    want, vals = np.full((2, ROWS, HKV, D), 9.0), values(codes, scales, fmt)
    for i, a, z in good(off):
        for t in range(z - a):
            at = starts[i] + t
            want[:, a + t] = vals[bt[i, at // P], :, :, at % P]
    out = [torch.full((ROWS, HKV, D), 9.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    err = err_of(dev)
    b.kv8_read(*where, pool, sc, i32(bt, dev), *out, dev_err=err)
    assert int(err.item()) == OFFSETS
    for kv in range(2):
        same(out[kv].double().cpu().numpy(), want[kv], "rows")
