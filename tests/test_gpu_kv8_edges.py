"""The 8-bit cache at the ends of its range: keys whose rotation overflows FP32 on the
way (GPU)."""
import numpy as np
import pytest
import torch

import oracle
from _gpu_util import binding, cuda_or_skip
from _kv8_util import D, FORMATS, as_pool, bits, decode, put_block, rotated
from _longctx_util import HKV, P
from test_gpu_kv8 import VALUE, bf16, err_of, i32, oracle_bits, random_cache, run_write, same

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- huge keys --

def keys_with_a_huge_pair(n, seed, at, dim, x1, x2):
    """N(0, 1) keys, one pair of token `at` and kv head 3 apart: dims dim and dim + 32."""
    rng = np.random.default_rng(seed)
    k, v = (rng.standard_normal((n, HKV, D)).astype(np.float32) for _ in range(2))
    k[at, 3, dim], k[at, 3, dim + 32] = x1, x2
    return oracle_bits(k), oracle_bits(v)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [0, 13, 31])
@pytest.mark.parametrize("start,n,at", [(0, 1, 0), (0, 20, 0), (5, 20, 9), (16, 16, 15),
                                        (2040, 20, 3), (40960, 17, 16)])
def test_write_of_a_huge_pair(fmt, dim, start, n, at):
    """|a| + |b| past FP32, the rotated pair within bf16: cached with the largest scale,
    and no error."""
    for x1, x2 in ((2e38, 2e38), (-2e38, 2e38), (2e38, -1.9e38), (1.6e38, 2.4e38)):
        k, v = keys_with_a_huge_pair(n, start + dim, at, dim, x1, x2)
        key = rotated(k, range(start, start + n), 500000.0)
        assert np.isfinite(key).all() and np.abs(key).max() > 2.0 ** 126
        width = (start + n + P - 1) // P
        codes, scales = random_cache(np.random.default_rng(dim), width + 2, fmt)
        bt = np.random.default_rng(1).permutation(width).astype(np.int32)[None]
        assert run_write(fmt, [n], [start], codes, scales, bt, k, v) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("position", [0, 7, 5000])
def test_append_and_write_of_a_huge_pair_agree(fmt, position):
    dev, b = cuda_or_skip(), binding()
    k, v = (bf16(x, dev) for x in keys_with_a_huge_pair(1, 4, 0, 20, 2e38, 2e38))
    width = position // P + 1
    bt, pos = i32([[0] * width], dev), i32([position], dev)
    rng = np.random.default_rng(position)
    codes, scales = random_cache(rng, 1, fmt)
    results = []
    for write in (False, True):
        pool, sc, err = as_pool(codes, fmt).to(dev), torch.from_numpy(scales).to(dev), err_of(dev)
        if write:
            b.kv8_write_prefill(k, v, i32([0, 1], dev), pos, pool, sc, bt, dev_err=err)
        else:
            b.kv8_append(k, v, pool, sc, bt, pos, dev_err=err)
        assert int(err.item()) == 0
        results.append((decode(bits(pool), fmt), bits(sc)))
    same(results[0][0], results[1][0], "values")
    same(results[0][1], results[1][1], "scales")


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_of_a_pair_that_overflows(fmt):
    """3e38 each, turned until a value passes bf16: that one is zero and reported, the
    pair's other one and the block's other keys are as they should be."""
    n = 16
    k, v = keys_with_a_huge_pair(n, 6, 1, 0, 3e38, 3e38)       # one radian: -9e37 and 4.1e38
    key = rotated(k, range(n), 500000.0)
    assert np.isinf(key).sum() == 1
    codes, scales = random_cache(np.random.default_rng(2), 3, fmt)
    assert run_write(fmt, [n], [0], codes, scales, np.array([[1]], np.int32), k, v) == VALUE
