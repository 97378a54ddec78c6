"""The 8-bit cache at the ends of its range: keys whose rotation overflows FP32 on the
way, values near the largest that it holds (GPU)."""
import numpy as np
import pytest
import torch

import oracle
from _gpu_util import binding, cuda_or_skip
from _kv8_util import (D, FORMATS, as_pool, bits, decode, make_cache8, put_block, random_codes,
                       rotated)
from _longctx_util import HKV, P
from test_gpu_kv8 import (VALUE, bf16, err_of, i32, oracle_bits, random_cache, run_chunk,
                          run_decode, run_write, same)
from test_gpu_kv8_use import wide

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


# --------------------------------------------------------------- huge values --

SCALES = {                                   # of V's blocks, page by page of a sequence
    "largest": lambda rng, n: np.full((n, HKV), 240),
    "rising": lambda rng, n: np.linspace(60, 240, n).astype(int)[:, None].repeat(HKV, 1),
    "falling": lambda rng, n: np.linspace(240, 3, n).astype(int)[:, None].repeat(HKV, 1),
    "any": lambda rng, n: rng.integers(3, 241, (n, HKV)),
}


def huge_cache(lens, fmt, kind, width=None):
    """A cache whose V reaches the largest magnitudes that the format and scales do."""
    rng = np.random.default_rng(len(lens))
    codes, sc, bt = make_cache8(lens, fmt, seed=len(lens), width=width)
    for b, n in enumerate(lens):
        pages = bt[b, :-(-n // P)]
        sc[pages, 1] = SCALES[kind](rng, len(pages))
        v = random_codes(rng, (len(pages), HKV, P, D), fmt, spread=200.0)
        hidden = np.arange(len(pages) * P).reshape(-1, P) >= n
        codes[pages, 1] = np.where(hidden[:, None, :, None], codes[pages, 1], v)
    return codes, sc, bt


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(SCALES))
@pytest.mark.parametrize("splits", [0, 1, 3, 20])
@pytest.mark.parametrize("lens", [[1], [2, 700, 0, 33], [300, 1300]], ids=str)
def test_values_of_any_magnitude(fmt, kind, splits, lens):
    assert run_decode(fmt, lens, splits=splits, cache=huge_cache(lens, fmt, kind)) == 0
    assert run_decode(fmt, lens, 150, 20, splits, cache=huge_cache(lens, fmt, kind)) == 0
    for n in (1, 2, 4):
        counts = [min(x, n) for x in lens]
        assert run_chunk(fmt, lens, counts, splits=splits, pad=0,
                         cache=huge_cache(lens, fmt, kind)) == 0
        assert run_chunk(fmt, lens, counts, 150, 20, splits=splits, pad=0,
                         cache=huge_cache(lens, fmt, kind)) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", list(SCALES))
def test_shared_values_of_any_magnitude(fmt, kind):
    cuda_or_skip()
    lens = [3000, 17, 0, 256, 900] * 3
    cache = huge_cache(lens, fmt, kind, width=wide(len(lens)))
    assert run_decode(fmt, lens, cache=cache) == 0
    counts = [min(n, 1 + i % 4) for i, n in enumerate(lens)]
    assert run_chunk(fmt, lens, counts, pad=0, cache=cache) == 0


@pytest.mark.parametrize("fmt,scale", [("e4m3", 225), ("int8", 227)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_longer_chunks_up_to_their_largest_values(fmt, scale, splits):
    """2^118 / 1300 is 2^107.7: codes of 448 with the scale 2^98, of 127 with 2^100."""
    lens = [1300, 90]
    codes, sc, bt = huge_cache(lens, fmt, "largest")
    sc[:, 1] = np.minimum(sc[:, 1], scale)
    for counts in ([40, 5], [300, 90], [5, 4]):
        assert run_chunk(fmt, lens, counts, splits=splits, cache=(codes, sc, bt)) == 0
