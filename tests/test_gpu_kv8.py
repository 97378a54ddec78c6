"""The operators over the 8-bit cache against plain 64-bit implementations (GPU)."""
import numpy as np
import pytest
import torch

import oracle
from _gpu_util import bf16_normal, binding, cuda_or_skip, special_bf16
from _kv8_util import (D, DTYPE, FORMATS, as_pool, attend8, bits, chunk_reference8, decode,
                       make_cache8, needed, put_block, random_codes, rotated, values)
from _longctx_util import HKV, HQ, P, check, normal, offsets, visible

pytestmark = pytest.mark.gpu

PAGE, SEQLEN, POSITION, OFFSETS, VALUE = 1, 2, 4, 16, 64
THETA = 500000.0


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def err_of(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def bf16(x, dev):
    return torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).to(dev)


def random_cache(rng, pages, fmt):
    return (random_codes(rng, (pages, 2, HKV, P, D), fmt),
            rng.integers(117, 124, (pages, 2, HKV)).astype(np.uint8))


def same(got, want, what):
    bad = np.argwhere(got != want)
    assert not len(bad), f"{what}: {len(bad)} differ, first at {tuple(bad[0])}: " \
                         f"{got[tuple(bad[0])]} not {want[tuple(bad[0])]}"


# ------------------------------------------------------------------- append --

def run_append(fmt, k, v, slots, positions, codes, scales, bt, *, separate=True, q=None):
    """Appends on the GPU and in the reference; returns the error bits."""
    dev, b = cuda_or_skip(), binding()
    pool, sc = as_pool(codes, fmt).to(dev), torch.from_numpy(scales).to(dev)
    err = err_of(dev)
    kw = {}
    if q is not None:
        kw = dict(q_in=bf16(q, dev), q_out=torch.empty((len(q), HQ, D), dtype=torch.bfloat16,
                                                      device=dev))
    b.kv8_append(bf16(k, dev), bf16(v, dev), pool, sc, i32(bt, dev), i32(positions, dev),
                 i32(slots, dev) if separate else None, rope_theta=THETA, dev_err=err, **kw)
    codes, scales = codes.copy(), scales.copy()
    for i, (s, p) in enumerate(zip(slots, positions)):
        if p < 0 or s < 0 or s >= bt.shape[1] * P or not 0 <= bt[i, s // P] < len(codes):
            continue
        page = bt[i, s // P]
        key = rotated(k[i:i + 1], [p], THETA)[0]
        for kv, x in enumerate((key, oracle.bf16_to_f64(v[i]))):
            x = np.where(np.isfinite(x), x, 0.0)
            for h in range(HKV):
                codes[page, kv, h], scales[page, kv, h] = put_block(
                    codes[page, kv, h], scales[page, kv, h], s % P, x[h:h + 1], fmt)
    same(bits(sc), scales, "scales")
    got = bits(pool)
    if fmt == "e4m3":                              # the sign of a zero code is free
        got, codes = np.where(got == 0x80, 0, got), np.where(codes == 0x80, 0, codes)
    same(got, codes, "codes")
    if q is not None:
        # (a negative position has no rotation to compare with)
        want = np.stack([np.stack([oracle.rope_rotate(q[i, j], int(p), THETA)
                                   for j in range(HQ)]) for i, p in enumerate(positions)])
        same(bits(kw["q_out"]), want, "queries")
    return int(err.item())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch,far", [(1, 0), (3, 9000), (70, 0), (33, 1 << 20)])
def test_append(fmt, batch, far):
    rng = np.random.default_rng(batch)
    codes, scales = random_cache(rng, 3 * batch + 2, fmt)
    bt = rng.permutation(3 * batch).reshape(batch, 3).astype(np.int32)
    slots = rng.integers(0, 3 * P, batch)
    slots[0] = 0
    if batch > 2:
        slots[1], slots[2] = 15, 16
    positions = rng.integers(0, far, batch) if far else slots
    # magnitudes from far below the old scales to far above
    size = 2.0 ** rng.integers(-12, 8, (batch, HKV, 1)).astype(np.float32)
    k, v = (oracle_bits(rng.standard_normal((batch, HKV, D)).astype(np.float32) * size)
            for _ in range(2))
    assert run_append(fmt, k, v, slots, positions, codes, scales, bt, separate=bool(far),
                      q=bf16_normal(rng, (batch, HQ, D))) == 0


def oracle_bits(x):
    return torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_token_by_token(fmt):
    # a page filled slot by slot: every growth rounds the earlier tokens again
    dev, b = cuda_or_skip(), binding()
    rng = np.random.default_rng(4)
    codes, scales = random_cache(rng, 4, fmt)
    pool, sc = as_pool(codes, fmt).to(dev), torch.from_numpy(scales).to(dev)
    bt = np.array([[2, 0]], np.int32)
    for t in range(2 * P):
        k, v = (oracle_bits(rng.standard_normal((1, HKV, D)).astype(np.float32) *
                            2.0 ** rng.integers(-3, 4)) for _ in range(2))
        b.kv8_append(bf16(k, dev), bf16(v, dev), pool, sc, i32(bt, dev), i32([t], dev),
                     rope_theta=THETA)
        for kv, x in enumerate((rotated(k, [t], THETA)[0], oracle.bf16_to_f64(v[0]))):
            page = bt[0, t // P]
            for h in range(HKV):
                codes[page, kv, h], scales[page, kv, h] = put_block(
                    codes[page, kv, h], scales[page, kv, h], t % P, x[h:h + 1], fmt)
    same(bits(sc), scales, "scales")
    same(decode(bits(pool), fmt), decode(codes, fmt), "codes")


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_special_values(fmt):
    # zeros, subnormals, the largest magnitudes, and values that are not finite
    rng = np.random.default_rng(5)
    batch = 24
    codes, scales = random_cache(rng, batch, fmt)
    scales[:] = rng.choice([0, 1, 100, 240, 255], scales.shape)
    bt = np.arange(batch, dtype=np.int32)[:, None]
    k, v = special_bf16(rng, (batch, HKV, D)), special_bf16(rng, (batch, HKV, D))
    k[0], v[0] = 0, 0x8000
    v[1] = 0x7F7F                                    # the largest finite value
    v[2] = 1                                         # the smallest
    slots = rng.integers(0, P, batch)
    slots[:4] = [0, 3, 0, 7]
    assert run_append(fmt, k, v, slots, slots, codes, scales, bt) == VALUE


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_bad_places(fmt):
    rng = np.random.default_rng(6)
    codes, scales = random_cache(rng, 6, fmt)
    bt = np.array([[0, 1], [6, -1], [2, -7], [3, 4]], np.int32)
    k, v = bf16_normal(rng, (4, HKV, D)), bf16_normal(rng, (4, HKV, D))
    assert run_append(fmt, k, v, [20, 3, 17, 5], [20, 3, 17, 5], codes, scales, bt) == PAGE
    assert run_append(fmt, k, v, [32, -1, 3, 5], [3, 3, 3, -2], codes, scales, bt) == POSITION


def test_scale_edges():
    # the thresholds of the scale: largest magnitudes just at and past T 2^e
    for fmt in FORMATS:
        rng = np.random.default_rng(7)
        batch = 64
        codes, scales = random_cache(rng, batch, fmt)
        v = np.zeros((batch, HKV, D), np.uint16)
        v[:, :, 3] = rng.integers(0, 0x7F80, (batch, HKV)).astype(np.uint16) | 0x8000
        v[:, 0, 3] = (np.arange(batch) % 32 + 100 << 7) | (96 if fmt == "e4m3" else 126)
        v[:, 1, 3] = v[:, 0, 3] + 1
        bt = np.arange(batch, dtype=np.int32)[:, None]
        zero = np.zeros(batch, np.int64)
        assert run_append(fmt, np.zeros_like(v), v, zero, zero, codes, scales, bt) == 0
    assert needed(448.0, "e4m3") == 127 and needed(127.5, "int8") == 128


# -------------------------------------------------------------- write, read --

def run_write(fmt, counts, starts, codes, scales, bt, k, v, off=None):
    dev, b = cuda_or_skip(), binding()
    pool, sc = as_pool(codes, fmt).to(dev), torch.from_numpy(scales).to(dev)
    err = err_of(dev)
    good = np.concatenate([[0], np.cumsum(counts)])
    b.kv8_write_prefill(bf16(k, dev), bf16(v, dev), i32(good if off is None else off, dev),
                        i32(starts, dev), pool, sc, i32(bt, dev), rope_theta=THETA, dev_err=err)
    codes, scales = codes.copy(), scales.copy()
    for i, (n, f) in enumerate(zip(counts, starts)):
        lo, hi = max(f, 0), min(f + n, bt.shape[1] * P)
        for page0 in range(lo // P * P, hi, P):
            a, z = max(lo, page0), min(hi, page0 + P)
            page = bt[i, page0 // P]
            if not 0 <= page < len(codes):
                continue
            at = good[i] + a - f
            key = rotated(k[at:at + z - a], range(a, z), THETA)
            for kv, x in enumerate((key, oracle.bf16_to_f64(v[at:at + z - a]))):
                x = np.where(np.isfinite(x), x, 0.0)
                for h in range(HKV):
                    codes[page, kv, h], scales[page, kv, h] = put_block(
                        codes[page, kv, h], scales[page, kv, h], a - page0, x[:, h], fmt)
    same(bits(sc), scales, "scales")
    got = bits(pool)
    if fmt == "e4m3":
        got, codes = np.where(got == 0x80, 0, got), np.where(codes == 0x80, 0, codes)
    same(got, codes, "codes")
    return int(err.item())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,starts", [
    ([1], [0]), ([1], [31]), ([16], [16]), ([17], [15]), ([33, 0, 5], [0, 3, 14]),
    ([0, 0, 70, 2, 0], [0, 5, 9, 16, 7]), ([40] * 9, list(range(9))),
    ([1 + i % 5 for i in range(60)], [i % 40 for i in range(60)]), ([30], [2050]),
])
def test_write(fmt, counts, starts):
    rng = np.random.default_rng(sum(counts))
    width = max((f + n + P - 1) // P for n, f in zip(counts, starts))
    batch = len(counts)
    codes, scales = random_cache(rng, batch * width + 2, fmt)
    bt = rng.permutation(batch * width).reshape(batch, width).astype(np.int32)
    rows = sum(counts)
    size = 2.0 ** rng.integers(-8, 8, (rows, HKV, 1)).astype(np.float32)
    k, v = (oracle_bits(rng.standard_normal((rows, HKV, D)).astype(np.float32) * size)
            for _ in range(2))
    assert run_write(fmt, counts, starts, codes, scales, bt, k, v) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_special_values(fmt):
    rng = np.random.default_rng(8)
    codes, scales = random_cache(rng, 8, fmt)
    scales[:] = rng.choice([0, 1, 100, 240, 255], scales.shape)
    k, v = special_bf16(rng, (50, HKV, D)), special_bf16(rng, (50, HKV, D))
    bt = np.arange(8, dtype=np.int32).reshape(2, 4)
    assert run_write(fmt, [30, 20], [3, 17], codes, scales, bt, k, v) == VALUE


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_bad_places(fmt):
    rng = np.random.default_rng(9)
    codes, scales = random_cache(rng, 6, fmt)
    k, v = bf16_normal(rng, (40, HKV, D)), bf16_normal(rng, (40, HKV, D))
    bt = np.array([[0, 1], [2, 7], [3, -1]], np.int32)
    assert run_write(fmt, [10, 20, 10], [3, 5, 15], codes, scales, bt, k, v) == PAGE
    bt = np.array([[0, 1], [2, 4], [3, 5]], np.int32)
    assert run_write(fmt, [10, 20, 10], [-4, 20, 31], codes, scales, bt, k, v) == POSITION


def test_write_bad_offsets():
    # a sequence with bad offsets is skipped, the others are written
    rng = np.random.default_rng(10)
    codes, scales = random_cache(rng, 6, "int8")
    k, v = bf16_normal(rng, (40, HKV, D)), bf16_normal(rng, (40, HKV, D))
    bt = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    dev, b = cuda_or_skip(), binding()
    for off in ([0, 10, 5, 40], [3, 10, 20, 40], [0, 10, 20, 39], [-1, 10, 20, 40],
                [0, 10, 20, 41]):
        pool, sc = as_pool(codes, "int8").to(dev), torch.from_numpy(scales).to(dev)
        err = err_of(dev)
        b.kv8_write_prefill(bf16(k, dev), bf16(v, dev), i32(off, dev), i32([0, 0, 0], dev), pool,
                            sc, i32(bt, dev), dev_err=err)
        assert int(err.item()) & OFFSETS, off


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,starts", [
    ([1], [0]), ([5], [14]), ([100, 0, 3, 64], [0, 7, 15, 33]), ([20] * 40, list(range(40))),
])
def test_read(fmt, counts, starts):
    dev, b = cuda_or_skip(), binding()
    lens = [n + f for n, f in zip(counts, starts)]
    codes, scales, bt = make_cache8(lens, fmt, seed=sum(counts), scales=(3, 240))
    vals = values(codes, scales, fmt)
    rows = sum(counts)
    out = [torch.full((rows, HKV, D), 9.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    err = err_of(dev)
    got = b.kv8_read(offsets(counts).to(dev), i32(starts, dev), as_pool(codes, fmt).to(dev),
                     torch.from_numpy(scales).to(dev), i32(bt, dev), *out, dev_err=err)
    assert int(err.item()) == 0 and got[0] is out[0] and got[1] is out[1]
    r = 0
    for i, (n, f) in enumerate(zip(counts, starts)):
        for t in range(f, f + n):
            for kv in range(2):
                # every value is a bf16 number
                same(got[kv][r].double().cpu().numpy(), vals[bt[i, t // P], kv, :, t % P],
                     f"sequence {i} token {t}")
            r += 1


def test_read_leaves_other_rows():
    dev, b = cuda_or_skip(), binding()
    codes, scales, bt = make_cache8([40, 40], "e4m3")
    bt[1, 1] = len(codes)
    pool, sc = as_pool(codes, "e4m3").to(dev), torch.from_numpy(scales).to(dev)
    out = [torch.full((60, HKV, D), 9.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    err = err_of(dev)
    b.kv8_read(i32([0, 20, 50], dev), i32([-5, 10], dev), pool, sc, i32(bt, dev), *out,
               dev_err=err)
    assert int(err.item()) == PAGE | POSITION | OFFSETS
    vals = values(codes, scales, "e4m3")
    want = np.full((60, HKV, D), 9.0)
    for r, (i, t) in enumerate([(0, t) for t in range(-5, 15)] + [(1, t) for t in range(10, 40)]):
        if t >= 0 and 0 <= bt[i, t // P] < len(codes):
            want[r] = vals[bt[i, t // P], 1, :, t % P]
    same(out[1].double().cpu().numpy(), want, "rows")


# ------------------------------------------------------------------- decode --

def run_decode(fmt, lens, window=0, sinks=0, splits=0, cache=None, seed=1, scale=None, q_scale=1.0,
               bad=()):
    dev, b = cuda_or_skip(), binding()
    codes, sc, bt = cache or make_cache8(lens, fmt, seed=seed)
    for i, p, page in bad:
        bt[i, p] = page
    q = normal((len(lens), HQ, D), seed + 1) * q_scale
    err = err_of(dev)
    out = b.paged8_decode_attention(q.to(dev), as_pool(codes, fmt).to(dev),
                                    torch.from_numpy(sc).to(dev), i32(bt, dev), i32(lens, dev),
                                    window=window, sinks=sinks, num_splits=splits, scale=scale,
                                    dev_err=err)
    vals = values(codes, sc, fmt)
    kw = {} if scale is None else {"scale": scale}
    both = [attend8(q[i], vals, bt[i], visible(min(max(n, 0), bt.shape[1] * P) - 1, window, sinks),
                    16, **kw) for i, n in enumerate(lens)]
    check(out, np.stack([x[0] for x in both]), np.stack([x[1] for x in both]),
          f"{fmt} {lens} window {window} sinks {sinks} splits {splits}")
    return int(err.item())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [0, 1, 3, 7])
@pytest.mark.parametrize("lens", [[1], [0, 3], [16], [17], [500, 1, 33, 129, 0], [1300],
                                  [40 + 7 * i for i in range(50)]])
def test_decode(fmt, lens, splits):
    assert run_decode(fmt, lens, splits=splits) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 3), (100, 200), (128, 16),
                                          (130, 0), (64, 129), (2 ** 31 - 1, 5), (700, 4)])
def test_decode_window(fmt, window, sinks, splits):
    assert run_decode(fmt, [700, 90, 33, 1], window, sinks, splits=splits) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_bad_pages_and_lengths(fmt):
    assert run_decode(fmt, [100, 40, 7], bad=[(0, 2, -1), (1, 0, 10 ** 9), (2, 0, -5)]) == PAGE
    codes, sc, bt = make_cache8([64, 64], fmt)
    assert run_decode(fmt, [65, -3], cache=(codes, sc, bt)) == SEQLEN


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [1, 4])
def test_decode_scales_of_any_size(fmt, splits):
    # blocks whose V scales lie 2^40 apart, queries 2^-30 .. 2^30, flat weights
    lens = [700, 33]
    codes, sc, bt = make_cache8(lens, fmt, seed=3)
    rng = np.random.default_rng(3)
    sc[:, 1] = rng.integers(100, 141, sc[:, 1].shape)
    run_decode(fmt, lens, splits=splits, cache=(codes, sc, bt))
    for up in (-30, 30):
        sc2 = sc.copy()
        sc2[:, 0] = np.clip(sc2[:, 0].astype(int) - up, 3, 240)
        run_decode(fmt, lens, splits=splits, cache=(codes, sc2, bt), q_scale=2.0 ** up)
    run_decode(fmt, lens, splits=splits, scale=2.0 ** -20)
    run_decode(fmt, lens, splits=splits, scale=3.0)


# ------------------------------------------------------------------- chunks --

def run_chunk(fmt, lens, counts, window=0, sinks=0, splits=0, seed=1, pad=2, cache=None, bad=(),
              scale=None):
    dev, b = cuda_or_skip(), binding()
    codes, sc, bt = cache or make_cache8(lens, fmt, seed=seed)
    for i, p, page in bad:
        bt[i, p] = page
    off = offsets(counts)
    rows = int(off[-1]) + pad
    q = normal((rows, HQ, D), seed + 1)
    out0 = torch.full((rows, HQ, D), 7.0, dtype=torch.bfloat16)
    out, err = out0.to(dev), err_of(dev)
    b.paged8_chunk_attention(q.to(dev), off.to(dev), as_pool(codes, fmt).to(dev),
                             torch.from_numpy(sc).to(dev), i32(bt, dev), i32(lens, dev), out,
                             window=window, sinks=sinks, num_splits=splits, scale=scale,
                             dev_err=err)
    want, tol = chunk_reference8(q, off, values(codes, sc, fmt), bt, lens, window, sinks, out0,
                                 **({} if scale is None else {"scale": scale}))
    check(out, want, tol, f"{fmt} {lens} {counts} window {window} sinks {sinks} splits {splits}")
    return int(err.item())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("lens,counts", [
    ([1], [1]), ([17], [17]), ([16], [1]), ([129], [128]), ([515], [5]), ([300], [300]),
    ([40, 3, 131], [5, 3, 1]), ([33, 7, 64, 5], [0, 7, 0, 1]), ([700, 64, 200], [130, 64, 33]),
    ([1100], [1]), ([257, 256, 255, 1], [9, 65, 31, 1]), ([4], [4]), ([5], [5]),
    ([500, 499, 17, 1300], [2, 3, 4, 1]),
])
def test_chunk_causal(fmt, lens, counts, splits):
    assert run_chunk(fmt, lens, counts, splits=splits) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("window,sinks", [
    (1, 0), (1, 1), (16, 3), (100, 200), (128, 16), (130, 0), (64, 129), (2 ** 31 - 1, 5),
    (700, 4),
])
def test_chunk_window(fmt, window, sinks, splits):
    assert run_chunk(fmt, [700, 90, 33], [140, 90, 2], window, sinks, splits=splits) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("lens,counts,window", [
    ([100] * 70, [2] * 70, 0), ([1 + i for i in range(64)], [1] * 64, 0),
    ([90 + 20 * i for i in range(40)], [1 + (i * 29) % 80 for i in range(40)], 0),
    ([200 + 7 * (i % 5) for i in range(45)], [(0, 1, 33, 64, 70)[i % 5] for i in range(45)], 60),
    ([8 + (i * 61) % 300 for i in range(90)], [1 + i % 4 if i % 9 else 5 for i in range(90)], 40),
])
def test_chunk_many(fmt, lens, counts, window, splits):
    assert run_chunk(fmt, lens, counts, window, 3 if window else 0, splits=splits) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_bad_inputs(fmt):
    # bad pages are skipped, chunks longer than their sequence start with zero rows
    assert run_chunk(fmt, [300, 40], [70, 4], bad=[(0, 3, -1), (1, 1, 10 ** 6)]) == PAGE
    codes, sc, bt = make_cache8([64, 64, 64], fmt)
    assert run_chunk(fmt, [3, 2, 64], [7, 4, 10], cache=(codes, sc, bt)) == POSITION
    codes, sc, bt = make_cache8([64, 64], fmt)
    assert run_chunk(fmt, [70, -1], [10, 3], cache=(codes, sc, bt)) == SEQLEN | POSITION


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[70, 5], [4, 2]])
def test_chunk_scales(fmt, counts):
    lens = [500, 90]
    codes, sc, bt = make_cache8(lens, fmt, seed=3)
    rng = np.random.default_rng(3)
    sc[:, 1] = rng.integers(100, 141, sc[:, 1].shape)
    run_chunk(fmt, lens, counts, cache=(codes, sc, bt))
    run_chunk(fmt, lens, counts, scale=2.0 ** -20)
    run_chunk(fmt, lens, counts, scale=3.0)
