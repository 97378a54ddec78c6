"""8-bit caches and 64-bit references for the tests of the operators over them."""
import numpy as np
import torch

import oracle
from _longctx_util import G, HKV, HQ, P, SCALE, visible

D = 64
TOP = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FORMATS = ("e4m3", "int8")
BIAS, LEAST, MOST = 127, 3, 240


def _e4m3_values():
    """Values of the codes 0 .. 0x7E."""
    e, m = np.divmod(np.arange(127), 8)
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3 = _e4m3_values()


def decode(codes, fmt):
    """Codes (uint8 bits) as 64-bit values (e4m3's NaN codes as NaN)."""
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    a = codes & 0x7F
    v = np.where(a == 0x7F, np.nan, E4M3[np.minimum(a, 126)])
    return np.where(codes & 0x80, -v, v)


def encode(x, fmt):
    """Values (already divided by the scale) as codes: nearest, ties to even,
    saturating."""
    x = np.clip(x, -TOP[fmt], TOP[fmt])
    if fmt == "int8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    a = np.abs(x)
    hi = np.searchsorted(E4M3, a)                    # first code at or above
    lo = np.maximum(hi - 1, 0)
    below, above = a - E4M3[lo], E4M3[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def needed(top, fmt):
    """The smallest scale with top <= TOP 2^(scale - 127)."""
    for e in range(LEAST, MOST):
        if top <= TOP[fmt] * 2.0 ** (e - BIAS):
            return e
    return MOST


def put_block(codes, scale, s0, rows, fmt):
    """A block [16][64] and its scale after the call that writes `rows` [n][64]
    (64-bit, finite) from slot s0: (codes, scale)."""
    codes = codes.copy()
    e = needed(np.abs(rows).max(initial=0.0), fmt)
    if s0 > 0:
        old = int(np.clip(scale, LEAST, MOST))
        e = max(e, old)
        if e > old:
            codes[:s0] = encode(decode(codes[:s0], fmt) * 2.0 ** (old - e), fmt)
    codes[s0:s0 + len(rows)] = encode(rows * 2.0 ** (BIAS - e), fmt)
    return codes, e


def rotated(k_bits, positions, theta):
    """Keys [n][8][64] (uint16 bf16 bits) rotated for positions [n], rounded to
    bf16, in 64 bits."""
    out = np.stack([np.stack([oracle.rope_rotate(k_bits[i, h], int(p), theta)
                              for h in range(HKV)]) for i, p in enumerate(positions)]) \
        if len(positions) else np.zeros((0, HKV, D), np.uint16)
    return oracle.bf16_to_f64(out)


def as_pool(codes, fmt):
    return torch.from_numpy(codes.copy()).view(DTYPE[fmt])


def bits(t):
    """A tensor's 8- or 16-bit patterns."""
    t = t.cpu()
    return (t.view(torch.uint8).numpy() if t.element_size() == 1 else
            t.view(torch.int16).numpy().view(np.uint16))


def random_codes(rng, shape, fmt, spread=40.0):
    return encode(rng.standard_normal(shape) * spread, fmt)


def make_cache8(lens, fmt, *, width=None, seed=0, spare=3, scales=(119, 122)):
    """(codes uint8 [pages][2][8][16][64], scales, tables): shuffled pages whose
    values are about N(0, 1/4); spare pages and the slots past each sequence's
    end hold e4m3's NaN code and scale 255."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // P) for n in lens]
    width = width or max(max(need, default=1), 1)
    pages = sum(need) + spare
    ids = rng.permutation(pages)
    bt = np.full((len(lens), width), -1, np.int32)
    codes = random_codes(rng, (pages, 2, HKV, P, D), fmt)
    sc = rng.integers(scales[0], scales[1] + 1, (pages, 2, HKV)).astype(np.uint8)
    at = 0
    used = np.zeros(pages, bool)
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
        used[bt[b, :n]] = True
        if lens[b] % P:
            codes[bt[b, n - 1], :, :, int(lens[b]) % P:] = 0x7F
    codes[~used] = 0x7F
    sc[~used] = 255
    return codes, sc, bt


def values(codes, scales, fmt):
    """What a pool stands for, in 64 bits."""
    s = np.clip(scales.astype(np.int64), LEAST, MOST)
    return decode(codes, fmt) * 2.0 ** (s - BIAS)[..., None, None]


def attend8(q, vals, bt_row, tokens, weight_bits, scale=SCALE):
    """One query [32][64] over tokens of a cache given as values: (out,
    tolerance), both [32][64].

    Tolerance, elementwise, with A = sum w |v| and T tokens:
      * a score is an FP32 sum of 64 products, exact but for q's f16 or bf16 form
        (exact too, or 2^-40 of the row's largest): off by at most 64 * 2^-23 *
        sum |q k| however it is summed, and 2^-22 of itself for the factors put
        on it; times scale it changes a weight by e^d; 2^x and its FP32 argument
        add 2^-21; the row sum is off by T * 2^-24 relative: all of it twice.
      * weights enter the product with V with `weight_bits` significant bits, as
        f16 numbers 2^(s - m + 7), m at most the row's largest score: the largest
        weight is 2^7 or more, and the two terms leave at most half of f16's
        smallest step, 2^-25: 2^-32 of the largest weight for each token.
      * the FP32 sums of T products: T * 2^-23 A.
      * the result rounded to bf16: 2^-8 |out|.
    """
    t = np.asarray(tokens, np.int64)
    pid = np.asarray(bt_row)[t // P]
    ok = (pid >= 0) & (pid < len(vals))
    t, pid = t[ok], pid[ok]
    if len(t) == 0:
        return np.zeros((HQ, D)), np.zeros((HQ, D))
    k, v = vals[pid, 0, :, t % P], vals[pid, 1, :, t % P]          # [T][8][64]
    q = q.double().numpy()
    kk, vv = np.repeat(k, G, 1), np.repeat(v, G, 1)
    s = np.einsum("jd,tjd->tj", q, kk) * scale
    big = scale * np.einsum("jd,tjd->tj", np.abs(q), np.abs(kk)).max(initial=0.0)
    d = (64 * 2.0 ** -23 + 2.0 ** -22) * big
    w = np.exp(s - s.max(0))
    w /= w.sum(0)
    out = np.einsum("tj,tjd->jd", w, vv)
    a = np.einsum("tj,tjd->jd", w, np.abs(vv))
    rel = 2 * (np.expm1(d) + 2.0 ** -21 + len(t) * 2.0 ** -24)
    tol = 2.0 ** -8 * np.abs(out) + a * (2.0 ** -weight_bits + rel + len(t) * 2.0 ** -23)
    tol += 2.0 ** -32 * w.max(0)[:, None] * np.abs(vv).sum(0)
    return out, tol * (1 + 2.0 ** -7) + 2.0 ** -126


def chunk_reference8(q, off, vals, bt, lens, window, sinks, out, scale=SCALE, short=16):
    """Every row's result and tolerance; rows of no token keep `out`'s.  Chunks
    of at most 4 tokens weigh V with `short` significant bits or more, longer
    ones with 8."""
    want = out.double().numpy().copy()
    tol = np.zeros_like(want)
    for b in range(len(lens)):
        n = int(off[b + 1]) - int(off[b])
        for i in range(n):
            pos = min(max(int(lens[b]), 0), bt.shape[1] * P) - n + i
            r = int(off[b]) + i
            toks = visible(pos, window, sinks) if pos >= 0 else np.zeros(0, np.int64)
            want[r], tol[r] = attend8(q[r], vals, bt[b], toks, short if n <= 4 else 8, scale)
    return want, tol
