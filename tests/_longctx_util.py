"""Caches and 64-bit references for the tests of the long-context operators."""
import numpy as np
import torch

HQ, HKV, G, D, P = 32, 8, 4, 64, 16
SCALE = D ** -0.5


def make_cache(lens, *, width=None, seed=0, spare=3, scale=1.0):
    """(pool, tables): bf16 pool with shuffled pages, its spare pages and the
    slots past each sequence's end filled with NaN, tables -1 past the end."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // P) for n in lens]
    width = width or max(max(need, default=1), 1)
    pages = sum(need) + spare
    ids = rng.permutation(pages)
    bt = np.full((len(lens), width), -1, np.int32)
    pool = torch.from_numpy(rng.standard_normal((pages, 2, P, HKV, D)).astype(np.float32) *
                            scale).to(torch.bfloat16)
    at = 0
    used = np.zeros(pages, bool)
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
        used[bt[b, :n]] = True
        if lens[b] % P:
            pool[int(bt[b, n - 1]), :, int(lens[b]) % P:] = float("nan")
    pool[torch.from_numpy(~used)] = float("nan")
    return pool, torch.from_numpy(bt)


def rows_of(pool, bt_row, tokens):
    """K and V [T][8][64] in 64 bits; tokens on bad pages are dropped."""
    t = np.asarray(tokens, np.int64)
    pid = np.asarray(bt_row)[t // P]
    ok = (pid >= 0) & (pid < pool.shape[0])
    t, pid = t[ok], pid[ok]
    r = pool[torch.from_numpy(pid.astype(np.int64)), :, torch.from_numpy(t % P)].double().numpy()
    return r[:, 0], r[:, 1], t


def visible(pos, window, sinks):
    t = np.arange(pos + 1)
    return t if not window else t[(t > pos - window) | (t < sinks)]


def attend(q, pool, bt_row, tokens, scale=SCALE):
    """One query [32][64]: (out [32][64], tolerance [32][64], weights
    {token: [32]} as (tokens, [T][32]), relative weight error).

    Tolerance, elementwise, with A = sum w |v| and T tokens:
      * a score is an FP32 sum of 64 exact products: off by at most 64 * 2^-23
        * sum |q k| however it is summed (truncation included); times scale
        it changes a weight by the factor e^d, d at most that; 2^x on the
        special-function unit and the FP32 argument add 2^-21 (|x| < 8: more
        is below every tolerance because the weight itself is below 2^-8 of
        the largest); the row sum is off by T * 2^-24 relative: all of it
        twice (numerator and denominator).
      * weights rounded to bf16 for the product with V: 2^-8 A.
      * the FP32 sum of T products: T * 2^-23 A.
      * the result rounded to bf16: 2^-8 |out|.
    """
    k, v, t = rows_of(pool, bt_row, tokens)
    q = q.double().numpy()
    if len(t) == 0:
        return np.zeros((HQ, D)), np.zeros((HQ, D)), (t, np.zeros((0, HQ))), 0.0
    kk, vv = np.repeat(k, G, 1), np.repeat(v, G, 1)               # [T][32][64]
    s = np.einsum("jd,tjd->tj", q, kk) * scale
    d = 64 * 2.0 ** -23 * scale * np.einsum("jd,tjd->tj", np.abs(q), np.abs(kk)).max(initial=0.0)
    w = np.exp(s - s.max(0))
    w /= w.sum(0)
    out = np.einsum("tj,tjd->jd", w, vv)
    a = np.einsum("tj,tjd->jd", w, np.abs(vv))
    rel = 2 * (np.expm1(d) + 2.0 ** -21 + len(t) * 2.0 ** -24)
    tol = 2.0 ** -8 * np.abs(out) + a * (2.0 ** -8 + rel + len(t) * 2.0 ** -23)
    return out, tol * (1 + 2.0 ** -7) + 2.0 ** -126, (t, w), rel


def check(got, want, tol, what=""):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) - tol, -1)), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance, worst at "
                             f"{i}: got {got[i]!r}, want {want[i]!r} within {tol[i]!r}")


def chunk_reference(q, off, pool, bt, lens, window, sinks, out, scale=SCALE):
    """Every row's result and tolerance; rows of no token keep `out`'s."""
    want = out.double().numpy().copy()
    tol = np.zeros_like(want)
    for b in range(len(lens)):
        n = int(off[b + 1]) - int(off[b])
        for i in range(n):
            pos = int(lens[b]) - n + i
            r = int(off[b]) + i
            toks = visible(pos, window, sinks) if pos >= 0 else np.zeros(0, np.int64)
            want[r], tol[r], _, _ = attend(q[r], pool, bt[b], toks, scale)
    return want, tol


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def normal(shape, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(
        np.float32)).to(torch.bfloat16)
