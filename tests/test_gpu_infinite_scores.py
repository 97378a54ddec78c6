"""Keys whose scores are -inf (a masked key that the model itself wrote: an
infinite component against a query of the other sign), on whole pages, on a
page's only token, on everything that one warp or one range sees, and on the
whole sequence (GPU).

Such a token has the weight 0 and leaves the row's other weights as they are;
a row whose scores are all -inf is zero.  Every attention call has to agree,
so each is compared with the 64-bit attention over the other tokens.
"""
import numpy as np
import pytest
import torch

from _gpu_util import binding, cuda_or_skip
from _longctx_util import G, HKV, HQ, P, attend, check, make_cache, normal, offsets, visible

pytestmark = pytest.mark.gpu

KINDS = ["none", "newest", "last page", "first page", "first pages", "every fourth page",
         "all but the newest", "all"]


def places(n, kind):
    t = np.arange(n)
    return t[{"none": t < 0, "newest": t == n - 1, "last page": t // P == (n - 1) // P,
              "first page": t < P, "first pages": t < min(128, n - n // 3),
              "every fourth page": t // P % 4 == 0, "all but the newest": t < n - 1,
              "all": t >= 0}[kind]]


def infinite_cache(lens, kinds, seed):
    """(pool, tables, the tokens of each sequence whose scores are -inf)."""
    pool, bt = make_cache(lens, seed=seed)
    where = []
    for b, n in enumerate(lens):
        t = places(n, kinds[b % len(kinds)])
        pool[bt[b, t // P].long(), 0, torch.from_numpy(t % P), :, 0] = float("-inf")
        where.append(t)
    return pool, bt, where


def queries(rows, seed):
    q = normal((rows, HQ, 64), seed)
    q[..., 0] = q[..., 0].abs() + 0.25      # against the infinite components
    return q


def reference(q, pool, bt, tokens, where):
    """(out, tolerance, (tokens, weights), weight error) of each row."""
    return [attend(q[i], pool, bt[i], np.setdiff1d(tokens[i], where[i]))
            for i in range(len(tokens))]


def check_rows(out, ref, what):
    check(out, np.stack([r[0] for r in ref]), np.stack([r[1] for r in ref]), what)


def on(dev, *tensors):
    return [t.to(dev) for t in tensors]


def lens_t(lens):
    return torch.tensor(lens, dtype=torch.int32)


ONE_BATCH = [17, 16, 100, 640, 1500, 33, 1, 700]


def one_batch(kind, seed=3):
    pool, bt, where = infinite_cache(ONE_BATCH, [kind], seed)
    return queries(len(ONE_BATCH), seed + 1), pool, bt, where


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("kind", KINDS)
def test_window(kind, splits):
    dev, b = cuda_or_skip(), binding()
    q, pool, bt, where = one_batch(kind)
    for window, sinks in ((2 ** 31 - 1, 0), (64, 20), (300, 0)):
        out = b.paged_window_attention(*on(dev, q, pool, bt, lens_t(ONE_BATCH)), window,
                                       sinks=sinks, num_splits=splits)
        seen = [visible(n - 1, window, sinks) for n in ONE_BATCH]
        check_rows(out, reference(q, pool, bt, seen, where), f"window {window} {kind}")


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("kind", KINDS)
def test_scored(kind, splits):
    dev, b = cuda_or_skip(), binding()
    q, pool, bt, where = one_batch(kind)
    before = torch.from_numpy(np.random.default_rng(7).random(
        (len(ONE_BATCH), HKV, bt.shape[1] * P)).astype(np.float32))
    mass = before.to(dev)
    out = b.paged_scored_attention(*on(dev, q, pool, bt, lens_t(ONE_BATCH)), mass,
                                   num_splits=splits)
    ref = reference(q, pool, bt, [np.arange(n) for n in ONE_BATCH], where)
    check_rows(out, ref, f"scored {kind}")
    want, tol = before.double().numpy().copy(), np.zeros(before.shape)
    for i, (_, _, (t, w), rel) in enumerate(ref):
        ws = w.reshape(len(t), HKV, G).sum(-1)
        want[i][:, t] += ws.T
        # the weights' relative errors, their sum's and the addition's roundings;
        # tokens of weight 0 keep their mass
        tol[i][:, t] = (ws * (rel + 2.0 ** -22)).T + 2.0 ** -24 * np.abs(want[i][:, t]) * 1.01
    check(mass, want, tol + 1e-38, f"mass {kind}")


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("kind", KINDS)
def test_decode(kind, splits):
    dev, b = cuda_or_skip(), binding()
    q, pool, bt, where = one_batch(kind)
    out = b.paged_decode_attention(*on(dev, q, pool, bt, lens_t(ONE_BATCH)), num_splits=splits)
    check_rows(out, reference(q, pool, bt, [np.arange(n) for n in ONE_BATCH], where),
               f"decode {kind}")


@pytest.mark.parametrize("count", [4, 70])
@pytest.mark.parametrize("kind", KINDS)
def test_chunk(kind, count):
    dev, b = cuda_or_skip(), binding()
    lens = [700, 100]
    pool, bt, where = infinite_cache(lens, [kind], 5)
    q = queries(2 * count, 6)
    for window, sinks, splits in ((0, 0, 0), (90, 20, 1), (0, 0, 3)):
        out = b.paged_chunk_attention(
            *on(dev, q, offsets([count, count]), pool, bt, lens_t(lens)), window=window,
            sinks=sinks, num_splits=splits)
        seen, seq = [], []
        for s, n in enumerate(lens):
            seen += [visible(n - count + i, window, sinks) for i in range(count)]
            seq += [s] * count
        ref = reference(q, pool, bt[seq], seen, [where[s] for s in seq])
        check_rows(out, ref, f"chunk {kind} window {window} splits {splits}")


@pytest.mark.parametrize("route", ["whole pages", "packed", "segments", "ranges"])
def test_planned_decode(route):
    dev, b = cuda_or_skip(), binding()
    batch = 160 if route in ("whole pages", "packed") else 48
    rng = np.random.default_rng(9)
    lens = rng.integers(1, 60 if route == "packed" else 500, batch).tolist()
    pool, bt, where = infinite_cache(lens, KINDS, 10)
    q = queries(batch, 11)
    args = on(dev, q, pool, bt, lens_t(lens))
    if route == "whole pages":
        assert b.attention_kernels(batch, bt.shape[1], 1) == "paged_decode_pagebox_kernel"
        out = b.paged_decode_attention(*args, num_splits=1)
    else:
        plan = b.Plan(np.asarray(lens, np.int32), bt.shape[1], device=dev,
                      num_sms=8 if route == "segments" else 0)
        if route == "segments":
            assert plan.num_segs > 0
        out = b.paged_decode_attention_planned(*args, plan)
    check_rows(out, reference(q, pool, bt, [np.arange(n) for n in lens], where), route)


@pytest.mark.parametrize("sms", [0, 8])
@pytest.mark.parametrize("kind", ["none", "first pages", "every other pair", "shared",
                                  "shared but one", "all"])
def test_shared_prefix_decode(kind, sms):
    """Pages that several sequences share, weighed by the tcgen05 kernel: its two
    copies of the rows take pages 0, 1 and 2, 3 of every four."""
    dev, b = cuda_or_skip(), binding()
    rng = np.random.default_rng(12)
    shared, members = 37, 16
    lens = (shared * P + rng.integers(1, 200, members)).tolist()
    pool, bt = make_cache(lens, seed=13)
    bt[1:, :shared] = bt[0, :shared]
    where = []
    for s, n in enumerate(lens):
        t = np.arange(n)
        t = t[{"none": t < 0, "first pages": t < 2 * P, "every other pair": t // P % 4 >= 2,
               "shared": t < shared * P, "shared but one": (t < shared * P) & (t != 100),
               "all": t >= 0}[kind]]
        pool[bt[s, t // P].long(), 0, torch.from_numpy(t % P), :, 0] = float("-inf")
        where.append(t)
    q = queries(members, 14)
    plan = b.Plan(np.asarray(lens, np.int32), bt.shape[1], device=dev, num_sms=sms,
                  block_tables=bt.numpy())
    assert plan.num_shared > 0
    out = b.paged_decode_attention_planned(*on(dev, q, pool, bt, lens_t(lens)), plan)
    check_rows(out, reference(q, pool, bt, [np.arange(n) for n in lens], where), kind)
