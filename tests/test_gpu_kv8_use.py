"""The 8-bit cache as it is used: batches whose pages are shared out, long tables and
pools, graphs, streams, waits that run out, the calls one after the other (GPU)."""
import numpy as np
import pytest
import torch

import oracle
from _gpu_util import binding, cuda_or_skip
from _kv8_util import (D, DTYPE, FORMATS, as_pool, attend8, bits, chunk_reference8, decode,
                       make_cache8, put_block, rotated, values)
from _longctx_util import HKV, HQ, P, check, normal, offsets, visible
from test_gpu_kv8 import (OFFSETS, PAGE, POSITION, SEQLEN, bf16, err_of, i32, oracle_bits,
                          run_chunk, run_decode, same)

pytestmark = pytest.mark.gpu

TIMEOUT = 8


# ----------------------------------------------- pages shared out among CTAs --

def wide(batch):
    """A table's width with which the batch's pages are shared out: 64 of them for
    each of two CTAs an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-64 * 2 * sms // max(batch - 1, 1))


def shared_cache(lens, fmt, seed=1):
    cuda_or_skip()
    return make_cache8(lens, fmt, seed=seed, width=max(wide(len(lens)), -(-max(lens) // P)))


SHARED = [
    [5000] + [17] * 40, [17] * 40 + [5000], [0] * 10, [1, 0], [64, 0, 65], [0] * 300 + [33] * 10,
    [i % 41 for i in range(600)], [100 * i for i in range(30)], [1500] * 20, [0, 0, 9000, 0],
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens", SHARED, ids=lambda x: f"{len(x)}x{max(x)}")
def test_shared_decode(fmt, lens):
    cache = shared_cache(lens, fmt)
    b = binding()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert b.decode8_workspace_bytes(len(lens), cache[2].shape[1]) == \
        2 * 2 * sms * HQ * (D + 2) * 4 + 8 * (len(lens) + 1)
    assert run_decode(fmt, lens, cache=cache) == 0


@pytest.mark.parametrize("lens", [
    [250 + i % 14 for i in range(120)], [256, 257] * 60, [17, 3000, 256, 0, 256, 16] * 12,
    [300] * 2 + [256] * 80, [256] * 80 + [2000, 1],
], ids=lambda x: f"{len(x)}x{max(x)}")
def test_shared_around_what_stays_whole(lens):
    """Sequences of 16 pages are not cut, those of 17 are."""
    assert run_decode("int8", lens, cache=shared_cache(lens, "int8")) == 0
    counts = [min(n, 1 + i % 4) for i, n in enumerate(lens)]
    assert run_chunk("e4m3", lens, counts, pad=0, cache=shared_cache(lens, "e4m3")) == 0


@pytest.mark.parametrize("window,sinks", [(5000, 0), (5000, 70), (6000, 3)])
def test_shared_windows(window, sinks):
    lens = [6100, 30, 5200, 0, 5001] + [40] * 60
    assert run_decode("e4m3", lens, window, sinks, cache=shared_cache(lens, "e4m3")) == 0
    counts = [4, 1, 3, 0, 2] + [1 + i % 4 for i in range(60)]
    assert run_chunk("int8", lens, counts, window, sinks, pad=0,
                     cache=shared_cache(lens, "int8")) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens", SHARED, ids=lambda x: f"{len(x)}x{max(x)}")
def test_shared_chunks(fmt, lens):
    counts = [min(n, (i * 7) % 5) for i, n in enumerate(lens)]
    counts[-1] = min(4, lens[-1])
    assert run_chunk(fmt, lens, counts, pad=0, cache=shared_cache(lens, fmt)) == 0
    # with a long chunk, and rows behind the last
    if max(lens) >= 40:
        counts[int(np.argmax(lens))] = 40
        assert run_chunk(fmt, lens, counts, pad=5, cache=shared_cache(lens, fmt)) == 0


@pytest.mark.parametrize("batch", [289, 1500, 65535])
def test_shared_large_batches(batch):
    """Up to the largest batch, of a few lengths in turn: each sequence as in a batch of its
    own kind."""
    dev, b = cuda_or_skip(), binding()
    kinds, width = 70, max(wide(batch), 2)
    lens = [i % 33 for i in range(kinds - 1)] + [500]
    codes, sc, few = make_cache8(lens, "e4m3", width=max(width, 32))
    pool, s = as_pool(codes, "e4m3").to(dev), torch.from_numpy(sc).to(dev)
    pick = torch.from_numpy(np.random.default_rng(batch).integers(0, kinds, batch)).to(dev)
    ln, bt = i32(lens, dev), i32(few, dev)
    q, err = normal((kinds, HQ, D), 3).to(dev), err_of(dev)
    want = b.paged8_decode_attention(q, pool, s, bt, ln, num_splits=1)
    got = b.paged8_decode_attention(q[pick], pool, s, bt[pick], ln[pick], dev_err=err)
    # (sequences that two CTAs share are summed in another order)
    short = ln[pick] <= 16
    assert torch.equal(got[short], want[pick][short])
    assert (got.float() - want[pick].float()).abs().max() <= 2 ** -7 * want.float().abs().max()
    off = torch.arange(batch + 1, dtype=torch.int32, device=dev)
    got = b.paged8_chunk_attention(q[pick], off, pool, s, bt[pick], ln[pick], dev_err=err)
    assert torch.equal(got[short], want[pick][short])
    assert (got.float() - want[pick].float()).abs().max() <= 2 ** -7 * want.float().abs().max()
    # (an empty sequence has no place for its chunk's token)
    assert int(err.item()) == POSITION


def test_shared_bad_inputs():
    lens = [300, 40, 17, 2000]
    assert run_decode("e4m3", lens, cache=shared_cache(lens, "e4m3"),
                      bad=[(0, 3, -1), (1, 1, 10 ** 6), (3, 100, -9)]) == PAGE
    codes, sc, bt = shared_cache(lens, "int8")
    assert run_decode("int8", [300, -4, 17, 2000], cache=(codes, sc, bt)) == SEQLEN
    assert run_chunk("int8", [3, 40, 17, -1], [4, 4, 0, 2], pad=0,
                     cache=(codes, sc, bt)) == SEQLEN | POSITION
    assert run_chunk("e4m3", lens, [4, 3, 2, 1], cache=shared_cache(lens, "e4m3"),
                     bad=[(0, 3, -1), (2, 0, 10 ** 6), (3, 7, -9)]) == PAGE


@pytest.mark.parametrize("splits", [0, 1])
def test_short_chunks_with_bad_offsets(splits):
    """Sequences with bad offsets are skipped, and their rows left as they were."""
    dev, b = cuda_or_skip(), binding()
    lens = [300, 200, 100, 50]
    codes, sc, bt = shared_cache(lens, "int8")
    q = normal((9, HQ, D), 3)
    cache = (as_pool(codes, "int8").to(dev), torch.from_numpy(sc).to(dev), i32(bt, dev))
    for off, good in (([0, 2, 5, 4, 4], (0, 1)), ([-1, 2, 4, 8, 9], (1, 2, 3)),
                      ([0, 3, 6, 9, 12], (0, 1, 2)), ([0, 3, 6, 2 ** 31 - 1, 9], (0, 1))):
        out, err = torch.full((9, HQ, D), 7.0, dtype=torch.bfloat16, device=dev), err_of(dev)
        b.paged8_chunk_attention(q.to(dev), i32(off, dev), *cache, i32(lens, dev), out,
                                 num_splits=splits, dev_err=err)
        assert int(err.item()) == OFFSETS
        want, tol = np.full((9, HQ, D), 7.0), np.zeros((9, HQ, D))
        vals = values(codes, sc, "int8")
        for i in good:
            n = off[i + 1] - off[i]
            for j in range(n):
                want[off[i] + j], tol[off[i] + j] = attend8(
                    q[off[i] + j], vals, bt[i], np.arange(lens[i] - n + j + 1), 16)
        check(out, want, tol, f"offsets {off}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch", [1, 2, 3, 8, 9, 20])
def test_many_ranges(fmt, batch):
    """Merges of more results than a warp's, by CTAs of each size."""
    lens = [(1100, 0, 1, 700, 33, 512)[i % 6] + i for i in range(batch)]
    for splits in (17, 40, 100):
        assert run_decode(fmt, lens, splits=splits) == 0
        assert run_chunk(fmt, lens, [min(n, 1 + i % 4) for i, n in enumerate(lens)], splits=splits,
                         pad=0) == 0


# ----------------------------------------------------------- long and large --

def test_widening_in_rounds():
    """Sequences whose pages do not fit the workspace at once: each as by itself."""
    dev, b = cuda_or_skip(), binding()
    batch, width, n = 40, 2048, 5
    lens = [width * P - 3 * i for i in range(batch)]
    rng = np.random.default_rng(5)
    codes, sc, _ = make_cache8([200 * P], "int8", spare=0)
    bt = np.stack([rng.integers(0, 200, width) for _ in range(batch)]).astype(np.int32)
    counts = [n if i != 7 else 2 for i in range(batch)]
    off = offsets(counts)
    q = normal((int(off[-1]), HQ, D), 6).to(dev)
    pool, s, t = as_pool(codes, "int8").to(dev), torch.from_numpy(sc).to(dev), i32(bt, dev)
    one = b.chunk8_workspace_bytes(n, 1, width, 1)
    assert b.chunk8_workspace_bytes(len(q), batch, width, 1) < 33 * one
    err = err_of(dev)
    out = b.paged8_chunk_attention(q, off.to(dev), pool, s, t, i32(lens, dev), num_splits=1,
                                   dev_err=err)
    assert int(err.item()) == 0
    for i in range(batch):
        a, z = int(off[i]), int(off[i + 1])
        want = b.paged8_chunk_attention(q[a:z], offsets([z - a]).to(dev), pool, s, t[i:i + 1],
                                        i32(lens[i:i + 1], dev), num_splits=1)
        assert torch.equal(out[a:z], want), i
    want, tol = chunk_reference8(q[-n:].cpu(), [0, n], values(codes, sc, "int8"), bt[-1:],
                                 lens[-1:], 0, 0, torch.zeros((n, HQ, D)))
    check(out[-n:], want, tol, "last sequence")


@pytest.mark.parametrize("fmt", FORMATS)
def test_pool_past_32_bits(fmt):
    """Pages beyond 2^32 bytes of codes, through every call."""
    dev, b = cuda_or_skip(), binding()
    pages, n = 2 ** 18 + 40, 90
    pool = torch.zeros((pages, 2, HKV, P, D), dtype=torch.int8, device=dev).view(DTYPE[fmt])
    sc = torch.full((pages, 2, HKV), 127, dtype=torch.uint8, device=dev)
    order = [pages - 1, 2 ** 18 + 7, pages - 9, 2 ** 18, 5, pages - 2]
    bt = i32([order], dev)
    k, v, err = normal((n, HKV, D), 1).to(dev), normal((n, HKV, D), 2).to(dev), err_of(dev)
    b.kv8_write_prefill(k[:-1], v[:-1], i32([0, n - 1], dev), i32([0], dev), pool, sc, bt,
                        dev_err=err)
    b.kv8_append(k[-1:], v[-1:], pool, sc, bt, i32([n - 1], dev), dev_err=err)
    # the same in a small pool
    small = torch.zeros((6, 2, HKV, P, D), dtype=torch.int8, device=dev).view(DTYPE[fmt])
    s2 = torch.full((6, 2, HKV), 127, dtype=torch.uint8, device=dev)
    t2 = i32([list(range(6))], dev)
    b.kv8_write_prefill(k[:-1], v[:-1], i32([0, n - 1], dev), i32([0], dev), small, s2, t2)
    b.kv8_append(k[-1:], v[-1:], small, s2, t2, i32([n - 1], dev))
    at = torch.tensor(order, device=dev)
    assert torch.equal(pool.view(torch.uint8)[at], small.view(torch.uint8))
    assert torch.equal(sc[at], s2)
    ln, off = i32([n], dev), i32([0, n], dev)
    q = normal((n, HQ, D), 3).to(dev)
    for c in (1, 4, n):
        o = i32([0, c], dev)
        assert torch.equal(b.paged8_chunk_attention(q[:c], o, pool, sc, bt, ln, dev_err=err),
                           b.paged8_chunk_attention(q[:c], o, small, s2, t2, ln))
    assert torch.equal(b.paged8_decode_attention(q[:1], pool, sc, bt, ln, dev_err=err),
                       b.paged8_decode_attention(q[:1], small, s2, t2, ln))
    got = b.kv8_read(off, i32([0], dev), pool, sc, bt, torch.empty_like(k), torch.empty_like(v),
                     dev_err=err)
    want = b.kv8_read(off, i32([0], dev), small, s2, t2, torch.empty_like(k), torch.empty_like(v))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int(err.item()) == 0


@pytest.mark.parametrize("counts", [[1], [3], [5]])
def test_largest_table(counts):
    """Positions up to the last one a table can name."""
    dev, b = cuda_or_skip(), binding()
    blocks, window, sinks, n = 2 ** 27 - 1, 200, 3, counts[0]
    L, last = blocks * 16 - 2, 16           # the table's pages that exist: 0 and the last 16
    codes, sc, _ = make_cache8([17 * P], "e4m3", spare=0)
    q = normal((n, HQ, D), 41)
    bt = torch.full((1, blocks), -1, dtype=torch.int32, device=dev)
    bt[0, 0] = last
    bt[0, blocks - last:] = torch.arange(last, dtype=torch.int32, device=dev)
    near = np.concatenate([[last], np.arange(last)]).astype(np.int32)
    want, tol = np.zeros((n, HQ, D)), np.zeros((n, HQ, D))
    for i in range(n):
        p = L - n + i
        t = np.concatenate([np.arange(sinks), 16 + np.arange(p - window + 1, p + 1) -
                            (blocks - last) * 16])
        want[i], tol[i] = attend8(q[i], values(codes, sc, "e4m3"), near, t, 16 if n < 5 else 8)
    pool, s, ln, err = as_pool(codes, "e4m3").to(dev), torch.from_numpy(sc).to(dev), \
        i32([L], dev), err_of(dev)
    got = b.paged8_chunk_attention(q.to(dev), offsets(counts).to(dev), pool, s, bt, ln,
                                   window=window, sinks=sinks, dev_err=err)
    check(got, want, tol, "chunk")
    if n == 1:
        got = b.paged8_decode_attention(q.to(dev), pool, s, bt, ln, window=window, sinks=sinks,
                                        dev_err=err)
        check(got, want, tol, "decode")
    # the last places written and read
    k = normal((3, HKV, D), 42).to(dev)
    b.kv8_write_prefill(k, k, i32([0, 3], dev), i32([blocks * 16 - 3], dev), pool, s, bt,
                        dev_err=err)
    b.kv8_append(k[:1], k[:1], pool, s, bt, i32([blocks * 16 - 1], dev), dev_err=err)
    _, v = b.kv8_read(i32([0, 3], dev), i32([blocks * 16 - 3], dev), pool, s, bt,
                      torch.empty_like(k), torch.empty_like(k), dev_err=err)
    assert (v[:2].float() - k[:2].float()).abs().max() <= 0.5
    assert (v[2].float() - k[0].float()).abs().max() <= 0.5
    assert int(err.item()) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("theta", [10000.0, 1e6, 1.0, 0.5, 1e30])
@pytest.mark.parametrize("start", [2040, 40961, 2 ** 21 + 5])
def test_write_far_positions(fmt, theta, start):
    dev, b = cuda_or_skip(), binding()
    n, width = 37, (start + 37) // P + 1
    rng = np.random.default_rng(start)
    k, v = (oracle_bits(rng.standard_normal((n + 1, HKV, D)).astype(np.float32))
            for _ in range(2))
    bt = np.full((1, width), -1, np.int32)
    first = start // P
    bt[0, first:] = np.arange(width - first)[::-1]
    pages = width - first
    codes, scales = np.zeros((pages, 2, HKV, P, D), np.uint8), np.full((pages, 2, HKV), 100,
                                                                      np.uint8)
    pool, sc, err = as_pool(codes, fmt).to(dev), torch.from_numpy(scales).to(dev), err_of(dev)
    b.kv8_write_prefill(bf16(k[:n], dev), bf16(v[:n], dev), i32([0, n], dev), i32([start], dev),
                        pool, sc, i32(bt, dev), rope_theta=theta, dev_err=err)
    b.kv8_append(bf16(k[n:], dev), bf16(v[n:], dev), pool, sc, i32(bt, dev), i32([start + n], dev),
                 rope_theta=theta, dev_err=err)
    assert int(err.item()) == 0
    key, val = rotated(k, range(start, start + n + 1), theta), oracle.bf16_to_f64(v)
    for a, z in [(max(start, p), min(start + n, p + P)) for p in range(first * P, start + n, P)] + \
            [(start + n, start + n + 1)]:
        page = bt[0, a // P]
        for kv, x in enumerate((key, val)):
            for h in range(HKV):
                codes[page, kv, h], scales[page, kv, h] = put_block(
                    codes[page, kv, h], scales[page, kv, h], a % P, x[a - start:z - start, h], fmt)
    same(bits(sc), scales, "scales")
    same(decode(bits(pool), fmt), decode(codes, fmt), "values")


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_and_read_with_offsets_that_fall(fmt):
    """Sequences are written as the definition says or not at all, reported either way,
    and no page of another one changes."""
    dev, b = cuda_or_skip(), binding()
    rng = np.random.default_rng(9)
    k, v = (oracle_bits(rng.standard_normal((100, HKV, D)).astype(np.float32)) for _ in range(2))
    bt = np.arange(28, dtype=np.int32).reshape(4, 7)
    codes, scales, _ = make_cache8([28 * P], fmt, spare=0)
    for off in ([0, 90, 5, 40, 100], [0, 100, 100, 0, 100], [0, 5, 100, 40, 50],
                [0, -7, 60, 80, 100], [0, 2 ** 31 - 1, -2 ** 31, 50, 100]):
        pool, sc, err = as_pool(codes, fmt).to(dev), torch.from_numpy(scales).to(dev), err_of(dev)
        b.kv8_write_prefill(bf16(k, dev), bf16(v, dev), i32(off, dev), i32([0] * 4, dev), pool, sc,
                            i32(bt, dev), rope_theta=1e4, dev_err=err)
        assert int(err.item()) == OFFSETS, off
        got, got_sc = bits(pool), bits(sc)
        for i in range(4):
            pages = bt[i]
            want, want_sc = codes.copy(), scales.copy()
            n = off[i + 1] - off[i]
            if off[i] >= 0 and 0 < n and off[i + 1] <= 100:
                key = rotated(k[off[i]:off[i + 1]], range(n), 1e4)
                for a in range(0, n, P):
                    for kv, x in enumerate((key, oracle.bf16_to_f64(v[off[i]:off[i + 1]]))):
                        for h in range(HKV):
                            page = pages[a // P]
                            want[page, kv, h], want_sc[page, kv, h] = put_block(
                                want[page, kv, h], want_sc[page, kv, h], 0, x[a:a + P, h], fmt)
            for p in pages:
                new = np.array_equal(got_sc[p], want_sc[p]) and np.array_equal(
                    decode(got[p], fmt), decode(want[p], fmt), equal_nan=True)
                old = np.array_equal(got_sc[p], scales[p]) and np.array_equal(got[p], codes[p])
                assert new or old, (off, i, p)
        out = torch.full((100, HKV, D), 9.0, dtype=torch.bfloat16, device=dev)
        out2, err = out.clone(), err_of(dev)
        b.kv8_read(i32(off, dev), i32([0] * 4, dev), pool, sc, i32(bt, dev), out, out2, dev_err=err)
        assert int(err.item()) == OFFSETS


# --------------------------------------------------- streams, graphs, waits --

def batch_of(fmt, lens, counts, seed=1, width=None):
    dev = cuda_or_skip()
    codes, sc, bt = make_cache8(lens, fmt, seed=seed, width=width)
    return (normal((sum(counts), HQ, D), seed).to(dev), offsets(counts).to(dev),
            as_pool(codes, fmt).to(dev), torch.from_numpy(sc).to(dev), i32(bt, dev),
            i32(lens, dev))


CALLS = [  # (num_splits, table's width: the shape of each call's work)
    (0, None), (3, None), (0, 20000)]


@pytest.mark.parametrize("splits,width", CALLS)
def test_waits_that_run_out(splits, width):
    """With a wait limit of 0 every kernel gives up at its first look at a copy that has
    not landed, reports it, and leaves the stream and the next calls as they should be.
    (Pages and rows come from memory, what a kernel reads before that look from L2, so
    such a copy is certain.)"""
    dev, b = cuda_or_skip(), binding()
    counts = [3, 70, 200, 1]
    q, off, pool, sc, bt, ln = batch_of("e4m3", [900, 70, 1500, 333], counts, width=width)
    kw = dict(num_splits=splits)
    k, v = normal((400, HKV, D), 7).to(dev), normal((400, HKV, D), 8).to(dev)
    wpool, wsc = torch.zeros_like(pool.view(torch.int8)), torch.full_like(sc, 127)
    woff, wstart = i32([0, 100, 200, 300, 400], dev), i32([0, 0, 3000, 8], dev)
    calls = [(lambda e: b.paged8_chunk_attention(q, off, pool, sc, bt, ln, dev_err=e, **kw)),
             (lambda e: b.paged8_chunk_attention(q[:16], i32([0, 4, 8, 12, 16], dev), pool, sc,
                                                 bt, ln, dev_err=e, **kw)),
             (lambda e: b.paged8_decode_attention(q[:4], pool, sc, bt, ln, dev_err=e, **kw))]
    if splits == 0 and width is None:
        wide_bt = torch.full((4, 200), -1, dtype=torch.int32, device=dev)
        wide_bt[:, :8] = torch.arange(32, device=dev).reshape(4, 8)
        wide_bt[2, 187:195] = torch.arange(40, 48, device=dev)

        def write(e):
            b.kv8_write_prefill(k, v, woff, wstart, wpool, wsc, wide_bt, dev_err=e)
            return wpool.clone()
        calls.append(write)
    for call in calls:
        want = call(None)
        old = b.set_wait_limit_ns(0)
        err = err_of(dev)
        torch.empty(1 << 28, dtype=torch.uint8, device=dev).zero_()
        for x in (q, off, bt, ln):
            x.clone()
        try:
            call(err)
        finally:
            b.set_wait_limit_ns(old)
        torch.cuda.synchronize()
        assert int(err.item()) & TIMEOUT
        err = err_of(dev)
        assert torch.equal(want, call(err)) and int(err.item()) == 0


@pytest.mark.parametrize("splits,width", CALLS)
def test_repeats_bit_for_bit_and_replays(splits, width):
    dev, b = cuda_or_skip(), binding()
    lens, counts = [900, 77, 300], [60, 1, 4]
    q, *rest = batch_of("int8", lens, counts, width=width)
    off, pool, sc, bt, ln = rest
    w = torch.empty(b.chunk8_workspace_bytes(len(q), 3, bt.shape[1], splits) + 16,
                    dtype=torch.uint8, device=dev)
    w2 = torch.empty(b.decode8_workspace_bytes(3, bt.shape[1], splits) + 16, dtype=torch.uint8,
                     device=dev)

    def run(out, out2):
        b.paged8_chunk_attention(q, *rest, out, num_splits=splits, workspace=w)
        b.paged8_decode_attention(q[:3], pool, sc, bt, ln, out2, num_splits=splits, workspace=w2)
        return out, out2
    first = run(torch.empty_like(q), torch.empty_like(q[:3]))
    for _ in range(3):
        w.fill_(255)                             # (NaN, and pages that are not there)
        w2.fill_(255)
        again = run(torch.empty_like(q), torch.empty_like(q[:3]))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    outs = torch.zeros_like(q), torch.zeros_like(q[:3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(*outs)
    # other queries, and other lengths: nothing of the first ones is kept
    q.copy_(normal(q.shape, 16).to(dev))
    ln.copy_(i32([400, 33, 290], dev))
    g.replay()
    torch.cuda.synchronize()
    want = run(torch.empty_like(q), torch.empty_like(q[:3]))
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_a_captured_step_replays():
    """Append, decode and read in a graph, its positions moved on between replays, against
    the same steps one by one."""
    dev, b = cuda_or_skip(), binding()
    batch, steps = 5, 20
    rng = np.random.default_rng(3)
    start = rng.integers(0, 60, batch)
    bt = i32(rng.permutation(batch * 6).reshape(batch, 6), dev)
    k, v = normal((steps, batch, HKV, D), 1).to(dev), normal((steps, batch, HKV, D), 2).to(dev)
    q = normal((steps, batch, HQ, D), 3).to(dev)

    def fresh():
        return (torch.zeros((batch * 6, 2, HKV, P, D), dtype=torch.int8, device=dev).view(
            DTYPE["e4m3"]), torch.full((batch * 6, 2, HKV), 120, dtype=torch.uint8, device=dev))

    def step(pool, sc, kk, vv, qq, pos, ws):
        qr = torch.empty_like(qq)
        b.kv8_append(kk, vv, pool, sc, bt, pos, q_in=qq, q_out=qr)
        return b.paged8_decode_attention(qr, pool, sc, bt, pos + 1, workspace=ws, num_splits=2)
    ws = torch.empty(b.decode8_workspace_bytes(batch, 6, 2), dtype=torch.uint8, device=dev)
    pool, sc = fresh()
    want = [step(pool, sc, k[i], v[i], q[i], i32(start + i, dev), ws) for i in range(steps)]
    p2, s2 = fresh()
    a, c, d, pos = k[0].clone(), v[0].clone(), q[0].clone(), i32(start, dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = step(p2, s2, a, c, d, pos, ws)
    for i in range(steps):
        a.copy_(k[i]), c.copy_(v[i]), d.copy_(q[i]), pos.copy_(i32(start + i, dev))
        g.replay()
        assert torch.equal(out, want[i]), i
    assert torch.equal(pool.view(torch.int8), p2.view(torch.int8)) and torch.equal(sc, s2)


def test_calls_on_other_streams():
    """Each call on two streams at once, with workspaces of their own."""
    dev, b = cuda_or_skip(), binding()
    lens, counts = [333, 40, 900], [50, 4, 1]
    q, *rest = batch_of("e4m3", lens, counts, width=8000)
    off, pool, sc, bt, ln = rest
    calls = (lambda **kw: b.paged8_chunk_attention(q, *rest, **kw),
             lambda **kw: b.paged8_chunk_attention(q, *rest, num_splits=2, **kw),
             lambda **kw: b.paged8_decode_attention(q[:3], pool, sc, bt, ln, **kw),
             lambda **kw: b.paged8_decode_attention(q[:3], pool, sc, bt, ln, num_splits=2, **kw))
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for f, w in zip(calls, want):
        for _ in range(3):
            freed = torch.empty_like(q)
            torch.cuda._sleep(1_000_000)
            freed.fill_(9)
            del freed
            got = [f(stream=s) for s in streams]
            torch.empty(1 << 20, dtype=torch.uint8, device=dev).fill_(0xFF)
            torch.cuda.synchronize()
            assert all(torch.equal(w, x) for x in got)


def test_write_and_read_on_another_stream():
    dev, b = cuda_or_skip(), binding()
    n = 200
    k, v = normal((n, HKV, D), 1).to(dev), normal((n, HKV, D), 2).to(dev)
    off, start, bt = i32([0, n], dev), i32([0], dev), i32([list(range(13))], dev)
    results = []
    for s in (None, torch.cuda.Stream()):
        pool = torch.zeros((13, 2, HKV, P, D), dtype=torch.int8, device=dev)
        sc = torch.full((13, 2, HKV), 127, dtype=torch.uint8, device=dev)
        out = torch.zeros_like(k), torch.zeros_like(v)
        torch.cuda.synchronize()
        b.kv8_write_prefill(k, v, off, start, pool, sc, bt, stream=s)
        b.kv8_append(k[:1], v[:1], pool, sc, bt, i32([n], dev), stream=s)
        b.kv8_read(off, start, pool, sc, bt, *out, stream=s)
        torch.cuda.synchronize()
        results.append((pool, sc, *out))
    for x, y in zip(*results):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ together --

@pytest.mark.parametrize("fmt", FORMATS)
def test_a_conversation(fmt):
    """A prompt written and attended in chunks, speculative tokens verified and partly
    rejected, decode steps, a windowed step, and the cache read back: every output
    against the 64-bit attention over the cache as it stands."""
    dev, b = cuda_or_skip(), binding()
    pages, err = 30, err_of(cuda_or_skip())
    pool = torch.full((pages, 2, HKV, P, D), 0x7F, dtype=torch.int8, device=dev).view(DTYPE[fmt])
    sc = torch.full((pages, 2, HKV), 255, dtype=torch.uint8, device=dev)
    bt = np.random.default_rng(61).permutation(pages).astype(np.int32)[:14][None]
    t = i32(bt, dev)

    def vals():
        return values(bits(pool), sc.cpu().numpy(), fmt)

    def chunk(n, at, seed):
        k, v, q = (normal((n, h, D), seed + h).to(dev) for h in (HKV, HKV, HQ))
        off = offsets([n]).to(dev)
        b.kv8_write_prefill(k, v, off, i32([at], dev), pool, sc, t, dev_err=err)
        out = b.paged8_chunk_attention(q, off, pool, sc, t, i32([at + n], dev), dev_err=err)
        want, tol = chunk_reference8(q.cpu(), off.cpu(), vals(), bt, [at + n], 0, 0,
                                     torch.zeros_like(q).cpu())
        check(out, want, tol, f"chunk of {n} at {at}")
    cached = 0
    for n in (64, 64, 22):
        chunk(n, cached, 62 + cached)
        cached += n
    for i in range(6):                           # four tokens tried, `i % 4 + 1` kept
        chunk(4, cached, 400 + i)
        cached += i % 4 + 1
    for i in range(20):
        k, v, q = (normal((1, h, D), 900 + i + h).to(dev) for h in (HKV, HKV, HQ))
        qr, window = torch.empty_like(q), 50 if i == 19 else 0
        b.kv8_append(k, v, pool, sc, t, i32([cached], dev), q_in=q, q_out=qr, dev_err=err)
        cached += 1
        out = b.paged8_decode_attention(qr, pool, sc, t, i32([cached], dev), window=window,
                                        sinks=3 if window else 0, dev_err=err)
        want, tol = attend8(qr[0].cpu(), vals(), bt[0],
                            visible(cached - 1, window, 3 if window else 0), 16)
        check(out[0], want, tol, f"step at {cached}")
    k, v = torch.empty((2, cached, HKV, D), dtype=torch.bfloat16, device=dev).unbind(0)
    b.kv8_read(i32([0, cached], dev), i32([0], dev), pool, sc, t, k, v, dev_err=err)
    x = vals()[bt[0]].transpose(0, 3, 1, 2, 4).reshape(-1, 2, HKV, D)[:cached]
    assert np.array_equal(k.double().cpu().numpy(), x[:, 0])
    assert np.array_equal(v.double().cpu().numpy(), x[:, 1])
    assert int(err.item()) == 0


def test_other_scales_and_devices_are_refused():
    dev, b = cuda_or_skip(), binding()
    q, off, pool, sc, bt, ln = batch_of("e4m3", [40], [1])
    kv = normal((1, HKV, D), 1).to(dev)
    for bad in (sc.cpu(), sc[:-1], sc.int(), sc[..., None], sc.transpose(1, 2), None):
        for f in (lambda: b.paged8_decode_attention(q, pool, bad, bt, ln),
                  lambda: b.paged8_chunk_attention(q, off, pool, bad, bt, ln),
                  lambda: b.kv8_append(kv, kv, pool, bad, bt, ln),
                  lambda: b.kv8_write_prefill(kv, kv, off, ln, pool, bad, bt),
                  lambda: b.kv8_read(off, ln, pool, bad, bt, kv, kv.clone())):
            with pytest.raises((TypeError, ValueError)):
                f()
