"""Timed cases and plain forms of the operators over an 8-bit paged KV cache.

The cache holds K and V as 8-bit codes (e4m3 floats or signed integers), 64
dims x 16 tokens of one kv head to a block, with one power-of-two scale a
block: pool [pages][K|V][8 kv heads][16 tokens][64], scales uint8
[pages][K|V][8], a value being code * 2^(scale - 127).

  append  one new token per sequence: K rotated for its position (and rounded
          to bf16, what a 16-bit cache holds), K and V rounded to the block's
          scale.  The block's scale is the smallest whose codes reach the
          largest magnitude it was given; where a token needs a larger one the
          block's earlier tokens are rounded again to it
  write   the same for a ragged batch of prompt tokens, each block's new tokens
          at once
  read    cached tokens as bf16 (codes times scales: exact)
  decode  one-token attention over the cache, optionally under a sliding
          window with sink tokens
  chunk   attention of a ragged chunk of new tokens, causal, optionally under
          a window

A pass of append or write ends with a read of the tokens in the blocks it
wrote, so its outputs are the values that the cache then stands for.
Geometry as everywhere in this library: 32 query heads, 8 kv heads of 64 dims,
pages of 16 tokens.
"""
import functools
import math

import torch

own = False

HQ, HKV, G, D, P = 32, 8, 4, 64, 16
SCALE = D ** -0.5
THETA = 500000.0
BIAS, LEAST, MOST = 127, 3, 240          # scale exponents: bias, smallest, largest
TOP = {"e4m3": 448.0, "int8": 127.0}     # largest code of each format


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the next token of one conversation far past its cache slots (latency)
        dict(name="append one", op="append", fmt="int8", batch=1, ctx=2048, far=131072),
        # the next token of a large decode batch
        dict(name="append batch", op="append", fmt="e4m3", batch=2048, ctx=2048, far=0),
        # a few short turns added behind caches that end inside a block
        dict(name="write turns", op="write", fmt="int8", batch=5, ctx=37, start=1000),
        # a batch of whole prompts
        dict(name="write prompts", op="write", fmt="e4m3", batch=64, ctx=2047, start=0),
        # one sequence's cache as bf16, to hand it on
        dict(name="read one", op="read", fmt="e4m3", batch=1, ctx=4093, start=0),
        # the newer part of a batch's caches
        dict(name="read batch", op="read", fmt="int8", batch=32, ctx=4096, start=777),
        # one long conversation decoding (latency, split over the cache)
        dict(name="decode one", op="decode", fmt="int8", batch=1, ctx=30011, window=0, sinks=0),
        # a full decode batch: the cache is read once (memory-bound)
        dict(name="decode batch", op="decode", fmt="e4m3", batch=256, ctx=2048, window=0, sinks=0),
        # a decode batch far past its window
        dict(name="decode window", op="decode", fmt="int8", batch=128, ctx=16384, window=1000,
             sinks=4),
        # verifying four drafted tokens of 64 sequences at once (memory-bound)
        dict(name="chunk verify", op="chunk", fmt="e4m3", batch=64, ctx=2048, tokens=4, singles=0,
             window=0, sinks=0, pad=3),
        # the second half of two long prompts (compute-bound, the largest case)
        dict(name="chunk prefill", op="chunk", fmt="int8", batch=2, ctx=8192, tokens=4096,
             singles=0, window=0, sinks=0, pad=0),
        # continuous batching: a prompt chunk beside 63 decoding sequences
        dict(name="chunk mixed", op="chunk", fmt="e4m3", batch=64, ctx=2047, tokens=509,
             singles=63, window=0, sinks=0, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "write", "read", "decode", "decode", "chunk", "chunk"])
    c = dict(op=op, fmt=rng.choice(["e4m3", "int8"]))
    window = _log(rng, 1, 8192) if rng.random() < 0.4 else 0
    sinks = rng.randrange(0, 200) if window and rng.random() < 0.7 else 0
    if op == "append":
        return dict(c, batch=_log(rng, 1, 2048), ctx=_log(rng, 1, 4096),
                    far=_log(rng, 4096, 1 << 20) if rng.random() < 0.5 else 0)
    if op in ("write", "read"):
        batch, ctx = _log(rng, 1, 128), _log(rng, 1, 8192)
        while batch * ctx > 1 << 17:
            batch //= 2
        return dict(c, batch=batch, ctx=ctx, start=_log(rng, 1, 4000) if rng.random() < 0.5 else 0)
    if op == "decode":
        batch, ctx = _log(rng, 1, 256), _log(rng, 1, 131072)
        while batch * (min(ctx, window + sinks) if window else ctx) > 1 << 19:
            batch //= 2
        return dict(c, batch=batch, ctx=ctx, window=window, sinks=sinks)
    batch, tokens = _log(rng, 1, 128), _log(rng, 1, 4096)
    ctx = max(tokens, _log(rng, 1, 16384))
    while batch * tokens * ctx > 2 * 4096 * 8192 or batch * ctx > 1 << 19:
        batch = max(1, batch // 2)
        if batch == 1:
            tokens = max(1, tokens // 2)
            ctx = max(tokens, ctx * 3 // 4)
    return dict(c, batch=batch, ctx=ctx, tokens=tokens,
                singles=rng.randrange(batch) if rng.random() < 0.4 else 0, window=window,
                sinks=sinks, pad=rng.randrange(0, 9))


def _lens(c):
    """Tokens of each sequence (cached, or written or read by the call): the
    first has ctx, the others spread over the upper half of the range."""
    return [max(1, c["ctx"] - (i * 617) % (c["ctx"] // 2 + 1)) for i in range(c["batch"])]


def _starts(c):
    """First token of each sequence that the call writes or reads."""
    return [max(0, c["start"] - (i * 397) % (c["start"] // 3 + 1)) for i in range(c["batch"])]


def _chunks(c):
    """New tokens of each sequence: the last `singles` decode one token, the
    others take ragged chunks of up to `tokens`."""
    few = c["batch"] - c["singles"]
    return [min(n, c["tokens"] - (i * 13) % (c["tokens"] // 4 + 1)) if i < few else 1
            for i, n in enumerate(_lens(c))]


def _visible(pos, window, sinks):
    """How many cached tokens position pos sees."""
    if not window or window > pos:
        return pos + 1
    first = pos - window + 1
    return window + min(sinks, first)


def work(c):
    B, half, row = c["batch"], HKV * D, HKV * D * 2      # 8-bit and 16-bit row bytes
    if c["op"] == "append":
        # K and V in, their codes out; then the tokens of the blocks written
        # (those before the new one also read by the append, if only to learn
        # that the scale stands) as codes in and bf16 out
        live = sum((L - 1) % P + 1 for L in _lens(c))
        return {"bytes": B * (2 * row + 2 * half + 2 * HQ * D * 2 + 2 * HKV + 12) +
                         live * (2 * half + 2 * row), "flops": 3 * B * (HQ + HKV) * D}
    if c["op"] in ("write", "read"):
        n, first = sum(_lens(c)), sum(s % P for s in _starts(c))
        pages = sum((s + L + P - 1) // P - s // P for s, L in zip(_starts(c), _lens(c)))
        read = n * (2 * half + 2 * row) + pages * (2 * HKV + 4)
        if c["op"] == "read":
            return {"bytes": read, "flops": 2 * n * HKV * D}
        return {"bytes": n * (2 * row + 2 * half) + pages * (2 * HKV + 4) + read +
                         first * (2 * half + 2 * row), "flops": 5 * n * HKV * D}
    if c["op"] == "decode":
        seen = sum(_visible(L - 1, c["window"], c["sinks"]) for L in _lens(c))
        return {"bytes": 2 * half * seen + seen // P * (2 * HKV + 4) + 2 * B * HQ * D * 2 + 4 * B,
                "flops": 4 * D * HQ * seen}
    seen = pairs = 0
    for L, n in zip(_lens(c), _chunks(c)):
        pairs += sum(_visible(p, c["window"], c["sinks"]) for p in range(L - n, L))
        lo = max(0, L - n - c["window"] + 1) if c["window"] else 0
        seen += L - lo + min(c["sinks"], lo)
    return {"bytes": 2 * half * seen + seen // P * (2 * HKV + 4) +
                     2 * sum(_chunks(c)) * HQ * D * 2 + 4 * (2 * B + 1),
            "flops": 4 * D * HQ * pairs}


# ------------------------------------------------------------------ inputs --

def _table(need, g, spare=3):
    """Block tables naming shuffled pages where need [B][width] is true, -1
    elsewhere, and the pages of a pool that holds them."""
    pages = int(need.sum()) + spare
    ids = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    at = (torch.cumsum(need.reshape(-1).long(), 0) - 1).clamp(min=0)
    return torch.where(need.reshape(-1), ids[at], -1).reshape(need.shape).contiguous(), pages


def _gains(g):
    """Magnitudes of K's and V's dims [2][8][64]: a few large channels of K."""
    x = torch.exp(0.6 * torch.randn((2, HKV, D), generator=g, device="cuda"))
    return x / x.square().mean(-1, keepdim=True).sqrt()


def _cache(pages, fmt, gains, g):
    """A pool of codes and its scales, as the writers would have left them."""
    pool = torch.empty((pages, 2, HKV, P, D), device="cuda",
                       dtype=torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)
    scales = torch.empty((pages, 2, HKV), dtype=torch.uint8, device="cuda")
    for a in range(0, pages, 4096):
        m = min(4096, pages - a)
        x = torch.randn((m, 2, HKV, P, D), generator=g, device="cuda").mul_(gains[:, :, None])
        x = x.to(torch.bfloat16).float()
        e = _exponent(x.abs().amax((3, 4)), fmt)
        pool[a:a + m] = _encode(x, e[..., None, None], fmt)
        scales[a:a + m] = e.to(torch.uint8)
    return pool, scales


def _buffers(n):
    """K and V of n tokens, for a read to fill."""
    return tuple(torch.empty((n, HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, B = torch.device("cuda"), c["batch"]
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    gains = _gains(g)
    s = {"case": c, "lens": lens}

    def rows(n, kv):
        x = torch.randn((n, HKV, D), generator=g, device=dev) * gains[kv]
        return x.to(torch.bfloat16)

    def queries(n):
        return torch.randn((n, HQ, D), generator=g, device=dev, dtype=torch.bfloat16)

    def offsets(counts):
        return torch.tensor([0] + list(counts), device=dev).cumsum(0).to(torch.int32)

    if c["op"] == "append":
        page = torch.arange(-(-c["ctx"] // P), device=dev)[None, :]
        slots = lens - 1
        s["bt"], pages = _table(page == (slots // P)[:, None], g)
        s["slots"] = slots.contiguous()
        s["pos"] = (torch.randint(0, c["far"], (B,), generator=g, device=dev, dtype=torch.int32)
                    if c["far"] else s["slots"])
        s["k"], s["v"], s["q"] = rows(B, 0), rows(B, 1), queries(B)
        s["q_out"] = torch.empty_like(s["q"])
        # the tokens of the blocks written, to be read back
        s["first"] = (slots // P * P).to(torch.int32)
        s["off"] = offsets([(L - 1) % P + 1 for L in _lens(c)])
        s["back"] = _buffers(sum((L - 1) % P + 1 for L in _lens(c)))
    elif c["op"] in ("write", "read"):
        starts = torch.tensor(_starts(c), dtype=torch.int32, device=dev)
        end = int((starts + lens).max())
        page = torch.arange(-(-end // P), device=dev)[None, :]
        s["bt"], pages = _table((page >= (starts // P)[:, None]) &
                                (page * P < (starts + lens)[:, None]), g)
        s["starts"] = starts
        s["total"] = sum(_lens(c))
        s["off"] = offsets(_lens(c))
        if c["op"] == "write":
            s["k"], s["v"] = rows(s["total"], 0), rows(s["total"], 1)
            # read back: the earlier tokens of a first block too
            s["first"] = (starts // P * P).to(torch.int32)
            counts = [L + f % P for L, f in zip(_lens(c), _starts(c))]
            s["back_off"], s["back"] = offsets(counts), _buffers(sum(counts))
        else:
            s["back"] = _buffers(s["total"])
    else:
        width = -(-c["ctx"] // P) + 1
        page = torch.arange(width, device=dev)[None, :]
        counts = _chunks(c) if c["op"] == "chunk" else [1] * B
        need = page * P < lens[:, None]
        if c["window"]:
            # a serving loop frees the pages that no later step can see
            first = (lens - torch.tensor(counts, device=dev) - c["window"] + 1).clamp(min=0)
            need = need & ((page >= (first // P)[:, None]) | (page * P < c["sinks"]))
        s["bt"], pages = _table(need, g)
        total = B
        if c["op"] == "chunk":
            s["off"] = offsets(counts)
            s["most"] = max(counts)
            total = sum(counts) + c["pad"]
        s["q"] = queries(total)
        s["out"] = torch.zeros_like(s["q"])
        if own:
            from paged_kv_decode_04_gb300 import binding
            n = (binding.chunk8_workspace_bytes(total, B, width, window=c["window"],
                                                sinks=c["sinks"]) if c["op"] == "chunk" else
                 binding.decode8_workspace_bytes(B, width, window=c["window"], sinks=c["sinks"]))
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    s["pool"], s["scales"] = _cache(pages, c["fmt"], gains, g)
    return s


# ------------------------------------------------------------ the own passes --

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _own_append(s):
    from paged_kv_decode_04_gb300 import binding
    binding.kv8_append(s["k"], s["v"], s["pool"], s["scales"], s["bt"], s["pos"], s["slots"],
                       rope_theta=THETA, q_in=s["q"], q_out=s["q_out"])
    k, v = binding.kv8_read(s["off"], s["first"], s["pool"], s["scales"], s["bt"], *s["back"])
    return {"k": k, "v": v, "scales": s["scales"], "q": s["q_out"]}


def _own_write(s):
    from paged_kv_decode_04_gb300 import binding
    binding.kv8_write_prefill(s["k"], s["v"], s["off"], s["starts"], s["pool"], s["scales"],
                              s["bt"], rope_theta=THETA)
    k, v = binding.kv8_read(s["back_off"], s["first"], s["pool"], s["scales"], s["bt"],
                            *s["back"])
    return {"k": k, "v": v, "scales": s["scales"]}


def _own_read(s):
    from paged_kv_decode_04_gb300 import binding
    return binding.kv8_read(s["off"], s["starts"], s["pool"], s["scales"], s["bt"], *s["back"])


def _own_decode(s):
    from paged_kv_decode_04_gb300 import binding
    c = s["case"]
    return binding.paged8_decode_attention(s["q"], s["pool"], s["scales"], s["bt"], s["lens"],
                                           s["out"], window=c["window"], sinks=c["sinks"],
                                           workspace=s["ws"])


def _own_chunk(s):
    from paged_kv_decode_04_gb300 import binding
    c = s["case"]
    return binding.paged8_chunk_attention(s["q"], s["off"], s["pool"], s["scales"], s["bt"],
                                          s["lens"], s["out"], window=c["window"],
                                          sinks=c["sinks"], workspace=s["ws"])


_OWN = dict(append=_own_append, write=_own_write, read=_own_read, decode=_own_decode,
            chunk=_own_chunk)


# ---------------------------------------------------------- the plain passes --

def _exponent(top, fmt):
    """Biased exponent of the smallest power of two s with top <= TOP * s."""
    m, x = torch.frexp(top)
    whole = TOP[fmt] / 2.0 ** math.ceil(math.log2(TOP[fmt]))
    e = x - math.ceil(math.log2(TOP[fmt])) + (m > whole).int() + BIAS
    return torch.where(top == 0, LEAST, e).clamp(LEAST, MOST)


def _pow2(e):
    """2^e in 32 bits (-126 <= e <= 127)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, e, fmt):
    """Codes of the values x under the scales 2^(e - BIAS) (an exact division)."""
    y = (x * _pow2(BIAS - e)).clamp(-TOP[fmt], TOP[fmt])
    return y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)


def _rotate(x, pos):
    """Rotate-half RoPE of [n][heads][64] at positions [n], angles in 64 bits,
    rounded to bf16."""
    half = D // 2
    f = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    a = pos.double()[:, None, None] * f
    c, n = a.cos(), a.sin()
    out = torch.empty_like(x)
    for h in range(x.shape[1]):
        x1, x2 = x[:, h:h + 1, :half].double(), x[:, h:h + 1, half:].double()
        out[:, h:h + 1, :half] = (x1 * c - x2 * n).to(x.dtype)
        out[:, h:h + 1, half:] = (x2 * c + x1 * n).to(x.dtype)
    return out


def _put(s, k, v, page, slot, first):
    """Write rows k, v [n][8][64] to (page, slot) [n]: every block named takes
    its rows at once.  `first` [n] is the lowest slot that its page is given;
    the slots before it hold earlier tokens."""
    fmt, pool, scales = s["case"]["fmt"], s["pool"], s["scales"]
    ids, block = torch.unique(page, return_inverse=True)                 # pages written
    n = ids.numel()
    before = torch.zeros(n, dtype=torch.long, device=page.device).scatter_(0, block, first)
    top = torch.zeros((n, 2, HKV), device=page.device)
    for kv, x in enumerate((k, v)):
        most = x.float().abs().amax(-1)                                  # [rows][8]
        top[:, kv].scatter_reduce_(0, block[:, None].expand_as(most), most, "amax")
    e = _exponent(top, fmt)
    old = scales[ids].int()
    e = torch.where((before > 0)[:, None, None], torch.maximum(e, old), e)
    # the earlier tokens under the new scale
    raw = pool.view(torch.uint8)
    codes = raw[ids]
    value = codes.view(pool.dtype).float() * _pow2(old - BIAS)[..., None, None]
    again = _encode(value, e[..., None, None], fmt)
    keep = (torch.arange(P, device=page.device) < before[:, None])[:, None, None, :, None]
    raw[ids] = torch.where(keep, again.view(torch.uint8), codes)
    scales[ids] = e.to(torch.uint8)
    for kv, x in enumerate((k, v)):
        raw[page, kv, :, slot] = _encode(x.float(), e[block, kv][..., None], fmt).view(torch.uint8)


def _rows_of(off, starts, bt, total):
    """Page, slot and position of each of `total` tokens, sequence b's
    off[b] .. off[b + 1] standing at starts[b] and on."""
    r = torch.arange(total, device=off.device)
    b = torch.searchsorted(off.long(), r, right=True) - 1
    pos = starts.long()[b] + r - off.long()[b]
    return bt[b, pos // P].long(), pos % P, pos, b


def _read(s, off, starts, total):
    page, slot, _, _ = _rows_of(off, starts, s["bt"], total)
    out = []
    for kv in range(2):
        codes = s["pool"].view(torch.uint8)[page, kv, :, slot].view(s["pool"].dtype)  # [n][8][64]
        scale = _pow2(s["scales"][page, kv].int() - BIAS)
        out.append((codes.float() * scale[..., None]).to(torch.bfloat16))
    return out[0], out[1]


def _plain_append(s):
    slot = s["slots"].long()
    page = torch.gather(s["bt"], 1, (slot // P)[:, None])[:, 0].long()
    _put(s, _rotate(s["k"], s["pos"]), s["v"], page, slot % P, slot % P)
    k, v = _read(s, s["off"], s["first"], s["back"][0].shape[0])
    return {"k": k, "v": v, "scales": s["scales"], "q": _rotate(s["q"], s["pos"])}


def _plain_write(s):
    page, slot, pos, b = _rows_of(s["off"], s["starts"], s["bt"], s["total"])
    first = torch.where(pos // P == s["starts"].long()[b] // P, s["starts"].long()[b] % P, 0)
    _put(s, _rotate(s["k"], pos), s["v"], page, slot, first)
    k, v = _read(s, s["back_off"], s["first"], s["back"][0].shape[0])
    return {"k": k, "v": v, "scales": s["scales"]}


def _plain_read(s):
    return _read(s, s["off"], s["starts"], s["total"])


def _cached(s, tokens):
    """K and V of the cached tokens [B][T] (positions) as [B][8][T][64]."""
    page = torch.gather(s["bt"], 1, tokens // P).long().clamp(min=0)
    slot = tokens % P
    raw = s["pool"].view(torch.uint8)
    out = []
    for kv in range(2):
        codes = raw[page, kv, :, slot].view(s["pool"].dtype).float()     # [B][T][8][64]
        scale = _pow2(s["scales"][page, kv].int() - BIAS)
        out.append((codes * scale[..., None]).permute(0, 2, 1, 3))
    return out


def _softmax(x, mask):
    """Softmax over the last axis of the masked scores, in place."""
    x.masked_fill_(~mask, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    return x.div_(x.sum(-1, keepdim=True).clamp(min=1e-30))


def _plain_decode(s):
    c, lens = s["case"], s["lens"].long()
    B, W = c["batch"], min(c["window"] or c["ctx"], c["ctx"])
    first = (lens - W).clamp(min=0)[:, None]
    near = first + torch.arange(W, device=lens.device)
    sink = torch.arange(min(c["sinks"], c["ctx"]), device=lens.device).expand(B, -1)
    tokens = torch.cat([sink, near], 1)
    mask = torch.cat([sink < first, near < lens[:, None]], 1)
    k, v = _cached(s, torch.where(mask, tokens, lens[:, None] - 1))
    q = s["q"].float().reshape(B, HKV, G, D)
    p = _softmax(torch.matmul(q, k.transpose(2, 3)).mul_(SCALE), mask[:, None, None])
    return torch.matmul(p, v).reshape(B, HQ, D).to(torch.bfloat16)


def _plain_chunk(s):
    c, lens, off = s["case"], s["lens"].long(), s["off"].long()
    B, N, T = c["batch"], s["most"], c["ctx"]
    dev = lens.device
    counts = off[1:] - off[:-1]
    i = torch.arange(N, device=dev)
    row = (off[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)           # [B][N] rows of q
    q = s["q"][row].float().reshape(B, N, HKV, G, D).permute(0, 2, 3, 1, 4)
    t = torch.arange(T, device=dev)
    k, v = _cached(s, t.expand(B, T))
    x = torch.matmul(q.reshape(B, HKV, G * N, D), k.transpose(2, 3)).mul_(SCALE)
    pos = (lens - counts)[:, None] + i                                   # [B][N]
    mask = t <= pos[..., None]
    if c["window"]:
        mask = mask & ((t > pos[..., None] - c["window"]) | (t < c["sinks"]))
    p = _softmax(x.reshape(B, HKV, G, N, T), mask[:, None, None])
    o = torch.matmul(p.reshape(B, HKV, G * N, T), v)
    o = o.reshape(B, HKV, G, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, HQ, D).to(torch.bfloat16)
    # each row of the output takes its token's result; rows of no token keep theirs
    r = torch.arange(s["q"].shape[0], device=dev)
    b = (torch.searchsorted(off, r, right=True) - 1).clamp(0, B - 1)
    j = (r - off[b]).clamp(max=N - 1)
    return torch.where((r < off[-1])[:, None, None], o[b, j], s["out"])


_PLAIN = dict(append=_plain_append, write=_plain_write, read=_plain_read, decode=_plain_decode,
              chunk=_plain_chunk)


# ------------------------------------------------- the definition in 64 bits --
# Values and scales in 64 bits; the roundings that the cache is defined by (a
# key to bf16, values to codes) are made explicitly, on numbers that 64 bits
# hold exactly.

@functools.lru_cache
def _powers(device):
    return torch.tensor([2.0 ** i for i in range(-400, 401)], dtype=torch.float64, device=device)


def _two_to(k):
    """2^k in 64 bits for whole k in [-400, 400]."""
    return _powers(k.device)[k.long() + 400]


def _round_code(y, fmt):
    """y rounded to the nearest code, ties to even, within the format's range."""
    y = y.clamp(-TOP[fmt], TOP[fmt])
    if fmt == "int8":
        return torch.round(y)
    # spacing of e4m3: 2^-9 below 2^-6, 2^(exponent - 3) above
    _, x = torch.frexp(y)
    step = _two_to((x - 4).clamp(min=-9))
    return torch.round(y / step) * step


def _round_bf16(y):
    """y rounded once to bf16's eight significant bits (normal numbers)."""
    _, x = torch.frexp(y)
    step = _two_to((x - 8).clamp(min=-133))
    return torch.round(y / step) * step


def _turn(x, pos):
    """RoPE of [n][heads][64] as a product of complex numbers."""
    f = torch.exp(-math.log(THETA) * torch.arange(D // 2, device=x.device, dtype=torch.float64) /
                  (D // 2))
    z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double())
    z = z * torch.polar(torch.ones_like(f), pos.double()[:, None, None] * f)
    return torch.cat([z.real, z.imag], -1)


def _exact_block(c, old, old_scale, rows):
    """A block [8][16][64] of earlier values `old` [8][m][64] (scale 2^(old_scale
    - 127) [8]) given the rows [8][r][64]: the values it stands for and its
    scale exponents."""
    reach = TOP[c["fmt"]] * _two_to(torch.arange(LEAST, MOST, device=rows.device) - BIAS)
    fit = torch.searchsorted(reach, rows.abs().amax((1, 2))) + LEAST      # smallest that reaches
    if old.shape[1]:
        fit = torch.maximum(fit, old_scale.long())
    s = _two_to(fit - BIAS)[:, None, None]
    return _round_code(torch.cat([old, rows], 1) / s, c["fmt"]) * s, fit


def _exact_written(s, c, keys, starts, counts):
    """Values of every token of the blocks that tokens starts[b] .. + counts[b]
    of each sequence went to, in order, and the scales of all blocks."""
    scales = s["scales"].clone()
    out = ([], [])
    at = 0
    for b, (f, n) in enumerate(zip(starts, counts)):
        for page0 in range(f // P * P, f + n, P):
            page = int(s["bt"][b, page0 // P])
            lo, hi = max(f, page0), min(f + n, page0 + P)
            for kv, x in enumerate((keys, s["v"].double())):
                rows = x[at + lo - f:at + hi - f].transpose(0, 1)
                e = s["scales"][page, kv]
                old = s["pool"][page, kv, :, :lo - page0].double() * _two_to(
                    e.long() - BIAS)[:, None, None]
                new, fit = _exact_block(c, old, e, rows)
                scales[page, kv] = fit.to(torch.uint8)
                out[kv].append(new.transpose(0, 1))
        at += n
    return {"k": torch.cat(out[0]), "v": torch.cat(out[1]), "scales": scales}


def _exact_rows(s, b, tokens):
    """K and V [8][T][64] of the cached tokens of sequence b, in 64 bits."""
    pages, slot = s["bt"][b].long()[tokens // P], tokens % P
    out = []
    for kv in range(2):
        codes = s["pool"].view(torch.uint8)[pages, kv, :, slot].view(s["pool"].dtype).double()
        scale = _two_to(s["scales"][pages, kv].long() - BIAS)
        out.append((codes * scale[..., None]).transpose(0, 1))
    return out


def _exact_attend(q, k, v, hide=None):
    """Outputs of query rows [8][R][64] over [8][T][64]."""
    z = q @ k.transpose(1, 2) / math.sqrt(D)
    if hide is not None:
        z = z.masked_fill(hide, -math.inf)
    return torch.softmax(z, -1) @ v


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    dev, lens = s["lens"].device, _lens(c)
    if c["op"] == "append":
        keys = _round_bf16(_turn(s["k"], s["pos"]))
        return dict(_exact_written(s, c, keys, [L - 1 for L in lens], [1] * len(lens)),
                    q=_turn(s["q"], s["pos"]))
    if c["op"] == "write":
        pos = torch.cat([f + torch.arange(n, device=dev) for f, n in zip(_starts(c), lens)])
        return _exact_written(s, c, _round_bf16(_turn(s["k"], pos)), _starts(c), lens)
    if c["op"] == "read":
        both = [_exact_rows(s, b, f + torch.arange(n, device=dev))
                for b, (f, n) in enumerate(zip(_starts(c), lens))]
        return tuple(torch.cat([r[kv].transpose(0, 1) for r in both]) for kv in range(2))
    if c["op"] == "decode":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        for b, L in enumerate(lens):
            t = torch.arange(L, device=dev)
            if c["window"]:
                t = t[(t >= L - c["window"]) | (t < c["sinks"])]
            k, v = _exact_rows(s, b, t)
            out[b] = _exact_attend(s["q"][b].double().reshape(HKV, G, D), k, v).reshape(HQ, D)
        return out
    out = s["out"].double()
    at = 0
    for b, (L, n) in enumerate(zip(lens, _chunks(c))):
        for a in range(0, n, 512):                                       # query tokens at a time
            m = min(512, n - a)
            lo = L - n + a
            back = max(0, lo - c["window"] + 1) if c["window"] else 0
            t = torch.cat([torch.arange(min(c["sinks"], back), device=dev),
                           torch.arange(back, lo + m, device=dev)])
            pos = torch.arange(lo, lo + m, device=dev)[:, None]
            hide = t > pos
            if c["window"]:
                hide = hide | ((pos - t >= c["window"]) & (t >= c["sinks"]))
            k, v = _exact_rows(s, b, t)
            q = s["q"][at + a:at + a + m].double().reshape(m, HKV, G, D)
            q = q.permute(1, 2, 0, 3).reshape(HKV, G * m, D)
            o = _exact_attend(q, k, v, hide.repeat(G, 1))
            out[at + a:at + a + m] = o.reshape(HKV, G, m, D).permute(2, 0, 1, 3).reshape(m, HQ, D)
        at += n
    return out
