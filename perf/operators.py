"""Timed cases of the long-context operators over the paged KV cache.

Five operators, each in its plain form (elementary torch operations in 32
bits, 64 where angles need them) and as the library call a serving loop makes:

  chunk   attention of a ragged chunk of new tokens over the paged cache,
          causal, optionally with a sliding window and sink tokens
  window  one-token decode attention with a sliding window and sink tokens
  scored  one-token decode attention that adds each cached token's attention
          weight to a running mass per (sequence, kv head)
  evict   keeping the sinks, the most recent tokens and the heaviest others of
          each kv head, packed into fresh pages
  append  the one-token append at a cache slot that is not the RoPE position
          (what a cache that has been evicted from needs)

Geometry as everywhere in this library: 32 query heads, 8 kv heads of 64 dims,
pages of 16 tokens, bf16 pool [pages][K|V][16][8][64].
"""
import math

import torch

own = False

HQ, HKV, G, D, P = 32, 8, 4, 64, 16
SCALE = D ** -0.5
THETA = 500000.0
NEVER = 2 ** 31 - 1


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # verifying four drafted tokens of 64 sequences at once: the cache is
        # read once for few rows (memory-bound)
        dict(name="chunk verify", op="chunk", batch=64, ctx=2048, tokens=4, singles=0, window=0,
             sinks=0, pad=3),
        # the second half of two long prompts, prefilled in one chunk each
        # (compute-bound, the largest case)
        dict(name="chunk prefill", op="chunk", batch=2, ctx=8192, tokens=4096, singles=0,
             window=0, sinks=0, pad=0),
        # continuous batching: a prompt chunk beside 63 decoding sequences
        dict(name="chunk mixed", op="chunk", batch=64, ctx=2047, tokens=509, singles=63, window=0,
             sinks=0, pad=0),
        # a whole long prompt under a sliding window with four sinks
        dict(name="chunk window", op="chunk", batch=1, ctx=8192, tokens=8192, singles=0,
             window=1024, sinks=4, pad=0),
        # one long conversation decoding under a window (latency)
        dict(name="window one", op="window", batch=1, ctx=30011, window=1024, sinks=4),
        # a full decode batch far past its window
        dict(name="window batch", op="window", batch=256, ctx=16384, window=1000, sinks=4),
        # one sequence whose weights are tracked (latency, split over the axis)
        dict(name="scored one", op="scored", batch=1, ctx=4093),
        # a decode batch whose weights are tracked
        dict(name="scored batch", op="scored", batch=128, ctx=2048),
        # halving one sequence's cache
        dict(name="evict one", op="evict", batch=1, ctx=2049, budget=1024, sinks=4, recent=128),
        # a batch brought back to a quarter of its cache
        dict(name="evict batch", op="evict", batch=64, ctx=4096, budget=1024, sinks=4, recent=256),
        # the next token of one evicted cache, with its query rotation
        dict(name="append one", op="append", batch=1, ctx=2048, far=9001),
        # the next token of a large batch at positions far past its slots
        dict(name="append batch", op="append", batch=2048, ctx=1024, far=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "window", "scored", "evict", "append"])
    if op == "chunk":
        batch = _log(rng, 1, 128)
        tokens = _log(rng, 1, 4096)
        ctx = max(tokens, _log(rng, 1, 16384))
        while batch * tokens * ctx > 2 * 4096 * 8192 or batch * ctx > 1 << 20:
            batch = max(1, batch // 2)
            if batch == 1:
                tokens = max(1, tokens // 2)
                ctx = max(tokens, ctx * 3 // 4)
        window = _log(rng, 1, 4096) if rng.random() < 0.5 else 0
        return dict(op=op, batch=batch, ctx=ctx, tokens=tokens,
                    singles=rng.randrange(batch) if rng.random() < 0.4 else 0, window=window,
                    sinks=rng.randrange(0, 200) if window and rng.random() < 0.7 else 0,
                    pad=rng.randrange(0, 9))
    if op == "window":
        batch, window, sinks = _log(rng, 1, 256), _log(rng, 1, 8192), rng.randrange(0, 130)
        while batch * (window + sinks) > 1 << 19:
            batch //= 2
        return dict(op=op, batch=batch, ctx=_log(rng, 1, 131072), window=window, sinks=sinks)
    if op == "scored":
        batch, ctx = _log(rng, 1, 128), _log(rng, 1, 32768)
        while batch * ctx > 1 << 19:
            batch //= 2
        return dict(op=op, batch=batch, ctx=ctx)
    if op == "evict":
        batch, ctx = _log(rng, 1, 64), _log(rng, 32, 32768)
        while batch * ctx > 1 << 19:
            batch //= 2
        budget = _log(rng, 16, ctx)
        sinks = rng.randrange(0, min(65, budget // 4 + 1))
        return dict(op=op, batch=batch, ctx=ctx, budget=budget, sinks=sinks,
                    recent=rng.randrange(0, (budget - sinks) // 2 + 1))
    return dict(op=op, batch=_log(rng, 1, 2048), ctx=_log(rng, 1, 4096),
                far=_log(rng, 4096, 1 << 20))


def _lens(c):
    """Cached tokens of each sequence: the first has ctx, the others spread
    over the upper half of the range."""
    return [max(1, c["ctx"] - (i * 617) % (c["ctx"] // 2 + 1)) for i in range(c["batch"])]


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
    B, row = c["batch"], HKV * D * 2
    if c["op"] == "chunk":
        read = pairs = 0
        for L, n in zip(_lens(c), _chunks(c)):
            pairs += sum(_visible(p, c["window"], c["sinks"]) for p in range(L - n, L))
            lo = max(0, L - n - c["window"] + 1) if c["window"] else 0
            read += L - lo + min(c["sinks"], lo)
        tokens = sum(_chunks(c))
        return {"bytes": 2 * row * read + 2 * tokens * HQ * D * 2 + 4 * (read // P + 2 * B + 1),
                "flops": 4 * D * HQ * pairs}
    if c["op"] == "window":
        read = sum(_visible(L - 1, c["window"], c["sinks"]) for L in _lens(c))
        return {"bytes": 2 * row * read + 2 * B * HQ * D * 2 + 4 * (read // P + B),
                "flops": 4 * D * HQ * read}
    if c["op"] == "scored":
        read = sum(_lens(c))
        return {"bytes": 2 * row * read + 8 * HKV * read + 2 * B * HQ * D * 2 + 4 * (read // P + B),
                "flops": 4 * D * HQ * read}
    if c["op"] == "evict":
        kept = sum(min(L, c["budget"]) for L in _lens(c))
        read = sum(_lens(c))
        return {"bytes": 4 * row * kept + 4 * HKV * read + 8 * HKV * kept +
                4 * (read // P + kept // P + 2 * B), "flops": 0}
    return {"bytes": B * (4 * row + 2 * HQ * D * 2 + 12), "flops": 3 * B * (HQ + HKV) * D}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(need, width, g, spare=7):
    """Block tables naming shuffled pages where need [B][width] is true, -1
    elsewhere, and the pages of a pool that holds them."""
    pages = int(need.sum()) + spare
    ids = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    at = (torch.cumsum(need.reshape(-1).long(), 0) - 1).clamp(min=0)
    return torch.where(need.reshape(-1), ids[at], -1).reshape(need.shape).contiguous(), pages


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def prepare(case, seed):
    c, g = case, _gen(seed)
    dev, B = torch.device("cuda"), case["batch"]
    lens_h = _lens(c)
    lens = torch.tensor(lens_h, dtype=torch.int32, device=dev)
    s = {"case": c, "lens": lens}
    width = -(-c["ctx"] // P) + 1
    page = torch.arange(width, device=dev)[None, :]
    live = page < ((lens + P - 1) // P)[:, None]
    if c["op"] == "chunk":
        counts = _chunks(c)
        off = [0]
        for n in counts:
            off.append(off[-1] + n)
        total = off[-1] + c["pad"]
        s["off"] = torch.tensor(off, dtype=torch.int32, device=dev)
        s["bt"], pages = _table(live, width, g)
        s["pool"] = _normal((pages, 2, P, HKV, D), g)
        s["q"] = _normal((total, HQ, D), g)
        s["out"] = torch.zeros((total, HQ, D), dtype=torch.bfloat16, device=dev)
        s["most"] = max(counts)
        if own:
            from paged_kv_decode_04_gb300 import binding
            s["ws"] = _workspace(binding.chunk_workspace_bytes(
                total, B, width, window=c["window"], sinks=c["sinks"]))
    elif c["op"] == "window":
        # a serving loop frees the pages that no later step can see
        first = (lens - c["window"]).clamp(min=0)
        need = live & ((page >= (first // P)[:, None]) | (page * P < c["sinks"]))
        s["bt"], pages = _table(need, width, g)
        s["pool"] = _normal((pages, 2, P, HKV, D), g)
        s["q"] = _normal((B, HQ, D), g)
        s["out"] = torch.empty_like(s["q"])
        if own:
            from paged_kv_decode_04_gb300 import binding
            s["ws"] = _workspace(binding.window_workspace_bytes(B, width, c["window"],
                                                                sinks=c["sinks"]))
    elif c["op"] == "scored":
        s["bt"], pages = _table(live, width, g)
        s["pool"] = _normal((pages, 2, P, HKV, D), g)
        s["q"] = _normal((B, HQ, D), g)
        s["out"] = torch.empty_like(s["q"])
        s["mass"] = torch.rand((B, HKV, width * P), generator=g, device=dev) * (
            torch.arange(width * P, device=dev)[None, None, :] < lens[:, None, None])
        if own:
            from paged_kv_decode_04_gb300 import binding
            s["ws"] = _workspace(binding.scored_workspace_bytes(B, width))
    elif c["op"] == "evict":
        wide = -(-c["budget"] // P)
        both, pages = _table(torch.cat([live, torch.ones((B, wide), dtype=torch.bool,
                                                         device=dev)], 1), width, g)
        s["bt"], s["dst"] = both[:, :width].contiguous(), both[:, width:].contiguous()
        s["pool"] = _normal((pages, 2, P, HKV, D), g)
        # summed attention weights: heavy-tailed, and equal for many tokens
        mass = torch.exp(1.5 * torch.randn((B, HKV, width * P), generator=g, device=dev))
        s["mass"] = torch.where(mass < 2.0, torch.round(mass * 64) / 64, mass)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
        s["new_mass"] = torch.empty((B, HKV, wide * P), device=dev)
        s["kept"] = torch.empty((B, HKV, c["budget"]), dtype=torch.int32, device=dev)
    else:
        slots = (lens - 1).to(torch.int32)
        need = page == (slots // P)[:, None]
        s["bt"], pages = _table(need, width, g)
        s["slots"] = slots.contiguous()
        s["pos"] = torch.randint(0, c["far"], (B,), generator=g, device=dev, dtype=torch.int32)
        s["pool"] = _normal((pages, 2, P, HKV, D), g)
        s["k"], s["v"] = _normal((B, HKV, D), g), _normal((B, HKV, D), g)
        s["q"] = _normal((B, HQ, D), g)
        s["q_out"] = torch.empty_like(s["q"])
    return s


def _workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


# --------------------------------------------------------------- the passes --

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_chunk(s):
    from paged_kv_decode_04_gb300 import binding
    c = s["case"]
    return binding.paged_chunk_attention(s["q"], s["off"], s["pool"], s["bt"], s["lens"],
                                         s["out"], window=c["window"], sinks=c["sinks"],
                                         workspace=s["ws"])


def _own_window(s):
    from paged_kv_decode_04_gb300 import binding
    c = s["case"]
    return binding.paged_window_attention(s["q"], s["pool"], s["bt"], s["lens"], c["window"],
                                          s["out"], sinks=c["sinks"], workspace=s["ws"])


def _own_scored(s):
    from paged_kv_decode_04_gb300 import binding
    out = binding.paged_scored_attention(s["q"], s["pool"], s["bt"], s["lens"], s["mass"],
                                         s["out"], workspace=s["ws"])
    return {"out": out, "mass": s["mass"]}


def _own_evict(s):
    from paged_kv_decode_04_gb300 import binding
    c = s["case"]
    lens, mass, kept = binding.kv_evict(s["mass"], s["pool"], s["bt"], s["lens"], s["dst"],
                                        s["new_lens"], s["new_mass"], s["kept"],
                                        budget=c["budget"], sinks=c["sinks"], recent=c["recent"])
    return {"lens": lens, "mass": mass, "kept": kept, "pool": s["pool"]}


def _own_append(s):
    from paged_kv_decode_04_gb300 import binding
    binding.kv_append_at(s["k"], s["v"], s["pool"], s["bt"], s["pos"], s["slots"],
                         rope_theta=THETA, q_in=s["q"], q_out=s["q_out"])
    return {"pool": s["pool"], "q": s["q_out"]}


_OWN = dict(chunk=_own_chunk, window=_own_window, scored=_own_scored, evict=_own_evict,
            append=_own_append)


def _cached(pool, bt, tokens):
    """K and V of the cached tokens [B][T] (positions), in 32 bits."""
    page = torch.gather(bt, 1, tokens // P).long().clamp(min=0)
    slot = tokens % P
    return pool[page, 0, slot].float(), pool[page, 1, slot].float()     # [B][T][8][64]


def _softmax(x, mask):
    """Softmax over the last axis of the masked scores, in place."""
    x.masked_fill_(~mask, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    return x.div_(x.sum(-1, keepdim=True).clamp(min=1e-30))


def _plain_chunk(s):
    c, lens, off = s["case"], s["lens"].long(), s["off"].long()
    B, N, T = c["batch"], s["most"], c["ctx"]
    dev = lens.device
    counts = off[1:] - off[:-1]
    i = torch.arange(N, device=dev)
    row = (off[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)           # [B][N] rows of q
    q = s["q"][row].float().reshape(B, N, HKV, G, D).permute(0, 2, 3, 1, 4)
    t = torch.arange(T, device=dev)
    k, v = _cached(s["pool"], s["bt"], t.expand(B, T))
    x = torch.matmul(q.reshape(B, HKV, G * N, D), k.permute(0, 2, 3, 1)).mul_(SCALE)
    pos = (lens - counts)[:, None] + i                                   # [B][N]
    mask = t <= pos[..., None]
    if c["window"]:
        mask = mask & ((t > pos[..., None] - c["window"]) | (t < c["sinks"]))
    p = _softmax(x.reshape(B, HKV, G, N, T), mask[:, None, None])
    o = torch.matmul(p.reshape(B, HKV, G * N, T), v.permute(0, 2, 1, 3))
    o = o.reshape(B, HKV, G, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, HQ, D).to(torch.bfloat16)
    # each row of the output takes its token's result; rows of no token keep theirs
    r = torch.arange(s["q"].shape[0], device=dev)
    b = (torch.searchsorted(off, r, right=True) - 1).clamp(0, B - 1)
    j = (r - off[b]).clamp(max=N - 1)
    return torch.where((r < off[-1])[:, None, None], o[b, j], s["out"])


def _plain_one(q, pool, bt, tokens, mask):
    """One query token per sequence over the cached tokens [B][T]: the output
    and the weights [B][8][4][T]."""
    B, T = tokens.shape
    k, v = _cached(pool, bt, tokens)
    x = torch.matmul(q.float().reshape(B, HKV, G, D), k.permute(0, 2, 3, 1)).mul_(SCALE)
    p = _softmax(x, mask[:, None, None])
    return torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(B, HQ, D).to(torch.bfloat16), p


def _plain_window(s):
    c, lens = s["case"], s["lens"].long()
    W = min(c["window"], c["ctx"])
    first = (lens - W).clamp(min=0)[:, None]
    near = first + torch.arange(W, device=lens.device)
    sink = torch.arange(min(c["sinks"], c["ctx"]), device=lens.device).expand(c["batch"], -1)
    tokens = torch.cat([sink, near], 1)
    mask = torch.cat([sink < first, near < lens[:, None]], 1)
    tokens = torch.where(mask, tokens, lens[:, None] - 1)
    return _plain_one(s["q"], s["pool"], s["bt"], tokens, mask)[0]


def _plain_scored(s):
    c, lens = s["case"], s["lens"].long()
    t = torch.arange(c["ctx"], device=lens.device).expand(c["batch"], -1)
    out, p = _plain_one(s["q"], s["pool"], s["bt"], t, t < lens[:, None])
    s["mass"][..., :c["ctx"]] += p.sum(2)
    return {"out": out, "mass": s["mass"]}


def _plain_evict(s):
    c, lens = s["case"], s["lens"].long()
    T, K = s["mass"].shape[2], c["budget"]
    t = torch.arange(T, device=lens.device)
    L = lens[:, None, None]
    always = (t < c["sinks"]) | (t >= L - c["recent"])
    rank = torch.where(always, math.inf, s["mass"])
    rank = torch.where(t < L, rank, -math.inf)
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)
    if K > T:
        order = torch.cat([order, order.new_full((*order.shape[:2], K - T), NEVER)], -1)
    kept = torch.where(order[..., :K] < L, order[..., :K], NEVER).sort(-1).values
    valid = kept < NEVER                                                 # [B][8][K]
    src = torch.where(valid, kept, 0)
    b = torch.arange(c["batch"], device=lens.device)[:, None, None]
    h = torch.arange(HKV, device=lens.device)[None, :, None]
    i = torch.arange(K, device=lens.device)
    dpage = s["dst"][:, i // P].long()[:, None, :].expand_as(kept)
    spage = s["bt"][b, src // P].long()
    page, slot = torch.where(valid, spage, dpage), torch.where(valid, src % P, i % P)
    rows = s["pool"][page, :, slot, h]                                   # [B][8][K][2][64]
    s["pool"][dpage, :, (i % P).expand_as(kept), h.expand_as(kept)] = rows
    mass = torch.zeros_like(s["new_mass"])
    mass[..., :K] = torch.where(valid, torch.gather(s["mass"], 2, src), 0.0)
    return {"lens": lens.clamp(max=K).to(torch.int32), "mass": mass,
            "kept": torch.where(valid, kept, -1).to(torch.int32), "pool": s["pool"]}


def _rotate(x, pos):
    """Rotate-half RoPE of [B][heads][64] at positions [B], angles in 64 bits."""
    half = D // 2
    f = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    a = pos.double()[:, None, None] * f
    x1, x2 = x[..., :half].double(), x[..., half:].double()
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()],
                     -1).to(torch.bfloat16)


def _plain_append(s):
    slot = s["slots"].long()
    page = torch.gather(s["bt"], 1, (slot // P)[:, None])[:, 0].long()
    s["pool"][page, 0, slot % P] = _rotate(s["k"], s["pos"])
    s["pool"][page, 1, slot % P] = s["v"]
    return {"pool": s["pool"], "q": _rotate(s["q"], s["pos"])}


_PLAIN = dict(chunk=_plain_chunk, window=_plain_window, scored=_plain_scored, evict=_plain_evict,
              append=_plain_append)


# ------------------------------------------------- the definition in 64 bits --

def _exact_rows(s, b, tokens):
    """K and V [8][T][64] of the cached tokens of sequence b, in 64 bits."""
    pages = s["bt"][b].long()[tokens // P]
    rows = s["pool"][pages, :, tokens % P].double()                      # [T][2][8][64]
    return rows[:, 0].transpose(0, 1), rows[:, 1].transpose(0, 1)


def _exact_attend(q, k, v, hide=None):
    """Weights and outputs of query rows [8][R][64] over [8][T][64]."""
    z = q @ k.transpose(1, 2) / math.sqrt(D)
    if hide is not None:
        z = z.masked_fill(hide, -math.inf)
    w = torch.softmax(z, -1)
    return w, w @ v


def exact(case, seed):
    s = prepare(case, seed)
    c, dev = case, s["lens"].device
    lens = _lens(c)
    if c["op"] == "chunk":
        out = s["out"].double()
        at = 0
        for b, (L, n) in enumerate(zip(lens, _chunks(c))):
            for a in range(0, n, 512):                                   # query tokens at a time
                m = min(512, n - a)
                lo = L - n + a
                hi = lo + m
                back = max(0, lo - c["window"] + 1) if c["window"] else 0
                t = torch.cat([torch.arange(min(c["sinks"], back), device=dev),
                               torch.arange(back, hi, device=dev)])
                pos = torch.arange(lo, hi, device=dev)[:, None]
                hide = t > pos
                if c["window"]:
                    hide = hide | ((pos - t >= c["window"]) & (t >= c["sinks"]))
                k, v = _exact_rows(s, b, t)
                q = s["q"][at + a:at + a + m].double().reshape(m, HKV, G, D)
                q = q.permute(1, 2, 0, 3).reshape(HKV, G * m, D)
                o = _exact_attend(q, k, v, hide.repeat(G, 1))[1]
                out[at + a:at + a + m] = o.reshape(HKV, G, m, D).permute(2, 0, 1, 3).reshape(
                    m, HQ, D)
            at += n
        return out
    if c["op"] in ("window", "scored"):
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        mass = s["mass"].double() if c["op"] == "scored" else None
        for b, L in enumerate(lens):
            t = torch.arange(L, device=dev)
            if c["op"] == "window":
                t = t[(t >= L - c["window"]) | (t < c["sinks"])]
            k, v = _exact_rows(s, b, t)
            w, o = _exact_attend(s["q"][b].double().reshape(HKV, G, D), k, v)
            out[b] = o.reshape(HQ, D)
            if mass is not None:
                mass[b, :, :L] += w.sum(1)
        return out if mass is None else {"out": out, "mass": mass}
    if c["op"] == "evict":
        # what is kept is whole; the masses and rows that come with it are copies
        mass = torch.zeros(s["new_mass"].shape, dtype=torch.float64, device=dev)
        pool = s["pool"].clone()
        kept_all = torch.full(s["kept"].shape, -1, dtype=torch.int32, device=dev)
        for b, L in enumerate(lens):
            n = min(L, c["budget"])
            for h in range(HKV):
                m = s["mass"][b, h, :L].double().clone()
                m[:min(c["sinks"], L)] = math.inf
                m[max(0, L - c["recent"]):] = math.inf
                top = torch.sort(-m, stable=True).indices[:n]
                kept = torch.sort(top).values
                kept_all[b, h, :n] = kept.to(torch.int32)
                mass[b, h, :n] = s["mass"][b, h][kept].double()
                at = torch.arange(n, device=dev)
                rows = s["pool"][s["bt"][b].long()[kept // P], :, kept % P, h]
                pool[s["dst"][b].long()[at // P], :, at % P, h] = rows
        return {"lens": torch.tensor([min(L, c["budget"]) for L in lens], dtype=torch.int32,
                                     device=dev), "mass": mass, "kept": kept_all, "pool": pool}
    # append: the rotation as a product of complex numbers
    f = torch.exp(-math.log(THETA) * torch.arange(D // 2, device=dev, dtype=torch.float64) /
                  (D // 2))
    turn = torch.polar(torch.ones_like(f), s["pos"].double()[:, None, None] * f)

    def rot(x):
        z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double()) * turn
        return torch.cat([z.real, z.imag], -1)

    pool = s["pool"].double()
    page = s["bt"].long()[torch.arange(c["batch"], device=dev), s["slots"].long() // P]
    pool[page, 0, s["slots"].long() % P] = rot(s["k"])
    pool[page, 1, s["slots"].long() % P] = s["v"].double()
    return {"pool": pool, "q": rot(s["q"])}
