"""Performance cases of the operators that serve from a block-scaled fp8 paged cache.

Four operators, used one after the other in a serving step:

  page_map  block tables and slot maps from request lengths and a free list
  append    bf16 key / value rows written into the fp8 cache, one power-of-two
            scale per (block of tokens, KV head)
  decode    one query per sequence over that cache, learned sinks in the softmax
  prefill   packed query rows over that cache

`run` computes a case with elementary torch operations in float32, or, with
`own` set, with this library's calls. `exact` computes it in float64 with
code of its own.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 60  # exponents of the scales that append writes


# ---------------------------------------------------------------- the cases

def _case(op, name, **kw):
    c = {"name": name, "op": op, "len_seed": 1}
    c.update(kw)
    return c


def listed():
    return [
        # one decode step's bookkeeping: 256 running requests, one new token each
        _case("page_map", "map_step", batch=256, new_lo=1, new_hi=1, old_lo=1024, old_hi=32768,
              page=16),
        # a large mixed batch: half a million new tokens in ragged chunks, many new pages
        _case("page_map", "map_chunks", batch=250, new_lo=1, new_hi=4096, old_lo=0, old_hi=8192,
              page=16),
        # a decode step's cache write: 64 requests, one token each, blocks that
        # already hold older tokens
        _case("append", "append_step", batch=64, new_lo=1, new_hi=1, old_lo=1024, old_hi=8192,
              page=16, block=16, hkv=8, dim=64, fused=True),
        # ragged chunks of 16 requests, head_dim 128, several blocks per page
        _case("append", "append_chunks", batch=16, new_lo=256, new_hi=2048, old_lo=0, old_hi=1000,
              page=64, block=32, hkv=8, dim=128, fused=False),
        # one long prompt
        _case("append", "append_prompt", batch=1, new_lo=131072, new_hi=131072, old_lo=0, old_hi=0,
              page=16, block=16, hkv=8, dim=64, fused=True),
        # one request's decode, where latency counts
        _case("decode", "decode_one", batch=1, old_lo=1000, old_hi=1000, page=16, block=16, hq=64,
              hkv=8, dim=64, window=0, sinks=True),
        # the serving batch: 256 requests with contexts of 1k to 32k tokens
        _case("decode", "decode_batch", batch=256, old_lo=1024, old_hi=32768, page=16, block=16,
              hq=64, hkv=8, dim=64, window=0, sinks=True),
        # the same requests in a sliding-window layer
        _case("decode", "decode_window", batch=256, old_lo=1024, old_hi=32768, page=16, block=16,
              hq=64, hkv=8, dim=64, window=128, sinks=True),
        # head_dim 128, large pages, a scale for each 32 tokens
        _case("decode", "decode_d128", batch=64, old_lo=1024, old_hi=8192, page=64, block=32,
              hq=64, hkv=8, dim=128, window=0, sinks=True),
        # a short prompt: 64 tokens, 4 query heads on one KV head
        _case("prefill", "prefill_short", batch=1, new_lo=64, new_hi=64, old_lo=0, old_hi=0,
              page=16, block=16, hq=4, hkv=1, dim=64, window=0, sinks=True),
        # ragged chunks of 16 requests on cached contexts, head_dim 128
        _case("prefill", "prefill_chunks", batch=16, new_lo=100, new_hi=1024, old_lo=500,
              old_hi=8192, page=64, block=32, hq=32, hkv=8, dim=128, window=0, sinks=True),
        # a chunk of a long context: 2048 new tokens, 131072 in all
        _case("prefill", "prefill_long", batch=1, new_lo=2048, new_hi=2048, old_lo=129024,
              old_hi=129024, page=16, block=16, hq=64, hkv=8, dim=64, window=0, sinks=True),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(x)))


def _layout(rng):
    page = rng.choice([8, 16, 16, 24, 32, 64, 100, 128, 256])
    blocks = [b for b in range(1, page + 1) if page % b == 0]
    return page, rng.choice(blocks[len(blocks) // 2:] + [page, 1])


def draw(rng):
    op = rng.choice(["page_map", "append", "decode", "prefill"])
    page, block = _layout(rng)
    while True:
        c = {"op": op, "len_seed": rng.randrange(1 << 30), "page": page}
        if op == "page_map":
            c.update(batch=_log_int(rng, 1, 600), new_lo=1, new_hi=_log_int(rng, 1, 8192),
                     old_lo=0, old_hi=_log_int(rng, 1, 32768))
            most = work(listed()[1])["bytes"]
        else:
            c.update(block=block, hkv=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([64, 128]))
        if op == "append":
            c.update(batch=_log_int(rng, 1, 256), new_lo=1, new_hi=_log_int(rng, 1, 131072),
                     old_lo=0, old_hi=_log_int(rng, 1, 4096), fused=rng.random() < 0.5)
            most = work(listed()[4])["bytes"]
        if op in ("decode", "prefill"):
            c.update(hq=c["hkv"] * rng.choice([1, 2, 3, 4, 8, 8, 16]),
                     window=rng.choice([0, 0, 0, 128, _log_int(rng, 1, 4096)]),
                     sinks=rng.random() < 0.8)
        if op == "decode":
            c.update(batch=_log_int(rng, 1, 256), old_lo=1, old_hi=_log_int(rng, 1, 32768))
            most = work(listed()[6])["bytes"]
        if op == "prefill":
            c.update(batch=_log_int(rng, 1, 16), new_lo=1, new_hi=_log_int(rng, 1, 2048),
                     old_lo=0, old_hi=_log_int(rng, 1, 32768))
            most = work(listed()[11])["flops"]
        w = work(c)
        if w["flops" if op == "prefill" else "bytes"] <= most and _padded(c) <= 1 << 33:
            return c


def _padded(c):
    """Elements of the plain form's largest padded tensor, or of the cache."""
    new, total = lengths(c)
    if c["op"] == "page_map":
        return sum(new)
    if c["op"] == "append":
        return sum(total) * c["hkv"] * c["dim"]
    if c["op"] == "decode":
        return len(total) * max(total) * max(c["hkv"] * c["dim"], c["hq"])
    return max(sum(total) * c["hkv"] * c["dim"],
               len(new) * max(new) * max(total) * (c["hq"] // c["hkv"]))


def lengths(c):
    """(new tokens, all tokens) of each sequence, fixed by the case."""
    r = random.Random(c["len_seed"])
    new = [r.randint(c.get("new_lo", 1), c.get("new_hi", 1)) for _ in range(c["batch"])]
    old = [r.randint(c["old_lo"], c["old_hi"]) for _ in range(c["batch"])]
    if c["op"] == "decode":  # old_lo..old_hi is the whole context there
        return new, old
    return new, [n + o for n, o in zip(new, old)]


def _ceil(a, b):
    return -(-a // b)


def work(case):
    c = case
    new, total = lengths(c)
    n, batch = sum(new), c["batch"]
    if c["op"] == "page_map":
        # lengths and offsets in, page offsets and slots out; a page id read
        # and a table entry written per new page
        pages = sum(_ceil(t, c["page"]) - _ceil(t - m, c["page"]) for m, t in zip(new, total))
        return {"bytes": 4 * batch + 8 * (batch + 1) + 8 * n + 8 * pages, "flops": 0}
    row = c["hkv"] * c["dim"]
    if c["op"] == "append":
        # bf16 k and v in, codes out, a scale per block and head out
        blocks = sum(_ceil(t, c["block"]) - (t - m) // c["block"] for m, t in zip(new, total))
        return {"bytes": n * (8 + 2 * row * (2 + 1)) + blocks * c["hkv"] * 2 * 4, "flops": 0}
    keys = 0   # key rows that some query sees
    pairs = 0  # visible (query, key) pairs
    w = c["window"]
    for m, t in zip(new, total):
        m = min(m, t)
        keys += t if w == 0 else min(t, m + w - 1)
        for p0 in range(t - m, t, 1 << 20):
            p1 = min(t, p0 + (1 << 20))
            # sum over positions p in [p0, p1) of min(p + 1, w)
            if w == 0:
                pairs += (p0 + 1 + p1) * (p1 - p0) // 2
            else:
                cut = min(max(w, p0), p1)
                pairs += (p0 + 1 + cut) * (cut - p0) // 2 + (p1 - cut) * w
    blocks = sum(_ceil(t, c["block"]) - max(0, t - min(m, t) - w + 1 if w else 0) // c["block"]
                 for m, t in zip(new, total))
    qrows = batch if c["op"] == "decode" else n
    return {"bytes": keys * 2 * row + blocks * c["hkv"] * 8 +
            qrows * c["hq"] * (2 * c["dim"] * 2 + 4),
            "flops": 4 * pairs * c["hq"] * c["dim"]}


# ---------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def _scale_exponent(amax):
    """Smallest e with amax <= 448 * 2^e, within the scales' range."""
    m, e = torch.frexp(amax)  # amax = m * 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP))
    return e.clamp(MIN_EXP, MAX_EXP)


def _to_e4m3(x):
    """float32 of magnitude up to 448 -> e4m3, round to nearest even."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).to(torch.float8_e4m3fn)


def _random_cache(g, pages, c):
    """Codes and scales of normal rows whose size varies from block to block."""
    hkv, page, dim, block = c["hkv"], c["page"], c["dim"], c["block"]
    codes = torch.empty((pages, hkv, page, dim), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, hkv, page // block), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (hkv * page * dim))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn((n, hkv, page // block, block * dim), generator=g, device="cuda")
        size = torch.exp(0.5 * torch.randn((n, hkv, page // block, 1), generator=g,
                                           device="cuda"))
        amax = x.abs().amax(-1) * size[..., 0]
        s = torch.ldexp(torch.ones_like(amax), _scale_exponent(amax))
        x *= size / s[..., None]
        codes[at:at + n] = x.to(torch.float8_e4m3fn).view(torch.uint8).view(n, hkv, page, dim)
        scales[at:at + n] = s
    return codes, scales


def _table(g, total, page, spare=1):
    """Block table over randomly permuted pages, and the number of pages."""
    need = [_ceil(t, page) for t in total]
    pages = sum(need) + spare
    width = max(max(need), 1)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor(_offsets(need)[:-1], device="cuda")[:, None]
    col = torch.arange(width, device="cuda")[None, :]
    used = col < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, perm[(start + col).clamp(max=pages - 1)], 0)
    return table.to(torch.int32).contiguous(), pages


def prepare(case, seed):
    c, g = case, _generator(seed)
    new, total = lengths(c)
    n, page = sum(new), c["page"]
    s = {"case": c}
    s["cu"] = _int32(_offsets(new))
    s["lens"] = _int32(total)
    if c["op"] == "page_map":
        # the pages of the earlier tokens are in the table, the others in the free list
        old = [_ceil(t - m, page) for m, t in zip(new, total)]
        table, pages = _table(g, total, page, spare=64)
        have = torch.arange(table.shape[1], device="cuda")[None, :] < _int32(old)[:, None]
        s["free"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["table"] = torch.where(have, table, -1).contiguous()
        s["head"] = _int32([5])
        s["n"] = n
        return s
    s["table"], pages = _table(g, total, page)
    s["k_cache"], s["k_scale"] = _random_cache(g, pages, c)
    s["v_cache"], s["v_scale"] = _random_cache(g, pages, c)
    if c["op"] == "append":
        # k and v as a projection leaves them: slices of one row, or tensors of their own
        hkv, dim = c["hkv"], c["dim"]
        if c["fused"]:
            x = torch.randn((n, 4 * hkv, dim), generator=g, device="cuda").to(torch.bfloat16)
            s["k"], s["v"] = x[:, 2 * hkv:3 * hkv], x[:, 3 * hkv:]
        else:
            s["k"], s["v"] = (torch.randn((n, hkv, dim), generator=g, device="cuda")
                              .to(torch.bfloat16) for _ in range(2))
        # the slot of each new token
        seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"),
                                      torch.tensor(new, device="cuda"))
        pos = torch.arange(n, device="cuda") - s["cu"][seq] + (s["lens"] - _int32(new))[seq]
        s["slots"] = s["table"][seq, pos // page].long() * page + pos % page
        return s
    rows = c["batch"] if c["op"] == "decode" else n
    s["q"] = torch.randn((rows, c["hq"], c["dim"]), generator=g, device="cuda").to(torch.bfloat16)
    s["sinks"] = torch.randn(c["hq"], generator=g, device="cuda") if c["sinks"] else None
    s["max_q"], s["max_k"] = max(new), max(total)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"page_map": _page_map, "append": _append, "decode": _decode,
            "prefill": _prefill}[op](state)


def _own(op, s):
    import attention_learned_sinks_gb300 as sa
    c = s["case"]
    if op == "page_map":
        slots, offs, head = sa.sinkattn_page_map(s["lens"], s["table"], s["free"], s["head"],
                                                 c["page"], cu_seqlens_q=s["cu"],
                                                 total_q=s["n"])
        return {"slots": slots, "offsets": offs, "head": head, "table": s["table"]}
    if op == "append":
        sa.sinkattn_append_fp8_block(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                                     s["k_scale"], s["v_scale"])
        return _cache_out(s)
    if op == "decode":
        out, lse = sa.sinkattn_decode_fp8_block(
            s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
            s["lens"], max_seqlen_k=s["max_k"], sinks=s["sinks"], window=c["window"])
    else:
        out, lse = sa.sinkattn_prefill_paged_fp8_block(
            s["q"], s["cu"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
            s["lens"], s["max_q"], s["max_k"], sinks=s["sinks"], window=c["window"])
    return {"out": out, "lse": lse}


def _cache_out(s):
    """The cache after an append: codes as the e4m3 values they are, and the scales."""
    e4m3 = torch.float8_e4m3fn
    return {"k": s["k_cache"].view(e4m3), "v": s["v_cache"].view(e4m3),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _page_map(s):
    page = s["case"]["page"]
    lens, cu = s["lens"].long(), s["cu"].long()
    old = (lens - (cu[1:] - cu[:-1])).clamp(min=0)
    have = (old + page - 1) // page
    need = (lens + page - 1) // page - have
    offs = torch.cat([s["head"].long(), s["head"].long() + torch.cumsum(need, 0)])
    seq = torch.searchsorted(cu, torch.arange(s["n"], device="cuda"), right=True) - 1
    pos = lens[seq] - cu[seq + 1] + torch.arange(s["n"], device="cuda")
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (offs[:-1, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    slots = table[seq, pos // page].long() * page + pos % page
    return {"slots": slots, "offsets": offs.int(), "head": offs[-1:].int(), "table": table}


def _append(s):
    for which in ("k", "v"):
        _append_one(s[which].float(), s["slots"], s[which + "_cache"], s[which + "_scale"],
                    s["case"]["block"])
    return _cache_out(s)


def _append_one(x, slots, cache, scale, block):
    pages, hkv, page, dim = cache.shape
    per = page // block
    blk, at = torch.unique(slots // block, return_inverse=True)
    amax = torch.zeros((blk.numel(), hkv), device="cuda")
    amax.scatter_reduce_(0, at[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    first = torch.full((blk.numel(),), block, device="cuda", dtype=torch.long)
    first.scatter_reduce_(0, at, slots % block, "amin")  # offset of the first new token
    fresh = torch.ldexp(torch.ones_like(amax), _scale_exponent(amax))
    bp, bi = blk // per, blk % per
    had = scale[bp, :, bi]
    now = torch.where((first > 0)[:, None], torch.maximum(fresh, had), fresh)
    scale[bp, :, bi] = now
    # older tokens of the blocks, under the new scale where it grew
    off = torch.arange(block, device="cuda")
    rows = (bi * block)[:, None] + off[None, :]
    codes = cache[bp[:, None], :, rows].view(torch.float8_e4m3fn)  # [blocks, block, hkv, dim]
    again = _to_e4m3(codes.float() * (had / now)[:, None, :, None])
    keep = (off[None, :] < first[:, None]).nonzero(as_tuple=True)
    cache[bp[keep[0]], :, rows[keep]] = again.view(torch.uint8)[keep]
    cache[slots // page, :, slots % page] = _to_e4m3(x / now[at][..., None]).view(torch.uint8)


def _values(cache, scale, table):
    """Dequantised rows of every sequence, padded: [batch, hkv, keys, dim] in float32."""
    page = cache.shape[2]
    x = cache[table].view(torch.float8_e4m3fn).float()      # [batch, pages, hkv, page, dim]
    x *= scale.repeat_interleave(page // scale.shape[2], 2)[table][..., None]
    b, p, h, _, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, p * page, d)


def _softmax_v(scores, visible, sinks, v):
    """softmax over [sink, visible scores] times v, and its log-sum-exp.
    scores [.., group, rows, keys], visible [.., 1, rows, keys], sinks [group, 1] or None."""
    scores.masked_fill_(~visible, -math.inf)
    top = scores.amax(-1)
    if sinks is not None:
        top = torch.maximum(top, sinks)
    top = torch.where(torch.isinf(top), 0.0, top)
    scores -= top[..., None]
    scores.exp_()
    den = scores.sum(-1)
    if sinks is not None:
        den = den + torch.exp(sinks - top)
    out = scores @ v
    out = torch.where(den[..., None] > 0, out / den[..., None], 0.0)
    return out, torch.log(den) + top


def _decode(s):
    c = s["case"]
    hkv, group, dim = c["hkv"], c["hq"] // c["hkv"], c["dim"]
    batch = c["batch"]
    q = s["q"].float().view(batch, hkv, group, dim) * dim ** -0.5
    scores = q @ _values(s["k_cache"], s["k_scale"], s["table"]).transpose(-1, -2)
    j = torch.arange(scores.shape[-1], device="cuda")[None, :]
    lens = s["lens"][:, None]
    see = j < lens
    if c["window"]:
        see &= j >= lens - c["window"]
    # the group of query heads takes the rows' place
    sinks = None if s["sinks"] is None else s["sinks"].view(hkv, group)
    out, lse = _softmax_v(scores, see[:, None, None, :], sinks,
                          _values(s["v_cache"], s["v_scale"], s["table"]))
    return {"out": out.reshape(batch, c["hq"], dim).to(torch.bfloat16),
            "lse": lse.reshape(batch, c["hq"])}


def _prefill(s):
    c = s["case"]
    hkv, group, dim, batch = c["hkv"], c["hq"] // c["hkv"], c["dim"], c["batch"]
    n, rows = s["q"].shape[0], s["max_q"]
    cu, lens = s["cu"].long(), s["lens"].long()
    seq = torch.searchsorted(cu, torch.arange(n, device="cuda"), right=True) - 1
    row = torch.arange(n, device="cuda") - cu[seq]
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(rows, device="cuda")[None, :]
    j = torch.arange(s["table"].shape[1] * c["page"], device="cuda")[None, None, :]
    see = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        see &= j > pos[..., None] - c["window"]
    out = torch.empty((n, hkv, group, dim), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, hkv, group), dtype=torch.float32, device="cuda")
    for h in range(hkv):  # one KV head at a time: the scores of all do not fit
        q = torch.zeros((batch, rows, group, dim), device="cuda")
        q[seq, row] = s["q"].view(n, hkv, group, dim)[:, h].float() * dim ** -0.5
        k = _values(s["k_cache"][:, h:h + 1], s["k_scale"][:, h:h + 1], s["table"])
        scores = q.transpose(1, 2) @ k.transpose(-1, -2)  # [batch, group, rows, keys]
        sinks = None if s["sinks"] is None else s["sinks"].view(hkv, group, 1)[h]
        o, l = _softmax_v(scores, see[:, None], sinks,
                          _values(s["v_cache"][:, h:h + 1], s["v_scale"][:, h:h + 1], s["table"]))
        del scores
        out[:, h] = o[seq, :, row].to(torch.bfloat16)
        lse[:, h] = l[seq, :, row]
    return {"out": out.view(n, c["hq"], dim), "lse": lse.view(n, c["hq"])}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "page_map":
        return None  # whole numbers
    if work(c)["flops"] > 6e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(s)
    return _exact_attention(s)


def _code_values():
    """The 256 e4m3 codes' values: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(math.nan if e == 15 and m == 7 else -x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _nearest_code_value(x, grid):
    """Nearest of the grid's values (positive, ascending; ties to the even code), in float64."""
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
    lo = hi - 1
    below, above = a - grid[lo], grid[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[pick], x)


def _exact_append(s):
    c, page, block = s["case"], s["case"]["page"], s["case"]["block"]
    new, total = lengths(c)
    values = _code_values()
    grid = values[:127]
    out = {}
    for which in ("k", "v"):
        cache = values[s[which + "_cache"].long()]
        scale = s[which + "_scale"].double()
        rows = s[which].double()
        at = 0
        for b, (m, t) in enumerate(zip(new, total)):
            old = t - m
            lo = old // block * block            # first position of the touched blocks
            n = _ceil(t, block) - lo // block
            pos = torch.arange(lo, lo + n * block, device="cuda")
            p = s["table"][b][(pos // page).clamp(max=s["table"].shape[1] - 1)].long()
            x = torch.zeros((n * block,) + rows.shape[1:], dtype=torch.float64, device="cuda")
            x[old - lo:t - lo] = rows[at:at + m]
            top = x.abs().view(n, block, *rows.shape[1:]).amax((1, 3))
            e = torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX))
            e = e.clamp(MIN_EXP, MAX_EXP)
            bp, bi = p[::block], pos[::block] % page // block
            had = scale[bp, :, bi]
            sc = torch.exp2(e)
            if old > lo:                         # the first block holds older tokens
                sc[0] = torch.maximum(sc[0], had[0])
                k = slice(0, old - lo)
                cache[p[k], :, pos[k] % page] = _nearest_code_value(
                    cache[p[k], :, pos[k] % page] * (had[0] / sc[0])[None, :, None], grid)
            scale[bp, :, bi] = sc
            k = slice(old - lo, t - lo)
            cache[p[k], :, pos[k] % page] = _nearest_code_value(
                x[k] / sc.repeat_interleave(block, 0)[k][..., None], grid)
            at += m
        out[which], out[which + "_scale"] = cache, scale
    return out


def _exact_attention(s):
    c, page, block = s["case"], s["case"]["page"], s["case"]["block"]
    new, total = lengths(c)
    group, dim = c["hq"] // c["hkv"], c["dim"]
    values = _code_values()
    outs, lses, at = [], [], 0
    for b, (m, t) in enumerate(zip(new, total)):
        m = 1 if c["op"] == "decode" else m
        lo = max(0, t - m - c["window"] + 1) if c["window"] else 0
        pos = torch.arange(lo, t, device="cuda")
        p, slot = s["table"][b][pos // page].long(), pos % page
        q = s["q"][at:at + m].double()
        at += m
        see = pos[None, :] <= torch.arange(t - m, t, device="cuda")[:, None]
        if c["window"]:
            see &= pos[None, :] > torch.arange(t - m, t, device="cuda")[:, None] - c["window"]
        o = torch.empty((m, c["hq"], dim), dtype=torch.float64, device="cuda")
        l = torch.empty((m, c["hq"]), dtype=torch.float64, device="cuda")
        for g in range(c["hkv"]):
            k = values[s["k_cache"][p, g, slot].long()] * \
                s["k_scale"][p, g, slot // block].double()[:, None]
            v = values[s["v_cache"][p, g, slot].long()] * \
                s["v_scale"][p, g, slot // block].double()[:, None]
            for h in range(g * group, (g + 1) * group):
                x = q[:, h] @ k.t() / math.sqrt(dim)
                x = torch.where(see, x, -math.inf)
                if s["sinks"] is not None:
                    x = torch.cat([s["sinks"][h].double().expand(m, 1), x], 1)
                l[:, h] = torch.logsumexp(x, 1)
                w = torch.exp(x - l[:, h, None])
                o[:, h] = (w[:, 1:] if s["sinks"] is not None else w) @ v
        outs.append(o)
        lses.append(l)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
