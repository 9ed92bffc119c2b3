"""Performance cases of the operators of one speculative decoding step over a bf16 paged cache.

A step checks a tree of drafted tokens for each sequence at once. Its operators, in order:

  rope     RMS norm of each query and key head and the rotation by position, keys and
           values written into the cache's pages; in training its gradients
  tree     attention of the drafted tokens over the cache: each sees the context, its
           ancestors and itself, learned sinks in the softmax
  verify   the accepted path through each tree and the next token, from the target's
           and the draft's probabilities and given random numbers
  compact  the accepted tokens' keys and values moved behind the context, the pages
           that are no longer needed given back

`run` computes a case with elementary torch operations (float32; float64 where sums
decide on whole numbers), or, with `own` set, with this library's calls. `exact`
computes it in float64 with code of its own.
"""
import math
import random

import torch

own = False

EPS = 1e-6
MAX_POS = 131072


# ---------------------------------------------------------------- the cases

def _case(op, name, **kw):
    c = {"name": name, "op": op, "len_seed": 1}
    c.update(kw)
    return c


def listed():
    return [
        # one step's queries, keys and values: 64 requests with 8 drafted tokens each, slices
        # of one fused projection, keys and values straight into the pages
        _case("rope", "rope_step", tokens=512, hq=64, hkv=8, dim=64, rot=64, norm=True,
              pairs=False, cache=True, grad=False, page=16, fused=True),
        # a prompt of 32768 tokens, written into the pages
        _case("rope", "rope_prompt", tokens=32768, hq=64, hkv=8, dim=64, rot=64, norm=True,
              pairs=False, cache=True, grad=False, page=16, fused=True),
        # the backward pass over a packed training batch, head_dim 128
        _case("rope", "rope_grad", tokens=32769, hq=32, hkv=8, dim=128, rot=128, norm=True,
              pairs=False, cache=False, grad=True, page=16, fused=False),
        # one request of 1000 cached tokens with a tree of 8, where latency counts
        _case("tree", "tree_one", batch=1, new_lo=8, new_hi=8, old_lo=1000, old_hi=1000, page=16,
              hq=64, hkv=8, dim=64, window=0, sinks=True, chain=False),
        # the serving batch: 64 requests with contexts of 1k to 8k tokens, trees of 16
        _case("tree", "tree_batch", batch=64, new_lo=16, new_hi=16, old_lo=1024, old_hi=8192,
              page=16, hq=64, hkv=8, dim=64, window=0, sinks=True, chain=False),
        # long contexts with wide trees, head_dim 128, large pages
        _case("tree", "tree_wide", batch=4, new_lo=50, new_hi=64, old_lo=16384, old_hi=65536,
              page=64, hq=32, hkv=8, dim=128, window=0, sinks=True, chain=False),
        # a sliding-window layer of a large batch, chains of up to 5 drafted tokens
        _case("tree", "tree_window", batch=256, new_lo=1, new_hi=5, old_lo=1024, old_hi=32768,
              page=16, hq=64, hkv=8, dim=64, window=128, sinks=True, chain=True),
        # one request's chain of 5 drafted tokens
        _case("verify", "verify_one", batch=1, new_lo=6, new_hi=6, vocab=32768, draft=True,
              chain=True, temp=2.0),
        # 64 requests with trees of 16 and a large vocabulary
        _case("verify", "verify_batch", batch=64, new_lo=16, new_hi=16, vocab=131072, draft=True,
              chain=False, temp=2.0),
        # trees from a draft that proposes its likeliest tokens: no draft probabilities; odd rows
        _case("verify", "verify_top", batch=32, new_lo=3, new_hi=12, vocab=50001, draft=False,
              chain=False, temp=3.0),
        # the end of a step of 64 requests
        _case("compact", "compact_step", batch=64, new_lo=16, new_hi=16, old_lo=100, old_hi=2048,
              page=16, hkv=8, dim=64, ended=False),
        # a large batch with wide trees, head_dim 128; some requests have ended
        _case("compact", "compact_large", batch=250, new_lo=1, new_hi=64, old_lo=0, old_hi=1500,
              page=16, hkv=8, dim=128, ended=True),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(x)))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "verify", "compact"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 100, 128, 256])
    while True:
        c = {"op": op, "len_seed": rng.randrange(1 << 30)}
        if op != "verify":
            c.update(page=page, hkv=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([64, 128]))
        if op in ("rope", "tree"):
            c.update(hq=c["hkv"] * rng.choice([1, 2, 3, 4, 8, 8, 16]))
        if op == "rope":
            grad = rng.random() < 0.4
            c.update(tokens=_log_int(rng, 1, 32769), norm=rng.random() < 0.8,
                     rot=rng.choice([c["dim"], c["dim"], c["dim"], c["dim"] // 2, 16, 0]),
                     pairs=rng.random() < 0.3, grad=grad,
                     cache=not grad and rng.random() < 0.5, fused=rng.random() < 0.5)
            if not c["norm"] and not c["rot"]:
                c["rot"] = c["dim"]
            most = work(listed()[2 if grad else 1])["bytes"]
        else:
            c.update(batch=_log_int(rng, 1, 256), new_lo=1, new_hi=_log_int(rng, 1, 64))
        if op == "tree":
            c.update(old_lo=0, old_hi=_log_int(rng, 1, 65536), chain=rng.random() < 0.3,
                     window=rng.choice([0, 0, 0, 128, _log_int(rng, 1, 4096)]),
                     sinks=rng.random() < 0.8)
            most = work(listed()[5])["flops"]
        if op == "verify":
            c.update(vocab=_log_int(rng, 1000, 200000), draft=rng.random() < 0.7,
                     chain=rng.random() < 0.4, temp=rng.choice([0.5, 1.0, 2.0, 4.0]))
            most = work(listed()[8])["bytes"]
        if op == "compact":
            c.update(old_lo=0, old_hi=_log_int(rng, 1, 2048), ended=rng.random() < 0.5)
            most = work(listed()[11])["bytes"]
        w = work(c)
        if w["flops" if op == "tree" else "bytes"] <= most and _largest(c) <= 1 << 31:
            return c


def _largest(c):
    """Elements of the plain form's largest padded tensor, or of the inputs."""
    if c["op"] == "rope":
        return c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["dim"]
    new, total = lengths(c)
    if c["op"] == "verify":
        return sum(new) * c["vocab"]
    if c["op"] == "compact":
        return sum(total) * c["hkv"] * c["dim"]
    return len(total) * max(total) * max(c["hkv"] * c["dim"], c["hq"] * max(new))


def lengths(c):
    """(new tokens, all tokens) of each sequence, fixed by the case."""
    r = random.Random(c["len_seed"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    old = [r.randint(c.get("old_lo", 0), c.get("old_hi", 0)) for _ in range(c["batch"])]
    return new, [n + o for n, o in zip(new, old)]


def _ceil(a, b):
    return -(-a // b)


def work(case):
    c = case
    if c["op"] == "rope":
        n, qk, v = c["tokens"], (c["hq"] + c["hkv"]) * c["dim"], c["hkv"] * c["dim"]
        table = n * (4 + 4 * c["rot"]) if c["rot"] else 0
        if c["grad"]:  # gradients and (for the norm) inputs in, gradients out
            return {"bytes": n * qk * 2 * (3 if c["norm"] else 2) + table, "flops": 16 * n * qk}
        rows = 2 * 2 * (qk + (v if c["cache"] else 0))
        return {"bytes": n * (rows + (8 if c["cache"] else 0)) + table, "flops": 8 * n * qk}
    new, total = lengths(c)
    n = sum(new)
    if c["op"] == "verify":
        # a row of each distribution for the final draw of each sequence; tokens, parents,
        # numbers and two probabilities for each drafted token
        rows = 2 if c["draft"] else 1
        return {"bytes": 4 * c["batch"] * c["vocab"] * rows + n * (8 + 4 + 4 + 4 * rows),
                "flops": 2 * c["batch"] * c["vocab"]}
    if c["op"] == "compact":
        # about half of each tree's rows read and written, and the bookkeeping
        return {"bytes": sum(m // 2 for m in new) * c["hkv"] * c["dim"] * 2 * 2 * 2 +
                c["batch"] * 20 + n * 4, "flops": 0}
    keys = pairs = 0  # key rows that some query sees; visible (query, key) pairs
    w = c["window"]
    for m, t in zip(new, total):
        context = t - m
        keys += min(context, w - 1) + m if w else t
        # a node of depth d sees d ancestors; the trees here are about m / 4 deep
        seen = m if c["chain"] else max(1, m // 4)
        pairs += m * (min(context, w - 1) if w else context) + m * max(1, seen // 2)
    return {"bytes": keys * 2 * c["hkv"] * c["dim"] * 2 + n * c["hq"] * (2 * c["dim"] * 2 + 4),
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


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _rope_table(rot):
    """[MAX_POS, rot] float32: the cosines of each position's rot / 2 angles, then the sines."""
    at = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None]
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    return torch.cat([torch.cos(at * freq), torch.sin(at * freq)], 1).float()


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


def _trees(c, seed):
    """The parent of each drafted token (an index into its own tree, -1 for the root)."""
    r = random.Random(seed * 7919 + c["len_seed"])
    out = []
    for m in lengths(c)[0]:
        reach = 1 if c.get("chain") else max(2, m // 3)
        out += [-1] + [r.randint(max(0, i - reach), i - 1) for i in range(1, m)]
    return _int32(out)


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = {"case": c}
    if c["op"] == "rope":
        return _prepare_rope(c, g, s)
    new, total = lengths(c)
    n = sum(new)
    s["cu"], s["lens"] = _int32(_offsets(new)), _int32(total)
    s["max_q"], s["max_k"] = max(new), max(total)
    if c["op"] == "verify":
        return _prepare_verify(c, g, s, seed, n)
    s["table"], pages = _table(g, total, c["page"])
    shape = (pages, c["hkv"], c["page"], c["dim"])
    s["k_cache"], s["v_cache"] = _normal(g, *shape), _normal(g, *shape)
    if c["op"] == "tree":
        s["q"] = _normal(g, n, c["hq"], c["dim"])
        s["sinks"] = torch.randn(c["hq"], generator=g, device="cuda") if c["sinks"] else None
        s["parents"] = None if c["chain"] else _trees(c, seed)
        return s
    # the accepted rows of each tree: its root and a share of the others, in order
    r = random.Random(seed * 104729 + c["len_seed"])
    path, num = [], []
    for m in new:
        kept = [0] + sorted(r.sample(range(1, m), r.randint(0, (m - 1) // 2)))
        path.append(kept + [-1] * (s["max_q"] - len(kept)))
        num.append(-1 if c["ended"] and r.random() < 0.1 else len(kept))
    s["path"], s["num"] = _int32(path), _int32(num)
    s["free"] = torch.randperm(pages + 64, generator=g, device="cuda").to(torch.int32)
    s["head"] = _int32([pages])
    return s


def _prepare_rope(c, g, s):
    n, hq, hkv, dim = c["tokens"], c["hq"], c["hkv"], c["dim"]
    if c["fused"]:
        x = _normal(g, n, hq + 2 * hkv, dim)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        s["q"], s["k"], s["v"] = (_normal(g, n, h, dim) for h in (hq, hkv, hkv))
    s["positions"] = torch.randint(0, MAX_POS, (n,), generator=g, device="cuda",
                                   dtype=torch.int32)
    s["cos_sin"] = _rope_table(c["rot"]) if c["rot"] else None
    s["wq"] = s["wk"] = None
    if c["norm"]:
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
                            for _ in range(2))
    if c["cache"]:
        pages = _ceil(n, c["page"]) + 16
        s["k_cache"] = _normal(g, pages, hkv, c["page"], dim)
        s["v_cache"] = _normal(g, pages, hkv, c["page"], dim)
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device="cuda")[:n]
    if c["grad"]:
        s["dq"], s["dk"] = _normal(g, n, hq, dim), _normal(g, n, hkv, dim)
    return s


def _prepare_verify(c, g, s, seed, n):
    vocab = c["vocab"]
    logits = c["temp"] * torch.randn((n, vocab), generator=g, device="cuda")
    s["p"] = torch.softmax(logits, 1)
    # a draft that is near the target
    logits += 0.5 * torch.randn((n, vocab), generator=g, device="cuda")
    q = torch.softmax(logits, 1)
    del logits
    s["parents"] = _trees(c, seed)
    row = torch.repeat_interleave(s["cu"][:-1], s["cu"][1:] - s["cu"][:-1]).long()
    row = row + s["parents"].clamp(min=0).long()  # the row each token was drafted from
    if c["draft"]:
        s["q"] = q
        s["tokens"] = torch.multinomial(q[row], 1, generator=g)[:, 0]
    else:  # one of the draft's eight likeliest
        s["q"] = None
        pick = torch.randint(0, 8, (n,), generator=g, device="cuda")
        s["tokens"] = torch.topk(q, 8, 1)[1][row, pick]
    s["u"] = torch.rand(n, generator=g, device="cuda")
    if c["chain"]:
        s["parents"] = None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"rope": _rope, "tree": _tree, "verify": _verify, "compact": _compact}[op](state)


def _own(op, s):
    import attention_learned_sinks_gb300 as sa
    c = s["case"]
    if op == "rope":
        kw = {"q_weight": s["wq"], "k_weight": s["wk"], "eps": EPS, "interleaved": c["pairs"]}
        if c["grad"]:
            dq, dk, dwq, dwk = sa.sinkattn_qk_norm_rope_backward(
                s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["cos_sin"], **kw)
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        if c["cache"]:
            q, _ = sa.sinkattn_qk_norm_rope(
                s["q"], s["k"], s["positions"], s["cos_sin"], v=s["v"], slot_mapping=s["slots"],
                k_cache=s["k_cache"], v_cache=s["v_cache"], **kw)
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        q, k = sa.sinkattn_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], **kw)
        return {"q": q, "k": k}
    if op == "tree":
        out, lse = sa.sinkattn_decode_tree(
            s["q"], s["cu"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["max_q"],
            s["max_k"], parents=s["parents"], sinks=s["sinks"], window=c["window"])
        return {"out": out, "lse": lse}
    if op == "verify":
        path, num, token = sa.sinkattn_verify_tree(
            s["p"], s["tokens"], s["u"], s["cu"], s["max_q"], draft_probs=s["q"],
            parents=s["parents"])
        return {"path": path, "num": num, "token": token}
    lens, head = sa.sinkattn_compact(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                                     s["path"], s["num"], s["free"], s["head"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": lens, "free": s["free"],
            "head": head}


def _turn(x, cos, sin, pairs):
    """Rotates the first 2 * cos.shape[-1] elements of each row of x [tokens, heads, dim]."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    a, b = ((x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs
            else (x[..., :half], x[..., half:2 * half]))
    first, second = a * cos - b * sin, b * cos + a * sin
    if pairs:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = first, second
    else:
        y[..., :half], y[..., half:2 * half] = first, second
    return y


def _angles(s):
    rot = s["case"]["rot"]
    t = s["cos_sin"][s["positions"].long()]
    return t[:, :rot // 2], t[:, rot // 2:]


def _rope_one(s, x, w):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if s["cos_sin"] is not None:
        x = _turn(x, *_angles(s), s["case"]["pairs"])
    return x.to(torch.bfloat16)


def _rope_grad_one(s, dz, x, w):
    dy = dz.float()
    if s["cos_sin"] is not None:
        cos, sin = _angles(s)
        dy = _turn(dy, cos, -sin, s["case"]["pairs"])
    if w is None:
        return dy.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dw = (dy * x * r).sum((0, 1), dtype=torch.float64).float()
    g = dy * w
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dw


def _rope(s):
    if s["case"]["grad"]:
        dq, dwq = _rope_grad_one(s, s["dq"], s["q"], s["wq"])
        dk, dwk = _rope_grad_one(s, s["dk"], s["k"], s["wk"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    q, k = _rope_one(s, s["q"], s["wq"]), _rope_one(s, s["k"], s["wk"])
    if not s["case"]["cache"]:
        return {"q": q, "k": k}
    page, at = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"]
    s["k_cache"][page, :, at] = k
    s["v_cache"][page, :, at] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _ancestors(s, seq, row):
    """sees [n, max_q]: the drafted tokens that each sees (itself among them), and depths [n]."""
    n, width = seq.numel(), s["max_q"]
    col = torch.arange(width, device="cuda")[None, :]
    if s["parents"] is None:
        return col <= row[:, None], row
    step = torch.zeros((s["case"]["batch"], width, width), device="cuda")
    step[seq, row, row] = 1.0
    at = s["parents"].long()
    has = (at >= 0).float()
    step[seq, row, at.clamp(min=0)] += has
    for _ in range(max(1, (width - 1).bit_length())):
        step = ((step @ step) > 0).float()
    sees = step[seq, row] > 0
    return sees, sees.sum(1) - 1


def _pages(cache, table):
    """The rows of every sequence, padded: [batch, hkv, keys, dim] in float32."""
    x = cache[table].float()  # [batch, pages, hkv, page, dim]
    b, p, h, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, p * page, d)


def _tree(s):
    c = s["case"]
    hkv, group, dim, batch = c["hkv"], c["hq"] // c["hkv"], c["dim"], c["batch"]
    n, rows = s["q"].shape[0], s["max_q"]
    cu, lens = s["cu"].long(), s["lens"].long()
    seq = torch.searchsorted(cu, torch.arange(n, device="cuda"), right=True) - 1
    row = torch.arange(n, device="cuda") - cu[seq]
    context = lens - (cu[1:] - cu[:-1])
    sees, depth = _ancestors(s, seq, row)
    j = torch.arange(s["table"].shape[1] * c["page"], device="cuda")[None, :]
    # [n, keys]: the context, and the drafted tokens behind it
    t = j - context[seq, None]
    drafted = (t >= 0) & (t < rows)
    at = t.clamp(0, rows - 1)
    see = (t < 0) | (drafted & torch.gather(sees, 1, at))
    see &= j < lens[seq, None]
    if c["window"]:
        depths = torch.zeros((batch, rows), dtype=torch.long, device="cuda")
        depths[seq, row] = depth
        place = torch.where(drafted, context[seq, None] + torch.gather(depths[seq], 1, at), j)
        see &= place > (context[seq] + depth)[:, None] - c["window"]
    mask = torch.zeros((batch, rows, j.shape[1]), dtype=torch.bool, device="cuda")
    mask[seq, row] = see
    q = torch.zeros((batch, rows, hkv, group, dim), device="cuda")
    q[seq, row] = s["q"].view(n, hkv, group, dim).float() * dim ** -0.5
    q = q.permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * rows, dim)
    scores = (q @ _pages(s["k_cache"], s["table"]).transpose(-1, -2)).view(
        batch, hkv, group, rows, -1)
    scores.masked_fill_(~mask[:, None, None], -math.inf)
    top = scores.amax(-1)
    if s["sinks"] is not None:
        sinks = s["sinks"].view(1, hkv, group, 1)
        top = torch.maximum(top, sinks)
    top = torch.where(torch.isinf(top), 0.0, top)
    scores -= top[..., None]
    scores.exp_()
    den = scores.sum(-1)
    if s["sinks"] is not None:
        den = den + torch.exp(sinks - top)
    out = scores.view(batch, hkv, group * rows, -1) @ _pages(s["v_cache"], s["table"])
    out = out.view(batch, hkv, group, rows, dim)
    out = torch.where(den[..., None] > 0, out / den[..., None], 0.0)
    lse = torch.log(den) + top
    return {"out": out[seq, :, :, row].reshape(n, c["hq"], dim).to(torch.bfloat16),
            "lse": lse[seq, :, :, row].reshape(n, c["hq"])}


def _verify(s):
    c = s["case"]
    batch, width = c["batch"], s["max_q"]
    first = s["cu"][:-1].long()
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    cur = torch.zeros(batch, dtype=torch.long, device="cuda")
    taken = torch.zeros(batch, dtype=torch.double, device="cuda")  # A: the draft's mass taken off
    left = torch.ones(batch, dtype=torch.double, device="cuda")    # S: what is left of the target
    path = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    num = torch.ones(batch, dtype=torch.int32, device="cuda")
    every = torch.arange(batch, device="cuda")
    gone = torch.zeros((batch, c["vocab"]), dtype=torch.bool, device="cuda")
    for t in range(1, width):  # a token's parent comes before it
        at = (first + t).clamp(max=s["tokens"].numel() - 1)
        parent = t - 1 if s["parents"] is None else s["parents"][at].long()
        ask = (t < count) & (cur == parent)
        token, u = s["tokens"][at], s["u"][at].double()
        p = s["p"][first + cur]
        if s["q"] is not None:
            q = s["q"][first + cur]
            drawn = q[every, token].double()
            v = (p[every, token].double() - taken * drawn).clamp(min=0)
        else:
            drawn = torch.ones_like(left)
            v = torch.where(gone[every, token], 0.0, p[every, token].double())
        good = ask & (u * left * drawn < v)
        bad = ask & ~good
        if s["q"] is not None:
            taken = torch.where(bad, taken + left, taken)
            rest = (p.double() - taken[:, None] * q.double()).clamp(min=0).sum(1)
            left = torch.where(bad, rest, left)
        else:
            gone[every, token] |= bad
            left = torch.where(bad, left - v, left)
        path[every, num.clamp(max=width - 1).long()] = torch.where(
            good, t, path[every, num.clamp(max=width - 1).long()])
        num = num + good.int()
        cur = torch.where(good, t, cur)
        taken = torch.where(good, 0.0, taken)
        left = torch.where(good, 1.0, left)
        gone &= ~good[:, None]
    v = s["p"][first + cur].double()
    if s["q"] is not None:
        v = (v - taken[:, None] * s["q"][first + cur].double()).clamp(min=0)
    else:
        v = torch.where(gone, 0.0, v)
    upto = torch.cumsum(v, 1)
    token = (upto <= s["u"][first].double()[:, None] * upto[:, -1:]).sum(1)
    return {"path": path, "num": num, "token": token}


def _compact(s):
    page = s["case"]["page"]
    lens, num, table = s["lens"].long(), s["num"].long(), s["table"]
    context = lens - (s["cu"][1:] - s["cu"][:-1])
    i = torch.arange(s["path"].shape[1], device="cuda")[None, :]
    seq, at = (i < num[:, None]).nonzero(as_tuple=True)
    src, dst = context[seq] + s["path"][seq, at], context[seq] + at
    for cache in (s["k_cache"], s["v_cache"]):
        cache[table[seq, dst // page].long(), :, dst % page] = \
            cache[table[seq, src // page].long(), :, src % page]
    now = torch.where(num < 0, 0, context + num)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    back = ((col >= ((now + page - 1) // page)[:, None]) &
            (col < ((lens + page - 1) // page)[:, None]))
    pages = table[back]
    head = s["head"].long() - pages.numel()
    s["free"][head + torch.arange(pages.numel(), device="cuda")] = pages
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": now.int(),
            "free": s["free"], "head": head.int()}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    c = case
    if c["op"] in ("verify", "compact"):
        return None  # whole numbers, and rows that are copied
    if work(c)["flops"] > 1e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "tree":
        return _exact_tree(s)
    z = torch.complex(*(t.double() for t in _exact_angles(s))) if c["rot"] else None
    if c["grad"]:
        dq, dwq = _exact_rope_grad(s, s["dq"], s["q"], s["wq"], z)
        dk, dwk = _exact_rope_grad(s, s["dk"], s["k"], s["wk"], z)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    q, k = _exact_rope(s, s["q"], s["wq"], z), _exact_rope(s, s["k"], s["wk"], z)
    if not c["cache"]:
        return {"q": q, "k": k}
    # rows of the pages, one after the other
    out = {"q": q}
    for name, rows in (("k_cache", k), ("v_cache", s["v"].double())):
        x = s[name].double().transpose(1, 2).flatten(0, 1).contiguous()
        x[s["slots"]] = rows
        out[name] = x.unflatten(0, (-1, c["page"])).transpose(1, 2).contiguous()
    return out


def _exact_angles(s):
    both = s["cos_sin"].index_select(0, s["positions"].long())
    return both.tensor_split(2, dim=1)


def _exact_spin(x, z, pairs):
    """The rotated elements as complex numbers, times z."""
    rot = 2 * z.shape[1]
    part = x[..., :rot].unflatten(-1, (rot // 2, 2) if pairs else (2, rot // 2))
    if not pairs:
        part = part.transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z[:, None])
    if not pairs:
        turned = turned.transpose(-1, -2)
    return torch.cat([turned.flatten(-2), x[..., rot:]], -1)


def _exact_rope(s, x, w, z):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    return x if z is None else _exact_spin(x, z, s["case"]["pairs"])


def _exact_rope_grad(s, dz, x, w, z):
    dy = dz.double() if z is None else _exact_spin(dz.double(), z.conj(), s["case"]["pairs"])
    if w is None:
        return dy, None
    x = x.double()
    size = torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
    unit = x / size
    dunit = dy * w.double()
    dx = (dunit - unit * (dunit * unit).sum(-1, keepdim=True) / x.shape[-1]) / size
    return dx, (dy * unit).flatten(0, 1).sum(0)


def _exact_tree(s):
    c, page = s["case"], s["case"]["page"]
    new, total = lengths(c)
    group, dim = c["hq"] // c["hkv"], c["dim"]
    parents = None if s["parents"] is None else s["parents"].tolist()
    outs, lses, at = [], [], 0
    for b, (m, t) in enumerate(zip(new, total)):
        context = t - m
        above = []  # each drafted token's line of ancestors, itself included
        for i in range(m):
            up = i - 1 if parents is None else parents[at + i]
            above.append([i] if up < 0 else above[up] + [i])
        see = torch.zeros((m, t), dtype=torch.bool)
        for i in range(m):
            lo = len(above[i]) - c["window"] if c["window"] else -t  # behind the context's end
            see[i, max(0, context + lo):context] = True
            see[i, [context + a for a in above[i] if len(above[a]) > lo]] = True
        see = see.cuda()
        first = 0
        if c["window"]:
            first = max(0, context - c["window"])
            see = see[:, first:]
        pos = torch.arange(first, t, device="cuda")
        p, slot = s["table"][b][pos // page].long(), pos % page
        q = s["q"][at:at + m].double()
        at += m
        o = torch.empty((m, c["hq"], dim), dtype=torch.float64, device="cuda")
        l = torch.empty((m, c["hq"]), dtype=torch.float64, device="cuda")
        for g in range(c["hkv"]):
            k, v = s["k_cache"][p, g, slot].double(), s["v_cache"][p, g, slot].double()
            h = slice(g * group, (g + 1) * group)
            x = torch.einsum("mhd,kd->mhk", q[:, h], k) / math.sqrt(dim)
            x = torch.where(see[:, None], x, -math.inf)
            if s["sinks"] is not None:
                x = torch.cat([s["sinks"][h].double()[None, :, None].expand(m, -1, 1), x], 2)
            l[:, h] = torch.logsumexp(x, 2)
            w = torch.exp(x - l[:, h, None])
            o[:, h] = (w[..., 1:] if s["sinks"] is not None else w) @ v
        outs.append(o)
        lses.append(l)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
