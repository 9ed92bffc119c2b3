"""The operators of a speculative decoding step in float64, written from their
definitions (numpy; no code shared with the library). Test infrastructure only.

Trees: parents[i] is the row (within the sequence) that row i follows, -1 for a root;
parents None means chains. The rows' keys are the last of their sequence's."""
import numpy as np


def _parents(parents, cu, b):
    n = int(cu[b + 1] - cu[b])
    if parents is None:
        return [i - 1 for i in range(n)]
    return [int(p) for p in parents[cu[b]:cu[b + 1]]]


def line(parents, i):
    """Row i and its ancestors, itself first."""
    out = [i]
    while parents[out[-1]] >= 0:
        out.append(parents[out[-1]])
    return out


# ---- norm and rotation ---------------------------------------------------------

def _partner(d, rope, interleaved):
    """For each element its partner's index, the sign of the sine, and its pair."""
    e = np.arange(d)
    if interleaved:
        other, first, pair = e ^ 1, e % 2 == 0, e // 2
    else:
        first = e < rope // 2
        other, pair = np.where(first, e + rope // 2, e - rope // 2), e % max(rope // 2, 1)
    turned = e < rope
    return (np.where(turned, other, e), np.where(turned, np.where(first, -1.0, 1.0), 0.0),
            np.where(turned, pair, 0))


def angles(positions, cos_sin, d, interleaved):
    """Partner index [d], cosines and signed sines [n, 1, d] of each row."""
    n_pos, rope = cos_sin.shape
    other, sign, pair = _partner(d, rope, interleaved)
    row = cos_sin[np.clip(positions, 0, n_pos - 1)].astype(np.float64)
    cos = np.where(np.arange(d) < rope, row[:, pair], 1.0)
    sin = row[:, rope // 2 + pair] * sign
    return other, cos[:, None], sin[:, None]


def norm_rope(x, w, eps, positions=None, cos_sin=None, interleaved=False):
    """x [n, heads, D] -> normed (w not None) and turned (cos_sin not None)."""
    y = np.asarray(x, dtype=np.float64)
    if w is not None:
        y = w * y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    if cos_sin is not None:
        other, cos, sin = angles(positions, cos_sin, y.shape[-1], interleaved)
        y = y * cos + y[..., other] * sin
    return y


def norm_rope_backward(dz, x, w, eps, positions=None, cos_sin=None, interleaved=False):
    """(dx, dw) of sum(dz * norm_rope(x, w, ..))."""
    dy = np.asarray(dz, dtype=np.float64)
    if cos_sin is not None:
        other, cos, sin = angles(positions, cos_sin, dy.shape[-1], interleaved)
        # element e enters z_e with cos and z_other with other's sine
        dy = dy * cos + (dy * sin)[..., other]
    if w is None:
        return dy, None
    x = np.asarray(x, dtype=np.float64)
    size = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u, g = x / size, w * dy
    return (g - u * (g * u).mean(-1, keepdims=True)) / size, (u * dy).sum((0, 1))


# ---- attention -------------------------------------------------------------------

def tree_attention(q, cu, parents, k_rows, v_rows, lens, sinks, window, scale):
    """q [n, hq, D]; k_rows / v_rows: for each sequence its keys [Lk, hkv, D] in order.
    Returns (out [n, hq, D], lse [n, hq]); rows behind cu[-1] are NaN."""
    n, hq, d = q.shape
    out, lse = np.full((n, hq, d), np.nan), np.full((n, hq), np.nan)
    for b, lk in enumerate(lens):
        par = _parents(parents, cu, b)
        context = lk - len(par)
        k, v = np.asarray(k_rows[b], np.float64), np.asarray(v_rows[b], np.float64)
        group = hq // k.shape[1]
        for i in range(len(par)):
            up = line(par, i)
            p = context + len(up) - 1
            keys = [j for j in range(max(context, 0)) if not window or j > p - window]
            # the ancestor t steps up stands at position p - t
            keys += [context + a for t, a in enumerate(up)
                     if (not window or t < window) and context + a >= 0]
            for h in range(hq):
                s = scale * (k[keys, h // group] @ q[cu[b] + i, h].astype(np.float64))
                if sinks is not None:
                    s = np.concatenate([[sinks[h]], s])
                if s.size == 0:
                    out[cu[b] + i, h], lse[cu[b] + i, h] = 0.0, -np.inf
                    continue
                top = s.max()
                w = np.exp(s - top)
                den = w.sum()
                lse[cu[b] + i, h] = top + np.log(den)
                w = w[1:] if sinks is not None else w
                out[cu[b] + i, h] = (w / den) @ v[keys, h // group]
    return out, lse


# ---- verification ----------------------------------------------------------------

def _probs(x):
    x = np.asarray(x, dtype=np.float64)
    return np.clip(np.where(np.isnan(x), 0.0, x), 0.0, 1.0)


def verify(p_all, q_all, tokens, parents, uniforms, cu, width):
    """(path [batch, width], num [batch], next [batch]), the residual kept as a vector."""
    batch = len(cu) - 1
    path = np.full((batch, width), -1, np.int64)
    num, token = np.zeros(batch, np.int64), np.full(batch, -1, np.int64)
    for b in range(batch):
        par = _parents(parents, cu, b)[:width]
        if not par:
            continue
        at = int(cu[b])
        kept = [0]
        while True:
            cur = kept[-1]
            p = _probs(p_all[at + cur])
            v, total, found = p.copy(), 1.0, None
            for c in range(cur + 1, len(par)):
                x = int(tokens[at + c])
                if par[c] != cur or not 0 <= x < v.size:
                    continue
                q = _probs(q_all[at + cur]) if q_all is not None else None
                if float(uniforms[at + c]) * total * (q[x] if q is not None else 1.0) < v[x]:
                    found = c
                    break
                if q is not None:
                    v = np.maximum(v - total * q, 0.0)
                    total = v.sum()
                else:
                    total -= v[x]
                    v[x] = 0.0
            if found is None:
                break
            kept.append(found)
        if v.sum() == 0.0:
            v = p
        if v.sum() > 0.0:
            upto = np.cumsum(v)
            token[b] = int(np.argmax(upto > float(uniforms[at]) * upto[-1]))
        path[b, :len(kept)], num[b] = kept, len(kept)
    return path, num, token


# ---- compaction ------------------------------------------------------------------

def compact(k_cache, v_cache, table, lens, cu, path, num, free, head):
    """New (k_cache, v_cache, lens, free, head) as copies."""
    k, v, free = k_cache.copy(), v_cache.copy(), np.array(free).copy()
    page = k.shape[2]
    new, back = [], []
    for b, lk in enumerate(int(x) for x in lens):
        context = lk - int(cu[b + 1] - cu[b])
        if num[b] < 0:
            now = 0
        else:
            now = context + int(num[b])
            rows = range(int(num[b])) if path is None else [int(r) for r in path[b, :num[b]]]
            src = [(table[b][(context + r) // page], (context + r) % page) for r in rows]
            for i, (pg, s) in enumerate(src):
                to = context + i
                k[table[b][to // page], :, to % page] = k_cache[pg, :, s]
                v[table[b][to // page], :, to % page] = v_cache[pg, :, s]
        new.append(now)
        back += [int(table[b][c]) for c in range(-(-now // page), -(-lk // page))
                 if 0 <= table[b][c] < k.shape[0]]
    head2 = head - len(back)
    for i, pg in enumerate(back):
        if 0 <= head2 + i < free.size:
            free[head2 + i] = pg
    return k, v, np.array(new), free, max(head2, 0)
