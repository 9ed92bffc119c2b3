"""The speculative decoding step on the GPU against its float64 definitions.

Whole numbers and copied rows have to be equal; attention is held to the parity bars of
helpers.py. Every cache slot that no token owns holds NaN, and every table entry that no
token needs a page id far outside the cache.

Norm and rotation: an element is r (x a + x' b) in fp32 with a = w cos, b = w' sin: the
sum of squares (at most 16 serial and 4 tree additions a lane), its root, and four
products lose at most 32 * 2^-24 = 2^-19 of |r x a| + |r x' b|, then half a bf16 step.
Gradients: dx = r (g - u mean(g u)) likewise, relative to r (|g| + |u| mean|g u|), at
most 64 * 2^-24 = 2^-18 of it; a weight gradient adds at most 64 terms in a row and joins
lanes, warps and blocks in 24 more steps: (64 + 24 + 40) 2^-24 = 2^-17 of the sum of
the terms' magnitudes."""
import numpy as np
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from helpers import bf16_spacing, check_close, to_np
from oracle import step as R

pytestmark = pytest.mark.gpu
FAR = 1 << 28
NAN = float("nan")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def bf(rng, *shape, scale=1.0):
    return torch.tensor(scale * rng.normal(size=shape)).to(torch.bfloat16)


# ---- norm and rotation ---------------------------------------------------------

def rope_table(rng, rows, rope):
    ang = rng.uniform(-np.pi, np.pi, size=(rows, rope // 2))
    return torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32)


def rope_case(n, hq, hkv, d, rope, norm, interleaved, fused, seed=0, scale=1.0):
    rng = np.random.default_rng(seed + n)
    if fused:
        x = bf(rng, n, hq + 2 * hkv + 1, d, scale=scale).cuda()
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    else:
        q, k, v = (bf(rng, n, h, d, scale=scale).cuda() for h in (hq, hkv, hkv))
    cs = rope_table(rng, 37, rope).cuda() if rope else None
    pos = i32(rng.integers(0, 37, n)) if rope else None
    wq, wk = ((torch.tensor(1 + 0.3 * rng.normal(size=d), dtype=torch.float32).cuda()
               for _ in range(2)) if norm else (None, None))
    return q, k, v, pos, cs, dict(q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved)


def np_of(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check_turned(got, x, w, kw, pos, cs, what):
    args = (kw["eps"], None if pos is None else pos.cpu().numpy(), np_of(cs), kw["interleaved"])
    ref = R.norm_rope(np_of(x), np_of(w), *args)
    # |r x a| + |r x' b|: the rotation of magnitudes with the magnitudes of cos and sin
    y = R.norm_rope(np_of(x), np_of(w), kw["eps"])
    size = np.abs(y)
    if cs is not None:
        other, cos, sin = R.angles(args[1], args[2], y.shape[-1], kw["interleaved"])
        size = np.abs(y * cos) + np.abs(y[..., other] * sin)
    bound = 0.5 * bf16_spacing(np.abs(ref) + 2.0 ** -19 * size) + 2.0 ** -19 * size
    err = np.abs(to_np(got) - ref)
    assert np.all(err <= bound), "%s: %g over its bound" % (what, (err / bound).max())


ROPE = [  # n, hq, hkv, d, rope, norm, interleaved, fused
    (1, 8, 1, 64, 64, True, False, False),
    (1, 1, 1, 128, 0, True, False, False),
    (3, 64, 8, 64, 64, True, False, True),
    (7, 3, 3, 64, 32, True, False, True),
    (5, 6, 2, 128, 128, True, True, True),
    (33, 32, 8, 128, 64, True, False, True),
    (9, 5, 1, 64, 16, False, True, False),
    (11, 4, 2, 128, 128, False, False, True),
    (700, 16, 2, 64, 64, True, True, True),
    (6001, 8, 1, 64, 64, True, False, True),
    (4000, 4, 4, 128, 128, True, False, False),
]


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_norm_rope(case):
    q, k, v, pos, cs, kw = rope_case(*case)
    n, hq, hkv, d = case[:4]
    qo, ko = sa.sinkattn_qk_norm_rope(q, k, pos, cs, **kw)
    check_turned(qo, q, kw["q_weight"], kw, pos, cs, "q")
    check_turned(ko, k, kw["k_weight"], kw, pos, cs, "k")
    # into a cache, some rows without a slot; k_out as before
    page, pages = 5, n // 5 + 3
    rng = np.random.default_rng(1)
    slots = rng.permutation(page * pages)[:n]
    slots[rng.random(n) < 0.2] = -1
    caches = [torch.full((pages, hkv, page, d), 7.0, dtype=torch.bfloat16, device="cuda")
              for _ in range(2)]
    for ask_k in (False, True):
        q2, k2 = sa.sinkattn_qk_norm_rope(
            q, k, pos, cs, v=v, k_cache=caches[0], v_cache=caches[1],
            slot_mapping=torch.tensor(slots).cuda(),
            k_out=torch.empty_like(ko) if ask_k else None, **kw)
        assert torch.equal(q2, qo)
        assert k2 is None if not ask_k else torch.equal(k2, ko)
        for cache, rows in ((caches[0], ko), (caches[1], v)):
            want = torch.full_like(cache, 7.0).transpose(1, 2).reshape(-1, hkv, d)
            want[torch.tensor(slots[slots >= 0]).cuda()] = rows[torch.tensor(slots >= 0).cuda()]
            assert torch.equal(cache.transpose(1, 2).reshape(-1, hkv, d), want)
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_norm_rope_backward(case):
    q, k, v, pos, cs, kw = rope_case(*case)
    n, hq, hkv, d = case[:4]
    rng = np.random.default_rng(5)
    dqo, dko = bf(rng, n, hq, d).cuda(), bf(rng, n, hkv, d).cuda()
    # the gradients as slices of one buffer
    wide = torch.full((n, hq + hkv + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dwq, dwk = sa.sinkattn_qk_norm_rope_backward(
        dqo, dko, q, k, pos, cs, dq=wide[:, :hq], dk=wide[:, hq:hq + hkv], **kw)
    assert torch.all(wide[:, -1] == 3.0)
    again = sa.sinkattn_qk_norm_rope_backward(dqo, dko, q, k, pos, cs, **kw)
    args = (kw["eps"], None if pos is None else pos.cpu().numpy(), np_of(cs), kw["interleaved"])
    for got, dw, dz, x, w, same in ((dq, dwq, dqo, q, kw["q_weight"], again[0::2]),
                                    (dk, dwk, dko, k, kw["k_weight"], again[1::2])):
        ref, ref_w = R.norm_rope_backward(np_of(dz), np_of(x), np_of(w), *args)
        mag = np.abs(np_of(dz))
        if cs is not None:  # |dz cos| + |dz' sin|
            other, cos, sin = R.angles(args[1], args[2], d, kw["interleaved"])
            mag = mag * np.abs(cos) + (mag * np.abs(sin))[..., other]
        size = mag
        if w is None:
            assert dw is None
        else:
            xs = np_of(x)
            r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + kw["eps"])
            u = xs * r
            g = np.abs(np_of(w)) * mag
            size = r * (g + np.abs(u) * (g * np.abs(u)).mean(-1, keepdims=True))
            terms = (np.abs(u) * mag).sum((0, 1))
            assert np.all(np.abs(to_np(dw) - ref_w) <= 2.0 ** -17 * terms)
            assert torch.equal(dw, same[1])  # the same call, the same bits
        bound = 0.5 * bf16_spacing(np.abs(ref) + 2.0 ** -18 * size) + 2.0 ** -18 * size
        assert np.all(np.abs(to_np(got) - ref) <= bound)
        assert torch.equal(got, same[0])


def test_norm_rope_gradient_by_differences():
    """The library's own forward, differenced in weight space, in which it is linear up
    to the outputs' rounding to bf16."""
    q, k, _, pos, cs, kw = rope_case(300, 8, 2, 64, 64, True, False, False)
    rng = np.random.default_rng(6)
    dqo, dko = bf(rng, 300, 8, 64).cuda(), bf(rng, 300, 2, 64).cuda()
    _, _, dwq, _ = sa.sinkattn_qk_norm_rope_backward(dqo, dko, q, k, pos, cs, **kw)
    h = 0.25
    step = torch.tensor(rng.choice([-1.0, 1.0], 64), dtype=torch.float32).cuda()
    f = lambda s: (sa.sinkattn_qk_norm_rope(
        q, k, pos, cs, **{**kw, "q_weight": kw["q_weight"] + s * step})[0].double() *
        dqo.double())
    up, down = f(h), f(-h)
    got = float(((up - down).sum()) / (2 * h))
    # each of the 153600 outputs is off by at most half a step, 2^-9 of it, of random sign:
    # six standard deviations of the sum
    noise = float(torch.sqrt((up ** 2 + down ** 2).sum())) * 2.0 ** -9 / (2 * h)
    assert abs(got - float((dwq.double() * step.double()).sum())) <= 6 * noise


def test_norm_rope_edges():
    q, k, v, pos, cs, kw = rope_case(4, 4, 2, 64, 64, True, False, False)
    # in place
    want = sa.sinkattn_qk_norm_rope(q, k, pos, cs, **kw)
    q2, k2 = q.clone(), k.clone()
    sa.sinkattn_qk_norm_rope(q2, k2, pos, cs, q_out=q2, k_out=k2, **kw)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    dz = [t.clone() for t in (q, k)]
    ref = sa.sinkattn_qk_norm_rope_backward(*dz, q, k, pos, cs, **kw)
    sa.sinkattn_qk_norm_rope_backward(*dz, q, k, pos, cs, dq=dz[0], dk=dz[1], **kw)
    assert torch.equal(dz[0], ref[0]) and torch.equal(dz[1], ref[1])
    # rows of zeros, tiny and huge ones (their squares overflow fp32)
    q2 = q.clone()
    q2[0] = 0
    q2[1] = q[1] * 1e-30
    q2[2] = q[2] * 1e30
    qo, _ = sa.sinkattn_qk_norm_rope(q2, k, pos, cs, **kw)
    check_turned(qo, q2, kw["q_weight"], kw, pos, cs, "sizes")
    assert torch.all(qo[0] == 0)
    dq = sa.sinkattn_qk_norm_rope_backward(q, k, q2, k, pos, cs, **kw)[0]
    ref = R.norm_rope_backward(np_of(q), np_of(q2), np_of(kw["q_weight"]), kw["eps"],
                               pos.cpu().numpy(), np_of(cs), False)[0]
    # huge rows: |dx| about 1e-30; half a step and the fp32 error, as a share of the row's size
    for t in range(4):
        size = np.abs(ref[t]).max()
        assert np.all(np.abs(to_np(dq[t]) - ref[t]) <=
                      0.5 * bf16_spacing(ref[t]) + 2.0 ** -14 * size), t
    # nothing to do; weights' gradients of no rows
    e = q[:0], k[:0]
    assert sa.sinkattn_qk_norm_rope(*e, pos[:0], cs, **kw)[0].shape == (0, 4, 64)
    g = sa.sinkattn_qk_norm_rope_backward(*e, *e, pos[:0], cs, **kw)
    assert torch.all(g[2] == 0) and torch.all(g[3] == 0)
    # positions and slots outside
    assert sa.sinkattn_get_device_error() == 0
    bad = pos.clone()
    bad[0], bad[1] = -3, 99
    got = sa.sinkattn_qk_norm_rope(q, k, bad, cs, **kw)
    assert sa.sinkattn_get_device_error() == 3
    assert torch.equal(got[0], sa.sinkattn_qk_norm_rope(q, k, bad.clamp(0, 36), cs, **kw)[0])
    cache = [torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.tensor([6, -1, 1 << 40, 5], device="cuda")
    sa.sinkattn_qk_norm_rope(q, k, pos, cs, v=v, k_cache=cache[0], v_cache=cache[1],
                             slot_mapping=slots, **kw)
    assert sa.sinkattn_get_device_error() == 2
    assert torch.equal(cache[0][1, :, 2], want[1][3]) and torch.equal(cache[1][1, :, 2], v[3])
    cache[0][1, :, 2] = 0
    assert torch.all(cache[0] == 0)
    with pytest.raises(ValueError):
        sa.sinkattn_qk_norm_rope(q, k, pos, cs, k_cache=cache[0], **kw)
    with pytest.raises(ValueError):
        sa.sinkattn_qk_norm_rope(q.float(), k, pos, cs, **kw)
    with pytest.raises(ValueError):
        sa.sinkattn_qk_norm_rope(q, k, pos.long(), cs, **kw)


# ---- tree attention --------------------------------------------------------------

def make_parents(rng, n, kind):
    if n == 0:
        return []
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    if kind == "mixed":
        return [-1] + [int(rng.integers(-1, i)) for i in range(1, n)]
    return [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]


class Tree:
    def __init__(self, new, old, page, hq, hkv, d, kind="tree", sinks=True, window=0, seed=0,
                 pad=0, spare_cols=1, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens = [max(n + o, 0) for n, o in zip(new, old)]
        self.cu = offsets(new)
        self.window, self.scale, self.hq = window, d ** -0.5, hq
        n = int(self.cu[-1]) + pad
        self.par = (None if kind is None else
                    np.concatenate([make_parents(rng, m, kind) for m in new] +
                                   [[0] * pad]).astype(np.int64))
        self.q = bf(rng, n, hq, d, scale=q_scale)
        need = [-(-l // page) for l in self.lens]
        pages = sum(need) + 2
        perm = rng.permutation(pages)
        width = max(max(need), 1) + spare_cols
        self.table = np.full((len(new), width), FAR)
        self.k = torch.full((pages, hkv, page, d), NAN, dtype=torch.bfloat16)
        self.v = torch.full((pages, hkv, page, d), NAN, dtype=torch.bfloat16)
        self.rows = [], []
        at = 0
        for b, l in enumerate(self.lens):
            kr, vr = bf(rng, l, hkv, d), bf(rng, l, hkv, d)
            self.rows[0].append(kr.double().numpy())
            self.rows[1].append(vr.double().numpy())
            self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            # positions that no row sees stay NaN
            first = 0
            if window and new[b]:
                first = max(0, l - new[b] - window + 1)
            pos = np.arange(first, l)
            p, s = torch.tensor(self.table[b][pos // page]), torch.tensor(pos % page)
            self.k[p, :, s], self.v[p, :, s] = kr[first:], vr[first:]
            if window:
                self.table[b, :first // page] = FAR
        self.max_q, self.max_k = max(max(new), 1), max(max(self.lens), 1)
        self.sinks = torch.tensor(rng.normal(size=hq), dtype=torch.float32) if sinks else None

    def args(self):
        return (self.q.cuda(), i32(self.cu), self.k.cuda(), self.v.cuda(), i32(self.table),
                i32(self.lens), self.max_q, self.max_k)

    def kw(self):
        return dict(parents=None if self.par is None else i32(self.par),
                    sinks=None if self.sinks is None else self.sinks.cuda(), window=self.window)

    def ref(self):
        return R.tree_attention(self.q.double().numpy(), self.cu, self.par, *self.rows, self.lens,
                                None if self.sinks is None else self.sinks.double().numpy(),
                                self.window, self.scale)

    def check(self, what="", **kw):
        n = int(self.cu[-1])
        out = torch.full(self.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], 5.0, device="cuda")
        sa.sinkattn_decode_tree(*self.args(), **self.kw(), out=out, lse=lse, **kw)
        assert sa.sinkattn_get_device_error() == 0
        ref = self.ref()
        check_close(out[:n], lse[:n], ref[0][:n], ref[1][:n], what)
        assert torch.all(out[n:] == 5.0) and torch.all(lse[n:] == 5.0)
        return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [None, "tree", "star", "roots", "mixed"])
def test_tree_shapes(kind, d):
    new = [1, 2, 7, 0, 16, 33, 3]
    old = [0, 5, 130, 9, 1, 500, 127]
    Tree(new, old, 16, 8, 1, d, kind).check()
    Tree(new, old, 16, 6, 2, d, kind, sinks=False, seed=1, pad=3).check()


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 256])
def test_tree_pages(page):
    Tree([5, 1, 12], [200, 31, 333], page, 8, 2, 64).check()
    Tree([5, 1, 12], [200, 31, 333], page, 4, 2, 128, window=50).check()


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 17])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_groups(group, d):
    Tree([1, 9, 20], [100, 300, 40], 16, 2 * group, 2, d).check()


@pytest.mark.parametrize("window", [1, 2, 3, 16, 100, 127, 128, 129, 300, 4000, 2 ** 31 - 1])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_windows(window, d):
    new, old = [1, 6, 40, 9], [0, 500, 129, 256]
    Tree(new, old, 16, 8, 2, d, window=window).check()
    Tree(new, old, 16, 4, 4, d, None, window=window, sinks=False).check()


@pytest.mark.parametrize("length", [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257,
                                    511, 512, 513])
def test_tree_context_lengths(length):
    Tree([4, 1], [length, length + 1], 16, 8, 1, 64).check()
    Tree([130], [length], 16, 2, 2, 128).check()


@pytest.mark.parametrize("splits", [0, 1, 2, 3, 7, 40, 64, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_splits(splits, d):
    t = Tree([5, 17, 1], [1500, 300, 20], 16, 8, 1, d)
    t.check(num_splits=splits)
    Tree([5, 17, 1], [1500, 300, 20], 16, 8, 1, d, window=200, sinks=False).check(
        num_splits=splits)


def test_tree_long_chain_and_wide_tree():
    Tree([300, 257], [100, 0], 16, 4, 2, 64, None).check()
    Tree([300, 257], [100, 0], 16, 2, 2, 128, "tree").check()


def test_tree_more_rows_than_keys():
    """Lq > Lk: the first rows have no key of their own, and may see nothing."""
    for sinks in (False, True):
        Tree([5, 3], [-2, -3], 16, 8, 2, 64, None, sinks=sinks).check()
        Tree([9], [-4], 16, 8, 2, 128, "tree", sinks=sinks).check()


def test_tree_large_scores_and_sinks():
    t = Tree([6, 9], [300, 700], 16, 8, 2, 64, q_scale=40.0)
    t.check("peaked")
    t = Tree([6, 9], [300, 700], 16, 8, 2, 64)
    t.sinks += 60.0
    t.check("sinks above")
    t.sinks -= 300.0
    t.check("sinks below")


def test_tree_wide_groups_and_many_sequences():
    Tree([3, 1], [70, 400], 16, 260, 2, 64).check("130 heads a group")
    Tree([2, 5], [20, 300], 16, 150, 1, 128, None).check("150 heads, one KV head")
    rng = np.random.default_rng(2)
    old = rng.integers(0, 40, 4200)
    old[::700] = 600  # above 4096 sequences items are not shared out
    Tree([1] * 4200, old.tolist(), 16, 2, 1, 64).check("4200 sequences")
    Tree([1, 0] * 1500, rng.integers(0, 400, 3000).tolist(), 16, 2, 2, 64).check("shares of many")


@pytest.mark.parametrize("splits", [0, 1])
def test_tree_sinks_beyond_log2_units(splits):
    """Sinks whose log2 value overflows fp32: a huge one leaves nothing to the keys, one at
    the other end changes nothing."""
    t = Tree([5, 17], [1500, 30], 16, 8, 2, 64)
    a, kw = t.args(), t.kw()
    none = sa.sinkattn_decode_tree(*a, **{**kw, "sinks": None}, num_splits=splits)
    for x in (3e38, float("inf")):
        out, lse = sa.sinkattn_decode_tree(
            *a, **{**kw, "sinks": torch.full((8,), x, device="cuda")}, num_splits=splits)
        assert torch.all(out == 0) and torch.all(lse == torch.tensor(x).cuda())
    for x in (-3e38, -float("inf")):
        out, lse = sa.sinkattn_decode_tree(
            *a, **{**kw, "sinks": torch.full((8,), x, device="cuda")}, num_splits=splits)
        assert torch.equal(out, none[0]) and torch.equal(lse, none[1])


def test_tree_equals_prefill():
    """A chain is the paged prefill's causal mask."""
    t = Tree([5, 17, 1], [1500, 300, 20], 16, 8, 2, 64, None)
    for c in (t.k, t.v):
        c.nan_to_num_(0.0)
    t.table[t.table == FAR] = 0
    out, lse = t.check()
    a = t.args()
    o, l = sa.sinkattn_prefill_paged(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7],
                                     sinks=t.sinks.cuda())
    assert (out.float() - o.float()).abs().max() <= 1e-2 and (lse - l).abs().max() <= 1e-3


def test_tree_bad_input_is_recorded():
    t = Tree([5, 3], [100, 200], 16, 8, 2, 64)
    a, kw = list(t.args()), t.kw()
    good = sa.sinkattn_decode_tree(*a, **kw)
    # a parent that is not below its row counts as none
    par = t.par.copy()
    par[3] = 3
    want = t.par.copy()
    want[3] = -1
    out = sa.sinkattn_decode_tree(*a, **{**kw, "parents": i32(par)})
    assert sa.sinkattn_get_device_error() == 2
    ref = sa.sinkattn_decode_tree(*a, **{**kw, "parents": i32(want)})
    assert sa.sinkattn_get_device_error() == 0 and torch.equal(out[0], ref[0])
    # a page outside the cache: its keys and values are zeros, others' rows are untouched
    table = t.table.copy()
    table[0, 2] = -7
    out = sa.sinkattn_decode_tree(*a[:4], i32(table), *a[5:], **kw)
    assert sa.sinkattn_get_device_error() == 2
    t.rows[0][0][32:48] = 0
    t.rows[1][0][32:48] = 0
    ref = t.ref()
    check_close(out[0], out[1], ref[0], ref[1])
    assert torch.equal(out[0][5:], good[0][5:])
    # lengths past their bounds are cut
    out = sa.sinkattn_decode_tree(*a[:6], 4, a[7], **kw)
    assert sa.sinkattn_get_device_error() == 3
    sa.sinkattn_decode_tree(*a[:7], 150, **kw)
    assert sa.sinkattn_get_device_error() == 3
    lens = i32([-5, 203])
    out = sa.sinkattn_decode_tree(*a[:5], lens, *a[6:], **kw)
    assert sa.sinkattn_get_device_error() == 3
    assert torch.all(out[0][:5] == 0) and torch.equal(out[0][5:], good[0][5:])
    with pytest.raises(ValueError):
        sa.sinkattn_decode_tree(a[0], *a[1:], **{**kw, "parents": i32(par[:-1])})
    with pytest.raises(ValueError):
        sa.sinkattn_decode_tree(a[0].float(), *a[1:], **kw)


def test_tree_repeats_and_shares_nothing():
    """Bitwise the same again, on another stream, and in two graphs that share a
    workspace."""
    t = Tree([5, 17, 1], [1500, 300, 20], 16, 8, 1, 64)
    a, kw = t.args(), t.kw()
    want = sa.sinkattn_decode_tree(*a, **kw, num_splits=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sa.sinkattn_decode_tree(*a, **kw, num_splits=4, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    u = Tree([5, 17, 1], [1500, 300, 20], 16, 8, 1, 64, seed=9)
    need = sa.sinkattn_decode_tree_workspace_size(3, 23, t.max_q, t.max_k, 8, 1, 64, 0, 4)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (t, u):
        args, kwx = x.args(), x.kw()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = sa.sinkattn_decode_tree(*args, **kwx, num_splits=4, workspace=ws)
        graphs.append((g, res, args, kwx))
    for i in (0, 1, 0):
        graphs[i][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], want[0])
    ref = u.ref()
    check_close(graphs[1][1][0], graphs[1][1][1], ref[0], ref[1])


# ---- verification ----------------------------------------------------------------

def probs(rng, n, vocab, temp):
    x = temp * rng.normal(size=(n, vocab))
    x = np.exp(x - x.max(1, keepdims=True))
    return (x / x.sum(1, keepdims=True)).astype(np.float32)


def verify_case(new, vocab, kind, draft, temp=2.0, seed=0, near=0.5):
    rng = np.random.default_rng(seed)
    cu, n = offsets(new), sum(new)
    par = np.concatenate([make_parents(rng, m, kind) for m in new]).astype(np.int64) if kind else None
    p = probs(rng, n, vocab, temp)
    q = p * np.exp(near * rng.normal(size=p.shape))
    q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    tokens = np.zeros(n, np.int64)
    for b, m in enumerate(new):
        for i in range(1, m):
            up = i - 1 if par is None else max(int(par[cu[b] + i]), 0)
            row = q[cu[b] + up].astype(np.float64)
            tokens[cu[b] + i] = (rng.choice(vocab, p=row / row.sum()) if draft else
                                 rng.choice(np.argsort(-row)[:6]))
    u = rng.random(n).astype(np.float32)
    return p, q if draft else None, tokens, par, u, cu


def check_verify(p, q, tokens, par, u, cu, width, code=0, **kw):
    ref = R.verify(p, q, tokens, par, u, cu, width)
    c = lambda x, t: None if x is None else torch.tensor(x, dtype=t).cuda()
    got = sa.sinkattn_verify_tree(c(p, torch.float32), c(tokens, torch.int64),
                                  c(u, torch.float32), i32(cu), width,
                                  draft_probs=c(q, torch.float32),
                                  parents=c(par, torch.int32), **kw)
    assert sa.sinkattn_get_device_error() == code
    for x, want in zip(got, ref):
        assert np.array_equal(x.cpu().numpy().astype(np.int64), want)
    return ref


@pytest.mark.parametrize("vocab", [1, 2, 5, 127, 128, 1000, 4099, 50001, 131072])
@pytest.mark.parametrize("draft", [False, True])
def test_verify_vocab(vocab, draft):
    for kind in (None, "tree", "star"):
        c = verify_case([1, 5, 2, 8], vocab, kind, draft)
        check_verify(*c, 8)


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("kind", [None, "tree", "star", "mixed", "roots"])
@pytest.mark.parametrize("temp", [0.0, 1.0, 6.0])
def test_verify_trees(kind, draft, temp):
    seen = 0
    for seed in range(3):
        c = verify_case([0, 1, 33, 64, 7, 2, 0, 40], 300, kind, draft, temp, seed, near=1.0)
        seen += int(check_verify(*c, 64)[1].sum())
    # the 18 roots, and some drafts where they are drawn near the target
    assert seen > (18 if draft and kind != "roots" else 17)


def test_verify_many_rejections():
    """Stars whose drafts come from a distribution far from the target."""
    for draft in (False, True):
        c = list(verify_case([200, 300], 64, "star", draft, 3.0, near=3.0))
        c[4][:] = np.maximum(c[4], 0.9)
        check_verify(*c, 300)
    c = list(verify_case([1024], 700, "star", True, 1.0, near=4.0))
    c[4][:] = 0.999
    check_verify(*c, 1024)
    c = verify_case([1024], 40, None, True, 0.5, near=0.0)  # the target's own drafts
    assert check_verify(*c, 1024)[1][0] == 1024


def test_verify_edges():
    # certain targets, both ends of the random numbers, and drafts with no chance
    eye = np.eye(8, dtype=np.float32)
    p, cu = eye[[1, 2, 3, 4]], np.array([0, 4])
    top = np.float32(1 - 2.0 ** -24)
    for u in (0.0, top):
        for q in (None, eye[[1, 2, 3, 4]]):
            ref = check_verify(p, q, np.array([0, 1, 2, 3]), None, np.full(4, u, np.float32), cu, 4)
            assert ref[1][0] == 4 and ref[2][0] == 4
        ref = check_verify(p, None, np.array([0, 7, 2, 3]), None, np.full(4, u, np.float32), cu, 4)
        assert ref[1][0] == 1 and ref[2][0] == 1
    # nothing left of the target: drawn from the target itself
    half = np.full((2, 2), 0.5, np.float32)
    check_verify(half, half * 2, np.array([0, 1]), None, np.float32([0.7, 0.6]), [0, 2], 2)
    # NaN, negative and large values; a row of zeros
    odd = np.float32([[NAN, 0.25, -1.0, 0.75], [0, 0, 0, 0]])
    check_verify(odd, None, np.array([0, 3]), None, np.float32([0.5, 0.9]), [0, 2], 2)
    check_verify(odd, None, np.array([0, 3]), None, np.float32([0.5, 0.1]), [0, 2], 2, code=5)
    # tokens outside the vocabulary, parents that do not come before
    p = probs(np.random.default_rng(0), 4, 8, 1.0)
    args = lambda t, par: (p, None, np.array(t), np.array(par), np.zeros(4, np.float32), [0, 4], 4)
    assert check_verify(*args([0, -1, 8, 2], [-1, 0, 0, 0]), code=2)[0][0].tolist() == [0, 3, -1, -1]
    check_verify(*args([0, 1, 1, 1], [-1, 2, 2, 0]), code=2)
    # more rows than the bound
    c = verify_case([6], 50, "tree", True, 0.1)
    check_verify(*c, 4, code=3)


def test_verify_graph():
    c = verify_case([5, 9, 16], 5000, "tree", True, seed=3)
    ref = R.verify(*c[:2], c[2], c[3], c[4], c[5], 16)
    d = [torch.tensor(c[0]).cuda(), torch.tensor(c[2]).cuda(), torch.tensor(c[4]).cuda(), i32(c[5])]
    kw = dict(draft_probs=torch.tensor(c[1]).cuda(), parents=i32(c[3]))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        res = sa.sinkattn_verify_tree(*d, 16, **kw)
    for _ in range(2):
        for t in res:
            t.fill_(99)
        g.replay()
        for x, want in zip(res, ref):
            assert np.array_equal(x.cpu().numpy().astype(np.int64), want)


# ---- compaction ------------------------------------------------------------------

def compact_case(new, old, page, hkv, d, seed=0, ended=0.3, path=True, width=None):
    rng = np.random.default_rng(seed)
    lens, cu = [n + o for n, o in zip(new, old)], offsets(new)
    need = [-(-l // page) for l in lens]
    pages = sum(need) + 3
    perm, at = rng.permutation(pages), 0
    table = np.full((len(new), max(max(need), 1) + 1), FAR)
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    width = width or max(max(new), 1)
    paths, num = np.full((len(new), width), -1), np.zeros(len(new), np.int64)
    for b, n in enumerate(new):
        kept = np.sort(rng.permutation(n)[:rng.integers(0, n + 1)])[:width]
        paths[b, :kept.size], num[b] = kept, kept.size
        if rng.random() < ended:
            num[b] = -1
    k, v = bf(rng, pages, hkv, page, d), bf(rng, pages, hkv, page, d)
    free = rng.permutation(pages + 5)
    return k, v, table, lens, cu, paths if path else None, num, free, sum(need) + 2


def check_compact(case, in_place=False, code=0):
    k, v, table, lens, cu, path, num, free, head = case
    ref = R.compact(k.float().numpy(), v.float().numpy(), table, lens, cu, path, num, free, head)
    kc, vc, ln, fr, hd = k.cuda(), v.cuda(), i32(lens), i32(free), i32([head])
    new, out = sa.sinkattn_compact(kc, vc, i32(table), ln, i32(cu),
                                   None if path is None else i32(path), i32(num), fr, hd,
                                   seqlens_out=ln if in_place else None,
                                   free_head_out=hd if in_place else None)
    assert sa.sinkattn_get_device_error() == code
    for got, want in zip((kc, vc, new, fr), ref):
        assert np.array_equal(got.float().cpu().numpy(), np.asarray(want, np.float32))
    assert out.item() == ref[4] and hd.item() == (ref[4] if in_place else head)


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_compact(page, d):
    new, old = [1, 0, 16, 64, 7, 33, 2], [0, 5, 100, 31, 64, 15, 0]
    for seed in range(3):
        check_compact(compact_case(new, old, page, 3, d, seed), in_place=seed == 1)
    check_compact(compact_case(new, old, page, 1, d, path=False))
    check_compact(compact_case(new, old, page, 8, d, width=5))


def test_compact_many_sequences():
    rng = np.random.default_rng(0)
    new, old = rng.integers(0, 4, 2500), rng.integers(0, 40, 2500)
    check_compact(compact_case(new.tolist(), old.tolist(), 4, 1, 64), in_place=True)
    check_compact(compact_case([3] * 1025, [700] * 1025, 16, 1, 64, ended=0.9))


def test_compact_edges():
    case = list(compact_case([4, 5], [30, 20], 8, 2, 64, ended=0.0))
    # pages that the list never gave are not put back
    case[2] = case[2].copy()
    case[5][1, :2], case[6][:] = [1, 3], [-1, 2]
    case[2][0, 2] = -1
    check_compact(case)
    # a path that does not increase ends there; counts past the rows are cut
    good = list(compact_case([4, 5], [30, 20], 8, 2, 64, ended=0.0))
    good[5] = np.array([[0, 2, 3, -1, -1], [0, 1, 2, 3, 4]])
    good[6] = np.array([2, 5])
    ref = R.compact(good[0].float().numpy(), good[1].float().numpy(), *good[2:])
    for path, num, code in (([[0, 2, 2, 3, 3], [0, 1, 2, 3, 4]], [4, 5], 2),
                            ([[0, 2, 4, 3, 3], [0, 1, 2, 3, 4]], [3, 5], 2),
                            ([[0, 2, -1, 3, 3], [0, 1, 2, 3, 4]], [2, 9], 3)):
        kc, vc, fr = good[0].cuda(), good[1].cuda(), i32(good[7])
        new, out = sa.sinkattn_compact(kc, vc, i32(good[2]), i32(good[3]), i32(good[4]),
                                       i32(path), i32(num), fr, i32([good[8]]))
        assert sa.sinkattn_get_device_error() == code
        for x, want in zip((kc, vc, new, fr), ref):
            assert np.array_equal(x.float().cpu().numpy(), np.asarray(want, np.float32))
    # a long path that stops increasing in its second batch of rows
    far = list(compact_case([60], [10], 16, 2, 64, ended=0.0))
    far[5] = np.arange(4, 60)[None, :].copy()
    far[6] = np.array([36])
    ref = R.compact(far[0].float().numpy(), far[1].float().numpy(), *far[2:])
    bad = far[5].copy()
    bad[0, 36] = bad[0, 35]
    kc, vc, fr = far[0].cuda(), far[1].cuda(), i32(far[7])
    new, out = sa.sinkattn_compact(kc, vc, i32(far[2]), i32(far[3]), i32(far[4]), i32(bad),
                                   i32([50]), fr, i32([far[8]]))
    assert sa.sinkattn_get_device_error() == 2
    for x, want in zip((kc, vc, new, fr), ref):
        assert np.array_equal(x.float().cpu().numpy(), np.asarray(want, np.float32))
    # more pages than the list has handed out
    short = list(compact_case([4, 5], [30, 20], 8, 2, 64, ended=1.1))
    short[8] = 2
    check_compact(short, code=4)
    # no sequences
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    kc = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    new, out = sa.sinkattn_compact(kc, kc.clone(), i32(np.zeros((0, 2))), e, i32([0]), None, e,
                                   i32([1, 2, 3]), i32([2]))
    assert new.numel() == 0 and out.item() == 2


# ---- together --------------------------------------------------------------------

def test_step_together():
    """Steps of a small batch as one captured graph, its state updated in place: map,
    norm + rotation + write, attention, verification, compaction. Attention is checked
    against the rows that the paths should have left in the cache."""
    rng = np.random.default_rng(11)
    batch, rows, hq, hkv, d, page, vocab, width = 3, 6, 4, 2, 64, 4, 50, 16
    par = np.array([-1, 0, 0, 1, 2, 3] * batch)
    depth = np.array([0, 1, 1, 2, 2, 3] * batch)
    at_rows = np.arange(batch + 1) * rows
    cu = i32(at_rows)
    pages = 40
    kc = torch.full((pages, hkv, page, d), NAN, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    free, head = i32(rng.permutation(pages)), i32([0])
    lens = i32([0] * batch)
    cs = rope_table(rng, 200, d).cuda()
    n = batch * rows
    x = torch.empty((n, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    p, q = (torch.empty((n, vocab), device="cuda") for _ in range(2))
    tok = torch.zeros(n, dtype=torch.int64, device="cuda")
    u = torch.zeros(n, device="cuda")
    w = torch.ones(d, device="cuda")
    parents, depths = i32(par), i32(depth)

    def step():
        old = lens.clone()
        lens.add_(rows)
        slots, _, _ = sa.sinkattn_page_map(lens, table, free, head, page, cu_seqlens_q=cu,
                                           total_q=n, free_head_out=head)
        pos = old.repeat_interleave(rows, output_size=n) + depths
        qo, _ = sa.sinkattn_qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], pos, cs, q_weight=w,
                                         k_weight=w, v=x[:, hq + hkv:], slot_mapping=slots,
                                         k_cache=kc, v_cache=vc)
        out, lse = sa.sinkattn_decode_tree(qo, cu, kc, vc, table, lens, rows, width * page,
                                           parents=parents)
        path, num, nxt = sa.sinkattn_verify_tree(p, tok, u, cu, rows, draft_probs=q,
                                                 parents=parents)
        sa.sinkattn_compact(kc, vc, table, lens, cu, path, num, free, head, seqlens_out=lens,
                            free_head_out=head)
        return pos, qo, out, lse, path, num, nxt

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        res = step()
    kept = [[np.zeros((0, hkv, d))] * 2 for _ in range(batch)]
    for it in range(4):
        x.copy_(bf(rng, n, hq + 2 * hkv, d))
        c = verify_case([rows] * batch, vocab, "tree", True, seed=it)
        p.copy_(torch.tensor(c[0]))
        q.copy_(torch.tensor(c[1]))
        tok.copy_(torch.tensor(c[2]))
        u.copy_(torch.tensor(c[4]))
        graph.replay()
        torch.cuda.synchronize()
        assert sa.sinkattn_get_device_error() == 0
        pos, qo, out, lse, path, num, nxt = res
        ref = R.verify(c[0], c[1], c[2], par, c[4], at_rows, rows)
        for got, want in zip((path, num, nxt), ref):
            assert np.array_equal(got.cpu().numpy().astype(np.int64), want)
        # keys rounded from float64: one that falls on the other side of a rounding border
        # than the cache's moves a score by 2^-8 of one of its 64 products
        kz = torch.tensor(R.norm_rope(np_of(x[:, hq:hq + hkv]), np.ones(d), 1e-6,
                                      pos.cpu().numpy(), np_of(cs))).to(torch.bfloat16)
        k_rows, v_rows = [], []
        for b in range(batch):
            at = slice(b * rows, (b + 1) * rows)
            k_rows.append(np.concatenate([kept[b][0], kz[at].double().numpy()]))
            v_rows.append(np.concatenate([kept[b][1], np_of(x[at, hq + hkv:])]))
        o, l = R.tree_attention(np_of(qo), at_rows, par, k_rows, v_rows,
                                [len(k) for k in k_rows], None, 0, d ** -0.5)
        check_close(out, lse, o, l, "step %d" % it)
        for b in range(batch):
            rows_b = ref[0][b][:ref[1][b]]
            base = len(kept[b][0])
            kept[b] = [np.concatenate([r[b][:base], r[b][base + rows_b]])
                       for r in (k_rows, v_rows)]
        assert lens.tolist() == [len(k[0]) for k in kept]
        used = [-(-len(k[0]) // page) for k in kept]
        assert head.item() == sum(used)
        held = [t for b in range(batch) for t in table[b, :used[b]].tolist()]
        assert sorted(free[sum(used):].tolist() + held) == list(range(pages))
