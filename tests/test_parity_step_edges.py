"""Edges of the speculative decoding step on the GPU: verification whose drafts have used
up a token's mass many times over or whose answer hangs on its last bits; values that are
not finite in the attention, the bits of its weights, long contexts; long sums of weight
gradients."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from helpers import to_np
from oracle import step as R
from test_parity_step import Tree, check_verify, i32

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


# ---- verification ----------------------------------------------------------------

def star(children, p, q, token, u, u0):
    """Stars of `children` drafts, all the same token, whose root has target p and draft q;
    u: the random numbers of the drafts, u0 those of the roots (one star each)."""
    batch, rows = len(u0), children + 1
    n = batch * rows
    uniforms = np.full(n, u, np.float32)
    uniforms[::rows] = u0
    par = np.tile([-1] + [0] * children, batch)
    tokens = np.full(n, token, np.int64)
    return (np.tile(np.float32(p), (n, 1)), np.tile(np.float32(q), (n, 1)), tokens, par, uniforms,
            np.arange(batch + 1) * rows)




@pytest.mark.parametrize("p,q", [
    ([0.5, 0.5], [1.0, 0.0]),        # after 31 rejections q has been taken off 16 times
    ([0.0625, 0.9375], [1.0, 0.0]),  # after 17 exactly 16 times
    ([0.0625, 0.4375, 0.5], [1.0, 0.0, 0.0]),
    ([0.0, 1.0], [1.0, 0.0]),
    ([0.05, 0.05, 0.3, 0.6], [0.9, 0.1, 0.0, 0.0]),
], ids=["half", "sixteenth", "three", "none", "share"])
@pytest.mark.parametrize("children", [1, 15, 16, 17, 18, 31, 33, 63, 64, 255, 300, 1023])
def test_verify_rejects_the_same_token_again_and_again(p, q, children):
    u0 = np.float32([0.0, 0.01, 0.05, 0.3, 0.5, 0.7, 0.93, 1 - 2.0 ** -24])
    for u in (0.5, 0.9, 1 - 2.0 ** -24):
        ref = check_verify(*star(children, p, q, 0, u, u0), children + 1)
        if ref[1][0] == 1 and children > 1 and float(p[0]) <= float(q[0]):
            assert not np.any(ref[2] == 0)  # its mass is gone


@pytest.mark.parametrize("children", [31, 63, 255])
def test_verify_stars_of_peaked_drafts(children):
    """Drafts drawn from a distribution with 0.98 on one token, of which the target has up
    to 0.4."""
    rng = np.random.default_rng(children)
    batch, rows, vocab = 2000, children + 1, 50
    n = batch * rows
    p = rng.dirichlet(np.full(vocab, 0.3), batch)
    top, share = rng.integers(0, vocab, batch), rng.uniform(0, 0.4, batch)
    p *= (1 - share)[:, None]
    p[np.arange(batch), top] += share
    p, top = p.astype(np.float32).repeat(rows, 0), top.repeat(rows)
    q = np.full((n, vocab), 0.02 / (vocab - 1), np.float32)
    q[np.arange(n), top] = 0.98
    tokens = np.where(rng.random(n) < 0.98, top, rng.integers(0, vocab, n))
    par = np.tile([-1] + [0] * children, batch)
    check_verify(p, q, tokens, par, rng.random(n).astype(np.float32), np.arange(batch + 1) * rows,
                 rows)


def one_root(p, q, tokens, u):
    """The next token of a star whose drafts are all rejected."""
    n = len(tokens) + 1
    full = lambda x: torch.tensor(np.tile(np.float32(x), (n, 1))).cuda()  # noqa: E731
    _, num, nxt = sa.sinkattn_verify_tree(
        full(p), torch.tensor([0] + tokens).cuda(), torch.tensor(np.float32(u)).cuda(),
        i32([0, n]), n, draft_probs=None if q is None else full(q), parents=i32([-1] + [0] * (n - 1)))
    assert num.item() == 1
    return nxt.item()


def test_verify_draw_is_exact():
    """Sums that differ below a double's 53 bits: the draw compares whole multiples of 2^-60."""
    one = 2.0 ** -60
    a, b = 2 ** 58 + 2 ** 35, 2 ** 29 + 2 ** 7
    p = [a, b, a, 2 ** 29 + 64, 63]
    # through token 1 the sum is a + b; half of all of it is 0.5 below that
    assert Fraction(sum(p), 2) == a + b - Fraction(1, 2)
    assert one_root([x * one for x in p], None, [], [0.5]) == 1
    p[4] = 64  # half of it is now just that: the sum has to exceed it
    assert Fraction(sum(p), 2) == a + b
    assert one_root([x * one for x in p], None, [], [0.5]) == 2
    p[4] = 65
    assert one_root([x * one for x in p], None, [], [0.5]) == 2


def test_verify_taken_mass_is_exact():
    """Two rejections of token 0 whose residual sum has bits down to 2^-60: they decide
    between tokens 1 and 2."""
    one, top = 2.0 ** -60, 1 - 2.0 ** -24
    # what is left of token 1 is (d - X) / 2 with X = p2 + p3; it exceeds half the sum while
    # d > 3 X
    for extra, want in ((3, 2), (-3, 1)):
        x = 2 ** 40 // 3 + extra
        p2 = x >> 16 << 16
        p = [0.5 - 2.0 ** -19, 0.5 + 2.0 ** -20, p2 * one, (x - p2) * one]
        assert [float(np.float32(v)) for v in p] == p
        q = [Fraction(1, 2), Fraction(1, 2), 0, 0]
        v = s = None
        for _ in range(2):
            before = (p, Fraction(1)) if v is None else (v, s)
            v = [max(Fraction(y) - before[1] * z, Fraction(0)) for y, z in zip(before[0], q)]
            s = sum(v)
        assert (v[0] + v[1] > s / 2) == (want == 1)
        assert one_root(p, [0.5, 0.5, 0.0, 0.0], [0, 0], [0.5, top, top]) == want


# ---- attention: what is not finite ---------------------------------------------------

@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_nan_of_a_sink_or_a_query_stays_one(d, splits, sinks):
    """A NaN sink is a NaN in every row of its head, a NaN query in its own; the others
    keep their bits."""
    t = Tree([5, 17, 1, 2], [1500, 300, 20, -2], 16, 8, 2, d, sinks=sinks)
    a, kw = list(t.args()), t.kw()
    out, lse = sa.sinkattn_decode_tree(*a, **kw, num_splits=splits)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    if sinks:
        kw["sinks"][3] = NAN
        hit[:, 3] = True
    a[0][2, 6, 11] = NAN
    a[0][9, 0, 0] = NAN
    hit[2, 6] = hit[9, 0] = True
    o, l = sa.sinkattn_decode_tree(*a, **kw, num_splits=splits)
    assert torch.equal(torch.isnan(l), hit) and torch.equal(l[~hit], lse[~hit])
    assert torch.all(torch.isnan(o[hit])) and torch.equal(o[~hit], out[~hit])
    assert sa.sinkattn_get_device_error() == 0


HIDDEN = [  # new, old, window, parents' kind
    ([6, 9, 3], [100, 700, 0], 0, "tree"),
    ([6, 9, 3], [100, 700, 0], 0, "star"),
    ([6, 40, 3], [61, 122, 63], 0, None),
    ([40, 70], [1000, 30], 0, "mixed"),
    ([40, 70], [1000, 30], 24, "tree"),
    ([6, 9, 64], [200, 700, 300], 100, None),
    ([6, 9, 64], [200, 700, 300], 64, "tree"),
    ([5], [40], 3, None),
    ([20, 1], [-5, 600], 0, "tree"),
    ([3, 7, 1] * 100, [50, 400, 333] * 100, 0, "tree"),
    ([2, 30] * 150, [500, 90] * 150, 40, "tree"),
]


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", HIDDEN, ids=lambda c: "%d-%s-%s" % (len(c[0]), c[2], c[3]))
def test_tree_values_that_are_not_finite_reach_only_rows_that_see_them(case, d, splits, value):
    new, old, window, kind = case
    t = Tree(new, old, 16, 6, 2, d, kind, window=window, sinks=False)
    rng = np.random.default_rng(1)
    bad = []  # (sequence, position, KV head, dim)
    for b, (n, lk) in enumerate(zip(new, t.lens)):
        last = [lk - 1, lk - 1 - n // 2, lk - n, lk - n - max(window - 2, 1), lk - n - window + 2]
        for pos in last + rng.integers(max(lk - n - (window or 80), 0), lk, 3).tolist():
            if max(0, lk - n - window + 1 if window else 0) <= pos < lk:
                bad.append((b, int(pos), int(rng.integers(2)), int(rng.integers(d))))
    a, kw = list(t.args()), t.kw()
    at = lambda b, pos: (int(t.table[b][pos // 16]), pos % 16)  # noqa: E731
    for b, pos, h, e in bad:
        pg, s = at(b, pos)
        a[3][pg, h, s, e] = 0.0
    out, lse = sa.sinkattn_decode_tree(*a, **kw, num_splits=splits)
    hit = np.zeros(out.shape, bool)  # elements whose row sees one of them
    for b, pos, h, e in bad:
        pg, s = at(b, pos)
        a[3][pg, h, s, e] = value
        par = [i - 1 for i in range(new[b])] if t.par is None else t.par[t.cu[b]:t.cu[b + 1]]
        context = t.lens[b] - new[b]
        for i in range(new[b]):
            up = R.line(par, i)
            place = pos if pos < context else None
            if pos >= context and pos - context in up:
                place = context + len(up) - 1 - up.index(pos - context)
            if place is not None and (not window or place > context + len(up) - 1 - window):
                hit[t.cu[b] + i, 3 * h:3 * h + 3, e] = True
    hit = torch.tensor(hit).cuda()
    assert 0 < int(hit.sum()) < hit.numel()
    o, l = sa.sinkattn_decode_tree(*a, **kw, num_splits=splits)
    assert sa.sinkattn_get_device_error() == 0
    assert torch.equal(l, lse) and torch.equal(o[~hit], out[~hit])
    assert not torch.any(torch.isfinite(o[hit]))


@pytest.mark.parametrize("splits", [0, 1])
def test_tree_keys_that_are_not_finite_reach_only_rows_that_see_them(splits):
    t = Tree([6, 9], [300, 700], 16, 8, 2, 64, "star")
    a, kw = list(t.args()), t.kw()
    out, lse = sa.sinkattn_decode_tree(*a, **kw, num_splits=splits)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    for b, row, h, x in ((0, 3, 0, NAN), (1, 8, 1, NAN), (1, 2, 0, NAN)):
        pos = t.lens[b] - int(t.cu[b + 1] - t.cu[b]) + row
        a[2][int(t.table[b][pos // 16]), h, pos % 16, 5] = x
        hit[int(t.cu[b]) + row, 4 * h:4 * h + 4] = True
    o, l = sa.sinkattn_decode_tree(*a, **kw, num_splits=splits)
    assert torch.equal(torch.isnan(l), hit) and torch.equal(l[~hit], lse[~hit])
    assert torch.all(torch.isnan(o[hit])) and torch.equal(o[~hit], out[~hit])


# ---- attention: weights and lengths ---------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
def test_tree_weights_keep_their_bits(d):
    """A row's weight p read back: two keys of weight 1 carry minus p's first bits (its bf16
    value, then that of the rest), the third has p and value 1, so that the output is what
    is left of p over p + 2.

    The first bf16 half of p is cut off, which leaves a rest below 2^-7 of p's power of two; the
    second rounds the rest by half a step, 2^-8 of the rest's power of two, which is 2^-8 of
    p's at most: 2^-16 p in all. exp2 and its argument (below 2 in magnitude) lose at most
    2^-21 p, the products' sum 2^-22, and the output's rounding half a step, 2^-8 of an
    output below 2^-15 / 2: 2^-24."""
    rng = np.random.default_rng(3)
    n = 300
    q = torch.zeros((n, 1, d), dtype=torch.bfloat16)
    q[:, 0, 0] = torch.tensor(rng.uniform(0.01, 1.3, n)).to(torch.bfloat16)
    scale = 0.7310585
    s = q[:, 0, 0].double().numpy() * float(np.float32(scale))
    p = np.exp(-s)
    h1 = torch.tensor(p).to(torch.bfloat16)
    h2 = (torch.tensor(p) - h1.double()).to(torch.bfloat16)
    # one sequence of one row each, so that every row has values of its own
    kc = torch.zeros((n, 1, 4, d), dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    kc[:, 0, 2, 0] = -1.0
    vc[:, 0, 0], vc[:, 0, 1], vc[:, 0, 2] = -h1[:, None], -h2[:, None], 1.0
    out, _ = sa.sinkattn_decode_tree(q.cuda(), i32(np.arange(n + 1)), kc.cuda(), vc.cuda(),
                                     i32(np.arange(n)[:, None]), i32([3] * n), 1, 4, scale=scale)
    ref = (p - h1.double().numpy() - h2.double().numpy()) / (p + 2)
    bound = (p * (2.0 ** -16 + 2.0 ** -21) + 2.0 ** -22) / (p + 2) + 2.0 ** -24
    err = np.abs(to_np(out)[:, 0, 0] - ref)
    assert np.all(err <= bound), (err / bound).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length", [8192, 8193, 20000, 65536, 131071])
def test_tree_long_contexts(length, d):
    """Shares of more than two tiles, items cut into up to 64 parts and their merges."""
    Tree([3], [length], 16, 4, 1, d, seed=length).check("one", num_splits=0)
    Tree([2], [length], 64, 2, 1, d, None, sinks=False).check("no sinks", num_splits=0)
    if d == 64:
        Tree([2, 5, 1], [length, 70, length // 3], 16, 2, 2, d).check("ragged", num_splits=0)
        Tree([2, 3], [length, 50], 16, 2, 1, d, window=length // 2).check("window", num_splits=0)


# ---- gradients of the norm's weights ------------------------------------------------------

@pytest.mark.parametrize("n,hq,d", [(32769, 32, 128), (600000, 64, 64), (300000, 64, 128),
                                    (700, 500, 64)])
def test_weight_gradient_of_many_equal_rows(n, hq, d):
    """Equal rows: the roundings of a running sum all go the same way.

    A term u dy takes 16 roundings at most (12 additions of squares, half of whose error
    reaches the root, the root and two products), 64 terms are added in a row, and 36 more
    steps join such sums, lanes, warps and blocks: 116 2^-24 < 2^-17 of the sum of the
    terms' magnitudes."""
    rng = np.random.default_rng(n)
    x = torch.tensor(rng.uniform(0.5, 2.0, d) * rng.choice([-1, 1], d)).to(torch.bfloat16)
    rows = x.cuda().expand(n, hq, d).contiguous()
    k = rows[:, :1].contiguous()
    w = torch.ones(d, device="cuda")
    _, _, dwq, dwk = sa.sinkattn_qk_norm_rope_backward(rows, k, rows, k, q_weight=w, k_weight=w,
                                                       eps=1e-6)
    xs = x.double().numpy()
    term = xs * xs / np.sqrt((xs * xs).mean() + 1e-6)
    for got, heads in ((dwq, hq), (dwk, 1)):
        ref = term * n * heads
        err = np.abs(to_np(got) - ref) / np.abs(ref)
        assert np.all(err <= 2.0 ** -17), err.max() * 2.0 ** 17
