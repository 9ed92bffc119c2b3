"""The speculative decoding step on the CPU: its float64 definitions against other
statements of them, and what the entry points refuse before any CUDA call."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import attention_learned_sinks_gb300 as sa
from attention_learned_sinks_gb300 import build as sbuild
from attention_learned_sinks_gb300 import sinkattn as B
from oracle import backward as OB
from oracle import step as R


@pytest.fixture(scope="module")
def lib():
    sbuild.build()
    return sa.load()


# ---- definitions -----------------------------------------------------------------

@pytest.mark.parametrize("rope,interleaved", [(8, False), (8, True), (4, False), (4, True)])
def test_rotation_turns_pairs(rope, interleaved):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 2, 8))
    ang = rng.uniform(0, 6, size=(5, rope // 2))
    z = R.norm_rope(x, None, 1.0, [4, 0, 2], np.concatenate([np.cos(ang), np.sin(ang)], 1),
                    interleaved)
    for t, pos in enumerate([4, 0, 2]):
        for i in range(rope // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rope // 2)
            turned = (x[t, :, a] + 1j * x[t, :, b]) * np.exp(1j * ang[pos, i])
            assert np.allclose(z[t, :, a], turned.real) and np.allclose(z[t, :, b], turned.imag)
    assert np.array_equal(z[..., rope:], x[..., rope:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,rope", [(True, 8), (True, 4), (True, 0), (False, 8)])
def test_norm_rope_gradient_by_differences(norm, rope, interleaved):
    rng = np.random.default_rng(2)
    x, dz, w = rng.normal(size=(2, 3, 8)), rng.normal(size=(2, 3, 8)), rng.normal(size=8)
    ang = rng.uniform(0, 6, size=(5, max(rope // 2, 1)))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1) if rope else None
    f = lambda x, w: (dz * R.norm_rope(x, w if norm else None, 1e-2, [3, 1], cs,
                                       interleaved)).sum()
    dx, dw = R.norm_rope_backward(dz, x, w if norm else None, 1e-2, [3, 1], cs, interleaved)
    h = 1e-5  # central differences: error h^2 times third derivatives, about 1e-9
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(8 if norm else 0):
        e = np.zeros(8)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


@pytest.mark.parametrize("window", [0, 1, 3, 100])
@pytest.mark.parametrize("with_sinks", [False, True])
def test_chain_is_causal_attention(window, with_sinks):
    """Chains are causal attention with the queries at the end."""
    rng = np.random.default_rng(3)
    cu, lens = np.array([0, 3, 4, 9]), [10, 1, 5]
    q = rng.normal(size=(9, 4, 8))
    k, v = ([rng.normal(size=(n, 2, 8)) for n in lens] for _ in range(2))
    sinks = rng.normal(size=4) if with_sinks else None
    out, lse = R.tree_attention(q, cu, None, k, v, lens, sinks, window, 0.3)
    cu_k = np.concatenate([[0], np.cumsum(lens)])
    o, l = OB.forward(q, np.concatenate(k), np.concatenate(v), cu, cu_k, hq=4, hkv=2,
                      sinks=sinks, causal=True, window=window, scale=0.3)[:2]
    assert np.allclose(out, o) and np.allclose(lse, l)


def test_tree_row_is_its_own_chain():
    """Each row of a tree attends as the last row of a chain made of its line alone."""
    rng = np.random.default_rng(4)
    parents = [-1, 0, 0, 1, 3, 2, 0, 6]
    lk, context = 13, 5
    q, k, v = rng.normal(size=(8, 2, 4)), rng.normal(size=(lk, 1, 4)), rng.normal(size=(lk, 1, 4))
    sinks = rng.normal(size=2)
    for window in (0, 2, 4):
        out, lse = R.tree_attention(q, [0, 8], parents, [k], [v], [lk], sinks, window, 0.5)
        for i in range(8):
            up = R.line(parents, i)[::-1]
            keys = list(range(context)) + [context + a for a in up]
            o, l = R.tree_attention(q[up], [0, len(up)], None, [k[keys]], [v[keys]], [len(keys)],
                                    sinks, window, 0.5)
            assert np.allclose(out[i], o[-1]) and np.allclose(lse[i], l[-1])


def _exact_choice(p, q, tokens, certain):
    """Distribution of the token that follows a root under the tests' rule, for `tokens`
    children drawn from q (or certain ones), enumerated in fractions."""
    n = len(p)
    out = [Fraction(0)] * n

    def go(k, v, total, weight):
        if weight == 0:
            return
        if k == tokens:
            for x in range(n):
                out[x] += weight * (v[x] / total if total else 0)
            return
        for x in range(n):
            draw = q[x] if certain is None else Fraction(int(certain[k] == x))
            if draw == 0:
                continue
            qx = q if certain is None else [Fraction(int(y == x)) for y in range(n)]
            accept = min(Fraction(1), v[x] / (total * qx[x])) if total else Fraction(0)
            out[x] += weight * draw * accept
            rest = [max(v[y] - total * qx[y], Fraction(0)) for y in range(n)]
            go(k + 1, rest, sum(rest), weight * draw * (1 - accept))

    go(0, list(p), Fraction(1), Fraction(1))
    return out


@pytest.mark.parametrize("certain", [None, [0, 2], [1, 1], [3, 0, 2]])
def test_verification_keeps_the_targets_distribution(certain):
    p = [Fraction(x, 20) for x in (3, 8, 7, 2)]
    q = [Fraction(x, 10) for x in (5, 1, 1, 3)]
    for children in ([1, 2, 3] if certain is None else [len(certain)]):
        assert _exact_choice(p, q, children, certain) == p


def test_verify_follows_the_rule():
    """The walk in numbers: a child rejected, its sibling tested by what is left."""
    p = np.array([[0.5, 0.25, 0.25, 0.0], [0.0, 0.0, 1.0, 0.0], [0.25] * 4])
    q = np.array([[0.75, 0.25, 0.0, 0.0], [0.25] * 4, [0.25] * 4])
    # root; child of token 0 (accepted below 2/3); child of token 1
    args = lambda u: (p, q, [9, 0, 1], [-1, 0, 0], np.array(u), [0, 3], 4)
    path, num, tok = R.verify(*args([0.5, 0.6, 0.9]))
    assert path.tolist() == [[0, 1, -1, -1]] and num[0] == 2 and tok[0] == 2
    # rejected: left is (0, 0, 1/4, 0); token 1 has nothing of it
    path, num, tok = R.verify(*args([0.99, 0.7, 0.0]))
    assert path.tolist() == [[0, -1, -1, -1]] and num[0] == 1 and tok[0] == 2


# ---- refusals ----------------------------------------------------------------------

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)
BAD, UNSUP, SMALL, OK = (B.SINKATTN_ERR_INVALID_ARGUMENT, B.SINKATTN_ERR_UNSUPPORTED,
                         B.SINKATTN_ERR_WORKSPACE_TOO_SMALL, B.SINKATTN_OK)


def test_qk_norm_rope_refusals(lib):
    def f(**kw):
        a = dict(q=FAKE, k=FAKE, v=None, qs=512, ks=128, vs=0, pos=FAKE, n=4, hq=8, hkv=2, d=64,
                 wq=FAKE, wk=FAKE, eps=1e-6, cs=FAKE, mp=10, rope=64, il=0, qo=FAKE, ko=FAKE,
                 slots=None, kc=None, vc=None, pages=0, page=0)
        a.update(kw)
        return lib.sinkattn_qk_norm_rope(*[a[x] for x in (
            "q k v qs ks vs pos n hq hkv d wq wk eps cs mp rope il qo ko slots kc vc pages "
            "page").split()], None)
    assert f(n=0) == OK
    assert f(d=96) == UNSUP and f(rope=24) == UNSUP
    for kw in (dict(rope=80), dict(rope=-16), dict(eps=0.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(mp=0), dict(pos=None), dict(qs=504), dict(qs=516),
               dict(ks=64), dict(hq=7), dict(hkv=0), dict(n=-1), dict(q=None), dict(ko=None),
               dict(qo=ODD), dict(q=ODD), dict(cs=ODD), dict(kc=FAKE), dict(slots=FAKE),
               dict(kc=FAKE, vc=FAKE, slots=FAKE, v=FAKE, vs=128, pages=3, page=0),
               dict(kc=FAKE, vc=FAKE, slots=FAKE, v=FAKE, vs=64, pages=3, page=16),
               dict(kc=FAKE, vc=FAKE, slots=FAKE, v=None, vs=128, pages=3, page=16),
               dict(kc=FAKE, vc=None, slots=FAKE, v=FAKE, vs=128, pages=3, page=16)):
        assert f(**kw) == BAD, kw
    assert f(n=1 << 31) == UNSUP


def test_qk_norm_rope_backward_refusals(lib):
    need = lib.sinkattn_qk_norm_rope_backward_workspace_size(64)
    assert need > 0 and lib.sinkattn_qk_norm_rope_backward_workspace_size(128) == 2 * need
    assert lib.sinkattn_qk_norm_rope_backward_workspace_size(96) == 0

    def f(**kw):
        a = dict(dqo=FAKE, dko=FAKE, q=FAKE, k=FAKE, qs=512, ks=128, pos=FAKE, n=4, hq=8, hkv=2,
                 d=64, wq=FAKE, wk=FAKE, eps=1e-6, cs=FAKE, mp=10, rope=64, il=0, dq=FAKE,
                 dk=FAKE, dqs=512, dks=128, dwq=FAKE, dwk=FAKE, ws=FAKE, wsb=need)
        a.update(kw)
        return lib.sinkattn_qk_norm_rope_backward(*[a[x] for x in (
            "dqo dko q k qs ks pos n hq hkv d wq wk eps cs mp rope il dq dk dqs dks dwq dwk ws "
            "wsb").split()], None)
    assert f(n=0, wq=None, wk=None) == OK
    assert f(ws=None) == SMALL and f(wsb=need - 1) == SMALL
    for kw in (dict(dqo=None), dict(q=None), dict(dqs=256), dict(dks=132), dict(qs=504),
               dict(ws=ctypes.c_void_p((1 << 20) + 64)), dict(dwq=ODD), dict(dk=ODD)):
        assert f(**kw) == BAD, kw


def test_decode_tree_refusals(lib):
    M = B.Mask(1, 0, 0.125)

    def f(**kw):
        a = dict(q=FAKE, cu=FAKE, par=None, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, pages=8,
                 maxp=4, page=16, batch=2, tq=10, mq=5, mk=64, hq=8, hkv=2, d=64, sinks=None,
                 mask=M, ns=0, out=FAKE, lse=None, ws=None, wsb=0)
        a.update(kw)
        return lib.sinkattn_decode_tree(*[a[x] for x in (
            "q cu par k v table lens pages maxp page batch tq mq mk hq hkv d sinks mask ns out "
            "lse ws wsb").split()], None)
    assert f(batch=0) == OK and f(tq=0) == OK and f(mq=0) == OK
    assert f(d=80) == UNSUP and f(batch=65536) == UNSUP
    assert f(tq=1 << 30) == UNSUP
    for kw in (dict(hq=7), dict(hkv=0), dict(page=0), dict(mk=65), dict(q=None), dict(cu=None),
               dict(lens=None), dict(table=None), dict(out=None), dict(k=None), dict(v=ODD),
               dict(par=ODD), dict(out=ODD), dict(mask=B.Mask(1, -1, 0.1)),
               dict(mask=B.Mask(1, 0, 0.0)), dict(mask=B.Mask(1, 0, float("inf"))), dict(ns=-1),
               dict(batch=-1), dict(pages=-1)):
        assert f(**kw) == BAD, kw


def test_verify_tree_refusals(lib):
    def f(**kw):
        a = dict(p=FAKE, q=None, tok=FAKE, par=None, u=FAKE, cu=FAKE, batch=2, tq=10, mq=5,
                 vocab=100, path=FAKE, num=FAKE, nxt=FAKE)
        a.update(kw)
        return lib.sinkattn_verify_tree(*[a[x] for x in (
            "p q tok par u cu batch tq mq vocab path num nxt").split()], None)
    assert f(batch=0) == OK
    assert f(mq=1025) == UNSUP and f(vocab=(1 << 30) + 1) == UNSUP
    for kw in (dict(vocab=0), dict(p=None), dict(tok=None), dict(u=None), dict(cu=None),
               dict(path=None), dict(num=None), dict(nxt=None), dict(p=ODD), dict(q=ODD),
               dict(nxt=ctypes.c_void_p((1 << 20) + 4)), dict(mq=-1), dict(batch=-1)):
        assert f(**kw) == BAD, kw


def test_compact_refusals(lib):
    def f(**kw):
        a = dict(k=FAKE, v=FAKE, table=FAKE, lens=FAKE, cu=FAKE, path=FAKE, num=FAKE, width=4,
                 batch=2, pages=8, maxp=4, page=16, hkv=2, d=64, lo=FAKE, free=FAKE, nf=8,
                 head=FAKE, ho=FAKE)
        a.update(kw)
        return lib.sinkattn_compact(*[a[x] for x in (
            "k v table lens cu path num width batch pages maxp page hkv d lo free nf head "
            "ho").split()], None)
    assert f(d=96) == UNSUP and f(batch=1 << 16, maxp=1 << 15) == UNSUP
    for kw in (dict(k=None), dict(v=ODD), dict(table=None), dict(lens=None), dict(cu=None),
               dict(num=None), dict(lo=None), dict(free=None), dict(head=None), dict(ho=None),
               dict(page=0), dict(hkv=0), dict(width=-1), dict(batch=-1), dict(nf=-1)):
        assert f(**kw) == BAD, kw
