"""Edges of the speculative decoding step on the GPU: verification whose drafts have used
up a token's mass many times over or whose answer hangs on its last bits."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from oracle import step as R
from test_parity_step import check_verify, i32

pytestmark = pytest.mark.gpu


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
