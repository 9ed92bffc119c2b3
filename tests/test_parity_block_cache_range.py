"""The block-scaled fp8 cache at the ends of its range, against the float64
definitions: scales far apart in one sequence, values that are not finite,
logits and queries outside half precision.

Bounds. Before its last rounding an output is sum_j p_j v_j / sum_j p_j with
every weight (decode: p_j times the value's scale; prefill: p_j) rounded to
fp16, half a step 2^-11 of the weight, and p_j = 2^x from a score |x| < 2^8 in
fp32 (an error of 2^-16 of p_j). With A = sum_j p_j |v_j| / sum_j p_j both add at
most (2^-11 + 2^-15) A, and rounding the output to bf16 at most 2^-8 of it."""
import numpy as np
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from helpers import cuda, to_np
from oracle import backward as OB
from oracle import block_cache as R
from test_parity_block_cache import Case, random_cache, run_append

pytestmark = pytest.mark.gpu


def references(c):
    """Output, lse and A (above) of a case, in float64."""
    k = [R.rows_of(c.kc, c.ks, c.table[b], n) for b, n in enumerate(c.lens)]
    v = [R.rows_of(c.vc, c.vs, c.table[b], n) for b, n in enumerate(c.lens)]
    k, v = np.concatenate(k), np.concatenate(v)
    cu_k = np.concatenate([[0], np.cumsum(c.lens)])
    kw = dict(hq=c.hq, hkv=c.hkv, sinks=c.sinks, causal=True, window=c.window, scale=c.scale)
    out, lse = OB.forward(c.q, k, v, c.cu, cu_k, **kw)
    absolute, _ = OB.forward(c.q, k, np.abs(v), c.cu, cu_k, **kw)
    return out, lse, absolute


def check(got, ref):
    out, lse, absolute = ref
    o, l = to_np(got[0]).reshape(out.shape), to_np(got[1]).reshape(lse.shape)
    assert np.isfinite(o).all()
    assert (np.abs(o - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -10 * absolute).all()
    seen = np.isfinite(lse)
    assert np.abs(l[seen] - lse[seen]).max(initial=0.0) <= 1e-3 and np.isneginf(l[~seen]).all()


def live(scale, value):
    """`scale` with `value` (broadcast) wherever a token lives."""
    return np.where(np.isnan(scale), np.nan, value).astype(np.float32)


# ---- decode: the denominator ------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (24, 8)])
@pytest.mark.parametrize("lens,num_splits", [([2000, 70], 1), ([2000, 300], 4), ([2000, 300], 0),
                                             ([9000, 700], 17), ([120, 90] * 330, 0)])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_decode_keeps_small_values_weights(d, page, block, lens, num_splits, where):
    """Value scales of 2^-60 but for one block with 2^60, whose key scores 4.5 to 8.5
    above the others': the small values vanish beside the large ones, their weights
    in the denominator do not, wherever the block stands."""
    c = Case(lens, 8, 2, d, page, block, seed=91, sinks=False)
    c.ks, c.vs = live(c.ks, 1.0), live(c.vs, 2.0 ** -60)
    c.kc[c.kc != 0x7F] = 0
    c.q *= 0.0
    c.q[:, :, 0] = torch.linspace(0.7, 1.3, 8).to(torch.bfloat16)
    c.scale = 1.0
    for b, n in enumerate(lens):
        j = int(round(where * (n - 1)))
        p, s = c.table[b, j // page], j % page
        c.vs[p, :, s // block] = 2.0 ** 60
        c.kc[p, :, s, 0] = R.encode_e4m3(6.5)
    got = c.decode(num_splits=num_splits, scale=1.0)
    out, lse, absolute = references(c)
    unit = 2.0 ** -60
    check((to_np(got[0]) * unit, got[1]), (out * unit, lse, absolute * unit))
    assert sa.sinkattn_get_device_error() == 0


# ---- prefill: the staged values -----------------------------------------------------

LAYOUTS = [(16, 16), (24, 8), (64, 32), (7, 1)]


def prefill_case(d, page, block, **kw):
    return Case([300, 40, 700, 128, 0], 8, 2, d, page, block, seed=92, new=[100, 40, 257, 1, 3],
                **kw)


def scaled(got, ref, unit):
    """Output and A in units of the rows' values (a power of two)."""
    return ((to_np(got[0]).reshape(ref[0].shape) / unit, got[1]),
            (ref[0] / unit, ref[1], ref[2] / unit))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", LAYOUTS)
@pytest.mark.parametrize("e", [-60, -27, 9, 60])
def test_prefill_scale_limits(d, page, block, e):
    """Value scales at both limits and where fp16 alone would round or clamp."""
    for num_splits, window in ((0, 0), (3, 0), (0, 150)):
        c = prefill_case(d, page, block, window=window)
        c.vs = live(c.vs, 2.0 ** e)
        check(*scaled(c.prefill(num_splits), references(c), 2.0 ** (e + 6)))
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("page,block", LAYOUTS)
def test_prefill_scales_differ_by_sequence_and_head(page, block):
    c = prefill_case(64, page, block)
    exps = np.array([[-60, 60], [3, -40], [50, 9], [-20, -60], [0, 0]])
    for b, n in enumerate(c.lens):
        for p in c.table[b, :-(-n // page)]:
            c.vs[p] = live(c.vs[p], 2.0 ** exps[b][:, None])
    unit = np.concatenate([np.repeat(2.0 ** (exps[b] + 6), 4)[None].repeat(m, 0)
                           for b, m in enumerate(c.new)])[..., None]
    check(*scaled(c.prefill(), references(c), unit))
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("page,block", LAYOUTS)
@pytest.mark.parametrize("e", [-50, 0, 40])
def test_prefill_early_values_keep_their_bits(page, block, e):
    """A prompt whose later blocks have scales 2^20 above the earlier ones': queries
    that see the earlier ones alone keep their own precision, and so do blocks of
    zeros under the smallest scale."""
    n, cut = 500, 5 * max(page, 24) // page * page
    c = Case([n, 50], 8, 2, 64, page, block, seed=93, new=[n, 50])
    c.vs = live(c.vs, 2.0 ** (e - 20))
    for p in c.table[0, cut // page:-(-n // page)]:
        c.vs[p] = live(c.vs[p], 2.0 ** e)
    p = c.table[0, 1]
    c.vs[p], c.vc[p] = 2.0 ** -60, 0
    ref = references(c)
    unit = np.where((np.arange(550) < cut) | (np.arange(550) >= n), 2.0 ** (e - 14), 2.0 ** (e + 6))
    got, ref = scaled(c.prefill(), ref, unit[:, None, None])
    # where both kinds are visible, in units of the larger
    check(got, ref)
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("page,block", [(16, 16), (24, 8)])
def test_prefill_scales_behind_the_window_do_not_count(page, block):
    c = Case([900, 500], 8, 2, 64, page, block, seed=94, new=[40, 500], window=100)
    c.vs = live(c.vs, 2.0 ** -45)
    for p in c.table[0, :(900 - 40 - 100) // page]:
        c.vs[p] = 2.0 ** 60
    check(*scaled(c.prefill(), references(c), 2.0 ** -39))
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("page,block", [(16, 16), (24, 8)])
def test_prefill_reports_values_that_it_cannot_hold(page, block):
    """A visible NaN value, and values 2^23 below their sequence's largest scale;
    other sequences' results do not change."""
    c = prefill_case(64, page, block)
    out, lse = c.prefill()
    assert sa.sinkattn_get_device_error() == 0
    keep = c.vc[c.table[0, 3], 1, 5, 9]
    c.vc[c.table[0, 3], 1, 5, 9] = 0xFF
    nout, nlse = c.prefill()
    assert sa.sinkattn_get_device_error() == 5
    assert torch.isfinite(nout).all()
    assert torch.equal(nout[100:], out[100:]) and torch.equal(nlse, lse)
    assert torch.equal(nout[:, :4], out[:, :4])  # the first KV head
    c.vc[c.table[0, 3], 1, 5, 9] = keep
    c.vs[c.table[0, 3]] = 2.0 ** -28
    c.vs[c.table[0, 4]] = 2.0 ** -5
    c.prefill()
    assert sa.sinkattn_get_device_error() == 5
    c.vc[c.table[0, 3]] = 0x80  # negative zeros
    got = c.prefill()
    check(got, references(c))
    assert sa.sinkattn_get_device_error() == 0


# ---- append: rows that are not finite -------------------------------------------------

def append_case(rng, seqs, page, hkv, d):
    """Slots of the new tokens of sequences (cached, new) on permuted pages, and the
    number of pages."""
    need = [-(-(o + n) // page) for o, n in seqs]
    ids = rng.permutation(sum(need))
    at = np.concatenate([[0], np.cumsum(need)])
    slots = [ids[a + np.arange(o, o + n) // page] * page + np.arange(o, o + n) % page
             for a, (o, n) in zip(at, seqs)]
    return np.concatenate(slots), len(ids)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (16, 1), (16, 2), (16, 4), (24, 8), (24, 24),
                                        (64, 64), (256, 256)])
def test_append_rows_that_are_not_finite(d, page, block):
    """Infinities and NaNs count as +-448 and NaN under the scale of the finite
    elements: older tokens of their block and the call's other rows keep their values."""
    rng = np.random.default_rng(page + block)
    hkv = 3
    seqs = [(page // 2, 1), (page - 1, 3), (0, 2 * page + 5), (3, 40), (0, 1), (5, page)]
    slots, pages = append_case(rng, seqs, page, hkv, d)
    n = len(slots)
    kc, ks = random_cache(rng, pages, hkv, page, d, block)
    k = torch.randn(n, hkv, d, generator=torch.Generator().manual_seed(page)).to(torch.bfloat16)
    v = k * 0.25
    k[0, 1, 7], k[1, 0, 0] = float("nan"), float("inf")        # single rows behind older ones
    k[6, 2, d - 1], v[6, 2, 5] = -float("inf"), float("nan")
    v[9, 0, 3], v[10, 0, 3] = float("inf"), float("nan")
    k[n - 2, 1] = float("inf")                                  # nothing finite in the row
    v[4, 2] = float("nan")
    run_append(k, v, slots, (kc, kc, ks, ks))
    assert sa.sinkattn_get_device_error() == 5
    run_append(torch.nan_to_num(k, 1.0, 2.0, -2.0), torch.nan_to_num(v, 1.0, 2.0, -2.0), slots,
               (kc, kc, ks, ks))
    assert sa.sinkattn_get_device_error() == 0


def test_append_of_a_nan_keeps_the_older_tokens():
    kc, ks = random_cache(np.random.default_rng(3), 2, 1, 16, 64, 16)
    k = torch.randn(1, 1, 64).to(torch.bfloat16)
    k[0, 0, 3] = float("nan")
    codes, _, scale, _ = run_append(k, k, [9], (kc, kc, ks, ks))
    old = R.rows_of(kc, ks, [0], 9)
    new = R.rows_of(codes.cpu().numpy(), scale.cpu().numpy(), [0], 10)
    grown = scale[0, 0, 0].item() / ks[0, 0, 0]
    # a code times a power of two is off by at most half a subnormal step, 2^-10 of the scale
    assert np.abs(new[:9] - old).max() <= (0 if grown == 1 else 2.0 ** -10 * scale[0, 0, 0].item())
    assert np.isnan(new[9, 0, 3]) and np.isfinite(np.delete(new[9, 0], 3)).all()
    assert sa.sinkattn_get_device_error() == 5


def test_append_long_runs_that_are_not_finite():
    """Blocks shared by several warps."""
    rng = np.random.default_rng(4)
    hkv, page = 8, 256
    slots, pages = append_case(rng, [(100, 9000), (0, 6000)], page, hkv, 64)
    kc, ks = random_cache(rng, pages, hkv, page, 64, page)
    k = torch.randn(15000, hkv, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    k[[5, 700, 701, 14999], [0, 3, 3, 7], [1, 2, 3, 4]] = torch.tensor(
        [float("nan"), float("inf"), -float("inf"), float("nan")]).to(torch.bfloat16)
    run_append(k, -k, slots, (kc, kc, ks, ks), fused=True)
    assert sa.sinkattn_get_device_error() == 5


# ---- decode: sinks and queries of any size ----------------------------------------------

PLANS = [([500, 3, 0, 2000], 1), ([500, 3, 0, 2000], 4), ([500, 3, 0, 2000], 0),
         ([500, 3, 0, 2000], 17), ([100, 0, 60] * 400, 0)]


@pytest.mark.parametrize("page,block", [(16, 16), (24, 8)])
@pytest.mark.parametrize("lens,num_splits", PLANS)
def test_decode_sinks_of_any_size(page, block, lens, num_splits):
    """Sinks that overflow in log2 units: a huge one takes all the weight (out = 0,
    lse = sink), a hugely negative one none, but is the lse of a row without keys.
    Other heads' results are the same bits."""
    c = Case(lens, 8, 2, 64, page, block, seed=95)
    out, lse = c.decode(num_splits)
    high, low = {0: float("inf"), 2: 3.3e38, 5: 2.3e38}, {1: -3.3e38, 6: -float("inf")}
    for h, s in {**high, **low}.items():
        c.sinks[h] = s
    got, glse = c.decode(num_splits)
    for h, s in high.items():
        # 2.3e38 comes through two products with rounded constants, four errors of 2^-24
        assert torch.all(got[:, h] == 0)
        want = np.float32(s)
        l = to_np(glse[:, h])
        assert np.all(l == want) or np.all(np.abs(l - want) <= 2.0 ** -22 * want) and s < 2.36e38
    for h, s in low.items():
        c.sinks[h] = -1e4
    ref = references(c)
    some = np.array(c.lens) > 0
    rest = [h for h in range(8) if h not in high]
    pick = np.ix_(some, rest)
    check((to_np(got)[pick], to_np(glse)[pick]), [x[pick] for x in ref])
    for h, s in low.items():
        assert torch.all(got[~torch.from_numpy(some), h] == 0)
        assert np.all(to_np(glse)[~some, h] == np.float32(s))
    same = [3, 4, 7]
    assert torch.equal(got[:, same], out[:, same]) and torch.equal(glse[:, same], lse[:, same])
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("page,block", [(16, 16), (24, 8)])
@pytest.mark.parametrize("lens,num_splits", PLANS)
def test_decode_queries_of_any_size(page, block, lens, num_splits):
    """Query heads of 2^-40 and 2^100 times ordinary ones, under a softmax scale that
    keeps the logits ordinary: the same bits, since every factor is a power of two. An
    infinite element makes its own head's row NaN and changes no other."""
    c = Case(lens, 8, 2, 64, page, block, seed=96, sinks=False)
    # heads of one size in a call: the softmax scale is one for all
    out, lse = c.decode(num_splits)
    for e in (-40, 100):
        big = torch.ldexp(c.q.float(), torch.tensor(e)).to(torch.bfloat16)
        got, glse = sa.sinkattn_decode_fp8_block(big.cuda(), **c.dev(), max_seqlen_k=max(c.lens),
                                                 num_splits=num_splits, scale=c.scale * 2.0 ** -e)
        assert torch.equal(got, out) and torch.equal(glse, lse)
    # heads of different sizes: the largest below what half precision alone holds
    mixed = c.q.clone()
    mixed[:, 2] *= 2.0 ** -30
    mixed[:, 5] *= 2.0 ** 20
    c.q = mixed
    got = c.decode(num_splits)
    ref = references(c)
    heads = [h for h in range(8) if h != 5]
    pick = np.ix_(range(len(c.lens)), heads)
    check((to_np(got[0])[pick], to_np(got[1])[pick]), [x[pick] for x in ref])
    # head 5: logits of 2^20 and more, whose fp32 sums (five joins of four products of
    # 16 dims each, cut off at 2^-22 or better) are off by at most 2^-19 of sum |q k|
    for b, n in enumerate(c.lens):
        if n:
            k = R.rows_of(c.kc, c.ks, c.table[b], n)[:, 1]
            size = c.scale * (np.abs(k) @ np.abs(c.q[b, 5].double().numpy())).max()
            assert abs(got[1][b, 5].item() - ref[1][b, 5]) <= 2.0 ** -19 * size
    c.q[0, 1, 7] = float("inf")
    inf, linf = c.decode(num_splits)
    assert torch.isnan(inf[0, 1]).all()
    keep = torch.ones_like(linf, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(inf[keep], got[0][keep]) and torch.equal(linf[keep], got[1][keep])
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("hq,d", [(8, 64), (6, 64), (8, 128)])
@pytest.mark.parametrize("num_splits", [1, 3])
def test_prefill_sinks_of_any_size(hq, d, num_splits):
    """Finite sinks that overflow in log2 units, also over rows without keys."""
    c = Case([300, 40, 700, 128, 0], hq, 2, d, 16, 16, seed=95, new=[100, 40, 257, 1, 3])
    out, lse = c.prefill(num_splits)
    c.sinks[1], c.sinks[2], c.sinks[5] = -3.3e38, 3.3e38, 2.3e38
    got, glse = c.prefill(num_splits)
    assert torch.all(got[:, [2, 5]] == 0)
    assert torch.all(glse[:, 2] == c.sinks[2].item())
    assert np.all(np.abs(to_np(glse[:, 5]) / 2.3e38 - 1) <= 2.0 ** -22)
    assert torch.all(got[-3:, 1] == 0) and torch.all(glse[-3:, 1] == c.sinks[1].item())
    c.sinks[1] = -1e4
    ref = references(c)
    check((to_np(got)[:-3, 1], to_np(glse)[:-3, 1]), [x[:-3, 1] for x in ref])
    same = [h for h in range(hq) if h not in (1, 2, 5)]
    assert torch.equal(got[:, same], out[:, same]) and torch.equal(glse[:, same], lse[:, same])
    assert sa.sinkattn_get_device_error() == 0


# ---- a padded batch ---------------------------------------------------------------------

@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_step(num_splits, d):
    """A step of fixed size with 37 padding rows and two empty sequences, from the page
    map to the attention: the padding writes no slot, and its output rows stay."""
    hq, hkv, page, pad = 8, 2, 16, 37
    new, lens = [100, 40, 0, 0], [100, 40, 0, 0]
    n, total = sum(new), sum(new) + pad
    gen = torch.Generator().manual_seed(99)
    k, v = (torch.randn(total, hkv, d, generator=gen).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(total, hq, d, generator=gen).to(torch.bfloat16)
    for x in (k, v, q):
        x[n:] = float("nan")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = [torch.full((12, hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda"),
             torch.full((12, hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda"),
             torch.full((12, hkv, 1), float("nan"), device="cuda"),
             torch.full((12, hkv, 1), float("nan"), device="cuda")]
    table = torch.full((4, 8), 1 << 28, dtype=torch.int32, device="cuda")
    cu, L = i32(np.concatenate([[0], np.cumsum(new)])), i32(lens)
    slots, _, _ = sa.sinkattn_page_map(L, table, i32(np.arange(12)[::-1].copy()), i32([0]), page,
                                       cu_seqlens_q=cu, total_q=total)
    sa.sinkattn_append_fp8_block(k.cuda(), v.cuda(), slots, *cache)
    out = torch.full((total, hq, d), 7.0, device="cuda").to(torch.bfloat16)
    lse = torch.full((total, hq), 7.0, device="cuda")
    sa.sinkattn_prefill_paged_fp8_block(q.cuda(), cu, *cache, table, L, max(new), 128,
                                        num_splits=num_splits, out=out, lse=lse)
    assert (slots[n:] == -1).all()
    assert torch.all(out[n:] == 7) and torch.all(lse[n:] == 7)
    c = [t.cpu().numpy() for t in cache]
    kr, vr = (np.concatenate([R.rows_of(c[i], c[i + 2], table[b].tolist(), m)
                              for b, m in enumerate(lens)]) for i in (0, 1))
    kw = dict(hq=hq, hkv=hkv, causal=True, scale=d ** -0.5)
    cu = cu.tolist()
    ro, rl = OB.forward(q[:n], kr, vr, cu, cu, **kw)
    ra, _ = OB.forward(q[:n], kr, np.abs(vr), cu, cu, **kw)
    check((out[:n], lse[:n]), (ro, rl, ra))
    assert sa.sinkattn_get_device_error() == 0
