"""GPU calls on a block-scaled fp8 paged cache against the float64 definitions.

Bookkeeping and codes are whole numbers and have to be equal. Attention is held
to the parity bars of helpers.py on the dequantised cache. The prefill stages
scale * code once, K as bf16 and V as fp16; its reference does the same, which
changes nothing for power-of-two scales. Every slot, scale and table entry that
no token owns is poisoned (NaN codes, NaN scales, page ids far outside)."""
import numpy as np
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from attention_learned_sinks_gb300 import synthetic as S
from helpers import check_close, cuda, to_np
from oracle import backward as OB
from oracle import block_cache as R
from oracle import fp8 as F

pytestmark = pytest.mark.gpu
FAR = 1 << 28  # a page id outside every cache


def t32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


# ---- page map ------------------------------------------------------------------

def run_page_map(lens, new, page, *, width, nfree, head=3, pad=0, decode=False, in_place=False,
                 seed=1):
    rng = np.random.default_rng(seed)
    batch = len(lens)
    cu = None if decode else np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    total = batch if decode else int(cu[-1]) + pad
    table = rng.integers(0, 1000, size=(batch, width))
    free = rng.permutation(nfree + 1000)[:nfree]
    ref = R.page_map(lens, cu, total, table, free, head, page)
    tb, hd = t32(table).cuda(), t32([head]).cuda()
    slots, offs, out = sa.sinkattn_page_map(
        t32(lens).cuda(), tb, t32(free).cuda(), hd, page,
        cu_seqlens_q=None if decode else t32(cu).cuda(), total_q=total,
        free_head_out=hd if in_place else None)
    code = sa.sinkattn_get_device_error()
    assert code == ref[4]
    for got, want in zip((slots, offs, out, tb), (ref[0], ref[1], [ref[2]], ref[3])):
        assert np.array_equal(got.cpu().numpy().astype(np.int64), np.asarray(want))
    assert hd.item() == (ref[2] if in_place else head)
    return ref


@pytest.mark.parametrize("page", [1, 3, 16, 24, 256])
def test_page_map_ragged(page):
    rng = np.random.default_rng(page)
    new = [0, 1, page, page + 1, 2 * page - 1, 700, 0, 1, 33, 2000]
    lens = [n + int(o) for n, o in zip(new, rng.integers(0, 600, len(new)))]
    lens[1], lens[2] = 1, page  # no cached tokens; a page filled exactly
    run_page_map(lens, new, page, width=2600 // page + 2, nfree=4000, pad=5)
    run_page_map(lens, new, page, width=2600 // page + 2, nfree=4000, in_place=True)


def test_page_map_decode_step_and_empty_sequences():
    lens = [1, 16, 17, 0, 300, 32, 33, 0]
    ref = run_page_map(lens, None, 16, width=20, nfree=10, head=0, decode=True)
    assert ref[0][3] == -1 and ref[2] == 3  # lengths 1, 17, 33 start a page


@pytest.mark.parametrize("batch", [1, 255, 1024, 1025, 3000, 9001])
def test_page_map_many_sequences(batch):
    rng = np.random.default_rng(batch)
    new = rng.integers(0, 40, batch)
    lens = new + rng.integers(0, 200, batch)
    run_page_map(lens, new, 16, width=16, nfree=4 * batch + 8)
    run_page_map(lens + 1, None, 16, width=16, nfree=batch + 8, decode=True)


def test_page_map_long_chunk():
    run_page_map([131072, 5], [100001, 5], 16, width=8192, nfree=7000, pad=1000)


def test_page_map_list_runs_out():
    ref = run_page_map([100, 50, 64], [100, 50, 4], 16, width=8, nfree=9, head=2)
    assert ref[4] == 4 and (ref[0] < 0).any() and ref[2] == 9
    run_page_map([100, 50], [100, 50], 16, width=8, nfree=0, head=0)


def test_page_map_lengths_outside_the_table():
    run_page_map([100, 40], [90, 40], 16, width=4, nfree=50)          # cut at 64
    run_page_map([-3, 40], [2, 3], 16, width=4, nfree=50)
    run_page_map([3, 40], [8, 40], 16, width=4, nfree=50)              # Lq > Lk
    run_page_map([500, 40], [3, 40], 16, width=4, nfree=50)            # all past the table


def test_page_map_no_sequences():
    slots, offs, head = sa.sinkattn_page_map(t32([]).cuda(), torch.zeros(
        (0, 4), dtype=torch.int32, device="cuda"), t32([7]).cuda(), t32([0]).cuda(), 16,
        cu_seqlens_q=t32([0]).cuda(), total_q=3)
    assert slots.tolist() == [-1, -1, -1] and offs.tolist() == [0] and head.item() == 0


# ---- append --------------------------------------------------------------------

def random_cache(rng, pages, hkv, page, d, block, scale_exp=(-8, -4)):
    """Cache whose content is finite codes (no NaN) and power-of-two scales."""
    codes = rng.integers(0, 127, (pages, hkv, page, d)) + 128 * rng.integers(
        0, 2, (pages, hkv, page, d))
    scale = 2.0 ** rng.integers(scale_exp[0], scale_exp[1] + 1, (pages, hkv, page // block))
    return codes.astype(np.uint8), scale.astype(np.float32)


def run_append(k, v, slots, cache, fused=False):
    """k, v bf16 [n, hkv, D] (CPU); cache = (kc, vc, ks, vs) arrays."""
    n, hkv, d = k.shape
    if fused:
        x = torch.randn(n, 3 * hkv, d, device="cuda").to(torch.bfloat16)
        kd, vd = x[:, hkv:2 * hkv], x[:, 2 * hkv:]
        kd.copy_(k)
        vd.copy_(v)
    else:
        kd, vd = k.cuda(), v.cuda()
    got = [torch.from_numpy(a.copy()).cuda() for a in cache]
    sl = torch.from_numpy(np.asarray(slots, dtype=np.int64)).cuda()
    sa.sinkattn_append_fp8_block(kd, vd, sl, *got)
    rk, rks = R.append(k.double().numpy(), slots, cache[0], cache[2])
    rv, rvs = R.append(v.double().numpy(), slots, cache[1], cache[3])
    for g, r in zip(got, (rk, rv, rks, rvs)):
        assert np.array_equal(g.cpu().numpy(), r, equal_nan=r.dtype == np.float32)
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (16, 4), (16, 1), (24, 24), (24, 3), (64, 32),
                                        (256, 256), (100, 50), (1, 1), (7, 7)])
def test_append_ragged(d, page, block):
    rng = np.random.default_rng(page * 1000 + block + d)
    hkv = 3
    # sequences: cached tokens, new tokens; pages in random order
    seqs = [(0, 1), (0, page), (5, 1), (page - 1, 1), (page, 2 * page + 3), (3, 70), (11, 300)]
    need = [-(-(o + n) // page) for o, n in seqs]
    ids = rng.permutation(sum(need) + 3)
    slots, at = [], 0
    for (o, n), m in zip(seqs, need):
        own = ids[at:at + m]
        at += m
        slots += [own[j // page] * page + j % page for j in range(o, o + n)]
    n = len(slots)
    kc, ks = random_cache(rng, len(ids), hkv, page, d, block)
    vc, vs = random_cache(rng, len(ids), hkv, page, d, block, (-12, 3))
    gen = torch.Generator().manual_seed(page + block)
    size = torch.exp2(torch.randint(-6, 7, (n, 1, 1), generator=gen).float())
    k = (torch.randn(n, hkv, d, generator=gen) * size).to(torch.bfloat16)
    v = (torch.randn(n, hkv, d, generator=gen) / size).to(torch.bfloat16)
    run_append(k, v, slots, (kc, vc, ks, vs))
    run_append(k, v, slots, (kc, vc, ks, vs), fused=True)
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("page,block,d", [(16, 16, 64), (16, 1, 64), (16, 2, 128), (512, 512, 64),
                                          (256, 256, 128), (100, 50, 64), (40, 40, 128),
                                          (8, 8, 64), (16, 1, 128)])
def test_append_long_calls(page, block, d):
    """Calls long enough to fill the GPU: other shares of the rows than short ones."""
    rng = np.random.default_rng(page + block)
    hkv = 3
    seqs = [(0, 20011), (page // 2, 1), (page - 1, 9000), (3, 11000), (0, 513)]
    need = [-(-(o + n) // page) for o, n in seqs]
    ids = rng.permutation(sum(need))
    slots, at = [], 0
    for (o, n), m in zip(seqs, need):
        j = np.arange(o, o + n)
        slots.append(ids[at + j // page] * page + j % page)
        at += m
    slots = np.concatenate(slots + [[-1, -1]])
    slots[[700, 30000]] = -1  # padding in the middle ends a run
    n = len(slots)
    kc, ks = random_cache(rng, len(ids), hkv, page, d, block)
    gen = torch.Generator().manual_seed(page)
    size = torch.exp2(torch.randint(-6, 7, (n, 1, 1), generator=gen).float())
    k = (torch.randn(n, hkv, d, generator=gen) * size).to(torch.bfloat16)
    # a run that a padding row cuts leaves its block to two writers: keep the rows
    # behind it out of that block
    for r in (700, 30000):
        while r + 1 < n and slots[r + 1] >= 0 and slots[r + 1] % block:
            r += 1
            slots[r] = -1
    run_append(k, -k, slots, (kc, kc, ks, ks), fused=True)
    assert sa.sinkattn_get_device_error() == 0


def test_append_skips_padding_and_reports_bad_slots():
    rng = np.random.default_rng(5)
    kc, ks = random_cache(rng, 4, 2, 16, 64, 16)
    vc, vs = random_cache(rng, 4, 2, 16, 64, 16)
    k = torch.randn(6, 2, 64).to(torch.bfloat16)
    v = torch.randn(6, 2, 64).to(torch.bfloat16)
    k[2] = float("nan")  # padding rows are not read
    run_append(k, v, [3, 4, -1, 0 + 32, -7, 63], (kc, vc, ks, vs))
    assert sa.sinkattn_get_device_error() == 0
    run_append(k[:2], v[:2], [64, 5], (kc, vc, ks, vs))
    assert sa.sinkattn_get_device_error() == 2
    run_append(k[:2], v[:2], [1 << 40, -1], (kc, vc, ks, vs))
    assert sa.sinkattn_get_device_error() == 2


def test_append_fresh_block_ignores_stale_contents():
    """A recycled page: NaN scales and codes of its last owner do not matter."""
    kc = np.full((2, 2, 16, 64), 0x7F, np.uint8)
    ks = np.full((2, 2, 2), np.nan, np.float32)
    k = torch.randn(10, 2, 64).to(torch.bfloat16)
    got = run_append(k, k * 3, list(range(16, 26)), (kc, kc, ks, ks))
    assert torch.isfinite(got[2][1]).all() and torch.isnan(got[2][0]).all()


def test_append_extreme_values():
    """Zeros, the largest and the smallest bf16, values on the edge of a scale."""
    vals = torch.tensor([0.0, 448.0, 449.0, 450.0, 3.3e38, 1e-38, 1e-40, 448 * 2.0 ** -60,
                         2.0 ** -75, -0.0, 224.0, 226.0])
    n = len(vals)
    k = (vals[:, None, None] * torch.linspace(-1, 1, 64)[None, None, :]).to(torch.bfloat16)
    kc = np.zeros((n, 1, 16, 64), np.uint8)
    ks = np.zeros((n, 1, 1), np.float32)
    run_append(k, -k, [16 * i for i in range(n)], (kc, kc, ks, ks))


def test_append_old_scale_of_any_value():
    """A scale that is not a power of two becomes one, and the older codes are
    re-encoded through an fp32 product. With x the exact product and x' = x (1 + d),
    |d| <= 2^-24, its fp32 value, the code a nearest to x' and the code r nearest to x
    satisfy |a - x| <= |r - x'| + |x' - x| <= |r - x| + 2^-23 |x|."""
    rng = np.random.default_rng(6)
    kc, ks = random_cache(rng, 5, 1, 16, 64, 16)
    ks = np.array([0.7, 1e-6, 0.0, 3.0, 2.0 ** 70], dtype=np.float32).reshape(5, 1, 1)
    k = torch.randn(5, 1, 64).to(torch.bfloat16)
    slots = [16 * i + 5 for i in range(5)]
    codes, scale = torch.from_numpy(kc.copy()).cuda(), torch.from_numpy(ks.copy()).cuda()
    vc, vs = codes.clone(), scale.clone()
    sa.sinkattn_append_fp8_block(k.cuda(), k.cuda(), torch.tensor(slots).cuda(), codes, vc, scale,
                                 vs)
    rk, rks = R.append(k.double().numpy(), slots, kc, ks)
    got = codes.cpu().numpy()
    assert np.array_equal(scale.cpu().numpy(), rks) and torch.equal(codes, vc)
    assert rks[0] == 1.0 and rks[3] == 4.0 and rks[4] == 2.0 ** 60
    assert np.array_equal(got[:, :, 5:], rk[:, :, 5:])
    x = np.clip(F.e4m3_to_float64(kc) * (ks.astype(np.float64) / rks)[..., None], -448, 448)[:, :, :5]
    a, r = F.e4m3_to_float64(got)[:, :, :5], F.e4m3_to_float64(rk)[:, :, :5]
    assert (np.abs(a - x) <= np.abs(r - x) + 2.0 ** -23 * np.abs(x)).all()


def test_append_in_steps_is_append_at_once():
    """The codes written token by token are those of one call wherever no value
    became subnormal in between; the scales are always the same."""
    rng = np.random.default_rng(8)
    n, hkv, d = 40, 2, 64
    vals = rng.choice([1.0, 1.25, -1.5, 1.75, -3.5], (n, hkv, d)) * 2.0 ** rng.integers(
        -2, 3, (n, 1, 1))
    k = torch.tensor(vals).to(torch.bfloat16)
    cache = [torch.zeros((3, hkv, 16, d), dtype=torch.uint8, device="cuda") for _ in range(2)] + [
        torch.full((3, hkv, 1), float("nan"), device="cuda") for _ in range(2)]
    once = [c.clone() for c in cache]
    slots = torch.arange(n, device="cuda")
    sa.sinkattn_append_fp8_block(k.cuda(), k.cuda(), slots, *once)
    for a, b in [(0, 1), (1, 7), (7, 8), (8, 9), (9, 30), (30, 31), (31, 40)]:
        sa.sinkattn_append_fp8_block(k[a:b].cuda(), k[a:b].cuda(), slots[a:b], *cache)
    for x, y in zip(cache, once):
        assert torch.equal(x, y)


def test_append_offsets_past_32_bits():
    """A cache of more than 2^32 codes: pages on both sides of the border."""
    pages = (1 << 32) // (8 * 64 * 128) + 70
    kc = torch.zeros((pages, 8, 64, 128), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.zeros((pages, 8, 4), device="cuda")
    vs = torch.zeros_like(ks)
    k = torch.randn(3, 8, 128).to(torch.bfloat16)
    slots = [0, (pages - 60) * 64 + 16, (pages - 1) * 64 + 48]
    sa.sinkattn_append_fp8_block(k.cuda(), (2 * k).cuda(), torch.tensor(slots).cuda(), kc, vc, ks,
                                 vs)
    for i, s in enumerate(slots):
        p, o = divmod(s, 64)
        for c, sc, m in ((kc, ks, 1.0), (vc, vs, 2.0)):
            for g in range(8):
                want = 2.0 ** R.scale_exponent(m * float(k[i, g].abs().max()))
                assert sc[p, g, o // 16].item() == want
                assert np.array_equal(c[p, g, o].cpu().numpy(),
                                      R.encode_e4m3(m * k[i, g].double().numpy() / want))
    # and the attention that reads them
    table = t32([[p // 64 for p in slots[1:]]]).cuda()
    kc[pages - 60, :, :16] = kc[pages - 60, :, 16:17]
    ks[pages - 60] = ks[pages - 60, :, 1:2]
    vs[pages - 60] = vs[pages - 60, :, 1:2]
    vc[pages - 60] = vc[pages - 60, :, 16:17]
    q = torch.randn(1, 8, 128).to(torch.bfloat16).cuda()
    ro, rl = None, None
    sub = [pages - 60, pages - 1]
    c = [x[sub].cpu().numpy() for x in (kc, vc, ks, vs)]
    kr, vr = R.rows_of(c[0], c[2], [0, 1], 64), R.rows_of(c[1], c[3], [0, 1], 64)
    ro, rl = OB.forward(q, kr, vr, [0, 1], [0, 64], hq=8, hkv=8, causal=True, scale=128 ** -0.5)
    lens = t32([64]).cuda()
    out, lse = sa.sinkattn_decode_fp8_block(q, kc, vc, ks, vs, table, lens, max_seqlen_k=64)
    check_close(out, lse, ro, rl, "decode past 2^32")
    out, lse = sa.sinkattn_prefill_paged_fp8_block(q, t32([0, 1]).cuda(), kc, vc, ks, vs, table,
                                                   lens, 1, 64)
    check_close(out, lse, ro, rl, "prefill past 2^32")


# ---- attention -----------------------------------------------------------------

class Case:
    """Random sequences in a poisoned paged cache."""

    def __init__(self, lens, hq, hkv, d, page, block, *, seed, new=None, spread=1, pow2=True,
                 sinks=True, window=0, extra=2):
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.window = list(lens), hq, hkv, d, window
        self.new = [1] * len(lens) if new is None else list(new)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        ids = rng.permutation(pages)
        width = max(max(need), 1) + extra
        self.table = np.full((len(lens), width), FAR)
        used = np.zeros((pages, page), bool)
        at = 0
        for b, (n, m) in enumerate(zip(lens, need)):
            self.table[b, :m] = ids[at:at + m]
            for j in range(n):
                used[ids[at + j // page], j % page] = True
            at += m
        self.cache = []
        for _ in range(2):
            x = rng.standard_normal((pages, hkv, page // block, block, d))
            sc = 2.0 ** rng.integers(-6 - spread, -5 + spread, (pages, hkv, page // block))
            if not pow2:
                sc = sc * rng.uniform(0.75, 1.5, sc.shape)
            codes = R.encode_e4m3(x * 2.0 ** 6).reshape(pages, hkv, page, d)
            codes[np.broadcast_to(~used[:, None, :, None], codes.shape)] = 0x7F
            sc = sc.astype(np.float32)
            dead = ~used.reshape(pages, page // block, block).any(-1)
            sc[np.broadcast_to(dead[:, None, :], sc.shape)] = np.nan
            self.cache.append((codes, sc))
        (self.kc, self.ks), (self.vc, self.vs) = self.cache
        gen = torch.Generator().manual_seed(seed)
        self.q = torch.randn(sum(self.new), hq, d, generator=gen).to(torch.bfloat16)
        self.sinks = torch.randn(hq, generator=gen) * 1.5 if sinks else None
        self.cu = np.concatenate([[0], np.cumsum(self.new)])
        self.scale = d ** -0.5

    def dev(self):
        g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return dict(k_cache=g(self.kc), v_cache=g(self.vc), k_scale=g(self.ks),
                    v_scale=g(self.vs), block_table=t32(self.table).cuda(),
                    seqlens_k=t32(self.lens).cuda())

    def reference(self, staged=False, causal=True):
        kr = [R.rows_of(self.kc, self.ks, self.table[b], n) for b, n in enumerate(self.lens)]
        vr = [R.rows_of(self.vc, self.vs, self.table[b], n) for b, n in enumerate(self.lens)]
        k, v = np.concatenate(kr), np.concatenate(vr)
        if staged:
            k = torch.from_numpy(k).float().to(torch.bfloat16).double().numpy()
            v = torch.from_numpy(v).float().to(torch.float16).double().numpy()
        cu_k = np.concatenate([[0], np.cumsum(self.lens)])
        self.vmax = float(np.abs(v).max()) if v.size else 0.0
        return OB.forward(self.q, k, v, self.cu, cu_k, hq=self.hq, hkv=self.hkv,
                          sinks=self.sinks, causal=causal, window=self.window, scale=self.scale)

    def decode(self, num_splits=0, **kw):
        return sa.sinkattn_decode_fp8_block(self.q.cuda(), **self.dev(),
                                            max_seqlen_k=max(max(self.lens), 0),
                                            sinks=cuda(self.sinks), window=self.window,
                                            num_splits=num_splits, **kw)

    def prefill(self, num_splits=0, causal=True, **kw):
        a = self.dev()
        return sa.sinkattn_prefill_paged_fp8_block(
            self.q.cuda(), t32(self.cu).cuda(), a["k_cache"], a["v_cache"], a["k_scale"],
            a["v_scale"], a["block_table"], a["seqlens_k"], max(self.new), max(self.lens),
            sinks=cuda(self.sinks), window=self.window, num_splits=num_splits, causal=causal, **kw)


LENS = [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 511, 513, 1000, 1537, 0, 2049]
LAYOUTS = [(16, 16), (16, 4), (16, 1), (24, 24), (24, 8), (64, 32), (7, 7), (1, 1), (256, 128),
           (48, 48), (32, 2)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", LAYOUTS)
def test_decode_layouts(d, page, block):
    for window in (0, 200):
        c = Case(LENS, 16, 2, d, page, block, seed=page + block + window, window=window)
        out, lse = c.decode()
        ro, rl = c.reference()
        check_close(out, lse, ro, rl, "decode d=%d %d/%d w=%d" % (d, page, block, window), c.vmax)
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (6, 2), (24, 3), (32, 2), (18, 2), (64, 8)])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 129])
def test_decode_heads_and_windows(hq, hkv, window):
    for d in (64, 128):
        c = Case(LENS, hq, hkv, d, 16, 16, seed=hq * 7 + window, window=window,
                 sinks=window != 100)
        out, lse = c.decode()
        ro, rl = c.reference()
        check_close(out, lse, ro, rl, "decode %d/%d w=%d d=%d" % (hq, hkv, window, d), c.vmax)


@pytest.mark.parametrize("num_splits", [1, 2, 5, 16, 40])
def test_decode_splits(num_splits):
    for d in (64, 128):
        c = Case([6000, 0, 1, 4097, 300], 16, 2, d, 16, 16, seed=num_splits)
        ro, rl = c.reference()
        out, lse = c.decode(num_splits=num_splits)
        check_close(out, lse, ro, rl, "decode splits=%d d=%d" % (num_splits, d), c.vmax)
        again = c.decode(num_splits=num_splits)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("page,block", [(16, 16), (24, 8), (64, 32)])
@pytest.mark.parametrize("window", [0, 1301, 2999])
def test_decode_even_shares(page, block, window):
    """All keys shared out evenly: sequences cut in many places, empty ones, ones of
    a single token, several head tiles, more sequences than threads of a block."""
    rng = np.random.default_rng(page)
    few = [9000, 0, 1, 4097, 300, 2999, 0]
    many = list(rng.integers(0, 60, 290)) + [5000, 1, 2500]
    for lens, hq, hkv, d in ((few, 16, 2, 64), (few, 8, 4, 128), (many, 18, 2, 64)):
        c = Case(lens, hq, hkv, d, page, block, seed=page + window, window=window)
        ro, rl = c.reference()
        for ns in (0, 17):
            out, lse = c.decode(num_splits=ns)
            check_close(out, lse, ro, rl, "shares %d/%d w=%d ns=%d" % (page, block, window, ns),
                        c.vmax)
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("page,block", [(16, 16), (24, 8)])
@pytest.mark.parametrize("batch,hq,hkv,window", [(330, 16, 2, 100), (330, 6, 2, 128),
                                                 (1300, 8, 1, 500), (140, 80, 5, 1),
                                                 (1300, 2, 1, 0)])
def test_decode_many_short_spans(page, block, batch, hq, hkv, window):
    """Enough (sequence, KV head) pairs for one warp each."""
    rng = np.random.default_rng(batch + window)
    lens = list(rng.integers(0, 120 if window == 0 else 700, batch))
    lens[3], lens[7] = 0, 1
    for d in (64, 128):
        c = Case(lens, hq, hkv, d, page, block, seed=page + window, window=window,
                 sinks=window != 1)
        out, lse = c.decode()
        ro, rl = c.reference()
        check_close(out, lse, ro, rl, "spans %d w=%d d=%d" % (batch, window, d), c.vmax)
        bound = sa.sinkattn_decode_fp8_block(  # lengths above the host's bound
            c.q.cuda(), **c.dev(), max_seqlen_k=40, sinks=cuda(c.sinks), window=window)
        check_close(*bound, ro, rl, "spans bound", c.vmax)
    assert sa.sinkattn_get_device_error() == 0


def test_decode_thousands_of_sequences():
    rng = np.random.default_rng(11)
    lens = list(rng.integers(0, 40, 4200))
    lens[17], lens[4100] = 1500, 2300
    c = Case(lens, 2, 1, 64, 16, 16, seed=41)
    ro, rl = c.reference()
    for ns in (0, 3, 17):
        out, lse = c.decode(num_splits=ns)
        check_close(out, lse, ro, rl, "4200 sequences ns=%d" % ns, c.vmax)


@pytest.mark.parametrize("page", [16, 24])
def test_attention_without_any_key(page):
    """Lengths of 0 under a bound of 0, and a cache without pages."""
    for pages in (0, 2):
        cache = dict(k_cache=torch.zeros((pages, 2, page, 64), dtype=torch.uint8, device="cuda"),
                     v_cache=torch.zeros((pages, 2, page, 64), dtype=torch.uint8, device="cuda"),
                     k_scale=torch.zeros((pages, 2, 1), device="cuda"),
                     v_scale=torch.zeros((pages, 2, 1), device="cuda"))
        q = torch.randn(3, 8, 64).to(torch.bfloat16).cuda()
        sinks = torch.randn(8).cuda()
        table, lens = t32(np.zeros((3, pages))).cuda(), t32([0, 0, 0]).cuda()
        for ns in (0, 2, 17):
            out, lse = sa.sinkattn_decode_fp8_block(q, **cache, block_table=table, seqlens_k=lens,
                                                    max_seqlen_k=0, sinks=sinks, num_splits=ns)
            assert torch.all(out == 0) and torch.allclose(lse, sinks.expand(3, 8), atol=1e-6)
        out, lse = sa.sinkattn_prefill_paged_fp8_block(
            q, t32([0, 1, 3, 3]).cuda(), cache["k_cache"], cache["v_cache"], cache["k_scale"],
            cache["v_scale"], table, lens, 2, 0, sinks=sinks)
        assert torch.all(out == 0) and torch.allclose(lse, sinks.expand(3, 8), atol=1e-6)
    assert sa.sinkattn_get_device_error() == 0


def test_decode_without_a_table_or_caches():
    """max_pages_per_seq 0: the C call takes null caches, whatever num_pages says."""
    from attention_learned_sinks_gb300 import sinkattn as B
    q, out = torch.ones(2, 8, 64).to(torch.bfloat16).cuda(), torch.empty(2, 8, 64).bfloat16().cuda()
    lens, lse = t32([0, 0]).cuda(), torch.empty(2, 8, device="cuda")
    for pages in (0, 4):
        out.fill_(1.0)
        st = B.load().sinkattn_decode_fp8_block(
            q.data_ptr(), None, None, None, None, 16, None, lens.data_ptr(), pages, 0, 16, 2, 0, 8,
            2, 64, None, B.Mask(1, 0, 0.125), 0, out.data_ptr(), lse.data_ptr(), None, 0,
            torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0
        assert torch.all(out == 0) and torch.isneginf(lse).all()
    assert sa.sinkattn_get_device_error() == 0


def test_decode_graphs_of_every_plan_share_a_workspace():
    """Captured calls of the three plans, replayed in turn with one workspace."""
    cases = [Case([3000, 50, 9000], 16, 2, 64, 16, 16, seed=63),          # even shares
             Case([900, 50, 1200], 16, 2, 64, 16, 16, seed=64),           # clusters
             Case([100, 50, 128] * 220, 16, 2, 128, 16, 16, seed=65)]     # one warp each
    ws = torch.empty(max(sa.sinkattn_decode_fp8_block_workspace_size(len(c.lens), max(c.lens),
                                                                     16, 2, c.d) for c in cases), dtype=torch.uint8, device="cuda")
    runs = []
    for c in cases:
        a, q, sk = c.dev(), c.q.cuda(), c.sinks.cuda()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        f = lambda a=a, q=q, sk=sk, out=out, lse=lse, c=c: sa.sinkattn_decode_fp8_block(  # noqa: E731
            q, **a, max_seqlen_k=max(c.lens), sinks=sk, out=out, lse=lse, workspace=ws)
        f()
        torch.cuda.synchronize()
        ref = (out.clone(), lse.clone())
        check_close(out, lse, *c.reference(), "graph", c.vmax)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        runs.append((g, out, lse, ref, f))  # f keeps the inputs
    for _ in range(5):
        for g, out, lse, _, _ in runs:
            out.zero_()
            lse.zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, out, lse, ref, _ in runs:
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_decode_long_context_of_small_pages():
    """One-token pages: a table entry per key."""
    c = Case([9000], 8, 1, 64, 1, 1, seed=3)
    for ns in (1, 2):
        out, lse = c.decode(num_splits=ns)
        ro, rl = c.reference()
        check_close(out, lse, ro, rl, "decode page 1 splits=%d" % ns, c.vmax)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_scales_of_any_value_and_spread(d):
    c = Case(LENS, 16, 2, d, 16, 4, seed=31, pow2=False)
    out, lse = c.decode()
    ro, rl = c.reference()
    check_close(out, lse, ro, rl, "decode any scale", c.vmax)


def test_decode_tiny_values_next_to_huge_ones():
    """Value scales 2^24 apart: a token that takes nearly all the weight has tiny
    values, its neighbours' values are huge but get no weight. Each of the 600
    keys adds at most 2^-11 |w v| by P's rounding, w v at most e^-40 2^24 there,
    so the output keeps bf16 precision relative to the tiny values."""
    c = Case([600], 8, 1, 64, 16, 16, seed=32, sinks=False)
    c.vs[:] = np.where(np.isnan(c.vs), np.nan, 2.0 ** 12)
    pick = c.table[0, 7]
    c.vs[pick] = 2.0 ** -12
    c.ks[:] = np.where(np.isnan(c.ks), np.nan, 2.0 ** -20)
    c.ks[pick] = 1.0
    rows = R.rows_of(c.kc, c.ks, c.table[0], 600)
    c.q[:] = torch.from_numpy(rows[117, 0]).to(torch.bfloat16)  # key 117 lies in that page
    out, lse = c.decode()
    ro, rl = c.reference()
    assert np.abs(ro).max() < 1.0
    err = np.abs(to_np(out) - ro)
    # bf16 rounding 2^-9 and P's rounding 2^-11 of the largest value
    assert err.max() <= (2.0 ** -9 + 2.0 ** -11) * np.abs(ro).max() * 1.01


def test_decode_scale_limits():
    """Scales at 2^-60 and 2^60, and 0 (a block of zeros)."""
    for e in (-60, 60):
        c = Case([300, 40], 8, 2, 64, 16, 16, seed=33)
        c.vs = np.where(np.isnan(c.vs), np.nan, np.float32(2.0 ** e)).astype(np.float32)
        out, lse = c.decode()
        ro, rl = c.reference()
        check_close(to_np(out) / 2.0 ** (e + 6), lse, ro / 2.0 ** (e + 6), rl, "scale 2^%d" % e)
    c = Case([300, 40], 8, 2, 64, 16, 16, seed=34)
    c.vs = np.where(np.isnan(c.vs), np.nan, np.float32(0)).astype(np.float32)
    c.vs[c.table[0, 3]] = 2.0 ** -6
    c.ks[c.table[1, 1]] = 0.0
    out, lse = c.decode()
    ro, rl = c.reference()
    check_close(out, lse, ro, rl, "zero scales", c.vmax)
    assert torch.all(out[1] == 0)


def test_decode_large_sink_and_none():
    for s in (-1e4, 60.0, 1e4):
        c = Case([500, 3, 0, 2000], 8, 1, 64, 16, 16, seed=35)
        c.sinks[:] = s
        out, lse = c.decode()
        ro, rl = c.reference()
        bar = 1e-3 * max(1.0, abs(s) * 1e-3)  # lse is fp32: 1e4 has a spacing of 2^-10
        assert np.abs(to_np(lse) - rl).max() <= bar
        assert np.abs(to_np(out) - ro).max() <= 1e-2
    c = Case([500, 3, 0, 2000], 8, 1, 64, 16, 16, seed=36, sinks=False)
    out, lse = c.decode()
    ro, rl = c.reference()
    check_close(out, lse, ro, rl, "no sinks", c.vmax)
    assert torch.all(out[2] == 0) and torch.all(torch.isneginf(lse[2]))


@pytest.mark.parametrize("page,block", [(16, 16), (24, 8)])
@pytest.mark.parametrize("lens,num_splits", [([500, 3, 0, 2000], 0), ([500, 3, 0, 2000], 1),
                                             ([500, 3, 0, 2000], 4), ([500, 3, 0, 2000], 17),
                                             ([100, 0, 60] * 400, 0)])
def test_decode_nan_stays_in_its_head(page, block, lens, num_splits):
    """A NaN sink and a NaN in a query make their own head's rows NaN, in every plan;
    the other heads' results are the same bits as without (the heads of a warp move
    their references together; with these inputs after the first keys only)."""
    c = Case(lens, 8, 2, 64, page, block, seed=39)
    out, lse = c.decode(num_splits)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    c.sinks[3] = float("nan")
    c.q[0, 5, 7] = float("nan")
    nout, nlse = c.decode(num_splits)
    bad = torch.zeros_like(lse, dtype=torch.bool)
    bad[:, 3] = True
    bad[0, 5] = True
    assert torch.isnan(nout[bad]).all() and torch.isnan(nlse[bad]).all()
    assert torch.equal(nout[~bad], out[~bad]) and torch.equal(nlse[~bad], lse[~bad])


@pytest.mark.parametrize("window", [0, 60])
def test_decode_bad_pages_and_lengths(window):
    c = Case([300, 40, 2000], 8, 2, 64, 16, 16, seed=37, window=window)
    c.table[0, 17] = -1
    c.table[2, 124] = len(c.kc)
    ro, rl = c.reference()
    out, lse = c.decode()
    check_close(out, lse, ro, rl, "bad pages", c.vmax)
    assert sa.sinkattn_get_device_error() == 2
    c = Case([300, 40, 320], 8, 2, 64, 16, 16, seed=38, window=window, extra=0)
    a = c.dev()
    a["seqlens_k"] = t32([300, -5, 900]).cuda()  # the table reaches 320 keys
    out, lse = sa.sinkattn_decode_fp8_block(c.q.cuda(), **a, max_seqlen_k=320,
                                            sinks=cuda(c.sinks), window=window)
    c.lens = [300, 0, 320]
    ro, rl = c.reference()
    check_close(out, lse, ro, rl, "bad lengths", c.vmax)
    assert sa.sinkattn_get_device_error() == 3
    assert sa.sinkattn_get_device_error() == 0


def test_decode_entries_outside_the_window_are_not_read():
    """Pages behind the window were given back: their entries are garbage."""
    for window in (17, 128, 500):
        c = Case([2000, 700, 5000], 16, 2, 64, 16, 16, seed=39, window=window)
        ro, rl = c.reference()
        for b, n in enumerate(c.lens):
            c.table[b, :max(0, n - window) // 16] = FAR
        out, lse = c.decode()
        check_close(out, lse, ro, rl, "window %d" % window, c.vmax)
    assert sa.sinkattn_get_device_error() == 0


def test_decode_length_above_the_host_bound():
    c = Case([3000, 50], 8, 2, 64, 16, 16, seed=40)
    ro, rl = c.reference()
    a = c.dev()
    for bound in (50, 700):
        out, lse = sa.sinkattn_decode_fp8_block(c.q.cuda(), **a, max_seqlen_k=bound,
                                                sinks=cuda(c.sinks))
        check_close(out, lse, ro, rl, "bound %d" % bound, c.vmax)


NEW = [1, 5, 16, 17, 31, 32, 1, 127, 100, 129, 300, 0, 200, 64, 0, 700]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", LAYOUTS)
def test_prefill_layouts(d, page, block):
    for window in (0, 150):
        c = Case(LENS, 16, 2, d, page, block, seed=page + block + window, new=NEW, window=window)
        out, lse = c.prefill()
        ro, rl = c.reference(staged=True)
        check_close(out, lse, ro, rl, "prefill d=%d %d/%d w=%d" % (d, page, block, window), c.vmax)
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (6, 2), (24, 8), (32, 2)])
def test_prefill_heads_splits_and_masks(hq, hkv):
    for d in (64, 128):
        for kw in (dict(num_splits=1), dict(num_splits=3), dict(causal=False)):
            c = Case([400, 9, 1200, 64], hq, hkv, d, 16, 16, seed=hq, new=[130, 12, 257, 64],
                     sinks=hq != 6)
            out, lse = c.prefill(**kw)
            ro, rl = c.reference(staged=True, causal=kw.get("causal", True))
            check_close(out, lse, ro, rl, "prefill %d/%d d=%d %s" % (hq, hkv, d, kw), c.vmax)


def test_prefill_scales_of_any_value():
    c = Case([400, 90, 1200], 16, 2, 64, 16, 4, seed=51, new=[130, 12, 257], pow2=False)
    out, lse = c.prefill()
    ro, rl = c.reference(staged=True)
    check_close(out, lse, ro, rl, "prefill any scale", c.vmax)


def test_prefill_entries_outside_the_window_are_not_read():
    for window, new in ((17, [5, 300, 1]), (128, [200, 64, 33]), (500, [700, 1, 40])):
        c = Case([2000, 700, 5000], 16, 2, 64, 16, 16, seed=52, new=new, window=window)
        ro, rl = c.reference(staged=True)
        for b, (n, m) in enumerate(zip(c.lens, new)):
            c.table[b, :max(0, n - m - window + 1) // 16] = FAR
        out, lse = c.prefill()
        check_close(out, lse, ro, rl, "prefill window %d" % window, c.vmax)
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("window", [2 ** 31 - 1, 1200, 1199])
def test_windows_of_every_length(window):
    """Windows at and above the lengths, also where queries stand before the first
    key (Lq > Lk), hide nothing."""
    c = Case([300, 9, 1200, 64], 8, 2, 64, 16, 16, seed=54, new=[130, 40, 257, 64],
             window=window)
    out, lse = c.prefill()
    c.window = 0 if window > 1199 else window
    check_close(out, lse, *c.reference(staged=True), "prefill window %d" % window, c.vmax)
    c = Case([300, 9, 1200, 64], 8, 2, 64, 16, 16, seed=55, window=window)
    out, lse = c.decode()
    c.window = 0 if window > 1199 else window
    check_close(out, lse, *c.reference(), "decode window %d" % window, c.vmax)
    assert sa.sinkattn_get_device_error() == 0


def test_prefill_bad_pages():
    c = Case([300, 40], 8, 2, 64, 16, 16, seed=53, new=[100, 40])
    c.table[0, 5] = -1
    ro, rl = c.reference(staged=True)
    out, lse = c.prefill()
    check_close(out, lse, ro, rl, "prefill bad page", c.vmax)
    assert sa.sinkattn_get_device_error() == 2


# ---- the calls together ----------------------------------------------------------

def serve(c_heads, d, page, block, graph, window=0, steps=40):
    """Two prompts prefilled, then `steps` decode steps: page map, append and
    attention each step, checked against the float64 definitions on the cache
    that the reference keeps from the same rows."""
    hq, hkv = c_heads
    prompts = [37, 150]
    pages, width = 64, 32
    gen = torch.Generator().manual_seed(7)
    draw = lambda n, h: torch.randn(n, h, d, generator=gen).to(torch.bfloat16)  # noqa: E731
    kc = torch.full((pages, hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks = torch.full((pages, hkv, page // block), float("nan"), device="cuda")
    vs = ks.clone()
    free = torch.randperm(pages, generator=gen).to(torch.int32).cuda()
    head = t32([0]).cuda()
    table = torch.full((2, width), FAR, dtype=torch.int32, device="cuda")
    sinks = torch.randn(hq, generator=gen).cuda()
    r = dict(kc=kc.cpu().numpy(), vc=vc.cpu().numpy(), ks=ks.cpu().numpy(), vs=vs.cpu().numpy(),
             table=table.cpu().numpy(), head=0)

    def reference(lens, cu, k, v, q):
        slots, _, r["head"], r["table"], code = R.page_map(
            lens, cu, len(q), r["table"], free.cpu().numpy(), r["head"], page)
        assert code == 0
        r["kc"], r["ks"] = R.append(k.double().numpy(), slots, r["kc"], r["ks"])
        r["vc"], r["vs"] = R.append(v.double().numpy(), slots, r["vc"], r["vs"])
        kr = np.concatenate([R.rows_of(r["kc"], r["ks"], r["table"][b], n)
                             for b, n in enumerate(lens)])
        vr = np.concatenate([R.rows_of(r["vc"], r["vs"], r["table"][b], n)
                             for b, n in enumerate(lens)])
        return OB.forward(q, kr, vr, np.arange(3) if cu is None else cu,
                          np.concatenate([[0], np.cumsum(lens)]), hq=hq, hkv=hkv,
                          sinks=sinks.cpu(), causal=True, window=window, scale=d ** -0.5)

    lens = list(prompts)
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v, q = draw(sum(lens), hkv), draw(sum(lens), hkv), draw(sum(lens), hq)
    L, cu_d = t32(lens).cuda(), t32(cu).cuda()
    slots, _, _ = sa.sinkattn_page_map(L, table, free, head, page, cu_seqlens_q=cu_d,
                                       total_q=len(q), free_head_out=head)
    sa.sinkattn_append_fp8_block(k.cuda(), v.cuda(), slots, kc, vc, ks, vs)
    out, lse = sa.sinkattn_prefill_paged_fp8_block(q.cuda(), cu_d, kc, vc, ks, vs, table, L,
                                                   max(lens), width * page, sinks=sinks,
                                                   window=window)
    ro, rl = reference(lens, cu, k, v, q)
    check_close(out, lse, ro, rl, "serve prefill")

    one = dict(k=draw(2, hkv).cuda(), v=draw(2, hkv).cuda(), q=draw(2, hq).cuda())
    slots = torch.empty(2, dtype=torch.int64, device="cuda")
    offs = torch.empty(3, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(one["q"]), torch.empty((2, hq), device="cuda")
    ws = torch.empty(max(1, sa.sinkattn_decode_fp8_block_workspace_size(
        2, width * page, hq, hkv, d, window)), dtype=torch.uint8, device="cuda")

    def step():
        L.add_(1)
        sa.sinkattn_page_map(L, table, free, head, page, free_head_out=head, slot_mapping=slots,
                             page_offsets=offs)
        sa.sinkattn_append_fp8_block(one["k"], one["v"], slots, kc, vc, ks, vs)
        sa.sinkattn_decode_fp8_block(one["q"], kc, vc, ks, vs, table, L,
                                     max_seqlen_k=width * page, sinks=sinks, window=window,
                                     out=out, lse=lse, workspace=ws)

    if graph:
        state = [t.clone() for t in (L, table, head, kc, vc, ks, vs)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        for t, s in zip((L, table, head, kc, vc, ks, vs), state):
            t.copy_(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    for i in range(steps):
        lens = [n + 1 for n in lens]
        big = 4.0 if i == 11 else 1.0  # a token that makes the scales grow
        k, v, q = (draw(2, hkv) * big).to(torch.bfloat16), draw(2, hkv), draw(2, hq)
        one["k"].copy_(k)
        one["v"].copy_(v)
        one["q"].copy_(q)
        g.replay() if graph else step()
        ro, rl = reference(lens, None, k, v, q)
        check_close(out, lse, ro, rl, "serve step %d" % i)
    assert np.array_equal(kc.cpu().numpy(), r["kc"]) and np.array_equal(vc.cpu().numpy(), r["vc"])
    assert np.array_equal(ks.cpu().numpy(), r["ks"], equal_nan=True)
    assert np.array_equal(table.cpu().numpy(), r["table"]) and head.item() == r["head"]
    assert sa.sinkattn_get_device_error() == 0


@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(graph):
    serve((8, 2), 64, 16, 16, graph)
    serve((16, 2), 128, 16, 8, graph, window=50, steps=20)
    serve((3, 3), 64, 24, 1, graph, steps=20)


def test_without_lse_and_with_another_scale():
    for lens, new in (([3000, 50, 9000], None), ([900, 50, 1200], None),
                      ([300, 50, 900], [100, 50, 3])):
        c = Case(lens, 16, 2, 64, 16, 16, seed=66, new=new)
        c.scale = 0.3
        f = c.decode if new is None else c.prefill
        out, lse = f(scale=0.3)
        check_close(out, lse, *c.reference(), "scale", c.vmax)
        again, none = f(scale=0.3, return_lse=False)
        assert none is None and torch.equal(out, again)


def test_calls_on_another_stream():
    """Outputs and scratch that the calls allocate belong to the stream given."""
    c = Case([3000, 50, 900], 16, 2, 64, 16, 16, seed=60, new=[300, 50, 64])
    dc = Case([3000, 50, 900], 16, 2, 64, 16, 16, seed=61)
    po, pl = c.prefill()
    do, dl = dc.decode()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = c.dev(), dc.dev()
    q, cu, sk = c.q.cuda(), t32(c.cu).cuda(), c.sinks.cuda()
    q2, sk2 = dc.q.cuda(), dc.sinks.cuda()
    torch.cuda.synchronize()
    for _ in range(3):
        o1, l1 = sa.sinkattn_prefill_paged_fp8_block(
            q, cu, a["k_cache"], a["v_cache"], a["k_scale"], a["v_scale"], a["block_table"],
            a["seqlens_k"], 300, 3000, sinks=sk, stream=side)
        o2, l2 = sa.sinkattn_decode_fp8_block(q2, **b, max_seqlen_k=3000, sinks=sk2, stream=side)
        junk = torch.full((1 << 24,), 7, dtype=torch.uint8, device="cuda")  # noqa: F841
    torch.cuda.synchronize()
    assert torch.equal(o1, po) and torch.equal(l1, pl)
    assert torch.equal(o2, do) and torch.equal(l2, dl)


def test_named_workload_paged_decode_heads():
    """The serving geometry (64 q / 8 kv heads, 16-token pages) at a few lengths
    of the paged decode workload."""
    lens = S.uniform_lengths(8, 1024, 32768, seed=4000)
    c = Case(lens, 64, 8, 64, 16, 16, seed=70)
    out, lse = c.decode()
    ro, rl = c.reference()
    check_close(out, lse, ro, rl, "paged decode heads", c.vmax)
