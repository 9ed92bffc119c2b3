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
from test_parity_block_cache import Case

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
    assert np.abs(l - lse)[seen].max(initial=0.0) <= 1e-3 and np.isneginf(l[~seen]).all()


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
