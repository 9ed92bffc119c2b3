"""Host-side checks of the block-scaled fp8 cache that need no GPU: the
reference definitions and every refusal of the four calls (all of them return
before any CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from attention_learned_sinks_gb300 import build as sbuild
from attention_learned_sinks_gb300 import sinkattn as B
from oracle import block_cache as R
from oracle import fp8 as F

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)
M = B.Mask(1, 0, 0.125)


@pytest.fixture(scope="module")
def lib():
    sbuild.build()
    return sa.load()


# ---- the reference ------------------------------------------------------------

def test_reference_encoding_is_torchs():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 60
    x = torch.cat([x, torch.tensor([0.0, -0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10,
                                    1.5 * 2.0 ** -9, 17.0, 19.0])]).clamp(-448, 448)
    assert np.array_equal(R.encode_e4m3(x.double().numpy()),
                          x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert R.encode_e4m3([1e9])[0] == 0x7E


def test_reference_scale_is_the_smallest_power_of_two():
    for amax in (1e-30, 0.001, 0.4375, 0.4376, 1.0, 448.0, 448.5, 3.0e38):
        e = R.scale_exponent(amax)
        assert -60 <= e <= 60
        assert e == 60 or amax <= 448 * 2.0 ** e
        assert e == -60 or amax > 448 * 2.0 ** (e - 1)
    assert R.scale_exponent(0.0) == -60


def test_reference_append_in_pieces_is_append_at_once():
    """With values whose codes are normal under every scale involved, writing a
    sequence token by token gives the codes and scales of one call."""
    rng = np.random.default_rng(2)
    rows = rng.choice([1.0, -1.5, 3.0, 40.0, -0.75], size=(12, 2, 8)) * 2.0 ** rng.integers(
        -2, 3, size=(12, 1, 1))
    cache0 = np.full((2, 2, 8, 8), 0x7F, np.uint8)
    scale0 = np.full((2, 2, 2), np.nan, np.float32)
    slots = np.arange(2, 14) - 2
    one = R.append(rows, slots, cache0, scale0)
    cache, scale = cache0, scale0
    for i in range(12):
        cache, scale = R.append(rows[i:i + 1], slots[i:i + 1], cache, scale)
    assert np.array_equal(one[0], cache)
    assert np.array_equal(one[1], scale, equal_nan=True)
    for g in range(2):
        back = F.e4m3_to_float64(cache[0, g, :4]) * float(scale[0, g, 0])
        assert np.abs(back - rows[:4, g]).max() <= 2.0 ** -4 * np.abs(rows[:4, g]).max()


# ---- refusals -----------------------------------------------------------------

def page_map(lib, **kw):
    a = dict(lens=FAKE, cu=FAKE, batch=2, tq=10, ps=16, maxp=4, free=FAKE, nfree=8, head=FAKE,
             head_out=FAKE, table=FAKE, slots=FAKE, offs=FAKE)
    a.update(kw)
    return lib.sinkattn_page_map(a["lens"], a["cu"], a["batch"], a["tq"], a["ps"], a["maxp"],
                                 a["free"], a["nfree"], a["head"], a["head_out"], a["table"],
                                 a["slots"], a["offs"], None)


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(tq=-1), dict(ps=0), dict(maxp=-1),
                                dict(nfree=-1), dict(cu=None), dict(lens=None), dict(slots=None),
                                dict(table=None), dict(free=None), dict(head=None),
                                dict(head_out=None), dict(offs=None), dict(lens=ODD),
                                dict(cu=ODD), dict(table=ODD), dict(head=ODD), dict(offs=ODD),
                                dict(slots=ctypes.c_void_p((1 << 20) + 4))])
def test_page_map_refusals(lib, kw):
    assert page_map(lib, **kw) == B.SINKATTN_ERR_INVALID_ARGUMENT


def test_page_map_refuses_offsets_past_int32(lib):
    assert page_map(lib, tq=2 ** 31 - 5, nfree=6) == B.SINKATTN_ERR_UNSUPPORTED


def append(lib, **kw):
    a = dict(k=FAKE, v=FAKE, ks=128, vs=128, slots=FAKE, n=5, kc=FAKE, vc=FAKE, ksc=FAKE,
             vsc=FAKE, sb=16, pages=4, ps=16, hkv=2, d=64)
    a.update(kw)
    return lib.sinkattn_append_fp8_block(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["n"],
                                         a["kc"], a["vc"], a["ksc"], a["vsc"], a["sb"],
                                         a["pages"], a["ps"], a["hkv"], a["d"], None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(pages=-1), dict(hkv=0), dict(sb=0), dict(sb=5),
                                dict(sb=32), dict(ps=0), dict(ks=120), dict(vs=127),
                                dict(ks=132), dict(k=None), dict(v=None), dict(slots=None),
                                dict(kc=None), dict(vsc=None),
                                dict(k=ctypes.c_void_p((1 << 20) + 8)), dict(ksc=ODD),
                                dict(slots=ctypes.c_void_p((1 << 20) + 4))])
def test_append_refusals(lib, kw):
    assert append(lib, **kw) == B.SINKATTN_ERR_INVALID_ARGUMENT


def test_append_unsupported_and_empty(lib):
    assert append(lib, d=96, ks=192, vs=192) == B.SINKATTN_ERR_UNSUPPORTED
    assert append(lib, hkv=70000, ks=70000 * 64, vs=70000 * 64) == B.SINKATTN_ERR_UNSUPPORTED
    assert append(lib, n=0) == B.SINKATTN_OK


def attend(lib, prefill, **kw):
    a = dict(q=FAKE, cu=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, sb=16, table=FAKE,
             lens=FAKE, pages=8, maxp=4000, ps=16, batch=2, tq=10, mq=5, mk=64000, hq=8, hkv=2,
             d=64, sinks=None, mask=M, ns=0, out=FAKE, lse=None, ws=None, wsb=0)
    a.update(kw)
    head = [a["q"]] + ([a["cu"]] if prefill else [])
    mid = [a["kc"], a["vc"], a["ksc"], a["vsc"], a["sb"], a["table"], a["lens"], a["pages"],
           a["maxp"], a["ps"], a["batch"]] + ([a["tq"], a["mq"]] if prefill else [])
    f = lib.sinkattn_prefill_paged_fp8_block if prefill else lib.sinkattn_decode_fp8_block
    return f(*head, *mid, a["mk"], a["hq"], a["hkv"], a["d"], a["sinks"], a["mask"], a["ns"],
             a["out"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw", [dict(sb=0), dict(sb=3), dict(sb=32), dict(ps=0), dict(batch=-1),
                                dict(hq=9), dict(hkv=0), dict(pages=0), dict(mk=64001),
                                dict(ns=-1), dict(mask=B.Mask(1, -1, 0.1)),
                                dict(mask=B.Mask(1, 0, float("nan"))), dict(q=None),
                                dict(kc=None), dict(ksc=None), dict(vsc=None), dict(table=None),
                                dict(lens=None), dict(out=None), dict(ksc=ODD), dict(lens=ODD),
                                dict(q=ctypes.c_void_p((1 << 20) + 8))])
def test_attention_refusals(lib, prefill, kw):
    assert attend(lib, prefill, **kw) == B.SINKATTN_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("prefill", [False, True])
def test_attention_unsupported_workspace_and_empty(lib, prefill):
    assert attend(lib, prefill, d=96) == B.SINKATTN_ERR_UNSUPPORTED
    assert attend(lib, prefill, batch=70000) == B.SINKATTN_ERR_UNSUPPORTED
    assert attend(lib, prefill) == B.SINKATTN_ERR_WORKSPACE_TOO_SMALL
    assert attend(lib, prefill, batch=0) == B.SINKATTN_OK
    need = (lib.sinkattn_prefill_paged_fp8_block_workspace_size(2, 10, 5, 64000, 8, 2, 64, 0, 0) if prefill
            else lib.sinkattn_decode_fp8_block_workspace_size(2, 64000, 8, 2, 64, 0, 0))
    assert need > 0
    assert attend(lib, prefill, ws=FAKE, wsb=need - 1) == B.SINKATTN_ERR_WORKSPACE_TOO_SMALL
    assert attend(lib, prefill, ws=ctypes.c_void_p((1 << 20) + 16), wsb=need) == \
        B.SINKATTN_ERR_INVALID_ARGUMENT
    assert lib.sinkattn_decode_fp8_block_workspace_size(2, 64000, 9, 2, 64, 0, 0) == 0
    assert lib.sinkattn_decode_fp8_block_workspace_size(2, 64000, 8, 2, 96, 0, 0) == 0


def test_binding_refuses_wrong_tensors(lib):
    """CPU tensors, types and shapes are refused by the binding itself."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    codes, scale = torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2, 1))
    rows, q = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 8, 64),
                                                                         dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sa.sinkattn_page_map(i32(2), i32(2, 4), i32(8), i32(1), 16)
    with pytest.raises(ValueError, match="total_q"):
        sa.sinkattn_page_map(i32(2), i32(2, 4), i32(8), i32(1), 16, cu_seqlens_q=i32(3))
    with pytest.raises(ValueError, match="CUDA"):
        sa.sinkattn_append_fp8_block(rows, rows, torch.zeros(3, dtype=torch.int64), codes, codes,
                                     scale, scale)
    with pytest.raises(ValueError, match="scales per page"):
        sa.sinkattn_append_fp8_block(rows, rows, torch.zeros(3, dtype=torch.int64), codes, codes,
                                     torch.zeros((4, 2, 3)), scale)
    with pytest.raises(ValueError, match="CUDA"):
        sa.sinkattn_decode_fp8_block(q, codes, codes, scale, scale, i32(2, 4), i32(2),
                                     max_seqlen_k=64)
    with pytest.raises(ValueError, match="CUDA"):
        sa.sinkattn_prefill_paged_fp8_block(q, i32(3), codes, codes, scale, scale, i32(2, 4),
                                            i32(2), 1, 64)
