"""Thin ctypes binding of libsinkattn.so (C ABI in include/sinkattn.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the launch stream, missing outputs/workspace are allocated with
torch. Every step of the computation runs in the library's CUDA kernels; there
is no fallback. If the library is missing or cannot be loaded, every call
raises.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libsinkattn.so")

SINKATTN_OK = 0
SINKATTN_ERR_INVALID_ARGUMENT = 1
SINKATTN_ERR_UNSUPPORTED = 2
SINKATTN_ERR_WORKSPACE_TOO_SMALL = 3
SINKATTN_ERR_CUDA = 4
# size of the fixed scratch array behind sinkattn_decode_noalloc (as in the header)
SINKATTN_NOALLOC_SCRATCH_BYTES = 32 << 20

EXPORTED = (
    "sinkattn_status_string",
    "sinkattn_last_cuda_error",
    "sinkattn_prefill_workspace_size",
    "sinkattn_prefill",
    "sinkattn_prefill_paged_workspace_size",
    "sinkattn_prefill_paged",
    "sinkattn_prefill_backward_workspace_size",
    "sinkattn_prefill_backward",
    "sinkattn_decode_workspace_size",
    "sinkattn_decode",
    "sinkattn_decode_fp8",
    "sinkattn_decode_noalloc",
    "sinkattn_prefill_paged_fp8",
    "sinkattn_page_map",
    "sinkattn_append_fp8_block",
    "sinkattn_decode_fp8_block_workspace_size",
    "sinkattn_decode_fp8_block",
    "sinkattn_prefill_paged_fp8_block_workspace_size",
    "sinkattn_prefill_paged_fp8_block",
    "sinkattn_qk_norm_rope",
    "sinkattn_qk_norm_rope_backward_workspace_size",
    "sinkattn_qk_norm_rope_backward",
    "sinkattn_decode_tree_workspace_size",
    "sinkattn_decode_tree",
    "sinkattn_verify_tree",
    "sinkattn_compact",
    "sinkattn_merge",
    "sinkattn_get_device_error",
    "sinkattn_debug_stall_waits",
)


class SinkAttnError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = "%s: %s (status %d)" % (what, _status_string(status), status)
        if status == SINKATTN_ERR_CUDA:
            try:
                msg += ": " + load().sinkattn_last_cuda_error().decode()
            except Exception:  # library missing: the status alone
                pass
        super().__init__(msg)


class Mask(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int), ("window", ctypes.c_int), ("scale", ctypes.c_float)]


_LIB = None


def load(path: str = LIB_PATH):
    """Load the library (once) and declare its signatures."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError("libsinkattn.so not built at %s: run "
                           "`python -m attention_learned_sinks_gb300.build`" % path)
    lib = ctypes.CDLL(path)
    P, I, L, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.sinkattn_status_string.argtypes = [I]
    lib.sinkattn_status_string.restype = ctypes.c_char_p
    lib.sinkattn_last_cuda_error.argtypes = []
    lib.sinkattn_last_cuda_error.restype = ctypes.c_char_p
    lib.sinkattn_prefill_workspace_size.argtypes = [I, L, L, I, I, I, I, I, I, I]
    lib.sinkattn_prefill_workspace_size.restype = S
    lib.sinkattn_prefill.argtypes = [P, P, P, P, P, I, L, L, I, I, I, I, I, P, Mask, I,
                                     P, P, P, S, P]
    lib.sinkattn_prefill.restype = I
    lib.sinkattn_prefill_paged_workspace_size.argtypes = [I, L, I, I, I, I, I, I, I]
    lib.sinkattn_prefill_paged_workspace_size.restype = S
    lib.sinkattn_prefill_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, L, I, I, I, I, I, P,
                                           Mask, I, P, P, P, S, P]
    lib.sinkattn_prefill_paged.restype = I
    lib.sinkattn_prefill_paged_fp8.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, L, I, I, I,
                                               I, I, P, Mask, I, P, P, P, S, P]
    lib.sinkattn_prefill_paged_fp8.restype = I
    lib.sinkattn_prefill_backward_workspace_size.argtypes = [I, L, L, I, I, I]
    lib.sinkattn_prefill_backward_workspace_size.restype = S
    lib.sinkattn_prefill_backward.argtypes = [P, P, P, P, P, P, P, P, I, L, L, I, I, I, I, I, P,
                                              Mask, P, P, P, P, P, S, P]
    lib.sinkattn_prefill_backward.restype = I
    lib.sinkattn_decode_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.sinkattn_decode_workspace_size.restype = S
    lib.sinkattn_decode.argtypes = [P, P, P, P, P, P, L, I, I, I, I, I, I, I, P, Mask, I,
                                    P, P, P, S, P]
    lib.sinkattn_decode.restype = I
    lib.sinkattn_decode_fp8.argtypes = [P, P, P, P, P, P, P, P, L, I, I, I, I, I, I, I, P, Mask,
                                        I, P, P, P, S, P]
    lib.sinkattn_decode_fp8.restype = I
    lib.sinkattn_decode_noalloc.argtypes = [P, P, P, P, P, P, L, I, I, I, I, I, I, I, P, Mask,
                                            I, P, P, P]
    lib.sinkattn_decode_noalloc.restype = I
    lib.sinkattn_page_map.argtypes = [P, P, I, L, I, I, P, I, P, P, P, P, P, P]
    lib.sinkattn_page_map.restype = I
    lib.sinkattn_append_fp8_block.argtypes = [P, P, L, L, P, L, P, P, P, P, I, I, I, I, I, P]
    lib.sinkattn_append_fp8_block.restype = I
    lib.sinkattn_decode_fp8_block_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.sinkattn_decode_fp8_block_workspace_size.restype = S
    lib.sinkattn_decode_fp8_block.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, P,
                                              Mask, I, P, P, P, S, P]
    lib.sinkattn_decode_fp8_block.restype = I
    lib.sinkattn_prefill_paged_fp8_block_workspace_size.argtypes = [I, L, I, I, I, I, I, I, I]
    lib.sinkattn_prefill_paged_fp8_block_workspace_size.restype = S
    lib.sinkattn_prefill_paged_fp8_block.argtypes = [P, P, P, P, P, P, I, P, P, I, I, I, I, L, I,
                                                     I, I, I, I, P, Mask, I, P, P, P, S, P]
    lib.sinkattn_prefill_paged_fp8_block.restype = I
    F = ctypes.c_float
    lib.sinkattn_qk_norm_rope.argtypes = [P, P, P, L, L, L, P, L, I, I, I, P, P, F, P, I, I, I, P,
                                          P, P, P, P, I, I, P]
    lib.sinkattn_qk_norm_rope.restype = I
    lib.sinkattn_qk_norm_rope_backward_workspace_size.argtypes = [I]
    lib.sinkattn_qk_norm_rope_backward_workspace_size.restype = S
    lib.sinkattn_qk_norm_rope_backward.argtypes = [P, P, P, P, L, L, P, L, I, I, I, P, P, F, P, I,
                                                   I, I, P, P, L, L, P, P, P, S, P]
    lib.sinkattn_qk_norm_rope_backward.restype = I
    lib.sinkattn_decode_tree_workspace_size.argtypes = [I, L, I, I, I, I, I, I, I]
    lib.sinkattn_decode_tree_workspace_size.restype = S
    lib.sinkattn_decode_tree.argtypes = [P, P, P, P, P, P, P, I, I, I, I, L, I, I, I, I, I, P,
                                         Mask, I, P, P, P, S, P]
    lib.sinkattn_decode_tree.restype = I
    lib.sinkattn_verify_tree.argtypes = [P, P, P, P, P, P, I, L, I, I, P, P, P, P]
    lib.sinkattn_verify_tree.restype = I
    lib.sinkattn_compact.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, I, P, P, P]
    lib.sinkattn_compact.restype = I
    lib.sinkattn_merge.argtypes = [P, P, I, L, I, I, P, P, P, P]
    lib.sinkattn_merge.restype = I
    lib.sinkattn_get_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
    lib.sinkattn_get_device_error.restype = I
    lib.sinkattn_debug_stall_waits.argtypes = [ctypes.c_uint64]
    lib.sinkattn_debug_stall_waits.restype = I
    _LIB = lib
    return lib


def _status_string(status):
    try:
        return load().sinkattn_status_string(status).decode()
    except Exception:  # library missing: still report the number
        return "status"


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status, what):
    if status != SINKATTN_OK:
        raise SinkAttnError(status, what)


def _req(t, dtype, name):
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA %s tensor" % (name, dtype))


def sinkattn_prefill_workspace_size(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, hq,
                                    hkv, head_dim=64, window=0, num_splits=0):
    return load().sinkattn_prefill_workspace_size(int(batch), int(total_q), int(total_k),
                                                  int(max_seqlen_q), int(max_seqlen_k), hq, hkv,
                                                  head_dim, int(window), int(num_splits))


def sinkattn_decode_workspace_size(batch, max_seqlen_k, hq, hkv, head_dim=64, window=0,
                                   num_splits=0):
    return load().sinkattn_decode_workspace_size(batch, max_seqlen_k, hq, hkv, head_dim,
                                                 window, num_splits)


def sinkattn_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, *,
                     sinks=None, causal=True, window=0, scale=None, num_splits=0, out=None,
                     lse=None, return_lse=True, workspace=None, total_q=None, total_k=None,
                     stream=None):
    """Sink-attention prefill over packed sequences. Returns (out, lse)."""
    lib = load()
    _req(q, torch.bfloat16, "q")
    _req(k, torch.bfloat16, "k")
    _req(v, torch.bfloat16, "v")
    _req(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _req(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    tq, hq, d = q.shape
    tk, hkv, _ = k.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((tq, hq), dtype=torch.float32, device=q.device)
    if sinks is not None:
        _req(sinks, torch.float32, "sinks")
    tk_ = tk if total_k is None else total_k
    tq_ = tq if total_q is None else total_q
    batch = cu_seqlens_q.numel() - 1
    if workspace is None:
        need = lib.sinkattn_prefill_workspace_size(batch, tq_, tk_, int(max_seqlen_q),
                                                   int(max_seqlen_k), hq, hkv, d, int(window),
                                                   int(num_splits))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask = Mask(1 if causal else 0, int(window), float(d ** -0.5 if scale is None else scale))
    st = lib.sinkattn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                              batch, tq_, tk_, int(max_seqlen_q), int(max_seqlen_k), hq, hkv, d,
                              _ptr(sinks), mask, int(num_splits), _ptr(out), _ptr(lse),
                              _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sinkattn_prefill")
    return out, lse


def sinkattn_prefill_paged_workspace_size(batch, total_q, max_seqlen_q, max_seqlen_k, hq, hkv,
                                          head_dim=64, window=0, num_splits=0):
    return load().sinkattn_prefill_paged_workspace_size(int(batch), int(total_q),
                                                        int(max_seqlen_q), int(max_seqlen_k), hq,
                                                        hkv, head_dim, int(window),
                                                        int(num_splits))


def sinkattn_prefill_paged(q, cu_seqlens_q, k_cache, v_cache, block_table, seqlens_k,
                           max_seqlen_q, max_seqlen_k, *, sinks=None, causal=True, window=0,
                           scale=None, num_splits=0, out=None, lse=None, return_lse=True,
                           workspace=None, stream=None):
    """Sink-attention prefill of packed queries against a paged KV cache
    [num_pages, hkv, page_size, head_dim] addressed by block_table / seqlens_k.
    Returns (out, lse)."""
    lib = load()
    _req(q, torch.bfloat16, "q")
    _req(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _req(k_cache, torch.bfloat16, "k_cache")
    _req(v_cache, torch.bfloat16, "v_cache")
    _req(block_table, torch.int32, "block_table")
    _req(seqlens_k, torch.int32, "seqlens_k")
    tq, hq, d = q.shape
    num_pages, hkv, page_size, _ = k_cache.shape
    batch = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((tq, hq), dtype=torch.float32, device=q.device)
    if sinks is not None:
        _req(sinks, torch.float32, "sinks")
    if workspace is None:
        need = lib.sinkattn_prefill_paged_workspace_size(batch, tq, int(max_seqlen_q),
                                                         int(max_seqlen_k), hq, hkv, d,
                                                         int(window), int(num_splits))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask = Mask(1 if causal else 0, int(window), float(d ** -0.5 if scale is None else scale))
    st = lib.sinkattn_prefill_paged(_ptr(q), _ptr(cu_seqlens_q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_table), _ptr(seqlens_k), num_pages,
                                    block_table.shape[1], page_size, batch, tq,
                                    int(max_seqlen_q), int(max_seqlen_k), hq, hkv, d,
                                    _ptr(sinks), mask, int(num_splits), _ptr(out), _ptr(lse),
                                    _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sinkattn_prefill_paged")
    return out, lse


def sinkattn_prefill_paged_fp8(q, cu_seqlens_q, k_cache, v_cache, block_table, seqlens_k,
                               max_seqlen_q, max_seqlen_k, *, k_scale=None, v_scale=None,
                               sinks=None, causal=True, window=0, scale=None, num_splits=0,
                               out=None, lse=None, return_lse=True, workspace=None,
                               stream=None):
    """sinkattn_prefill_paged over an fp8 e4m3 cache: k_cache / v_cache hold
    uint8 codes [num_pages, hkv, page_size, head_dim]; k_scale / v_scale are
    float32 [hkv] (None = 1). Returns (out, lse)."""
    lib = load()
    _req(q, torch.bfloat16, "q")
    _req(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _req(k_cache, torch.uint8, "k_cache")
    _req(v_cache, torch.uint8, "v_cache")
    _req(block_table, torch.int32, "block_table")
    _req(seqlens_k, torch.int32, "seqlens_k")
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale"), (sinks, "sinks")):
        if t is not None:
            _req(t, torch.float32, n)
    tq, hq, d = q.shape
    num_pages, hkv, page_size, _ = k_cache.shape
    batch = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((tq, hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = lib.sinkattn_prefill_paged_workspace_size(batch, tq, int(max_seqlen_q),
                                                         int(max_seqlen_k), hq, hkv, d,
                                                         int(window), int(num_splits))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask = Mask(1 if causal else 0, int(window), float(d ** -0.5 if scale is None else scale))
    st = lib.sinkattn_prefill_paged_fp8(_ptr(q), _ptr(cu_seqlens_q), _ptr(k_cache),
                                        _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                        _ptr(block_table), _ptr(seqlens_k), num_pages,
                                        block_table.shape[1], page_size, batch, tq,
                                        int(max_seqlen_q), int(max_seqlen_k), hq, hkv, d,
                                        _ptr(sinks), mask, int(num_splits), _ptr(out), _ptr(lse),
                                        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sinkattn_prefill_paged_fp8")
    return out, lse


def sinkattn_prefill_backward_workspace_size(batch, total_q, total_k, hq, hkv, head_dim=64):
    return load().sinkattn_prefill_backward_workspace_size(int(batch), int(total_q),
                                                           int(total_k), hq, hkv, head_dim)


def sinkattn_prefill_backward(q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                              max_seqlen_k, *, sinks=None, causal=True, window=0, scale=None,
                              dq=None, dk=None, dv=None, dsinks=None, workspace=None,
                              stream=None):
    """Gradients of sinkattn_prefill with respect to q, k, v and the sinks,
    given the forward's out and lse and the output gradient dout.
    Returns (dq, dk, dv, dsinks); dsinks is None without sinks."""
    lib = load()
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _req(t, torch.bfloat16, name)
    _req(lse, torch.float32, "lse")
    _req(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _req(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    tq, hq, d = q.shape
    tk, hkv, _ = k.shape
    batch = cu_seqlens_q.numel() - 1
    if sinks is not None:
        _req(sinks, torch.float32, "sinks")
        if dsinks is None:
            dsinks = torch.empty(hq, dtype=torch.float32, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        need = lib.sinkattn_prefill_backward_workspace_size(batch, tq, tk, hq, hkv, d)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask = Mask(1 if causal else 0, int(window), float(d ** -0.5 if scale is None else scale))
    st = lib.sinkattn_prefill_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout),
                                       _ptr(lse), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), batch,
                                       tq, tk, int(max_seqlen_q), int(max_seqlen_k), hq, hkv, d,
                                       _ptr(sinks), mask, _ptr(dq), _ptr(dk), _ptr(dv),
                                       _ptr(dsinks if sinks is not None else None),
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sinkattn_prefill_backward")
    return dq, dk, dv, (dsinks if sinks is not None else None)


def sinkattn_decode(q, k_cache, v_cache, *, kv_indptr=None, block_table=None, seqlens_k=None,
                    max_seqlen_k, sinks=None, window=0, scale=None, num_splits=0, out=None,
                    lse=None, return_lse=True, workspace=None, stream=None):
    """Sink-attention decode over a contiguous (kv_indptr) or paged
    (block_table + seqlens_k) KV cache. Returns (out, lse)."""
    lib = load()
    _req(q, torch.bfloat16, "q")
    _req(k_cache, torch.bfloat16, "k_cache")
    _req(v_cache, torch.bfloat16, "v_cache")
    batch, hq, d = q.shape
    hkv = k_cache.shape[1]
    if block_table is not None:
        _req(block_table, torch.int32, "block_table")
        _req(seqlens_k, torch.int32, "seqlens_k")
        kv_rows, page_size, max_pages = k_cache.shape[0], k_cache.shape[2], block_table.shape[1]
    else:
        _req(kv_indptr, torch.int32, "kv_indptr")
        kv_rows, page_size, max_pages = k_cache.shape[0], 0, 0
    if sinks is not None:
        _req(sinks, torch.float32, "sinks")
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((batch, hq), dtype=torch.float32, device=q.device)
    need = lib.sinkattn_decode_workspace_size(batch, int(max_seqlen_k), hq, hkv, d, int(window),
                                              int(num_splits))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask = Mask(1, int(window), float(d ** -0.5 if scale is None else scale))
    st = lib.sinkattn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_indptr),
                             _ptr(block_table), _ptr(seqlens_k), kv_rows, max_pages, page_size,
                             batch, int(max_seqlen_k), hq, hkv, d, _ptr(sinks), mask,
                             int(num_splits), _ptr(out), _ptr(lse), _ptr(workspace),
                             workspace.numel(), _stream(stream))
    _check(st, "sinkattn_decode")
    return out, lse


def sinkattn_decode_fp8(q, k_cache, v_cache, *, k_scale=None, v_scale=None, kv_indptr=None,
                        block_table=None, seqlens_k=None, max_seqlen_k, sinks=None, window=0,
                        scale=None, num_splits=0, out=None, lse=None, return_lse=True,
                        workspace=None, stream=None):
    """sinkattn_decode over an fp8 e4m3 cache (uint8 codes, same layouts) with
    optional per-KV-head scales. Returns (out, lse)."""
    lib = load()
    _req(q, torch.bfloat16, "q")
    _req(k_cache, torch.uint8, "k_cache")
    _req(v_cache, torch.uint8, "v_cache")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale"), (sinks, "sinks")):
        if t is not None:
            _req(t, torch.float32, name)
    batch, hq, d = q.shape
    hkv = k_cache.shape[1]
    if block_table is not None:
        _req(block_table, torch.int32, "block_table")
        _req(seqlens_k, torch.int32, "seqlens_k")
        kv_rows, page_size, max_pages = k_cache.shape[0], k_cache.shape[2], block_table.shape[1]
    else:
        _req(kv_indptr, torch.int32, "kv_indptr")
        kv_rows, page_size, max_pages = k_cache.shape[0], 0, 0
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((batch, hq), dtype=torch.float32, device=q.device)
    need = lib.sinkattn_decode_workspace_size(batch, int(max_seqlen_k), hq, hkv, d, int(window),
                                              int(num_splits))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    mask = Mask(1, int(window), float(d ** -0.5 if scale is None else scale))
    st = lib.sinkattn_decode_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                 _ptr(v_scale), _ptr(kv_indptr), _ptr(block_table),
                                 _ptr(seqlens_k), kv_rows, max_pages, page_size, batch,
                                 int(max_seqlen_k), hq, hkv, d, _ptr(sinks), mask,
                                 int(num_splits), _ptr(out), _ptr(lse), _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _check(st, "sinkattn_decode_fp8")
    return out, lse


def sinkattn_decode_noalloc(q, k_cache, v_cache, *, kv_indptr=None, block_table=None,
                            seqlens_k=None, max_seqlen_k, sinks=None, window=0, scale=None,
                            num_splits=0, out, lse=None, stream=None):
    """sinkattn_decode without a workspace: the library's fixed scratch array is
    used instead (for callers that may not allocate device memory). `out` (and
    `lse`, if wanted) must be given; nothing is allocated here."""
    lib = load()
    batch, hq, d = q.shape
    hkv = k_cache.shape[1]
    if block_table is not None:
        kv_rows, page_size, max_pages = k_cache.shape[0], k_cache.shape[2], block_table.shape[1]
    else:
        kv_rows, page_size, max_pages = k_cache.shape[0], 0, 0
    mask = Mask(1, int(window), float(d ** -0.5 if scale is None else scale))
    st = lib.sinkattn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_indptr),
                                     _ptr(block_table), _ptr(seqlens_k), kv_rows, max_pages,
                                     page_size, batch, int(max_seqlen_k), hq, hkv, d, _ptr(sinks),
                                     mask, int(num_splits), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "sinkattn_decode_noalloc")
    return out, lse


# ---- block-scaled fp8 paged cache -------------------------------------------
# These calls check shapes and devices, run on the tensors' device, and take
# what they allocate from the stream that they launch on.

class _Unchanged:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_UNCHANGED = _Unchanged()


def _scope(device, stream):
    """Makes `stream` (or the device's current stream) the current one."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return _UNCHANGED
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    return torch.cuda.stream(stream)


def _at(t):
    return None if t is None else t.data_ptr()


def _current(device):
    """The device's current stream as an integer (a Stream object costs 3 us)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _tensor(t, dtype, shape, device, name):
    if (t.dtype is not dtype or t.shape != shape or t.device != device
            or not t.is_contiguous() or not t.is_cuda):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, tuple(shape), device if device.type == "cuda"
                            else "a CUDA device"))


def _block_cache(k_cache, v_cache, k_scale, v_scale, device):
    """Checks a block-scaled cache; returns (num_pages, hkv, page_size, D, scale_block)."""
    if k_cache.dim() != 4 or k_scale.dim() != 3:
        raise ValueError("k_cache must be [num_pages, hkv, page_size, D] and k_scale "
                         "[num_pages, hkv, page_size / scale_block]")
    pages, hkv, page, d = k_cache.shape
    per = k_scale.shape[2]
    if per <= 0 or page % per != 0:
        raise ValueError("k_scale has %d scales per page, which does not divide %d" % (per, page))
    codes, scales = (pages, hkv, page, d), (pages, hkv, per)
    _tensor(k_cache, torch.uint8, codes, device, "k_cache")
    _tensor(v_cache, torch.uint8, codes, device, "v_cache")
    _tensor(k_scale, torch.float32, scales, device, "k_scale")
    _tensor(v_scale, torch.float32, scales, device, "v_scale")
    return pages, hkv, page, d, page // per


def sinkattn_page_map(seqlens_k, block_table, free_pages, free_head, page_size, *,
                      cu_seqlens_q=None, total_q=None, free_head_out=None, slot_mapping=None,
                      page_offsets=None, stream=None):
    """Block tables and slot maps from request lengths: gives each sequence's new
    tokens pages from free_pages (from entry free_head on), writes the new pages
    into block_table [batch, max_pages] in place, and returns (slot_mapping int64
    [total_q], page_offsets int32 [batch + 1], free_head_out int32 [1]).

    cu_seqlens_q None: one new token per sequence. total_q (rows of
    slot_mapping) is needed with cu_seqlens_q unless slot_mapping is given;
    rows past cu_seqlens_q[-1] get -1. free_head_out may be free_head."""
    lib = load()
    device = seqlens_k.device
    batch = seqlens_k.numel()
    if total_q is None:
        if slot_mapping is not None:
            total_q = slot_mapping.numel()
        elif cu_seqlens_q is None:
            total_q = batch
        else:
            raise ValueError("total_q is needed with cu_seqlens_q")
    total_q, num_free = int(total_q), free_pages.numel()
    _tensor(seqlens_k, torch.int32, (batch,), device, "seqlens_k")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages]")
    max_pages = block_table.shape[1]
    _tensor(block_table, torch.int32, (batch, max_pages), device, "block_table")
    _tensor(free_pages, torch.int32, (num_free,), device, "free_pages")
    _tensor(free_head, torch.int32, (1,), device, "free_head")
    if cu_seqlens_q is not None:
        _tensor(cu_seqlens_q, torch.int32, (batch + 1,), device, "cu_seqlens_q")
    with _scope(device, stream):
        if slot_mapping is None:
            slot_mapping = torch.empty(total_q, dtype=torch.int64, device=device)
        if page_offsets is None:
            page_offsets = torch.empty(batch + 1, dtype=torch.int32, device=device)
        if free_head_out is None:
            free_head_out = torch.empty_like(free_head)
        _tensor(slot_mapping, torch.int64, (total_q,), device, "slot_mapping")
        _tensor(page_offsets, torch.int32, (batch + 1,), device, "page_offsets")
        _tensor(free_head_out, torch.int32, (1,), device, "free_head_out")
        st = lib.sinkattn_page_map(_at(seqlens_k), _at(cu_seqlens_q), batch, total_q,
                                   int(page_size), max_pages, _at(free_pages), num_free,
                                   _at(free_head), _at(free_head_out), _at(block_table),
                                   _at(slot_mapping), _at(page_offsets), _current(device))
    _check(st, "sinkattn_page_map")
    return slot_mapping, page_offsets, free_head_out


def _token_rows(t, n, hkv, d, device, name):
    """Token stride of bf16 rows [n, hkv, D] that may be a slice of wider rows."""
    if t.dtype != torch.bfloat16 or t.device != device or t.shape != (n, hkv, d):
        raise ValueError("%s must be a bfloat16 tensor of shape %s on %s"
                         % (name, (n, hkv, d), device))
    if d > 1 and t.stride(2) != 1 or hkv > 1 and t.stride(1) != d:
        raise ValueError("%s: each token's [hkv, D] must be contiguous" % name)
    return t.stride(0) if n > 1 else hkv * d


def sinkattn_append_fp8_block(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, *,
                              stream=None):
    """Writes key and value rows (bf16 [n, hkv, D], any token stride that is a
    multiple of 8) into a block-scaled fp8 cache in place: codes uint8
    [num_pages, hkv, page_size, D], scales float32 [num_pages, hkv, scales per
    page]. Rows with a negative slot are skipped."""
    lib = load()
    device = k_cache.device
    pages, hkv, page, d, block = _block_cache(k_cache, v_cache, k_scale, v_scale, device)
    n = slot_mapping.numel()
    _tensor(slot_mapping, torch.int64, (n,), device, "slot_mapping")
    ks = _token_rows(k, n, hkv, d, device, "k")
    vs = _token_rows(v, n, hkv, d, device, "v")
    with _scope(device, stream):
        st = lib.sinkattn_append_fp8_block(_at(k), _at(v), ks, vs, _at(slot_mapping), n,
                                           _at(k_cache), _at(v_cache), _at(k_scale),
                                           _at(v_scale), block, pages, page, hkv, d,
                                           _current(device))
    _check(st, "sinkattn_append_fp8_block")


def sinkattn_decode_fp8_block_workspace_size(batch, max_seqlen_k, hq, hkv, head_dim=64, window=0,
                                             num_splits=0):
    return load().sinkattn_decode_fp8_block_workspace_size(
        int(batch), int(max_seqlen_k), hq, hkv, head_dim, int(window), int(num_splits))


def _outputs(q, rows, hq, device, out, lse, return_lse):
    if out is None:
        out = torch.empty_like(q)
    else:
        _tensor(out, torch.bfloat16, q.shape, device, "out")
    if lse is not None:
        _tensor(lse, torch.float32, (rows, hq), device, "lse")
    elif return_lse:
        lse = torch.empty((rows, hq), dtype=torch.float32, device=device)
    return out, lse


def _scratch(workspace, need, device):
    """The caller's workspace, or `need` bytes (None for 0)."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _tensor(workspace, torch.uint8, (workspace.numel(),), device, "workspace")
    return workspace


def sinkattn_decode_fp8_block(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, *,
                              max_seqlen_k, sinks=None, window=0, scale=None, num_splits=0,
                              out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """Sink-attention decode over a paged fp8 cache with a scale for each (block
    of tokens, KV head): uint8 codes [num_pages, hkv, page_size, D], float32
    scales [num_pages, hkv, scales per page]. Returns (out, lse)."""
    lib = load()
    device = q.device
    pages, hkv, page, d, block = _block_cache(k_cache, v_cache, k_scale, v_scale, device)
    batch, hq, _ = q.shape
    _tensor(q, torch.bfloat16, (batch, hq, d), device, "q")
    max_pages = block_table.shape[-1]
    _tensor(block_table, torch.int32, (batch, max_pages), device, "block_table")
    _tensor(seqlens_k, torch.int32, (batch,), device, "seqlens_k")
    if sinks is not None:
        _tensor(sinks, torch.float32, (hq,), device, "sinks")
    max_seqlen_k, window, num_splits = int(max_seqlen_k), int(window), int(num_splits)
    mask = Mask(1, window, float(d ** -0.5 if scale is None else scale))
    with _scope(device, stream):
        out, lse = _outputs(q, batch, hq, device, out, lse, return_lse)
        need = 0
        if workspace is None:
            need = lib.sinkattn_decode_fp8_block_workspace_size(batch, max_seqlen_k, hq, hkv, d,
                                                                window, num_splits)
        workspace = _scratch(workspace, need, device)
        st = lib.sinkattn_decode_fp8_block(_at(q), _at(k_cache), _at(v_cache), _at(k_scale),
                                           _at(v_scale), block, _at(block_table),
                                           _at(seqlens_k), pages, max_pages, page, batch,
                                           max_seqlen_k, hq, hkv, d, _at(sinks), mask,
                                           num_splits, _at(out), _at(lse), _at(workspace),
                                           0 if workspace is None else workspace.numel(),
                                           _current(device))
    _check(st, "sinkattn_decode_fp8_block")
    return out, lse


def sinkattn_prefill_paged_fp8_block_workspace_size(batch, total_q, max_seqlen_q, max_seqlen_k,
                                                    hq, hkv, head_dim=64, window=0, num_splits=0):
    return load().sinkattn_prefill_paged_fp8_block_workspace_size(
        int(batch), int(total_q), int(max_seqlen_q), int(max_seqlen_k), hq, hkv, head_dim,
        int(window), int(num_splits))


def sinkattn_prefill_paged_fp8_block(q, cu_seqlens_q, k_cache, v_cache, k_scale, v_scale,
                                     block_table, seqlens_k, max_seqlen_q, max_seqlen_k, *,
                                     sinks=None, causal=True, window=0, scale=None, num_splits=0,
                                     out=None, lse=None, return_lse=True, workspace=None,
                                     stream=None):
    """sinkattn_prefill_paged over a block-scaled fp8 cache: uint8 codes
    [num_pages, hkv, page_size, D], float32 scales [num_pages, hkv, scales per
    page]. Returns (out, lse)."""
    lib = load()
    device = q.device
    pages, hkv, page, d, block = _block_cache(k_cache, v_cache, k_scale, v_scale, device)
    tq, hq, _ = q.shape
    batch = cu_seqlens_q.numel() - 1
    _tensor(q, torch.bfloat16, (tq, hq, d), device, "q")
    _tensor(cu_seqlens_q, torch.int32, (batch + 1,), device, "cu_seqlens_q")
    max_pages = block_table.shape[-1]
    _tensor(block_table, torch.int32, (batch, max_pages), device, "block_table")
    _tensor(seqlens_k, torch.int32, (batch,), device, "seqlens_k")
    if sinks is not None:
        _tensor(sinks, torch.float32, (hq,), device, "sinks")
    max_seqlen_q, max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    window, num_splits = int(window), int(num_splits)
    mask = Mask(1 if causal else 0, window, float(d ** -0.5 if scale is None else scale))
    with _scope(device, stream):
        out, lse = _outputs(q, tq, hq, device, out, lse, return_lse)
        need = 0
        if workspace is None:
            need = lib.sinkattn_prefill_paged_fp8_block_workspace_size(
                batch, tq, max_seqlen_q, max_seqlen_k, hq, hkv, d, window, num_splits)
        workspace = _scratch(workspace, need, device)
        st = lib.sinkattn_prefill_paged_fp8_block(
            _at(q), _at(cu_seqlens_q), _at(k_cache), _at(v_cache), _at(k_scale),
            _at(v_scale), block, _at(block_table), _at(seqlens_k), pages, max_pages, page,
            batch, tq, max_seqlen_q, max_seqlen_k, hq, hkv, d, _at(sinks), mask, num_splits,
            _at(out), _at(lse), _at(workspace), 0 if workspace is None else workspace.numel(),
            _current(device))
    _check(st, "sinkattn_prefill_paged_fp8_block")
    return out, lse


# ---- speculative decoding over the paged bf16 cache ----------------------------
# Checks, devices and streams as for the block-scaled cache above.

def _bf16_cache(k_cache, v_cache, device):
    """Checks a paged bf16 cache; returns (num_pages, hkv, page_size, D)."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, hkv, page_size, D]")
    shape = k_cache.shape
    _tensor(k_cache, torch.bfloat16, shape, device, "k_cache")
    _tensor(v_cache, torch.bfloat16, shape, device, "v_cache")
    return shape


def _rope_inputs(q_shape, k_shape, positions, cos_sin, q_weight, k_weight, device):
    """Checks what the head norm's forward and backward share; returns (n, hq, hkv, D,
    max_positions, rope_dim)."""
    if len(q_shape) != 3 or len(k_shape) != 3:
        raise ValueError("q must be [total, hq, D] and k [total, hkv, D]")
    n, hq, d = q_shape
    hkv = k_shape[1]
    max_pos = rope = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_positions, rope_dim]")
        max_pos, rope = cos_sin.shape
        _tensor(cos_sin, torch.float32, (max_pos, rope), device, "cos_sin")
        if positions is None:
            raise ValueError("positions are needed with cos_sin")
    if positions is not None:
        _tensor(positions, torch.int32, (n,), device, "positions")
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _tensor(t, torch.float32, (d,), device, name)
    return n, hq, hkv, d, max_pos, rope


def sinkattn_qk_norm_rope(q, k, positions=None, cos_sin=None, *, q_weight=None, k_weight=None,
                          eps=1e-6, interleaved=False, v=None, slot_mapping=None, k_cache=None,
                          v_cache=None, q_out=None, k_out=None, stream=None):
    """RMS norm of each query and key head (weights float32 [D], None: no norm) and
    rotation by position (cos_sin float32 [max_positions, rope_dim], cosines then
    sines; None: no rotation). q [n, hq, D] and k [n, hkv, D] are bf16 with any token
    stride that is a multiple of 8.

    With k_cache / v_cache (bf16 [num_pages, hkv, page_size, D]), slot_mapping int64 [n]
    and v, the turned keys and the values are written to their slots too, and k_out is
    made only if given. Returns (q_out, k_out)."""
    lib = load()
    device = q.device
    n, hq, hkv, d, max_pos, rope = _rope_inputs(q.shape, k.shape, positions, cos_sin, q_weight,
                                                k_weight, device)
    qs = _token_rows(q, n, hq, d, device, "q")
    ks = _token_rows(k, n, hkv, d, device, "k")
    cache = (k_cache, v_cache, slot_mapping, v)
    pages = page = vs = 0
    if any(t is not None for t in cache):
        if any(t is None for t in cache):
            raise ValueError("k_cache, v_cache, slot_mapping and v go together")
        pages, heads, page, dim = _bf16_cache(k_cache, v_cache, device)
        if (heads, dim) != (hkv, d):
            raise ValueError("k_cache is for %d heads of %d elements, k has %d of %d"
                             % (heads, dim, hkv, d))
        _tensor(slot_mapping, torch.int64, (n,), device, "slot_mapping")
        vs = _token_rows(v, n, hkv, d, device, "v")
    with _scope(device, stream):
        if q_out is None:
            q_out = torch.empty((n, hq, d), dtype=torch.bfloat16, device=device)
        if k_out is None and k_cache is None:
            k_out = torch.empty((n, hkv, d), dtype=torch.bfloat16, device=device)
        _tensor(q_out, torch.bfloat16, (n, hq, d), device, "q_out")
        if k_out is not None:
            _tensor(k_out, torch.bfloat16, (n, hkv, d), device, "k_out")
        st = lib.sinkattn_qk_norm_rope(_at(q), _at(k), _at(v), qs, ks, vs, _at(positions), n, hq,
                                       hkv, d, _at(q_weight), _at(k_weight), eps, _at(cos_sin),
                                       max_pos, rope, 1 if interleaved else 0, _at(q_out),
                                       _at(k_out), _at(slot_mapping), _at(k_cache),
                                       _at(v_cache), pages, page, _current(device))
    _check(st, "sinkattn_qk_norm_rope")
    return q_out, k_out


def sinkattn_qk_norm_rope_backward_workspace_size(head_dim=64):
    return load().sinkattn_qk_norm_rope_backward_workspace_size(int(head_dim))


def sinkattn_qk_norm_rope_backward(dq_out, dk_out, q, k, positions=None, cos_sin=None, *,
                                   q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                                   dq=None, dk=None, dq_weight=None, dk_weight=None,
                                   workspace=None, stream=None):
    """Gradients of sinkattn_qk_norm_rope with respect to q, k and the weights, given the
    forward's inputs and the gradients of q_out and k_out. dq and dk may be slices of
    wider rows, as q and k. Returns (dq, dk, dq_weight, dk_weight); a weight gradient is
    None without the weight."""
    lib = load()
    device = dq_out.device
    n, hq, hkv, d, max_pos, rope = _rope_inputs(dq_out.shape, dk_out.shape, positions, cos_sin,
                                                q_weight, k_weight, device)
    _tensor(dq_out, torch.bfloat16, (n, hq, d), device, "dq_out")
    _tensor(dk_out, torch.bfloat16, (n, hkv, d), device, "dk_out")
    qs = ks = 0
    if q_weight is not None:
        qs = _token_rows(q, n, hq, d, device, "q")
    if k_weight is not None:
        ks = _token_rows(k, n, hkv, d, device, "k")
    with _scope(device, stream):
        if dq is None:
            dq = torch.empty((n, hq, d), dtype=torch.bfloat16, device=device)
        if dk is None:
            dk = torch.empty((n, hkv, d), dtype=torch.bfloat16, device=device)
        dqs = _token_rows(dq, n, hq, d, device, "dq")
        dks = _token_rows(dk, n, hkv, d, device, "dk")
        grads = []
        for weight, grad, name in ((q_weight, dq_weight, "dq_weight"),
                                   (k_weight, dk_weight, "dk_weight")):
            if weight is None:
                grad = None
            elif grad is None:
                grad = torch.empty_like(weight)
            else:
                _tensor(grad, torch.float32, (d,), device, name)
            grads.append(grad)
        dq_weight, dk_weight = grads
        need = 0
        if workspace is None and not (dq_weight is None and dk_weight is None):
            need = lib.sinkattn_qk_norm_rope_backward_workspace_size(d)
        workspace = _scratch(workspace, need, device)
        st = lib.sinkattn_qk_norm_rope_backward(
            _at(dq_out), _at(dk_out), _at(q) if qs else None, _at(k) if ks else None, qs, ks,
            _at(positions), n, hq, hkv, d, _at(q_weight), _at(k_weight), eps, _at(cos_sin),
            max_pos, rope, 1 if interleaved else 0, _at(dq), _at(dk), dqs, dks, _at(dq_weight),
            _at(dk_weight), _at(workspace), 0 if workspace is None else workspace.numel(),
            _current(device))
    _check(st, "sinkattn_qk_norm_rope_backward")
    return dq, dk, dq_weight, dk_weight


def sinkattn_decode_tree_workspace_size(batch, total_q, max_seqlen_q, max_seqlen_k, hq, hkv,
                                        head_dim=64, window=0, num_splits=0):
    return load().sinkattn_decode_tree_workspace_size(
        int(batch), int(total_q), int(max_seqlen_q), int(max_seqlen_k), hq, hkv, head_dim,
        int(window), int(num_splits))


def sinkattn_decode_tree(q, cu_seqlens_q, k_cache, v_cache, block_table, seqlens_k, max_seqlen_q,
                         max_seqlen_k, *, parents=None, sinks=None, window=0, scale=None,
                         num_splits=0, out=None, lse=None, return_lse=True, workspace=None,
                         stream=None):
    """Sink-attention of drafted tokens over a paged bf16 cache [num_pages, hkv, page_size,
    D] that holds their keys and values behind their sequences' contexts: each row of q
    [total_q, hq, D] sees its sequence's context, its ancestors and itself. parents int32
    [total_q]: the row in its sequence that each row follows, -1 for row 0 (None: chains).
    Returns (out, lse)."""
    lib = load()
    device = q.device
    pages, hkv, page, d = _bf16_cache(k_cache, v_cache, device)
    tq, hq, _ = q.shape
    batch = cu_seqlens_q.numel() - 1
    _tensor(q, torch.bfloat16, (tq, hq, d), device, "q")
    _tensor(cu_seqlens_q, torch.int32, (batch + 1,), device, "cu_seqlens_q")
    max_pages = block_table.shape[-1]
    _tensor(block_table, torch.int32, (batch, max_pages), device, "block_table")
    _tensor(seqlens_k, torch.int32, (batch,), device, "seqlens_k")
    if parents is not None:
        _tensor(parents, torch.int32, (tq,), device, "parents")
    if sinks is not None:
        _tensor(sinks, torch.float32, (hq,), device, "sinks")
    max_seqlen_q, max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    window, num_splits = int(window), int(num_splits)
    mask = Mask(1, window, float(d ** -0.5 if scale is None else scale))
    with _scope(device, stream):
        out, lse = _outputs(q, tq, hq, device, out, lse, return_lse)
        need = 0
        if workspace is None:
            need = lib.sinkattn_decode_tree_workspace_size(
                batch, tq, max_seqlen_q, max_seqlen_k, hq, hkv, d, window, num_splits)
        workspace = _scratch(workspace, need, device)
        st = lib.sinkattn_decode_tree(
            _at(q), _at(cu_seqlens_q), _at(parents), _at(k_cache), _at(v_cache),
            _at(block_table), _at(seqlens_k), pages, max_pages, page, batch, tq, max_seqlen_q,
            max_seqlen_k, hq, hkv, d, _at(sinks), mask, num_splits, _at(out), _at(lse),
            _at(workspace), 0 if workspace is None else workspace.numel(), _current(device))
    _check(st, "sinkattn_decode_tree")
    return out, lse


def sinkattn_verify_tree(target_probs, tokens, uniforms, cu_seqlens_q, max_seqlen_q, *,
                         draft_probs=None, parents=None, path=None, num_path=None,
                         next_tokens=None, stream=None):
    """The accepted path of each sequence's drafted tree and its next token, from the
    target's probabilities after each row (float32 [total_q, vocab]), the drafted tokens
    (int64 [total_q]) and given random numbers (float32 [total_q] in [0, 1); a sequence's
    first draws its next token). draft_probs: what each row's children were drawn from
    (None: drafts are certain); parents as for sinkattn_decode_tree. Returns (path int32
    [batch, max_seqlen_q], rows of the accepted path then -1; num_path int32 [batch];
    next_tokens int64 [batch])."""
    lib = load()
    device = target_probs.device
    if target_probs.dim() != 2:
        raise ValueError("target_probs must be [total_q, vocab]")
    tq, vocab = target_probs.shape
    batch, width = cu_seqlens_q.numel() - 1, int(max_seqlen_q)
    _tensor(target_probs, torch.float32, (tq, vocab), device, "target_probs")
    if draft_probs is not None:
        _tensor(draft_probs, torch.float32, (tq, vocab), device, "draft_probs")
    _tensor(tokens, torch.int64, (tq,), device, "tokens")
    _tensor(uniforms, torch.float32, (tq,), device, "uniforms")
    _tensor(cu_seqlens_q, torch.int32, (batch + 1,), device, "cu_seqlens_q")
    if parents is not None:
        _tensor(parents, torch.int32, (tq,), device, "parents")
    with _scope(device, stream):
        if path is None:
            path = torch.empty((batch, width), dtype=torch.int32, device=device)
        if num_path is None:
            num_path = torch.empty(batch, dtype=torch.int32, device=device)
        if next_tokens is None:
            next_tokens = torch.empty(batch, dtype=torch.int64, device=device)
        _tensor(path, torch.int32, (batch, width), device, "path")
        _tensor(num_path, torch.int32, (batch,), device, "num_path")
        _tensor(next_tokens, torch.int64, (batch,), device, "next_tokens")
        st = lib.sinkattn_verify_tree(_at(target_probs), _at(draft_probs), _at(tokens),
                                      _at(parents), _at(uniforms), _at(cu_seqlens_q), batch, tq,
                                      width, vocab, _at(path), _at(num_path), _at(next_tokens),
                                      _current(device))
    _check(st, "sinkattn_verify_tree")
    return path, num_path, next_tokens


def sinkattn_compact(k_cache, v_cache, block_table, seqlens_k, cu_seqlens_q, path, num_path,
                     free_pages, free_head, *, seqlens_out=None, free_head_out=None,
                     stream=None):
    """Keeps the rows of each sequence's path (int32 [batch, width], increasing; None: the
    first num_path rows) of the step's rows: moves their keys and values behind the
    context, in place, and gives the pages that are then empty back to free_pages, in
    place, in front of entry free_head. num_path < 0 ends a sequence. Returns (seqlens_out
    int32 [batch], free_head_out int32 [1]), which may be seqlens_k and free_head."""
    lib = load()
    device = k_cache.device
    pages, hkv, page, d = _bf16_cache(k_cache, v_cache, device)
    batch = seqlens_k.numel()
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages]")
    max_pages, num_free, width = block_table.shape[1], free_pages.numel(), 0
    _tensor(block_table, torch.int32, (batch, max_pages), device, "block_table")
    _tensor(seqlens_k, torch.int32, (batch,), device, "seqlens_k")
    _tensor(cu_seqlens_q, torch.int32, (batch + 1,), device, "cu_seqlens_q")
    if path is not None:
        if path.dim() != 2:
            raise ValueError("path must be [batch, width]")
        width = path.shape[1]
        _tensor(path, torch.int32, (batch, width), device, "path")
    _tensor(num_path, torch.int32, (batch,), device, "num_path")
    _tensor(free_pages, torch.int32, (num_free,), device, "free_pages")
    _tensor(free_head, torch.int32, (1,), device, "free_head")
    with _scope(device, stream):
        if seqlens_out is None:
            seqlens_out = torch.empty_like(seqlens_k)
        if free_head_out is None:
            free_head_out = torch.empty_like(free_head)
        _tensor(seqlens_out, torch.int32, (batch,), device, "seqlens_out")
        _tensor(free_head_out, torch.int32, (1,), device, "free_head_out")
        st = lib.sinkattn_compact(_at(k_cache), _at(v_cache), _at(block_table), _at(seqlens_k),
                                  _at(cu_seqlens_q), _at(path), _at(num_path), width, batch,
                                  pages, max_pages, page, hkv, d, _at(seqlens_out),
                                  _at(free_pages), num_free, _at(free_head),
                                  _at(free_head_out), _current(device))
    _check(st, "sinkattn_compact")
    return seqlens_out, free_head_out


def sinkattn_merge(partial_o, partial_lse, *, sinks=None, out=None, lse=None, return_lse=True,
                   stream=None):
    """Merge split-KV partials [S, rows, hq, D] / [S, rows, hq] by log-sum-exp (D 64 or 128)."""
    lib = load()
    _req(partial_o, torch.float32, "partial_o")
    _req(partial_lse, torch.float32, "partial_lse")
    ns, rows, hq, d = partial_o.shape
    if out is None:
        out = torch.empty((rows, hq, d), dtype=torch.bfloat16, device=partial_o.device)
    if lse is None and return_lse:
        lse = torch.empty((rows, hq), dtype=torch.float32, device=partial_o.device)
    if sinks is not None:
        _req(sinks, torch.float32, "sinks")
    st = lib.sinkattn_merge(_ptr(partial_o), _ptr(partial_lse), ns, rows, hq, d, _ptr(sinks),
                            _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "sinkattn_merge")
    return out, lse


def sinkattn_get_device_error(stream=None) -> int:
    """Synchronise, read and clear the device error word (0 = no error)."""
    code = ctypes.c_int(0)
    _check(load().sinkattn_get_device_error(_stream(stream), ctypes.byref(code)),
           "sinkattn_get_device_error")
    return code.value


def sinkattn_debug_stall_waits(limit_ns: int) -> None:
    """Testing hook: later prefill / backward / block-scaled decode / tree attention
    calls make one wait of at most limit_ns on a barrier nothing completes, so every CTA (every
    warp of the decode) takes its timeout path (0 turns it off)."""
    _check(load().sinkattn_debug_stall_waits(int(limit_ns)), "sinkattn_debug_stall_waits")
