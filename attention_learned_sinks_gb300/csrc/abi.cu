// C ABI of libsinkattn.so (declared in include/sinkattn.h): argument
// validation, split planning and dispatch to the kernels. No device memory is
// allocated and no stream is synchronised here (except by
// sinkattn_get_device_error, which exists to read a device word back).
#include <math.h>
#include <stdint.h>

#include "../../include/sinkattn.h"
#include "launch.h"

using namespace sinkattn;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool mask_ok(const sinkattn_mask_t &m) {
  return m.window >= 0 && isfinite(m.scale) && m.scale > 0.f;
}

// A scale block of a paged cache lies within one page.
bool scale_block_ok(int scale_block, int page_size) {
  return page_size > 0 && scale_block > 0 && page_size % scale_block == 0;
}

// The CUDA error behind the calling thread's last SINKATTN_ERR_CUDA.
thread_local cudaError_t t_last_cuda_error = cudaSuccess;

sinkattn_status_t from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return SINKATTN_OK;
  t_last_cuda_error = e;
  return SINKATTN_ERR_CUDA;
}

}  // namespace

namespace sinkattn {
int cuda_status(cudaError_t e) { return from_cuda(e); }
}  // namespace sinkattn

extern "C" {

const char *sinkattn_last_cuda_error(void) {
  return t_last_cuda_error == cudaSuccess ? "no CUDA error" : cudaGetErrorName(t_last_cuda_error);
}

const char *sinkattn_status_string(sinkattn_status_t s) {
  switch (s) {
    case SINKATTN_OK:
      return "ok";
    case SINKATTN_ERR_INVALID_ARGUMENT:
      return "invalid argument";
    case SINKATTN_ERR_UNSUPPORTED:
      return "unsupported configuration";
    case SINKATTN_ERR_WORKSPACE_TOO_SMALL:
      return "workspace too small";
    case SINKATTN_ERR_CUDA:
      return "CUDA error";
  }
  return "unknown status";
}

size_t sinkattn_prefill_workspace_size(int batch, int64_t total_q, int64_t total_k,
                                       int max_seqlen_q, int max_seqlen_k, int hq, int hkv,
                                       int head_dim, int window, int num_splits) {
  if (batch < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 ||
      hq <= 0 || hkv <= 0 || hq % hkv != 0 || !prefill_head_dim_ok(head_dim) || window < 0 ||
      num_splits < 0)
    return 0;
  const int splits = prefill_plan_splits(num_splits, batch, total_q, max_seqlen_q, max_seqlen_k,
                                         hq, hkv, window, head_dim);
  return prefill_workspace_bytes(batch, total_q, total_k, hq, hkv, splits, head_dim);
}

sinkattn_status_t sinkattn_prefill(const void *q, const void *k, const void *v,
                                   const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                   int batch, int64_t total_q, int64_t total_k, int max_seqlen_q,
                                   int max_seqlen_k, int hq, int hkv, int head_dim,
                                   const float *sinks, sinkattn_mask_t mask, int num_splits,
                                   void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  if (batch < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || hq <= 0 ||
      hkv <= 0 || hq % hkv != 0 || num_splits < 0 || !mask_ok(mask))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!prefill_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return SINKATTN_OK;
  if (!q || !k || !v || !cu_seqlens_q || !cu_seqlens_k || !out)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) || (sinks && !aligned(sinks, 4)) ||
      (lse && !aligned(lse, 4)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch > 65535 || hq > 65535 || total_q > INT32_MAX || total_k > INT32_MAX ||
      (max_seqlen_q + 127) / 128 > 65535)
    return SINKATTN_ERR_UNSUPPORTED;
  const int splits = prefill_plan_splits(num_splits, batch, total_q, max_seqlen_q, max_seqlen_k,
                                         hq, hkv, mask.window, head_dim);
  if (splits > 1 && static_cast<int64_t>(splits) * total_q * hq > INT32_MAX)
    return SINKATTN_ERR_UNSUPPORTED;
  const size_t need = prefill_workspace_bytes(batch, total_q, total_k, hq, hkv, splits, head_dim);
  if (workspace == nullptr || workspace_bytes < need) return SINKATTN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return SINKATTN_ERR_INVALID_ARGUMENT;
  PrefillLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.batch = batch;
  a.total_q = total_q;
  a.total_k = total_k;
  a.max_seqlen_q = max_seqlen_q;
  a.max_seqlen_k = max_seqlen_k;
  a.hq = hq;
  a.hkv = hkv;
  a.sinks = sinks;
  a.causal = mask.causal != 0;
  a.window = mask.window;
  a.scale = mask.scale;
  a.out = out;
  a.lse = lse;
  a.num_splits = splits;
  a.head_dim = head_dim;
  a.v_f16 = workspace;
  bool encode_failed = false;
  cudaError_t e = launch_prefill(a, static_cast<cudaStream_t>(stream), &encode_failed);
  if (encode_failed) return SINKATTN_ERR_CUDA;
  return from_cuda(e);
}

size_t sinkattn_prefill_paged_workspace_size(int batch, int64_t total_q, int max_seqlen_q,
                                             int max_seqlen_k, int hq, int hkv, int head_dim,
                                             int window, int num_splits) {
  if (batch < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || hq <= 0 || hkv <= 0 ||
      hq % hkv != 0 || !prefill_head_dim_ok(head_dim) || window < 0 || num_splits < 0)
    return 0;
  const int splits = prefill_plan_splits(num_splits, batch, total_q, max_seqlen_q, max_seqlen_k,
                                         hq, hkv, window, head_dim);
  return prefill_paged_workspace_bytes(batch, total_q, max_seqlen_k, hq, hkv, splits, head_dim);
}

}  // extern "C"

namespace {

sinkattn_status_t prefill_paged_impl(const void *q, const int32_t *cu_seqlens_q,
                                     const void *k_cache, const void *v_cache, bool fp8,
                                     const float *k_scale, const float *v_scale,
                                     int scale_block, const int32_t *block_table,
                                     const int32_t *seqlens_k, int num_pages,
                                     int max_pages_per_seq, int page_size, int batch,
                                     int64_t total_q, int max_seqlen_q, int max_seqlen_k, int hq,
                                     int hkv, int head_dim, const float *sinks,
                                     sinkattn_mask_t mask, int num_splits, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, void *stream) {
  if (batch < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || hq <= 0 || hkv <= 0 ||
      hq % hkv != 0 || num_pages < 0 || max_pages_per_seq < 0 || page_size <= 0 ||
      num_splits < 0 || !mask_ok(mask))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!prefill_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_seqlen_k) > static_cast<int64_t>(max_pages_per_seq) * page_size)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return SINKATTN_OK;
  if (!q || !cu_seqlens_q || !seqlens_k || !out) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (max_seqlen_k > 0 && (!k_cache || !v_cache || !block_table || num_pages == 0))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (scale_block > 0 && max_seqlen_k > 0 && (!k_scale || !v_scale))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(cu_seqlens_q, 4) || !aligned(block_table, 4) || !aligned(seqlens_k, 4) ||
      (sinks && !aligned(sinks, 4)) || (lse && !aligned(lse, 4)) ||
      (k_scale && !aligned(k_scale, 4)) || (v_scale && !aligned(v_scale, 4)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch > 65535 || hq > 65535 || total_q > INT32_MAX || (max_seqlen_q + 127) / 128 > 65535 ||
      static_cast<int64_t>(batch) * max_seqlen_k + 128 > INT32_MAX)
    return SINKATTN_ERR_UNSUPPORTED;
  const auto plan = scale_block > 0 ? prefill_block_plan_splits : prefill_plan_splits;
  const int splits = plan(num_splits, batch, total_q, max_seqlen_q, max_seqlen_k, hq, hkv,
                          mask.window, head_dim);
  if (splits > 1 && static_cast<int64_t>(splits) * total_q * hq > INT32_MAX)
    return SINKATTN_ERR_UNSUPPORTED;
  const auto bytes =
      scale_block > 0 ? prefill_block_workspace_bytes : prefill_paged_workspace_bytes;
  const size_t need = bytes(batch, total_q, max_seqlen_k, hq, hkv, splits, head_dim);
  if (workspace == nullptr || workspace_bytes < need) return SINKATTN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return SINKATTN_ERR_INVALID_ARGUMENT;
  PrefillPagedLaunch a;
  a.base.q = q;
  a.base.k = nullptr;
  a.base.v = nullptr;
  a.base.cu_q = cu_seqlens_q;
  a.base.cu_k = nullptr;
  a.base.batch = batch;
  a.base.total_q = total_q;
  a.base.total_k = 0;
  a.base.max_seqlen_q = max_seqlen_q;
  a.base.max_seqlen_k = max_seqlen_k;
  a.base.hq = hq;
  a.base.hkv = hkv;
  a.base.sinks = sinks;
  a.base.causal = mask.causal != 0;
  a.base.window = mask.window;
  a.base.scale = mask.scale;
  a.base.out = out;
  a.base.lse = lse;
  a.base.num_splits = splits;
  a.base.head_dim = head_dim;
  if (scale_block > 0) {
    // a window of at least every length hides nothing
    if (mask.window >= max_seqlen_k) a.base.window = 0;
    a.scale_block = scale_block;
    a.k_block_scale = k_scale;
    a.v_block_scale = v_scale;
  } else {
    a.base.k_scale = k_scale;
    a.base.v_scale = v_scale;
  }
  a.base.v_f16 = nullptr;
  a.fp8 = fp8;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.seqlens_k = seqlens_k;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.workspace = workspace;
  bool encode_failed = false;
  cudaError_t e = launch_prefill_paged(a, static_cast<cudaStream_t>(stream), &encode_failed);
  if (encode_failed) return SINKATTN_ERR_CUDA;
  return from_cuda(e);
}

}  // namespace

extern "C" {

sinkattn_status_t sinkattn_prefill_paged(const void *q, const int32_t *cu_seqlens_q,
                                         const void *k_cache, const void *v_cache,
                                         const int32_t *block_table, const int32_t *seqlens_k,
                                         int num_pages, int max_pages_per_seq, int page_size,
                                         int batch, int64_t total_q, int max_seqlen_q,
                                         int max_seqlen_k, int hq, int hkv, int head_dim,
                                         const float *sinks, sinkattn_mask_t mask,
                                         int num_splits, void *out, float *lse, void *workspace,
                                         size_t workspace_bytes, void *stream) {
  return prefill_paged_impl(q, cu_seqlens_q, k_cache, v_cache, false, nullptr, nullptr, 0,
                            block_table, seqlens_k, num_pages, max_pages_per_seq, page_size,
                            batch, total_q, max_seqlen_q, max_seqlen_k, hq, hkv, head_dim, sinks,
                            mask, num_splits, out, lse, workspace, workspace_bytes, stream);
}

sinkattn_status_t sinkattn_prefill_paged_fp8(
    const void *q, const int32_t *cu_seqlens_q, const void *k_cache, const void *v_cache,
    const float *k_scale, const float *v_scale, const int32_t *block_table,
    const int32_t *seqlens_k, int num_pages, int max_pages_per_seq, int page_size, int batch,
    int64_t total_q, int max_seqlen_q, int max_seqlen_k, int hq, int hkv, int head_dim,
    const float *sinks, sinkattn_mask_t mask, int num_splits, void *out, float *lse,
    void *workspace, size_t workspace_bytes, void *stream) {
  return prefill_paged_impl(q, cu_seqlens_q, k_cache, v_cache, true, k_scale, v_scale, 0,
                            block_table, seqlens_k, num_pages, max_pages_per_seq, page_size,
                            batch, total_q, max_seqlen_q, max_seqlen_k, hq, hkv, head_dim, sinks,
                            mask, num_splits, out, lse, workspace, workspace_bytes, stream);
}

size_t sinkattn_prefill_paged_fp8_block_workspace_size(int batch, int64_t total_q,
                                                       int max_seqlen_q, int max_seqlen_k, int hq,
                                                       int hkv, int head_dim, int window,
                                                       int num_splits) {
  if (batch < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || hq <= 0 || hkv <= 0 ||
      hq % hkv != 0 || !prefill_head_dim_ok(head_dim) || window < 0 || num_splits < 0)
    return 0;
  const int splits = prefill_block_plan_splits(num_splits, batch, total_q, max_seqlen_q,
                                               max_seqlen_k, hq, hkv, window, head_dim);
  return prefill_block_workspace_bytes(batch, total_q, max_seqlen_k, hq, hkv, splits, head_dim);
}

sinkattn_status_t sinkattn_prefill_paged_fp8_block(
    const void *q, const int32_t *cu_seqlens_q, const void *k_cache, const void *v_cache,
    const float *k_scale, const float *v_scale, int scale_block, const int32_t *block_table,
    const int32_t *seqlens_k, int num_pages, int max_pages_per_seq, int page_size, int batch,
    int64_t total_q, int max_seqlen_q, int max_seqlen_k, int hq, int hkv, int head_dim,
    const float *sinks, sinkattn_mask_t mask, int num_splits, void *out, float *lse,
    void *workspace, size_t workspace_bytes, void *stream) {
  if (!scale_block_ok(scale_block, page_size)) return SINKATTN_ERR_INVALID_ARGUMENT;
  return prefill_paged_impl(q, cu_seqlens_q, k_cache, v_cache, true, k_scale, v_scale, scale_block,
                            block_table, seqlens_k, num_pages, max_pages_per_seq, page_size,
                            batch, total_q, max_seqlen_q, max_seqlen_k, hq, hkv, head_dim, sinks,
                            mask, num_splits, out, lse, workspace, workspace_bytes, stream);
}

size_t sinkattn_decode_workspace_size(int batch, int max_seqlen_k, int hq, int hkv, int head_dim,
                                      int window, int num_splits) {
  if (batch <= 0 || hq <= 0 || hkv <= 0 || !decode_head_dim_ok(head_dim) || max_seqlen_k < 0 ||
      window < 0 || num_splits < 0)
    return 0;
  const DecodePlan plan = plan_decode(batch, hq, hkv, max_seqlen_k, window, num_splits);
  return decode_workspace_layout(batch, hq, hkv, plan, head_dim).bytes;
}

}  // extern "C"

namespace {

sinkattn_status_t decode_impl(const void *q, const void *k_cache, const void *v_cache, bool fp8,
                              const float *k_scale, const float *v_scale,
                              const int32_t *kv_indptr, const int32_t *block_table,
                              const int32_t *seqlens_k, int64_t kv_rows, int max_pages_per_seq,
                              int page_size, int batch, int max_seqlen_k, int hq, int hkv,
                              int head_dim, const float *sinks, sinkattn_mask_t mask,
                              int num_splits, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream) {
  if (batch < 0 || max_seqlen_k < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0 || num_splits < 0 ||
      kv_rows < 0 || !mask_ok(mask))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!decode_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  const bool paged = block_table != nullptr;
  if (paged == (kv_indptr != nullptr)) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (paged && (seqlens_k == nullptr || page_size <= 0 || max_pages_per_seq <= 0))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!paged && seqlens_k != nullptr) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch == 0) return SINKATTN_OK;
  if (!q || !k_cache || !v_cache || !out) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      (kv_indptr && !aligned(kv_indptr, 4)) || (block_table && !aligned(block_table, 4)) ||
      (seqlens_k && !aligned(seqlens_k, 4)) || (sinks && !aligned(sinks, 4)) ||
      (lse && !aligned(lse, 4)) || (k_scale && !aligned(k_scale, 4)) ||
      (v_scale && !aligned(v_scale, 4)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch > 65535 || static_cast<int64_t>(hkv) * decode_head_tiles(hq, hkv) > 65535)
    return SINKATTN_ERR_UNSUPPORTED;
  const DecodePlan plan = plan_decode(batch, hq, hkv, max_seqlen_k, mask.window, num_splits);
  if (plan.max_splits > 1) {
    const size_t need = decode_workspace_layout(batch, hq, hkv, plan, head_dim).bytes;
    if (workspace == nullptr || workspace_bytes < need) return SINKATTN_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 256)) return SINKATTN_ERR_INVALID_ARGUMENT;
  }
  DecodeLaunch a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.kv_indptr = kv_indptr;
  a.block_table = block_table;
  a.seqlens_k = seqlens_k;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.batch = batch;
  a.max_seqlen_k = max_seqlen_k;
  a.hq = hq;
  a.hkv = hkv;
  a.window = mask.window;
  a.sinks = sinks;
  a.scale = mask.scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.plan = plan;
  a.fp8 = fp8;
  a.head_dim = head_dim;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return from_cuda(launch_decode(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

sinkattn_status_t sinkattn_decode(const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *kv_indptr, const int32_t *block_table,
                                  const int32_t *seqlens_k, int64_t kv_rows, int max_pages_per_seq,
                                  int page_size, int batch, int max_seqlen_k, int hq, int hkv,
                                  int head_dim, const float *sinks, sinkattn_mask_t mask,
                                  int num_splits, void *out, float *lse, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  return decode_impl(q, k_cache, v_cache, false, nullptr, nullptr, kv_indptr, block_table,
                     seqlens_k, kv_rows, max_pages_per_seq, page_size, batch, max_seqlen_k, hq,
                     hkv, head_dim, sinks, mask, num_splits, out, lse, workspace,
                     workspace_bytes, stream);
}

sinkattn_status_t sinkattn_decode_fp8(const void *q, const void *k_cache, const void *v_cache,
                                      const float *k_scale, const float *v_scale,
                                      const int32_t *kv_indptr, const int32_t *block_table,
                                      const int32_t *seqlens_k, int64_t kv_rows,
                                      int max_pages_per_seq, int page_size, int batch,
                                      int max_seqlen_k, int hq, int hkv, int head_dim,
                                      const float *sinks, sinkattn_mask_t mask, int num_splits,
                                      void *out, float *lse, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  return decode_impl(q, k_cache, v_cache, true, k_scale, v_scale, kv_indptr, block_table,
                     seqlens_k, kv_rows, max_pages_per_seq, page_size, batch, max_seqlen_k, hq,
                     hkv, head_dim, sinks, mask, num_splits, out, lse, workspace,
                     workspace_bytes, stream);
}

size_t sinkattn_decode_fp8_block_workspace_size(int batch, int max_seqlen_k, int hq, int hkv,
                                                int head_dim, int window, int num_splits) {
  if (batch <= 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0 || !decode_head_dim_ok(head_dim) ||
      max_seqlen_k < 0 || window < 0 || num_splits < 0)
    return 0;
  return decode_block_workspace_bytes(
      plan_decode_block(batch, hq, hkv, head_dim, max_seqlen_k, window, num_splits), head_dim);
}

sinkattn_status_t sinkattn_decode_fp8_block(
    const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
    const float *v_scale, int scale_block, const int32_t *block_table, const int32_t *seqlens_k,
    int num_pages, int max_pages_per_seq, int page_size, int batch, int max_seqlen_k, int hq,
    int hkv, int head_dim, const float *sinks, sinkattn_mask_t mask, int num_splits, void *out,
    float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  if (batch < 0 || max_seqlen_k < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0 || num_splits < 0 ||
      num_pages < 0 || max_pages_per_seq < 0 || !mask_ok(mask) ||
      !scale_block_ok(scale_block, page_size))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!decode_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_seqlen_k) > static_cast<int64_t>(max_pages_per_seq) * page_size)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch == 0) return SINKATTN_OK;
  if (!q || !seqlens_k || !out) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (max_pages_per_seq > 0 &&
      (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || num_pages == 0))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
      !aligned(seqlens_k, 4) || (sinks && !aligned(sinks, 4)) || (lse && !aligned(lse, 4)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  const int64_t heads = static_cast<int64_t>(hkv) * decode_head_tiles(hq, hkv);
  if (batch > 65535 || heads > 65535 || batch * heads > INT32_MAX) return SINKATTN_ERR_UNSUPPORTED;
  const DecodeBlockPlan plan =
      plan_decode_block(batch, hq, hkv, head_dim, max_seqlen_k, mask.window, num_splits);
  const size_t need = decode_block_workspace_bytes(plan, head_dim);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return SINKATTN_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 256)) return SINKATTN_ERR_INVALID_ARGUMENT;
  }
  DecodeBlockLaunch a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.seqlens_k = seqlens_k;
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.scale_block = scale_block;
  a.batch = batch;
  a.hq = hq;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.window = mask.window;
  a.sinks = sinks;
  a.scale = mask.scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.plan = plan;
  return from_cuda(launch_decode_block(a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status_t sinkattn_page_map(const int32_t *seqlens_k, const int32_t *cu_seqlens_q,
                                    int batch, int64_t total_q, int page_size,
                                    int max_pages_per_seq, const int32_t *free_pages, int num_free,
                                    const int32_t *free_head, int32_t *free_head_out,
                                    int32_t *block_table, int64_t *slot_mapping,
                                    int32_t *page_offsets, void *stream) {
  if (batch < 0 || total_q < 0 || page_size <= 0 || max_pages_per_seq < 0 || num_free < 0)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (cu_seqlens_q == nullptr && total_q != batch) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!free_head || !free_head_out || !page_offsets) return SINKATTN_ERR_INVALID_ARGUMENT;
  if ((batch > 0 && !seqlens_k) || (total_q > 0 && !slot_mapping) ||
      (batch > 0 && max_pages_per_seq > 0 && !block_table) || (num_free > 0 && !free_pages) ||
      (batch == 0 && total_q > 0 && !cu_seqlens_q))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(seqlens_k, 4) || !aligned(cu_seqlens_q, 4) || !aligned(free_pages, 4) ||
      !aligned(free_head, 4) || !aligned(free_head_out, 4) || !aligned(block_table, 4) ||
      !aligned(slot_mapping, 8) || !aligned(page_offsets, 4))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  // page_offsets holds free-list positions up to num_free + one page per new token
  if (total_q + num_free > INT32_MAX) return SINKATTN_ERR_UNSUPPORTED;
  PageMapLaunch a;
  a.seqlens_k = seqlens_k;
  a.cu_q = cu_seqlens_q;
  a.batch = batch;
  a.total_q = total_q;
  a.page_size = page_size;
  a.max_pages = max_pages_per_seq;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.free_head = free_head;
  a.free_head_out = free_head_out;
  a.block_table = block_table;
  a.page_offsets = page_offsets;
  a.slots = slot_mapping;
  return from_cuda(launch_page_map(a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status_t sinkattn_append_fp8_block(const void *k, const void *v, int64_t k_stride,
                                            int64_t v_stride, const int64_t *slot_mapping,
                                            int64_t total, void *k_cache, void *v_cache,
                                            float *k_scale, float *v_scale, int scale_block,
                                            int num_pages, int page_size, int hkv, int head_dim,
                                            void *stream) {
  if (total < 0 || num_pages < 0 || hkv <= 0 || !scale_block_ok(scale_block, page_size))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!decode_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(hkv) * head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (total == 0) return SINKATTN_OK;
  if (!k || !v || !slot_mapping) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (num_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_mapping, 8) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (hkv > 65535 || total > INT32_MAX) return SINKATTN_ERR_UNSUPPORTED;
  AppendLaunch a;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slot_mapping;
  a.total = total;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.scale_block = scale_block;
  a.hkv = hkv;
  a.head_dim = head_dim;
  return from_cuda(launch_append(a, static_cast<cudaStream_t>(stream)));
}

// Token rows of `width` elements that stand `stride` apart.
static bool rows_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; }

// What the forward and the backward call of the head norm share.
static sinkattn_status_t rope_check(const int32_t *positions, int64_t total, int hq, int hkv,
                                    int head_dim, const float *q_weight, const float *k_weight,
                                    float eps, const float *cos_sin, int max_positions,
                                    int rope_dim) {
  if (total < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!decode_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if ((q_weight || k_weight) && !(isfinite(eps) && eps > 0.f)) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (cos_sin) {
    if (max_positions <= 0 || rope_dim <= 0 || rope_dim > head_dim)
      return SINKATTN_ERR_INVALID_ARGUMENT;
    if (rope_dim % 16 != 0) return SINKATTN_ERR_UNSUPPORTED;
    if (total > 0 && !positions) return SINKATTN_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(cos_sin, 16) ||
      !aligned(positions, 4))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (hq > 65535 || total > INT32_MAX) return SINKATTN_ERR_UNSUPPORTED;
  return SINKATTN_OK;
}

sinkattn_status_t sinkattn_qk_norm_rope(
    const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, const int32_t *positions, int64_t total, int hq, int hkv, int head_dim,
    const float *q_weight, const float *k_weight, float eps, const float *cos_sin,
    int max_positions, int rope_dim, int interleaved, void *q_out, void *k_out,
    const int64_t *slot_mapping, void *k_cache, void *v_cache, int num_pages, int page_size,
    void *stream) {
  const sinkattn_status_t st = rope_check(positions, total, hq, hkv, head_dim, q_weight, k_weight,
                                          eps, cos_sin, max_positions, rope_dim);
  if (st != SINKATTN_OK) return st;
  const int64_t row = static_cast<int64_t>(hkv) * head_dim;
  const bool cache = k_cache || v_cache || slot_mapping;
  if (!rows_ok(q_stride, static_cast<int64_t>(hq) * head_dim) || !rows_ok(k_stride, row) ||
      (cache && (!rows_ok(v_stride, row) || num_pages < 0 || page_size <= 0)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (total == 0) return SINKATTN_OK;
  if (!q || !k || !q_out || (!cache && !k_out)) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (cache && (!v || !slot_mapping || !k_cache || !v_cache)) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(k_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 8))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  RopeLaunch a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.positions = positions;
  a.total = total;
  a.hq = hq;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_positions = max_positions;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved != 0;
  a.q_out = q_out;
  a.k_out = k_out;
  a.slots = slot_mapping;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_pages = num_pages;
  a.page_size = page_size;
  return from_cuda(launch_rope(a, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_qk_norm_rope_backward_workspace_size(int head_dim) {
  return decode_head_dim_ok(head_dim) ? rope_backward_workspace_bytes(head_dim) : 0;
}

sinkattn_status_t sinkattn_qk_norm_rope_backward(
    const void *dq_out, const void *dk_out, const void *q, const void *k, int64_t q_stride,
    int64_t k_stride, const int32_t *positions, int64_t total, int hq, int hkv, int head_dim,
    const float *q_weight, const float *k_weight, float eps, const float *cos_sin,
    int max_positions, int rope_dim, int interleaved, void *dq, void *dk, int64_t dq_stride,
    int64_t dk_stride, float *dq_weight, float *dk_weight, void *workspace,
    size_t workspace_bytes, void *stream) {
  const sinkattn_status_t st = rope_check(positions, total, hq, hkv, head_dim, q_weight, k_weight,
                                          eps, cos_sin, max_positions, rope_dim);
  if (st != SINKATTN_OK) return st;
  const int64_t qrow = static_cast<int64_t>(hq) * head_dim;
  const int64_t krow = static_cast<int64_t>(hkv) * head_dim;
  if ((q_weight && !rows_ok(q_stride, qrow)) || (k_weight && !rows_ok(k_stride, krow)) ||
      !rows_ok(dq_stride, qrow) || !rows_ok(dk_stride, krow))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (total > 0 && (!dq_out || !dk_out || !dq || !dk || (q_weight && !q) || (k_weight && !k)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(q, 16) || !aligned(k, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!q_weight) dq_weight = nullptr;
  if (!k_weight) dk_weight = nullptr;
  if (dq_weight || dk_weight) {
    if (!workspace || workspace_bytes < rope_backward_workspace_bytes(head_dim))
      return SINKATTN_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 256)) return SINKATTN_ERR_INVALID_ARGUMENT;
  }
  RopeLaunch a{};
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.positions = positions;
  a.total = total;
  a.hq = hq;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_positions = max_positions;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved != 0;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.dq = dq;
  a.dk = dk;
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.dq_weight = dq_weight;
  a.dk_weight = dk_weight;
  a.workspace = workspace;
  return from_cuda(launch_rope_backward(a, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_decode_tree_workspace_size(int batch, int64_t total_q, int max_seqlen_q,
                                           int max_seqlen_k, int hq, int hkv, int head_dim,
                                           int window, int num_splits) {
  if (batch <= 0 || total_q <= 0 || max_seqlen_q <= 0 || max_seqlen_k < 0 || hq <= 0 ||
      hkv <= 0 || hq % hkv != 0 || !decode_head_dim_ok(head_dim) || window < 0 || num_splits < 0)
    return 0;
  const DecodeTreePlan plan = plan_decode_tree(batch, max_seqlen_q, max_seqlen_k, hq, hkv,
                                               head_dim, window, num_splits);
  return decode_tree_workspace_bytes(plan, head_dim);
}

sinkattn_status_t sinkattn_decode_tree(
    const void *q, const int32_t *cu_seqlens_q, const int32_t *parents, const void *k_cache,
    const void *v_cache, const int32_t *block_table, const int32_t *seqlens_k, int num_pages,
    int max_pages_per_seq, int page_size, int batch, int64_t total_q, int max_seqlen_q,
    int max_seqlen_k, int hq, int hkv, int head_dim, const float *sinks, sinkattn_mask_t mask,
    int num_splits, void *out, float *lse, void *workspace, size_t workspace_bytes,
    void *stream) {
  if (batch < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || hq <= 0 || hkv <= 0 ||
      hq % hkv != 0 || num_splits < 0 || !mask_ok(mask) || page_size <= 0 ||
      max_pages_per_seq < 0 || num_pages < 0)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!decode_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_pages_per_seq) * page_size < max_seqlen_k)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return SINKATTN_OK;
  if (!q || !cu_seqlens_q || !seqlens_k || !out || (num_pages > 0 && (!k_cache || !v_cache)) ||
      (max_pages_per_seq > 0 && !block_table))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(cu_seqlens_q, 4) || !aligned(parents, 4) || !aligned(block_table, 4) ||
      !aligned(seqlens_k, 4) || !aligned(sinks, 4) || !aligned(lse, 4))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  // (row, query head) pairs and rows of the cache are counted in 32 bits
  if (batch > 65535 || hkv > 65535 || total_q * hq > INT32_MAX ||
      static_cast<int64_t>(max_seqlen_q) * (hq / hkv) > INT32_MAX / 2 ||
      static_cast<double>(num_pages) * hkv * page_size > 4e9 || max_seqlen_k > INT32_MAX - 128)
    return SINKATTN_ERR_UNSUPPORTED;
  const DecodeTreePlan plan = plan_decode_tree(batch, max_seqlen_q, max_seqlen_k, hq, hkv,
                                               head_dim, mask.window, num_splits);
  const size_t need = decode_tree_workspace_bytes(plan, head_dim);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return SINKATTN_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 256)) return SINKATTN_ERR_INVALID_ARGUMENT;
  }
  DecodeTreeLaunch a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.cu_q = cu_seqlens_q;
  a.parents = parents;
  a.block_table = block_table;
  a.seqlens_k = seqlens_k;
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.batch = batch;
  a.max_seqlen_q = max_seqlen_q;
  a.max_seqlen_k = max_seqlen_k;
  a.hq = hq;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.window = mask.window;
  a.sinks = sinks;
  a.scale = mask.scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.plan = plan;
  return from_cuda(launch_decode_tree(a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status_t sinkattn_verify_tree(const float *target_probs, const float *draft_probs,
                                       const int64_t *tokens, const int32_t *parents,
                                       const float *uniforms, const int32_t *cu_seqlens_q,
                                       int batch, int64_t total_q, int max_seqlen_q, int vocab,
                                       int32_t *path, int32_t *num_path, int64_t *next_tokens,
                                       void *stream) {
  if (batch < 0 || total_q < 0 || max_seqlen_q < 0 || vocab <= 0)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (max_seqlen_q > kVerifyMaxTokens || vocab > (1 << 30) || batch > (1 << 24))
    return SINKATTN_ERR_UNSUPPORTED;
  if (batch == 0) return SINKATTN_OK;
  if (!cu_seqlens_q || !num_path || !next_tokens || (max_seqlen_q > 0 && !path) ||
      (total_q > 0 && (!target_probs || !tokens || !uniforms)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(target_probs, 16) || !aligned(draft_probs, 16) || !aligned(tokens, 8) ||
      !aligned(parents, 4) || !aligned(uniforms, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(path, 4) || !aligned(num_path, 4) || !aligned(next_tokens, 8))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  VerifyLaunch a;
  a.target_probs = target_probs;
  a.draft_probs = draft_probs;
  a.tokens = tokens;
  a.parents = parents;
  a.cu_q = cu_seqlens_q;
  a.uniforms = uniforms;
  a.batch = batch;
  a.vocab = vocab;
  a.max_seqlen_q = max_seqlen_q;
  a.path = path;
  a.num_path = num_path;
  a.next_tokens = next_tokens;
  return from_cuda(launch_verify(a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status_t sinkattn_compact(void *k_cache, void *v_cache, const int32_t *block_table,
                                   const int32_t *seqlens_k, const int32_t *cu_seqlens_q,
                                   const int32_t *path, const int32_t *num_path, int path_width,
                                   int batch, int num_pages, int max_pages_per_seq,
                                   int page_size, int hkv, int head_dim, int32_t *seqlens_out,
                                   int32_t *free_pages, int num_free, const int32_t *free_head,
                                   int32_t *free_head_out, void *stream) {
  if (batch < 0 || num_pages < 0 || max_pages_per_seq < 0 || page_size <= 0 || hkv <= 0 ||
      num_free < 0 || path_width < 0)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!decode_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if (!free_head || !free_head_out || (num_free > 0 && !free_pages))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch > 0 && (!seqlens_k || !cu_seqlens_q || !num_path || !seqlens_out ||
                    (max_pages_per_seq > 0 && !block_table) ||
                    (num_pages > 0 && (!k_cache || !v_cache))))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_table, 4) ||
      !aligned(seqlens_k, 4) || !aligned(cu_seqlens_q, 4) || !aligned(path, 4) ||
      !aligned(num_path, 4) || !aligned(seqlens_out, 4) || !aligned(free_pages, 4) ||
      !aligned(free_head, 4) || !aligned(free_head_out, 4))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  // every page of every table may come back
  if (hkv > 65535 || static_cast<int64_t>(batch) * max_pages_per_seq > INT32_MAX)
    return SINKATTN_ERR_UNSUPPORTED;
  CompactLaunch a;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.seqlens_k = seqlens_k;
  a.cu_q = cu_seqlens_q;
  a.path = path;
  a.num_path = num_path;
  a.seqlens_out = seqlens_out;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.free_head_out = free_head_out;
  a.batch = batch;
  a.path_width = path_width;
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.hkv = hkv;
  a.head_dim = head_dim;
  a.num_free = num_free;
  return from_cuda(launch_compact(a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status_t sinkattn_merge(const float *partial_o, const float *partial_lse, int num_splits,
                                 int64_t rows, int hq, int head_dim, const float *sinks, void *out,
                                 float *lse, void *stream) {
  if (num_splits < 0 || rows < 0 || hq <= 0) return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!prefill_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if (rows == 0) return SINKATTN_OK;
  if (!out || (num_splits > 0 && (!partial_o || !partial_lse)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if ((partial_o && !aligned(partial_o, 16)) || (partial_lse && !aligned(partial_lse, 4)) ||
      !aligned(out, 16) || (sinks && !aligned(sinks, 4)) || (lse && !aligned(lse, 4)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if ((rows * hq + 7) / 8 > INT32_MAX) return SINKATTN_ERR_UNSUPPORTED;
  return from_cuda(launch_merge(partial_o, partial_lse, num_splits, rows, hq, head_dim, sinks, out,
                                lse, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_prefill_backward_workspace_size(int batch, int64_t total_q, int64_t total_k,
                                                int hq, int hkv, int head_dim) {
  if (batch < 0 || total_q < 0 || total_k < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0 ||
      !backward_head_dim_ok(head_dim))
    return 0;
  return backward_workspace_bytes(batch, total_q, total_k, hq, hkv, head_dim);
}

sinkattn_status_t sinkattn_prefill_backward(
    const void *q, const void *k, const void *v, const void *out, const void *dout,
    const float *lse, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int batch,
    int64_t total_q, int64_t total_k, int max_seqlen_q, int max_seqlen_k, int hq, int hkv,
    int head_dim, const float *sinks, sinkattn_mask_t mask, void *dq, void *dk, void *dv,
    float *dsinks, void *workspace, size_t workspace_bytes, void *stream) {
  if (batch < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || hq <= 0 ||
      hkv <= 0 || hq % hkv != 0 || !mask_ok(mask))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!backward_head_dim_ok(head_dim)) return SINKATTN_ERR_UNSUPPORTED;
  if (batch == 0 || (total_q == 0 && total_k == 0)) return SINKATTN_OK;
  if (!q || !k || !v || !out || !dout || !lse || !cu_seqlens_q || !cu_seqlens_k || !dq || !dk ||
      !dv)
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(lse, 4) || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) ||
      (sinks && !aligned(sinks, 4)) || (dsinks && !aligned(dsinks, 4)))
    return SINKATTN_ERR_INVALID_ARGUMENT;
  if (batch > 65535 || total_q > INT32_MAX || total_k > INT32_MAX ||
      (max_seqlen_q + 127) / 128 > 65535 || (max_seqlen_k + 127) / 128 > 65535 ||
      (total_q / 128 + batch) * hq * (head_dim / 64) > INT32_MAX ||
      (total_k / 128 + batch) * hkv * (head_dim / 64) > INT32_MAX)
    return SINKATTN_ERR_UNSUPPORTED;
  const size_t need = backward_workspace_bytes(batch, total_q, total_k, hq, hkv, head_dim);
  if (workspace == nullptr || workspace_bytes < need) return SINKATTN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return SINKATTN_ERR_INVALID_ARGUMENT;
  BackwardLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.dout = dout;
  a.lse = lse;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.batch = batch;
  a.total_q = total_q;
  a.total_k = total_k;
  a.max_seqlen_q = max_seqlen_q;
  a.max_seqlen_k = max_seqlen_k;
  a.hq = hq;
  a.hkv = hkv;
  a.sinks = sinks;
  a.causal = mask.causal != 0;
  a.window = mask.window;
  a.scale = mask.scale;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dsinks = dsinks;
  a.workspace = workspace;
  a.head_dim = head_dim;
  bool encode_failed = false;
  cudaError_t e = launch_backward(a, static_cast<cudaStream_t>(stream), &encode_failed);
  if (encode_failed) return SINKATTN_ERR_CUDA;
  return from_cuda(e);
}

sinkattn_status_t sinkattn_debug_stall_waits(uint64_t limit_ns) {
  cudaError_t e = prefill_set_stall(limit_ns);
  if (e == cudaSuccess) e = backward_set_stall(limit_ns);
  if (e == cudaSuccess) e = decode_block_set_stall(limit_ns);
  if (e == cudaSuccess) e = decode_tree_set_stall(limit_ns);
  return from_cuda(e);
}

sinkattn_status_t sinkattn_get_device_error(void *stream, int *code) {
  if (code == nullptr) return SINKATTN_ERR_INVALID_ARGUMENT;
  *code = 0;
  cudaError_t e = prefill_read_error(static_cast<cudaStream_t>(stream), code);
  // the first nonzero word is reported; every word is read and cleared
  const auto also = [&](cudaError_t (*read)(cudaStream_t, int *)) {
    int other = 0;
    if (e == cudaSuccess) e = read(static_cast<cudaStream_t>(stream), &other);
    if (*code == 0) *code = other;
  };
  also(backward_read_error);
  also(decode_block_read_error);
  also(cache_read_error);
  also(rope_read_error);
  also(decode_tree_read_error);
  also(verify_read_error);
  return from_cuda(e);
}

}  // extern "C"
