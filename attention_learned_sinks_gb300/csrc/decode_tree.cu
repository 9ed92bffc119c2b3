// Attention of a tree of drafted tokens over a paged bf16 cache.
//
// Row i of a sequence with Lk keys and Lq drafted tokens sees the C = Lk - Lq keys of
// its context (within the window) and, of the Lq keys behind it, those of its ancestors
// and its own; its position is C + depth(i). One warp per (row, query head): the keys one
// by one, the running maximum and denominator in registers.
#include <math.h>

#include "launch.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

__device__ int g_tree_error;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeParams {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *cu_q, *parents, *table, *seqlens_k;
  int num_pages, max_pages, page_size, batch;
  int64_t total_q;
  int max_q, max_k, hq, hkv, window;
  const float *sinks;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
};

template <int D>
__global__ void __launch_bounds__(128) tree_rows_kernel(const TreeParams p) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t row = idx / p.hq;
  const int h = static_cast<int>(idx % p.hq), g = h / (p.hq / p.hkv);
  if (row >= p.cu_q[p.batch] || row >= p.total_q) return;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid] <= row) lo = mid; else hi = mid;
  }
  const int b = lo, first = p.cu_q[b];
  const int i = static_cast<int>(row - first);
  if (i >= p.max_q) {
    if (lane == 0) atomicExch(&g_tree_error, kErrBadLength);
    return;
  }
  const int lq = min(p.cu_q[b + 1] - first, p.max_q);
  const int raw = p.seqlens_k[b];
  const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int lk = static_cast<int>(min(static_cast<int64_t>(min(max(raw, 0), p.max_k)), room));
  if (lk != raw && lane == 0) atomicExch(&g_tree_error, kErrBadLength);
  const int context = lk - lq;
  const auto up = [&](int a) -> int {
    if (p.parents == nullptr) return a - 1;
    const int x = p.parents[first + a];
    if (x >= a || x < -1) {
      if (lane == 0) atomicExch(&g_tree_error, kErrBadPage);
      return -1;
    }
    return x;
  };
  float qv[kPer], acc[kPer] = {};
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    qv[e] = __bfloat162float(p.q[(row * p.hq + h) * D + lane * kPer + e]) * p.scale_log2;
  float m = p.sinks != nullptr ? p.sinks[h] * kLog2e : -INFINITY;
  float d = p.sinks != nullptr ? 1.f : 0.f;
  const auto take = [&](int pos) {
    const int page = p.table[static_cast<int64_t>(b) * p.max_pages + pos / p.page_size];
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && lane == 0) atomicExch(&g_tree_error, kErrBadPage);
    const int64_t at = ((static_cast<int64_t>(ok ? page : 0) * p.hkv + g) * p.page_size +
                        pos % p.page_size) * D + lane * kPer;
    float s = 0.f, vv[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      s += ok ? qv[e] * __bfloat162float(p.k[at + e]) : 0.f;
      vv[e] = ok ? __bfloat162float(p.v[at + e]) : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float m_new = fmaxf(m, s);
    const float alpha = exp2f(m - m_new), w = exp2f(s - m_new);
    m = m_new;
    d = d * alpha + w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * alpha + w * vv[e];
  };
  int depth = 0;
  for (int a = up(i); a >= 0; a = up(a)) ++depth;
  const int64_t from = p.window > 0 ? static_cast<int64_t>(context) + depth - p.window + 1 : 0;
  for (int j = static_cast<int>(max(from, static_cast<int64_t>(0))); j < context; ++j) take(j);
  int left = p.window > 0 ? p.window : INT32_MAX;
  for (int a = i; a >= 0 && left > 0; a = up(a), --left)
    if (context + a >= 0) take(context + a);
  const float inv = d > 0.f ? 1.f / d : 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    p.out[(row * p.hq + h) * D + lane * kPer + e] = __float2bfloat16(acc[e] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[row * p.hq + h] = d > 0.f ? (m + log2f(d)) * kLn2 : -INFINITY;
}

}  // namespace

DecodeTreePlan plan_decode_tree(int, int, int max_seqlen_k, int, int, int, int, int) {
  return {max_seqlen_k, 1};
}
size_t decode_tree_workspace_bytes(const DecodeTreePlan &, int64_t, int, int) { return 0; }

cudaError_t launch_decode_tree(const DecodeTreeLaunch &a, cudaStream_t stream) {
  TreeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v);
  p.cu_q = a.cu_q, p.parents = a.parents, p.table = a.block_table, p.seqlens_k = a.seqlens_k;
  p.num_pages = a.num_pages, p.max_pages = a.max_pages, p.page_size = a.page_size;
  p.batch = a.batch, p.total_q = a.total_q, p.max_q = a.max_seqlen_q, p.max_k = a.max_seqlen_k;
  p.hq = a.hq, p.hkv = a.hkv, p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  const unsigned blocks = static_cast<unsigned>((a.total_q * a.hq + 3) / 4);
  if (a.head_dim == 128)
    tree_rows_kernel<128><<<blocks, 128, 0, stream>>>(p);
  else
    tree_rows_kernel<64><<<blocks, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t decode_tree_read_error(cudaStream_t stream, int *code) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_tree_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(int));
  return e;
}

}  // namespace sinkattn
