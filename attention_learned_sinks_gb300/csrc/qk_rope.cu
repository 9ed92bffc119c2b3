// RMS norm of each query and key head and the rotation by position in one pass,
// with the write of keys and values into a paged bf16 cache, and its gradients.
//
// For one head's row x of D elements, weights w and the angle table's row (cos, sin)
// of the token's position:
//
//   r = (mean(x^2) + eps)^(-1/2),   y = r w x,   z = R y
//
// where R turns each pair (a, b) of the first rope_dim elements into
// (a cos - b sin, b cos + a sin). Since r is one number per row, element e is
//
//   z_e = r (x_e A_e + x_{e'} B_e),  A_e = w_e cos,  B_e = -+ w_{e'} sin,
//
// e' its partner: A and B are the same for all heads of a token, so a warp takes a
// token, keeps them in registers and streams the token's rows past them, 16 bytes
// (8 elements) per lane. The partner's elements come from another lane (halves) or
// the same one (interleaved pairs) as packed bf16.
//
// Backward: dy = R^T dz, dw = sum over rows of u dy, g = w dy,
//   dx = r (g - u mean(g u)),  u = r x.
// The rows are read again instead of keeping r: 4 bytes per row would have to be
// written and read for a reduction that the row's own load feeds anyway.
//
// Bound by HBM: each row is read once and written once, no product is reused.
#include <float.h>
#include <math.h>

#include "launch.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

__device__ int g_rope_error;

constexpr int kWarps = 8;  // warps per block

struct RopeParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *positions;
  int64_t total;
  int hq, hkv;
  const float *wq, *wk;
  float eps;
  const float *table;
  int max_pos, rope_dim, interleaved;
  __nv_bfloat16 *q_out, *k_out;
  const int64_t *slots;
  __nv_bfloat16 *k_cache, *v_cache;
  int64_t num_slots;
  int page_size;
  int parts;  // warps per token
  // backward: incoming gradients in q_out's and k_out's layout
  const __nv_bfloat16 *dq_out, *dk_out;
  __nv_bfloat16 *dq, *dk;
  int64_t dq_stride, dk_stride;
  float *partial;  // [blocks][2][D]
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z), x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint4 shfl4(const uint4 &u, int lane) {
  return make_uint4(__shfl_sync(0xffffffffu, u.x, lane), __shfl_sync(0xffffffffu, u.y, lane),
                    __shfl_sync(0xffffffffu, u.z, lane), __shfl_sync(0xffffffffu, u.w, lane));
}
// The two halves of each packed pair change places.
__device__ __forceinline__ uint4 swap_pairs(const uint4 &u) {
  return make_uint4(__funnelshift_l(u.x, u.x, 16), __funnelshift_l(u.y, u.y, 16),
                    __funnelshift_l(u.z, u.z, 16), __funnelshift_l(u.w, u.w, 16));
}
// Sum over the kLanes lanes of a row (a power of two), in all of them.
template <int kLanes>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The squares of elements of 2^63 and above overflow: rows in which that happened are
// scaled by this power of two before they are summed, with eps scaled alike.
constexpr float kDown = 0x1p-70f;

// r of the row whose 8 elements x this lane holds; a row whose squares overflow has its
// elements scaled by *scale = kDown, so that r x stays what it is. Called by whole warps.
template <int D>
__device__ __forceinline__ float row_rms(float (&x)[8], float eps, float *scale) {
  constexpr int kRow = D / 8;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
  s = row_sum<kRow>(s);
  *scale = 1.f;
  if (__any_sync(0xffffffffu, !(s <= FLT_MAX))) {
    const bool over = !(s <= FLT_MAX);
    float t = 0.f;
    if (over) *scale = kDown;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= *scale;
      t = fmaf(x[i], x[i], t);
    }
    t = row_sum<kRow>(t);
    if (over) s = t, eps *= kDown * kDown;
  }
  return rsqrtf(s * (1.f / D) + eps);
}

// Where a lane's 8 elements stand in the rotation: their partners' lane and the
// cosine and signed sine of each.
struct Turn {
  int partner;           // lane that holds the partners (this one: none, or interleaved)
  float cos[8], sin[8];  // sin carries the sign: z = x cos + x' sin
};

template <int D>
__device__ __forceinline__ Turn load_turn(const RopeParams &p, int64_t token, int lane) {
  constexpr int kRow = D / 8;
  Turn t;
  t.partner = lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) t.cos[i] = 1.f, t.sin[i] = 0.f;
  const int half = p.rope_dim / 2;
  const int e0 = (lane % kRow) * 8;
  if (e0 >= p.rope_dim) return t;
  int pos = p.positions[token];
  if (pos < 0 || pos >= p.max_pos) {
    atomicExch(&g_rope_error, kErrBadLength);
    pos = min(max(pos, 0), p.max_pos - 1);
  }
  const float *row = p.table + static_cast<int64_t>(pos) * p.rope_dim;
  if (p.interleaved) {
    const float4 c = *reinterpret_cast<const float4 *>(row + e0 / 2);
    const float4 s = *reinterpret_cast<const float4 *>(row + half + e0 / 2);
    t.cos[0] = t.cos[1] = c.x, t.cos[2] = t.cos[3] = c.y;
    t.cos[4] = t.cos[5] = c.z, t.cos[6] = t.cos[7] = c.w;
    t.sin[0] = -s.x, t.sin[1] = s.x, t.sin[2] = -s.y, t.sin[3] = s.y;
    t.sin[4] = -s.z, t.sin[5] = s.z, t.sin[6] = -s.w, t.sin[7] = s.w;
    return t;
  }
  const bool first = e0 < half;
  const int at = first ? e0 : e0 - half;
  t.partner = first ? lane + half / 8 : lane - half / 8;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 c = *reinterpret_cast<const float4 *>(row + at + i);
    const float4 s = *reinterpret_cast<const float4 *>(row + half + at + i);
    t.cos[i] = c.x, t.cos[i + 1] = c.y, t.cos[i + 2] = c.z, t.cos[i + 3] = c.w;
    t.sin[i] = s.x, t.sin[i + 1] = s.y, t.sin[i + 2] = s.z, t.sin[i + 3] = s.w;
  }
  if (first) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t.sin[i] = -t.sin[i];
  }
  return t;
}

// A lane's 8 weights (1 without weights).
__device__ __forceinline__ void load_weights(const float *w, int e0, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = w != nullptr ? __ldg(w + e0 + i) : 1.f;
}

// The partner elements of `u`.
__device__ __forceinline__ uint4 partners(const RopeParams &p, const Turn &t, const uint4 &u) {
  const uint4 other = shfl4(u, t.partner);
  return p.interleaved ? swap_pairs(u) : other;
}

// Rows [lo, hi) of `src` (one token's heads), kU at a time per lane group.
template <int D, typename Dst>
__device__ __forceinline__ void turn_rows(const RopeParams &p, const Turn &t,
                                          const __nv_bfloat16 *src, const float *w, int lo, int hi,
                                          int lane, Dst dst) {
  constexpr int kRow = D / 8, kStep = 32 / kRow, kU = 2;
  const int e0 = (lane % kRow) * 8;
  float a[8], b[8];
  load_weights(w, e0, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float other = __shfl_sync(0xffffffffu, a[i], t.partner);
    b[i] = t.sin[i] * (p.interleaved ? a[i ^ 1] : other);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] *= t.cos[i];
  for (int h0 = lo; h0 < hi; h0 += kStep * kU) {
    uint4 u[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int h = h0 + j * kStep + lane / kRow;
      u[j] = h < hi ? *reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(h) * D + e0)
                    : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int h = h0 + j * kStep + lane / kRow;
      float x[8], o[8];
      unpack8(u[j], x);
      unpack8(partners(p, t, u[j]), o);
      float r = 1.f, scale = 1.f;
      if (w != nullptr) r = row_rms<D>(x, p.eps, &scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = r * fmaf(x[i], a[i], scale * o[i] * b[i]);
      if (h < hi) dst(h, e0, pack8(x));
    }
  }
}

// Four blocks per SM: warps hide the loads, not loads within a warp (32768 tokens of 80
// rows of 64: 141 us with two steps of rows in flight a warp and four blocks, 147 with
// four steps and three blocks, 179 with four steps and two).
template <int D>
__global__ void __launch_bounds__(kWarps * 32, 4) rope_kernel(const RopeParams p) {
  constexpr int kRow = D / 8, kStep = 32 / kRow;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t token = item / p.parts;
  const int part = static_cast<int>(item - token * p.parts);
  if (token >= p.total) return;
  // this warp's rows of the token: [lo, hi) of its query, key and value heads in a row
  const int vrows = p.v_cache != nullptr ? p.hkv : 0;
  const int rows = p.hq + p.hkv + vrows;
  const int per = (rows + p.parts - 1) / p.parts;
  const int lo = part * per, hi = min(lo + per, rows);
  if (lo >= hi) return;
  const Turn t = load_turn<D>(p, token, lane);
  if (lo < p.hq) {
    __nv_bfloat16 *out = p.q_out + token * p.hq * D;
    turn_rows<D>(p, t, p.q + token * p.q_stride, p.wq, lo, min(hi, p.hq), lane,
                 [&](int h, int e0, const uint4 &z) {
                   *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(h) * D + e0) = z;
                 });
  }
  if (hi <= p.hq) return;
  // element offset of KV head 0's row in the pages, -1 without one
  int64_t at = -1;
  if (p.k_cache != nullptr) {
    const int64_t slot = p.slots[token];
    if (slot >= p.num_slots) {
      if (lane == 0) atomicExch(&g_rope_error, kErrBadPage);
    } else if (slot >= 0) {
      const int64_t page = slot / p.page_size;
      at = (page * p.hkv * p.page_size + (slot - page * p.page_size)) * D;
    }
  }
  const int64_t head = static_cast<int64_t>(p.page_size) * D;
  const int k0 = max(lo - p.hq, 0), k1 = min(hi - p.hq, p.hkv);
  if (k0 < k1 && (at >= 0 || p.k_out != nullptr)) {
    turn_rows<D>(p, t, p.k + token * p.k_stride, p.wk, k0, k1, lane,
                 [&](int h, int e0, const uint4 &z) {
                   if (p.k_out != nullptr)
                     *reinterpret_cast<uint4 *>(p.k_out + (token * p.hkv + h) * D + e0) = z;
                   if (at >= 0)
                     *reinterpret_cast<uint4 *>(p.k_cache + at + h * head + e0) = z;
                 });
  }
  const int v0 = max(lo - p.hq - p.hkv, 0), v1 = hi - p.hq - p.hkv;
  if (at >= 0) {
    const int e0 = (lane % kRow) * 8;
    for (int h = v0 + lane / kRow; h < v1; h += kStep)
      *reinterpret_cast<uint4 *>(p.v_cache + at + h * head + e0) =
          *reinterpret_cast<const uint4 *>(p.v + token * p.v_stride + static_cast<int64_t>(h) * D +
                                           e0);
  }
}

// ---- backward ---------------------------------------------------------------
// Rows [lo, hi) of one token; dw collects this lane's 8 weight gradients.
template <int D>
__device__ __forceinline__ void grad_rows(const RopeParams &p, const Turn &t,
                                          const __nv_bfloat16 *dz, const __nv_bfloat16 *src,
                                          const float *w, __nv_bfloat16 *dx, int lo, int hi,
                                          int lane, float (&dw)[8]) {
  constexpr int kRow = D / 8, kStep = 32 / kRow, kU = 2;
  const int e0 = (lane % kRow) * 8;
  float wt[8];
  load_weights(w, e0, wt);
  for (int h0 = lo; h0 < hi; h0 += kStep * kU) {
    uint4 uz[kU], ux[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int h = h0 + j * kStep + lane / kRow;
      uz[j] = ux[j] = make_uint4(0, 0, 0, 0);
      if (h < hi) {
        uz[j] = *reinterpret_cast<const uint4 *>(dz + static_cast<int64_t>(h) * D + e0);
        if (w != nullptr)
          ux[j] = *reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(h) * D + e0);
      }
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int h = h0 + j * kStep + lane / kRow;
      float dy[8], o[8];
      unpack8(uz[j], dy);
      unpack8(partners(p, t, uz[j]), o);
      // the transposed turn: the sines change sign
#pragma unroll
      for (int i = 0; i < 8; ++i) dy[i] = fmaf(dy[i], t.cos[i], -o[i] * t.sin[i]);
      if (w != nullptr) {
        float x[8], gx = 0.f, scale;
        unpack8(ux[j], x);
        const float r = row_rms<D>(x, p.eps, &scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= r;
          gx = fmaf(wt[i] * dy[i], x[i], gx);
        }
        const float c = row_sum<kRow>(gx) * (1.f / D);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = wt[i] * dy[i];
          dw[i] = fmaf(dy[i], x[i], dw[i]);
          dy[i] = r * scale * fmaf(-c, x[i], g);
        }
      }
      if (h < hi)
        *reinterpret_cast<uint4 *>(dx + static_cast<int64_t>(h) * D + e0) = pack8(dy);
    }
  }
}

// Terms that a lane adds up before it hands their sum on: a running sum's roundings grow with
// its length, and all go one way where the rows are alike.
constexpr int kTerms = 64;

// Hands the sums dw on to `held`: for each a sum and what its roundings have lost.
__device__ __forceinline__ void hold(float2 (*held)[kWarps * 32], float (&dw)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 &h = held[i][threadIdx.x];
    const float s = h.x + dw[i], t = s - h.x;
    h = make_float2(s, h.y + ((h.x - (s - t)) + (dw[i] - t)));
    dw[i] = 0.f;
  }
}

// Each warp takes (token, part) items at a stride; the block's weight gradients go to
// `partial`, summed in a fixed order so that the same call gives the same bits.
template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2) rope_backward_kernel(const RopeParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kRow = D / 8, kStep = 32 / kRow;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int rows = p.hq + p.hkv;
  const int per = (rows + p.parts - 1) / p.parts;
  __shared__ float2 held[16][kWarps * 32];  // each thread's own: dwq, dwk
  float dwq[8] = {}, dwk[8] = {};
#pragma unroll
  for (int i = 0; i < 16; ++i) held[i][threadIdx.x] = make_float2(0.f, 0.f);
  const int each = (per + kStep - 1) / kStep;  // terms of an item, at most
  int terms = 0;
  const int64_t items = p.total * p.parts;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + wid; item < items;
       item += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t token = item / p.parts;
    const int part = static_cast<int>(item - token * p.parts);
    const int lo = part * per, hi = min(lo + per, rows);
    if (lo >= hi) continue;
    if (terms + each > kTerms && p.partial != nullptr) {
      hold(held, dwq);
      hold(held + 8, dwk);
      terms = 0;
    }
    terms += each;
    const Turn t = load_turn<D>(p, token, lane);
    if (lo < p.hq)
      grad_rows<D>(p, t, p.dq_out + token * p.hq * D, p.q + token * p.q_stride, p.wq,
                   p.dq + token * p.dq_stride, lo, min(hi, p.hq), lane, dwq);
    if (hi > p.hq)
      grad_rows<D>(p, t, p.dk_out + token * p.hkv * D, p.k + token * p.k_stride, p.wk,
                   p.dk + token * p.dk_stride, max(lo - p.hq, 0), hi - p.hq, lane, dwk);
  }
  if (p.partial == nullptr) return;
  __shared__ float sums[kWarps][2][D];
  hold(held, dwq);
  hold(held + 8, dwk);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 q = held[i][threadIdx.x], k = held[8 + i][threadIdx.x];
    dwq[i] = q.x + q.y, dwk[i] = k.x + k.y;
#pragma unroll
    for (int o = kRow; o < 32; o <<= 1) {
      dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
      dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
    }
  }
  if (lane < kRow) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[wid][0][lane * 8 + i] = dwq[i];
      sums[wid][1][lane * 8 + i] = dwk[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) s += sums[j][i / D][i % D];
    p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
  }
}

// Weight gradient i = the sum of the blocks' partials, one warp each.
__global__ void __launch_bounds__(256) rope_weight_grad_kernel(const float *partial, int blocks,
                                                               int dim, float *dwq, float *dwk) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= 2 * dim) return;
  float s = 0.f;
  for (int b = lane; b < blocks; b += 32) s += partial[static_cast<int64_t>(b) * 2 * dim + i];
  s = row_sum<32>(s);
  float *dw = i < dim ? dwq : dwk;
  if (lane == 0 && dw != nullptr) dw[i % dim] = s;
}

constexpr int kGradBlocks = 152 * 4;  // at most: two waves of two blocks of 8 warps per SM

RopeParams params(const RopeLaunch &a) {
  RopeParams p{};
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v);
  p.q_stride = a.q_stride, p.k_stride = a.k_stride, p.v_stride = a.v_stride;
  p.positions = a.positions;
  p.total = a.total;
  p.hq = a.hq, p.hkv = a.hkv;
  p.wq = a.q_weight, p.wk = a.k_weight;
  p.eps = a.eps;
  p.table = a.cos_sin;
  p.max_pos = a.max_positions;
  p.rope_dim = a.cos_sin != nullptr ? a.rope_dim : 0;
  p.interleaved = p.rope_dim > 0 && a.interleaved;
  return p;
}

// Warps per token: one where the tokens alone give every SM 32 warps, else as many as
// that takes, down to 8 rows each.
int token_parts(int64_t total, int rows) {
  const int64_t want = 152 * 32, most = (rows + 7) / 8;
  const int64_t parts = (want + total - 1) / total;
  return static_cast<int>(parts < 1 ? 1 : parts > most ? most : parts);
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch &a, cudaStream_t stream) {
  RopeParams p = params(a);
  p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
  p.k_out = static_cast<__nv_bfloat16 *>(a.k_out);
  p.slots = a.slots;
  p.k_cache = static_cast<__nv_bfloat16 *>(a.k_cache);
  p.v_cache = static_cast<__nv_bfloat16 *>(a.v_cache);
  p.num_slots = static_cast<int64_t>(a.num_pages) * a.page_size;
  p.page_size = a.page_size;
  p.parts = token_parts(a.total, a.hq + a.hkv + (p.v_cache != nullptr ? a.hkv : 0));
  const int64_t blocks = (a.total * p.parts + kWarps - 1) / kWarps;
  if (a.head_dim == 128)
    rope_kernel<128><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
  else
    rope_kernel<64><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

size_t rope_backward_workspace_bytes(int head_dim) {
  return static_cast<size_t>(kGradBlocks) * 2 * head_dim * sizeof(float);
}

cudaError_t launch_rope_backward(const RopeLaunch &a, cudaStream_t stream) {
  RopeParams p = params(a);
  p.dq_out = static_cast<const __nv_bfloat16 *>(a.dq_out);
  p.dk_out = static_cast<const __nv_bfloat16 *>(a.dk_out);
  p.dq = static_cast<__nv_bfloat16 *>(a.dq);
  p.dk = static_cast<__nv_bfloat16 *>(a.dk);
  p.dq_stride = a.dq_stride, p.dk_stride = a.dk_stride;
  p.partial = a.dq_weight != nullptr || a.dk_weight != nullptr ? static_cast<float *>(a.workspace)
                                                               : nullptr;
  const int rows = a.hq + a.hkv, most = kTerms * (256 / a.head_dim);  // rows of kTerms terms
  p.parts = a.total > 0 ? token_parts(a.total, rows) : 1;
  if (p.parts * most < rows) p.parts = (rows + most - 1) / most;
  int64_t blocks = (a.total * p.parts + kWarps - 1) / kWarps;
  if (blocks > kGradBlocks) blocks = kGradBlocks;
  if (blocks > 0) {
    if (a.head_dim == 128)
      rope_backward_kernel<128><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
    else
      rope_backward_kernel<64><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.partial == nullptr) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * a.head_dim / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_weight_grad_kernel,
                            static_cast<const float *>(p.partial), static_cast<int>(blocks),
                            a.head_dim, a.dq_weight, a.dk_weight);
}

cudaError_t rope_read_error(cudaStream_t stream, int *code) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_rope_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(int));
  return e;
}

}  // namespace sinkattn
