// Paged-cache bookkeeping: block tables and slot maps from request lengths,
// and the write of new key / value rows into a block-scaled fp8 cache.
//
// Page "Fast embeddings on GPUs", section "ROSE": paged KV for serving. The
// attention calls read a block table and lengths; page_map makes the table and
// append makes the pages' contents.
#include <math.h>

#include <type_traits>

#include "launch.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

__device__ int g_cache_error;

// ---- page map ---------------------------------------------------------------
// Sequence b holds old_b tokens and gets Lk_b - old_b more. The pages
// [ceil(old_b / ps), ceil(Lk_b / ps)) are new; over all sequences they take
// consecutive entries of the free list, in order. Both the entry index of a
// page and the slot of a token then follow from an exclusive prefix sum of the
// new-page counts.

struct PageMapParams {
  const int32_t *seqlens_k, *cu_q, *free_pages, *free_head;
  int32_t *free_head_out, *table, *page_offsets;
  int64_t *slots;
  int batch, page_size, max_pages, num_free;
  int64_t total_q;
};

constexpr int64_t kOneBlockRows = 1024;  // rows that one block fills itself (4096: 8.8 us, two launches 4.7)

struct SeqPages {
  int first_pos;  // position of the sequence's first new token (negative: Lq > Lk)
  int have, end;  // pages [have, end) are new
};

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

__device__ __forceinline__ SeqPages seq_pages(const PageMapParams &p, int b, bool *bad) {
  const int lk_raw = p.seqlens_k[b];
  const int lk = max(lk_raw, 0);
  const int lq = p.cu_q != nullptr ? max(p.cu_q[b + 1] - p.cu_q[b], 0) : 1;
  SeqPages s;
  s.first_pos = lk - lq;
  const int old = max(s.first_pos, 0);
  const int have = ceil_div(old, p.page_size), end = ceil_div(lk, p.page_size);
  s.have = min(have, p.max_pages);
  s.end = min(end, p.max_pages);
  *bad = lk_raw < 0 || end > p.max_pages;
  return s;
}

// Token row i: its slot, and the table entry of the page that it starts. Every new
// page is started by exactly one new token.
__device__ __forceinline__ void fill_row(const PageMapParams &p, int64_t i) {
  int b = static_cast<int>(i);
  if (p.cu_q != nullptr) {
    if (p.batch == 0 || i >= p.cu_q[p.batch]) {  // padding rows behind the last sequence
      p.slots[i] = -1;
      return;
    }
    int lo = 0, hi = p.batch;  // cu_q[lo] <= i < cu_q[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_q[mid] <= i) lo = mid; else hi = mid;
    }
    b = lo;
  }
  bool bad;
  const SeqPages s = seq_pages(p, b, &bad);
  const int pos = s.first_pos + (p.cu_q != nullptr ? static_cast<int>(i - p.cu_q[b]) : 0);
  int64_t slot = -1;
  if (pos >= 0) {
    const int pg = pos / p.page_size, off = pos - pg * p.page_size;
    int page = -1;
    if (pg < s.have) {
      page = p.table[static_cast<size_t>(b) * p.max_pages + pg];
    } else if (pg < s.end) {
      const int at = p.page_offsets[b] + pg - s.have;
      if (at >= 0 && at < p.num_free) page = p.free_pages[at];
      if (off == 0) p.table[static_cast<size_t>(b) * p.max_pages + pg] = page;
    }
    if (page >= 0) slot = static_cast<int64_t>(page) * p.page_size + off;
  }
  p.slots[i] = slot;
}

// One block: page_offsets (free-list index of each sequence's first new page) and
// the advanced head; on short calls (kFill) the rows too. Bound by latency: 256
// sequences of one token 3.2 us (two launches 4.8 us).
template <bool kFill>
__global__ void __launch_bounds__(1024) page_offsets_kernel(const PageMapParams p) {
  if (!kFill) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int warp_sums[32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int head = *p.free_head;
  int carry = head;
  for (int base = 0; base < p.batch; base += blockDim.x) {
    const int b = base + threadIdx.x;
    int need = 0;
    if (b < p.batch) {
      bool bad;
      const SeqPages s = seq_pages(p, b, &bad);
      if (bad) atomicExch(&g_cache_error, kErrBadLength);
      need = s.end - s.have;
    }
    int incl = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[wid] = incl;
    __syncthreads();
    if (wid == 0) {
      int v = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      warp_sums[lane] = v;
    }
    __syncthreads();
    const int before = wid > 0 ? warp_sums[wid - 1] : 0;
    if (b < p.batch) p.page_offsets[b] = carry + before + incl - need;
    carry += warp_sums[31];
    __syncthreads();  // warp_sums is reused by the next chunk
  }
  if (threadIdx.x == 0) {
    p.page_offsets[p.batch] = carry;
    if (head < 0 || carry > p.num_free) atomicExch(&g_cache_error, kErrNoPages);
    *p.free_head_out = min(carry, p.num_free);
  }
  if (kFill) {
    __syncthreads();  // page_offsets are written
    for (int64_t i = threadIdx.x; i < p.total_q; i += blockDim.x) fill_row(p, i);
  }
}

// The rows of longer calls, launched while the offsets are computed: 250 sequences
// with 503k new tokens in 7.9 us for both kernels (4.3 MB).
__global__ void __launch_bounds__(256) page_fill_kernel(const PageMapParams p) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // page_offsets
  if (i < p.total_q) fill_row(p, i);
}

// ---- append -----------------------------------------------------------------
// Rows of one scale block stand together in the call (consecutive rows,
// consecutive slots): a run. Its first row leads; one warp writes a run's codes
// and scale for one KV head of K or of V.
//
// The scale of a block is a power of two, the smallest 2^e with
// amax <= 448 * 2^e. e4m3 is a floating format, so a coarser choice of scale
// costs no relative precision above its subnormals, and x / 2^e as well as the
// re-encoding of older codes under a grown scale are exact until a value
// becomes subnormal: the codes do not depend on how the tokens of a block were
// split over calls, but for those.
//
// One element that is not finite must not set the scale, which would turn the other
// tokens of its block to zeros: where a maximum is not finite (never, in a working
// model), it is taken again over the finite elements.

constexpr int kAppendWarps = 4;
constexpr int kWideRows = 256;   // token rows per block where its warps share runs
constexpr int kMinScaleExp = -60, kMaxScaleExp = 60;

struct AppendParams {
  const __nv_bfloat16 *k, *v;
  int64_t k_stride, v_stride;
  const int64_t *slots;
  int64_t total, num_slots;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int hkv, page_size, scale_block;
  int rows;         // token rows per warp, at most 32
  int64_t warps;
  int per_page;     // scale blocks per page
  // slot -> page, scale block within it, offset within that
  __device__ void split(int64_t slot, int *page, int *bi, int *o1) const {
    int off;
    if (num_slots <= UINT32_MAX) {
      const uint32_t x = static_cast<uint32_t>(slot), ps = static_cast<uint32_t>(page_size);
      *page = static_cast<int>(x / ps);
      off = static_cast<int>(x % ps);
    } else {
      *page = static_cast<int>(slot / page_size);
      off = static_cast<int>(slot % page_size);
    }
    *bi = off / scale_block;
    *o1 = off - *bi * scale_block;
  }
};

// Packed |bf16| maxima of 8 values (finite: the 15 magnitude bits order as integers).
__device__ __forceinline__ uint32_t absmax8(uint4 x, uint32_t m) {
  const uint32_t mask = 0x7fff7fffu;
  m = __vmaxu2(m, x.x & mask);
  m = __vmaxu2(m, x.y & mask);
  m = __vmaxu2(m, x.z & mask);
  return __vmaxu2(m, x.w & mask);
}

// The same over the finite ones among them (magnitude bits below 0x7f80).
__device__ __forceinline__ uint32_t absmax8_finite(uint4 x, uint32_t m) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fff7fffu;
    m = __vmaxu2(m, a & __vcmpltu2(a, 0x7f807f80u));
  }
  return m;
}
__device__ __forceinline__ uint32_t upper_of(uint32_t m) { return max(m & 0xffffu, m >> 16); }
__device__ __forceinline__ bool not_finite(uint32_t m) { return upper_of(m) >= 0x7f80u; }

// Smallest e with s <= 2^e, within the scales' range.
__device__ __forceinline__ int ceil_exponent(float s) {
  const int bits = __float_as_int(fmaxf(s, 0.f));
  return min(max((bits >> 23) - 127 + ((bits & 0x7fffff) != 0 ? 1 : 0), kMinScaleExp),
             kMaxScaleExp);
}

// Smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8), amax as bf16 bits.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return min(max(e, kMinScaleExp), kMaxScaleExp);
}

// 8 bf16 values times inv, a power of two -> 8 e4m3 codes, round to nearest even.
__device__ __forceinline__ uint2 encode8(uint4 x, float inv) {
  return make_uint2(e4m3x4(bf16_lo(x.x) * inv, bf16_hi(x.x) * inv, bf16_lo(x.y) * inv,
                           bf16_hi(x.y) * inv),
                    e4m3x4(bf16_lo(x.z) * inv, bf16_hi(x.z) * inv, bf16_lo(x.w) * inv,
                           bf16_hi(x.w) * inv));
}

// 4 codes times f, re-encoded.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float f) {
  uint32_t lo, hi;
  e4m3x4_to_f16x4(c, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  return e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// One warp per (p.rows token rows, KV head, K or V), with no barrier: it reads
// 32 slots at once, finds the runs by ballot, and writes those that start in its
// rows. D / 8 lanes per row, 8 elements each; kTeam = lanes per run, in steps of
// kTeam * 8 / D rows. The first kKeep steps of a run stay in registers between
// the maximum and the encoding; longer runs are read twice (from L2).
// Bound by HBM latency and traffic (6 D bytes per token and head, K and V):
// 131072 tokens of 8 heads at head_dim 64, 404 MB in 70 us (5.8 TB/s; a block of
// 8 warps that shared its run finding took 76 us); 18k tokens at head_dim 128 with
// 32-token scales 23.7 us (29 us with 8 steps kept); a decode step of 64 rows
// 2.7 us, about 1.4 us more where the scales grow. Register caps trade resident
// warps against rows in flight and spills: 48 registers for 4 steps (10 blocks per
// SM, 48 bytes of spills; 12 blocks take 78 us), 48 to 64 for scale blocks of 2 to 8
// tokens (64 to 96 bytes; 65536 tokens with a scale per 4 tokens 46 us).
// kWide: the warps of a block share a run, for scale blocks that one warp cannot
// keep (65536 tokens of 256-token blocks: 92 -> 56 us; a run's rows are loaded
// and written between two barriers, so that loads and stores alternate).
template <int D, int kTeam, int kKeep, bool kWide, int kMinBlocks>
__global__ void __launch_bounds__(kAppendWarps * 32, kMinBlocks)
    append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = kTeam / kLanes * (kWide ? kAppendWarps : 1);
  constexpr int kTeams = 32 / kTeam;
  __shared__ uint32_t s_max[kAppendWarps];
  __shared__ int64_t s_slots[kWide ? kWideRows + 1 : 1];
  const int lane = threadIdx.x & 31;
  const int64_t unit = kWide ? blockIdx.x
                             : blockIdx.x * static_cast<int64_t>(kAppendWarps) + (threadIdx.x >> 5);
  if (unit >= p.warps) return;
  const int64_t chunk = p.warps <= UINT32_MAX
                            ? static_cast<uint32_t>(unit) / static_cast<uint32_t>(2 * p.hkv)
                            : unit / (2 * p.hkv);
  const int in = static_cast<int>(unit - chunk * 2 * p.hkv);
  const bool is_v = in >= p.hkv;
  const int g = is_v ? in - p.hkv : in;
  const int64_t unit_row = chunk * p.rows;
  if (kWide) {  // the slots of the unit's rows and of the one before, read at once
    for (int i = threadIdx.x; i <= kWideRows; i += kAppendWarps * 32) {
      const int64_t r = unit_row - 1 + i;
      s_slots[i] = r < 0 ? -2 : r < p.total ? p.slots[r] : -1;
    }
    __syncthreads();
  }
  for (int w0 = 0; w0 < (kWide ? kWideRows : 1); w0 += 32) {
    const int64_t row0 = unit_row + w0;
    // cont: the row continues the run of the row before it. Of a slot, the page,
    // the scale block in it (bi) and the offset in that block (o1) are kept.
    int my_page, my_bi, my_o1;
    unsigned conts, leads;
    {
      int64_t my, prev;
      if (kWide) {
        my = s_slots[w0 + lane + 1];
        prev = s_slots[w0 + lane];
      } else {
        my = row0 + lane < p.total ? p.slots[row0 + lane] : -1;
        prev = __shfl_up_sync(0xffffffffu, my, 1);
        if (lane == 0) prev = row0 > 0 ? p.slots[row0 - 1] : -2;
      }
      const bool valid = my >= 0 && my < p.num_slots;
      if (my >= p.num_slots) atomicExch(&g_cache_error, kErrBadPage);
      p.split(valid ? my : 0, &my_page, &my_bi, &my_o1);
      const bool cont = valid && prev == my - 1 && my_o1 != 0;
      conts = __ballot_sync(0xffffffffu, cont);
      leads = __ballot_sync(0xffffffffu, valid && !cont);
    }
    if (p.rows < 32) leads &= (1u << p.rows) - 1u;
    if (leads == 0u) continue;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const __nv_bfloat16 *base = is_v ? p.v : p.k;
    uint8_t *cache = is_v ? p.v_cache : p.k_cache;
    float *scales = is_v ? p.v_scale : p.k_scale;
    const unsigned team_mask =
        kTeam == 32 ? 0xffffffffu : ((1u << (kTeam & 31)) - 1u) << (lane / kTeam * kTeam);
    const int sub = lane % kTeam / kLanes + (kWide ? (threadIdx.x >> 5) * (32 / kLanes) : 0);
    const int col = (lane % kLanes) * 8;
    const int team = lane / kTeam;
    while (leads != 0u) {
      // teams take the next leads in order; a team without one idles
      int i0 = -1;
#pragma unroll
      for (int k = 0; k < kTeams; ++k) {
        if (k == team && leads != 0u) i0 = __ffs(leads) - 1;
        leads &= leads - 1u;
      }
      const bool has = i0 >= 0;
      i0 = max(i0, 0);
      const int o1 = __shfl_sync(0xffffffffu, my_o1, i0);  // older tokens of the block
      const int bi = __shfl_sync(0xffffffffu, my_bi, i0);
      const int64_t head = static_cast<int64_t>(__shfl_sync(0xffffffffu, my_page, i0)) * p.hkv + g;
      const int64_t r = row0 + i0;
      const int most = p.scale_block - o1;
      // rows of the run: set bits behind its lead, then, past these 32, the slots
      const unsigned after = ~(i0 == 31 ? 0u : conts >> (i0 + 1));
      int n = has ? 1 + (after == 0u ? 31 : __ffs(after) - 1) : 0;
      if (i0 + n == 32 && n < most) {
        const int64_t slot = p.slots[r];
        constexpr int kBatch = kTeam == 32 ? 8 : 1;  // loads in flight, kTeam slots each
        bool more = true;
        while (more && n < most) {
          bool ok[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int at = n + j * kTeam + lane % kTeam;
            ok[j] = at < most && r + at < p.total && p.slots[r + at] == slot + at;
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const unsigned w = ~(__ballot_sync(team_mask, ok[j]) >> (lane / kTeam * kTeam));
            const int k = w == 0u ? kTeam : min(__ffs(w) - 1, kTeam);
            if (more) n += k;
            more = more && k == kTeam;
          }
        }
      }
      __syncwarp();
      const __nv_bfloat16 *src = base + r * stride + static_cast<size_t>(g) * D + col;
      uint4 keep[kKeep];
      uint32_t m = 0u;
#pragma unroll
      for (int c = 0; c < kKeep; ++c) {
        const int i = c * kRows + sub;
        keep[c] = i < n ? *reinterpret_cast<const uint4 *>(src + i * stride)
                        : make_uint4(0u, 0u, 0u, 0u);
      }
      float *sp = scales + head * p.per_page + bi;
      const float had = has && o1 > 0 ? *sp : 0.f;
#pragma unroll
      for (int c = 0; c < kKeep; ++c) m = absmax8(keep[c], m);
      for (int i = kKeep * kRows + sub; i < n; i += kRows)
        m = absmax8(*reinterpret_cast<const uint4 *>(src + i * stride), m);
      auto join = [&] {
#pragma unroll
        for (int o = kTeam / 2; o > 0; o >>= 1)
          m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (kWide) {  // the block's warps hold parts of one run
          __syncthreads();  // s_max is free
          if (lane == 0) s_max[threadIdx.x >> 5] = m;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < kAppendWarps; ++w) m = __vmaxu2(m, s_max[w]);
        }
      };
      join();
      if (__builtin_expect(__any_sync(0xffffffffu, not_finite(m)), 0)) {  // kWide: in all warps
        if (not_finite(m)) atomicExch(&g_cache_error, kErrBadValue);
        m = 0u;
        for (int i = sub; i < n; i += kRows)
          m = absmax8_finite(*reinterpret_cast<const uint4 *>(src + i * stride), m);
        __syncwarp();
        join();
      }
      int e = scale_exponent(upper_of(m));
      uint8_t *dst = cache +
                     (head * p.page_size + static_cast<int64_t>(bi) * p.scale_block) * D + col;
      if (has && o1 > 0) {
        e = max(e, ceil_exponent(had));
        const float f = had * __int_as_float((127 - e) << 23);
        if (f != 1.f) {  // the scale changed
          for (int i = sub; i < o1; i += kRows) {
            uint2 *c = reinterpret_cast<uint2 *>(dst + static_cast<int64_t>(i) * D);
            const uint2 x = *c;
            *c = make_uint2(rescale4(x.x, f), rescale4(x.y, f));
          }
        }
      }
      const float inv = __int_as_float((127 - e) << 23);
      dst += static_cast<int64_t>(o1) * D;
#pragma unroll
      for (int c = 0; c < kKeep; ++c) {
        const int i = c * kRows + sub;
        if (i < n)
          *reinterpret_cast<uint2 *>(dst + static_cast<int64_t>(i) * D) = encode8(keep[c], inv);
      }
      for (int i = kKeep * kRows + sub; i < n; i += kRows)
        *reinterpret_cast<uint2 *>(dst + static_cast<int64_t>(i) * D) =
            encode8(*reinterpret_cast<const uint4 *>(src + i * stride), inv);
      __syncwarp();  // every lane has read the old scale (kWide: before the barrier)
      if (has && lane % kTeam == 0 && (!kWide || threadIdx.x == 0))
        *sp = __int_as_float((e + 127) << 23);
    }
  }
}

// A scale per token: no runs and no older tokens, so a warp takes 256 / D rows at
// a time and walks their heads; the page of a row is looked up once (65536 tokens,
// head_dim 64: 84 us by runs, which the instructions bound, 39 us so; 128: 124 and
// 66 us).
template <int D>
__global__ void __launch_bounds__(256) append_rows_kernel(const AppendParams p, int heads) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int64_t r = (blockIdx.x * int64_t(8) + (threadIdx.x >> 5)) * kRows + lane / kLanes;
  const int col = lane % kLanes * 8;
  const int64_t slot = r < p.total ? p.slots[r] : -1;
  if (slot >= p.num_slots) atomicExch(&g_cache_error, kErrBadPage);
  const bool ok = slot >= 0 && slot < p.num_slots;
  int page, off, o1;
  p.split(ok ? slot : 0, &page, &off, &o1);
  const int g0 = blockIdx.y * heads, g1 = min(p.hkv, g0 + heads);
  const __nv_bfloat16 *k = p.k + (ok ? r : 0) * p.k_stride + col;
  const __nv_bfloat16 *v = p.v + (ok ? r : 0) * p.v_stride + col;
#pragma unroll 4
  for (int g = g0; g < g1; ++g) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4 kx = ok ? *reinterpret_cast<const uint4 *>(k + static_cast<size_t>(g) * D) : zero;
    const uint4 vx = ok ? *reinterpret_cast<const uint4 *>(v + static_cast<size_t>(g) * D) : zero;
    uint32_t km = absmax8(kx, 0u), vm = absmax8(vx, 0u);
    auto join = [&] {
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        km = __vmaxu2(km, __shfl_xor_sync(0xffffffffu, km, o));
        vm = __vmaxu2(vm, __shfl_xor_sync(0xffffffffu, vm, o));
      }
    };
    join();
    if (__builtin_expect(__any_sync(0xffffffffu, not_finite(__vmaxu2(km, vm))), 0)) {
      if (not_finite(km) || not_finite(vm)) atomicExch(&g_cache_error, kErrBadValue);
      km = absmax8_finite(kx, 0u);
      vm = absmax8_finite(vx, 0u);
      join();
    }
    const int ke = scale_exponent(upper_of(km));
    const int ve = scale_exponent(upper_of(vm));
    if (!ok) continue;
    const int64_t at = (static_cast<int64_t>(page) * p.hkv + g) * p.page_size + off;
    *reinterpret_cast<uint2 *>(p.k_cache + at * D + col) =
        encode8(kx, __int_as_float((127 - ke) << 23));
    *reinterpret_cast<uint2 *>(p.v_cache + at * D + col) =
        encode8(vx, __int_as_float((127 - ve) << 23));
    if (col == 0) {
      p.k_scale[at] = __int_as_float((ke + 127) << 23);
      p.v_scale[at] = __int_as_float((ve + 127) << 23);
    }
  }
}

}  // namespace

cudaError_t launch_page_map(const PageMapLaunch &a, cudaStream_t stream) {
  PageMapParams p;
  p.seqlens_k = a.seqlens_k;
  p.cu_q = a.cu_q;
  p.free_pages = a.free_pages;
  p.free_head = a.free_head;
  p.free_head_out = a.free_head_out;
  p.table = a.block_table;
  p.page_offsets = a.page_offsets;
  p.slots = a.slots;
  p.batch = a.batch;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.num_free = a.num_free;
  p.total_q = a.total_q;
  if (a.total_q <= kOneBlockRows) {
    page_offsets_kernel<true><<<1, 1024, 0, stream>>>(p);
    return cudaGetLastError();
  }
  page_offsets_kernel<false><<<1, 1024, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.total_q + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, page_fill_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_append(const AppendLaunch &a, cudaStream_t stream) {
  AppendParams p;
  p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v);
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.slots = a.slots;
  p.total = a.total;
  p.num_slots = static_cast<int64_t>(a.num_pages) * a.page_size;
  p.k_cache = static_cast<uint8_t *>(a.k_cache);
  p.v_cache = static_cast<uint8_t *>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.hkv = a.hkv;
  p.page_size = a.page_size;
  p.scale_block = a.scale_block;
  p.per_page = a.page_size / a.scale_block;
  // Rows per warp: 32 once that still gives every SM about 48 warps; down to one
  // for a decode step, where each row is a run of its own.
  const int64_t want = a.total * a.hkv * 2 / (152 * 48);
  p.rows = 1;
  while (p.rows < 32 && p.rows * 2 <= want) p.rows *= 2;
  p.warps = (a.total + p.rows - 1) / p.rows * a.hkv * 2;
  const int64_t blocks = (p.warps + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  const int threads = kAppendWarps * 32;
  auto run_rows = [&](auto kernel, int step) {
    // all heads of a row by one warp once the rows fill the GPU
    const int heads = a.total >= 8192 ? a.hkv : 1;
    const int64_t per_block = 8 * step;
    kernel<<<dim3(static_cast<unsigned>((a.total + per_block - 1) / per_block),
                  static_cast<unsigned>((a.hkv + heads - 1) / heads)),
             256, 0, stream>>>(p, heads);
  };
  auto run_wide = [&](auto kernel) {
    p.rows = kWideRows;
    p.warps = (a.total + p.rows - 1) / p.rows * a.hkv * 2;
    kernel<<<static_cast<unsigned>(p.warps), threads, 0, stream>>>(p);
  };
  const int sb = a.scale_block;
  auto go = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    constexpr int kRow = D / 8, kStep = 256 / D;  // lanes per row, rows per warp step
    auto run = [&](auto kernel) { kernel<<<grid, threads, 0, stream>>>(p); };
    if (sb == 1)
      run_rows(append_rows_kernel<D>, kStep);
    else if (sb <= 2)
      run(append_kernel<D, kRow, 2, false, 10>);
    else if (sb <= 4)
      run(append_kernel<D, kRow, 4, false, 10>);
    else if (sb <= 8)
      run(append_kernel<D, kRow, 8, false, 8>);
    else if (sb <= 4 * kStep)
      run(append_kernel<D, 32, 4, false, 10>);
    else if (sb <= 8 * kStep)
      run(append_kernel<D, 32, 8, false, 6>);
    else if (sb <= 16 * kStep || p.rows < 32)  // a short call's runs are short too
      run(append_kernel<D, 32, 16, false, 4>);
    else
      run_wide(append_kernel<D, 32, 16, true, 4>);
  };
  if (a.head_dim == 128)
    go(std::integral_constant<int, 128>());
  else
    go(std::integral_constant<int, 64>());
  return cudaGetLastError();
}

cudaError_t cache_read_error(cudaStream_t stream, int *code) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_cache_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_cache_error, &zero, sizeof(int));
  return e;
}

}  // namespace sinkattn
