// Attention of a tree of drafted tokens over a paged bf16 cache, on the sm_103a tensor
// cores (tcgen05 + TMEM).
//
// Row i of a sequence with Lk keys and Lq drafted tokens sees the C = Lk - Lq keys of
// its context (within the window) and, of the Lq keys behind it, those of its ancestors
// and its own; its position is C + depth(i). The rows of a KV head's query heads,
// (i, head of the group), are packed into tiles of 128, so that one read of the keys
// serves Lq * group rows: a decode step's eight become up to 128, and the products need
// the tensor cores. With up to 128 rows HBM is the floor (128 keys of 64
// elements take 0.73 us of an SM's share of the bandwidth, their products 0.5 us).
//
// One CTA, two per SM, works through (KV head, 128 rows, range of keys) segments, 64 keys
// at a time:
//   warps 0-3  softmax: thread r owns row r of the tile (TMEM lane r)
//   warp 4     issues O += P V, owns TMEM
//   warp 5     issues S = Q K^T
//   warps 6-7  producers: page lookups and 16-byte cp.async copies of K and V rows into a
//              ring of 128-byte-swizzled slots (any page size; a row outside the visible
//              range is filled with zeros, whatever its page holds)
// TMEM (256 columns): two S buffers of 64 columns, O in D columns behind them. The softmax
// writes P over its S as two bf16 halves, P = hi + lo (16 significant bits, each product
// fp32): one bf16 P would round every weight to 2^-9, as much as the output's own
// rounding, and V has no exact fp16 form. Q K^T of the next tile runs during the
// softmax of this one. O is rescaled only where a row's maximum grows by more than 2^8.
//
// Instructions: the roles run different code on the same schedulers, and a warp of each
// role has to keep step with the others. Producers that looked pages up four steps at a
// time in an unrolled loop slowed every role (197 -> 253 us on 64 sequences of 1k to 8k
// keys), so their body is short: one lookup, one shuffle and one address for K and V (two
// loops 187 us, one 176 us). Bound now, at head_dim 64, by the softmax (1.5 k cycles per
// step and warp, about 500 of them issues; 57% of HBM on that case), at 128 by the copies.
//
// Shares: the tiles of all (sequence, KV head, row tile) items stand in one line, of which
// every CTA takes an equal piece, so that ragged batches end together. An item that a
// piece's border cuts leaves its parts (fp32 O, maximum, denominator) in the
// workspace, at most two per CTA, and a second kernel joins them.
#include <float.h>
#include <math.h>

#include <atomic>

#include "launch.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

__device__ int g_tree_error;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

constexpr int kRows = 128;  // rows of a tile
constexpr int kKeys = 64;   // keys per step
constexpr int kSoftmaxWarps = 4, kPvWarp = 4, kQkWarp = 5, kProducerWarp = 6;
constexpr int kProducers = 64;
constexpr int kThreads = kProducerWarp * 32 + kProducers;
constexpr int kSms = 152;
constexpr int kBlocks = 2 * kSms;  // resident at once
constexpr int kMaxShared = 4096;   // sequences whose tiles a CTA counts to find its share
constexpr int kMaxParts = 64;      // CTAs that share one item, at most
// Items of up to so many tiles are never cut. Of 256 sequences with windows of three and four
// tiles (chains of up to 5): 42 and 49 us whole, 48 and 70 us in shares; of 8: 8.1 and 8.9
// whole, 12.6 and 11.6 in shares. (At seven tiles whole ones are still ahead, 72 against 87
// and 10.8 against 14.8 us.)
constexpr int kWholeTiles = 4;

template <int D>
struct Cfg {
  static constexpr int kSlotBytes = kKeys * D * 2;  // K or V of one step
  static constexpr int kSlots = D == 64 ? 11 : 5;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffCtl = kOffRing + kSlots * kSlotBytes;
  static constexpr int kCtlBytes = 1024;
  static constexpr int kSmemBytes = kOffCtl + kCtlBytes;
  static constexpr int kTmemO = 2 * kKeys;
  static constexpr int kTmemCols = 256;
};
constexpr int kMaxSlots = 11;
// two CTAs per SM: 228 KB, of which 1 KB per CTA is the system's
static_assert(2 * (Cfg<64>::kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
static_assert(2 * (Cfg<128>::kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");

constexpr uint32_t kIdescQK = idesc_f32acc(kRows, kKeys, /*bf16=*/true, false, false);
constexpr uint32_t kIdescPV = idesc_f32acc(kRows, 64, /*bf16=*/true, false, true);

// An item that starts in CTA c's share and goes on into the next ones.
struct Header {
  int parts, b, g, rt;
};

struct TreeParams {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *cu_q, *parents, *table, *seqlens_k;
  int num_pages, max_pages, page_size, page_shift, batch;
  int max_q, max_k, hq, hkv, group, window;
  const float *sinks;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
  int shared, min_share;
  Header *headers;  // [blocks]
  float2 *part_md;  // [2 blocks][128]: maximum (log2 units), denominator
  float *part_o;    // [2 blocks][128][D], not normalised
  uint64_t stall_ns;
};

struct Ctl {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t s_full[2];   // S of step J in buffer J % 2
  uint64_t p_full[2];   // P of step J written
  uint64_t pv_done[2];  // P V of step J has completed
  uint64_t q_full, q_empty;
  uint64_t o_free;      // the segment's epilogue has read O
  uint64_t drain[2], never;
  int64_t begin, end, share;  // this CTA's tiles, and every CTA's number of them
  int b0;                     // sequence of its first tile
  int off_g, off_rt, off_t;   // KV head, row tile and tile within the sequence
  uint32_t tmem;
  int abort;
  int odd;  // a tile that rows see in part may have values that are not finite
  int64_t sums[kThreads / 32];
};
static_assert(sizeof(Ctl) <= 1024, "control block");

__device__ __forceinline__ void cp_async_mbar_arrive_noinc(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// One arrival for the whole warp, behind what its lanes did.
__device__ __forceinline__ void arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Seq {
  int first, lq, lk;  // first row, rows, keys
  int lo;             // first key that a row sees
  int tiles, row_tiles;
};

__device__ __forceinline__ Seq load_seq(const TreeParams &p, int b, bool report) {
  Seq s;
  s.first = p.cu_q[b];
  const int lq = p.cu_q[b + 1] - s.first, lk = p.seqlens_k[b];
  s.lq = min(max(lq, 0), p.max_q);
  s.lk = min(max(lk, 0), p.max_k);
  if (report && (s.lq != lq || s.lk != lk)) atomicExch(&g_tree_error, kErrBadLength);
  const int context = s.lk - s.lq;
  s.lo = p.window > 0 && p.window <= context ? context - (p.window - 1) : 0;
  s.tiles = max(1, (s.lk - s.lo + kKeys - 1) / kKeys);
  s.row_tiles = ceil_div(s.lq * p.group, kRows);
  return s;
}

// The segments of one CTA, in order: each role of the CTA walks them by itself.
struct Walk {
  Seq s;
  int b, g, rt;   // the segment's item
  int t0, t1;     // and its tiles [t0, t1)
  int64_t left;   // shares: tiles from t0 on
  int64_t item;   // whole items: index of the next one
  bool on;

  __device__ __forceinline__ void start(const TreeParams &p, const Ctl *c) {
    on = false;
    if (p.shared) {
      left = c->end - c->begin;
      if (left <= 0) return;
      b = c->b0, g = c->off_g, rt = c->off_rt, t0 = c->off_t;
      s = load_seq(p, b, false);
      t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), t0 + left));
      on = true;
    } else {
      item = blockIdx.x;
      next_item(p);
    }
  }
  __device__ __forceinline__ void next(const TreeParams &p) {
    if (!p.shared) {
      next_item(p);
      return;
    }
    left -= t1 - t0;
    on = left > 0;
    if (!on) return;
    t0 = 0;
    if (++rt == s.row_tiles) {
      rt = 0;
      if (++g == p.hkv) {
        g = 0;
        do {
          s = load_seq(p, ++b, false);
        } while (s.lq == 0);  // tiles are left, so a sequence with rows follows
      }
    }
    t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), left));
  }
  __device__ __forceinline__ void next_item(const TreeParams &p) {
    const int rt_max = ceil_div(p.max_q * p.group, kRows);
    const int64_t items = static_cast<int64_t>(p.batch) * p.hkv * rt_max;
    on = false;
    for (; item < items && !on; item += gridDim.x) {
      const int64_t pair = item / rt_max;
      rt = static_cast<int>(item - pair * rt_max);
      b = static_cast<int>(pair / p.hkv);
      g = static_cast<int>(pair - static_cast<int64_t>(b) * p.hkv);
      s = load_seq(p, b, false);
      on = rt < s.row_tiles;
    }
    t0 = 0, t1 = s.tiles;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == s.tiles; }
};

// This CTA's share of the line of tiles. Every thread counts the tiles of a run of
// sequences; the one whose run holds the share's first tile finds its place.
__device__ __forceinline__ void find_share(const TreeParams &p, Ctl *c) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int per = ceil_div(p.batch, kThreads);
  const int b0 = min(static_cast<int>(threadIdx.x) * per, p.batch), b1 = min(b0 + per, p.batch);
  int64_t mine = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const Seq s = load_seq(p, b, blockIdx.x == 0);
    mine += static_cast<int64_t>(s.tiles) * s.row_tiles * p.hkv;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) c->sums[wid] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < wid) before += c->sums[w];
    total += c->sums[w];
  }
  const int64_t share = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(p.min_share));
  const int64_t begin = min(blockIdx.x * share, total), end = min(begin + share, total);
  if (threadIdx.x == 0) c->begin = begin, c->end = end, c->share = share;
  if (begin < end && before <= begin && begin < before + mine) {
    int64_t at = begin - before;
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq(p, b, false);
      const int64_t n = static_cast<int64_t>(s.tiles) * s.row_tiles * p.hkv;
      if (at < n) {
        const int64_t head = static_cast<int64_t>(s.tiles) * s.row_tiles;
        c->b0 = b;
        c->off_g = static_cast<int>(at / head);
        at -= c->off_g * head;
        c->off_rt = static_cast<int>(at / s.tiles);
        c->off_t = static_cast<int>(at - static_cast<int64_t>(c->off_rt) * s.tiles);
        break;
      }
      at -= n;
    }
  }
}

// 32 scores -> 2^(x c - m), split into bf16 halves hi + lo, as 16 pairs each; row sums
// (of the unsplit values) into acc. hi is cut off, not rounded (its pair is one byte
// permutation of the values themselves), lo rounds the rest: hi + lo is 2^-16 from the value
// at most, far below the bf16 output's own 2^-8. (hi rounded: 2^-17, 176 -> 182 us on 64
// sequences of 1k to 8k keys.)
__device__ __forceinline__ void exp32(const float (&sv)[32], float2 c2, float2 nb2,
                                      float2 (&acc)[2], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 a = __ffma2_rn(make_float2(sv[2 * i], sv[2 * i + 1]), c2, nb2);
    const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
    acc[i & 1] = __fadd2_rn(acc[i & 1], e);
    const uint32_t ux = __float_as_uint(e.x), uy = __float_as_uint(e.y);
    hi[i] = __byte_perm(ux, uy, 0x7632);
    const float2 cut = make_float2(__uint_as_float(ux & 0xffff0000u), __uint_as_float(uy & 0xffff0000u));
    const float2 left = __ffma2_rn(cut, make_float2(-1.f, -1.f), e);
    lo[i] = pack_bf16x2(left.x, left.y);
  }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max32(const float (&s)[32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(s[8 * i], s[8 * i + 1], s[8 * i + 2]);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(m[i], s[8 * i + 3], s[8 * i + 4]);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(m[i], s[8 * i + 5], s[8 * i + 6]);
  return max3(max3(m[0], s[7], s[15]), max3(m[1], s[23], s[31]), fmaxf(m[2], m[3]));
}
__device__ __forceinline__ void hide32(float (&s)[32], uint32_t visible) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!(visible & (1u << i))) s[i] = -INFINITY;
}
// Bits [a, b) of a 64-bit word (either may lie outside).
__device__ __forceinline__ uint64_t bits(int a, int b) {
  a = max(a, 0), b = min(b, 64);
  if (a >= b) return 0;
  return (~0ull >> (64 - (b - a))) << a;
}

// The parent of row i, -1 without one (or with one that is not below it).
__device__ __forceinline__ int parent_of(const int32_t *parents, int i) {
  if (parents == nullptr) return i - 1;
  const int x = __ldg(parents + i);
  if (x >= i || x < -1) {
    atomicExch(&g_tree_error, kErrBadPage);
    return -1;
  }
  return x;
}

// The keys (bit = key of the tile that starts at key0) that row `tok` sees: those of the
// context from lo on, its ancestors within the window, itself.
__device__ __forceinline__ uint64_t visible_keys(const int32_t *parents, int tok, int lo,
                                                 int context, int key0, int window) {
  uint64_t vis = bits(lo - key0, context - key0);
  if (key0 + kKeys <= context) return vis;
  if (window <= 0) window = INT32_MAX;  // ancestors that are near enough
  if (parents == nullptr) {
    const int from = tok >= window ? tok - window + 1 : 0;
    return vis | bits(context + from - key0, context + tok + 1 - key0);
  }
  for (int i = tok; i >= 0 && window > 0; i = parent_of(parents, i), --window) {
    const int k = context + i - key0;
    if (k < 0) break;  // ancestors come before
    if (k < kKeys) vis |= 1ull << k;
  }
  return vis;
}

// Both halves of a packed pair that are infinite or NaN, as 0xffff each.
__device__ __forceinline__ uint32_t not_finite2(uint32_t x) {
  return (((x & 0x7f807f80u) + 0x00800080u) >> 15 & 0x00010001u) * 0xffffu;
}
__device__ __forceinline__ uint4 not_finite8(const uint4 &x) {
  return make_uint4(not_finite2(x.x), not_finite2(x.y), not_finite2(x.z), not_finite2(x.w));
}

// The first key of the context that row `tok` sees.
__device__ __forceinline__ int first_key(const int32_t *parents, int tok, int context, int window) {
  if (window <= 0) return 0;
  int depth = tok;
  if (parents != nullptr) {
    depth = 0;
    for (int i = parent_of(parents, tok); i >= 0; i = parent_of(parents, i)) ++depth;
  }
  return window - 1 <= context + depth ? context + depth - (window - 1) : 0;
}

// Whether one of 32 elements is not finite: 0 x + 0 x' .. tells.
__device__ __forceinline__ bool any_not_finite(const float (&o)[32]) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 32; e += 2)
    s = __ffma2_rn(make_float2(o[e], o[e + 1]), make_float2(0.f, 0.f), s);
  return s.x + s.y != 0.f;
}

// Whether some row of the sequence hides a key of the tile that another sees.
__device__ __forceinline__ bool mixed(const Seq &s, int key0, int window) {
  return s.lq > 1 && (key0 + kKeys > s.lk - s.lq || (window > 0 && key0 < s.lk - window));
}

// Makes the elements of a slot of values that are not finite zeros (called by a warp): with
// the weight 0 of a row that hides their key they would be NaN.
template <int D>
__device__ __forceinline__ void clear_values(uint8_t *slot) {
  uint4 *v = reinterpret_cast<uint4 *>(slot);
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < Cfg<D>::kSlotBytes / 16; i += 32) {
    const uint4 x = v[i], m = not_finite8(x);
    v[i] = make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
  }
}

// Values that are not finite: one of a key that some row hides and another sees reaches the
// row that hides it as 0 * NaN. So where a CTA's results are not all finite it walks its
// segments a second time, with such values set to zero in the tiles that some row sees only
// in part (clear_values), and then adds them to the results of the rows that see
// them (their weights are positive, so the values themselves will do). Thread r: row r of
// each segment, as in the softmax. (Looking every such tile over in the first walk: 50 -> 54 us
// on 256 sequences of window 128; noticing it in the results 50.4.)
template <int D>
__device__ __forceinline__ void put_values(const TreeParams &p, const Ctl *c) {
  Walk w;
#pragma unroll 1
  for (w.start(p, c); w.on; w.next(p)) {
    const int at = w.rt * kRows + threadIdx.x, context = w.s.lk - w.s.lq;
    if (at >= w.s.lq * p.group) continue;
    const int tok = at / p.group, h = w.g * p.group + (at - tok * p.group);
    const int32_t *parents = p.parents != nullptr ? p.parents + w.s.first : nullptr;
    const int32_t *table = p.table + static_cast<int64_t>(w.b) * p.max_pages;
    const int lo = first_key(parents, tok, context, p.window);
    __nv_bfloat16 *out = p.out + (static_cast<size_t>(w.s.first + tok) * p.hq + h) * D;
    float *part = p.part_o + ((2 * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * static_cast<size_t>(kRows) +
                              threadIdx.x) * D;
#pragma unroll 1
    for (int t = w.t0; t < w.t1; ++t) {
      const int key0 = w.s.lo + t * kKeys;
      if (!mixed(w.s, key0, p.window)) continue;
      const uint64_t vis = visible_keys(parents, tok, lo, context, key0, p.window);
#pragma unroll 1
      for (int k = 0; k < kKeys; ++k) {
        if (!(vis >> k & 1)) continue;
        const int pos = key0 + k, pg = pos / p.page_size, page = table[pg];
        if (page < 0 || page >= p.num_pages) continue;
        const __nv_bfloat16 *v = p.v + ((static_cast<int64_t>(page) * p.hkv + w.g) * p.page_size +
                                        (pos - pg * p.page_size)) * D;
#pragma unroll 1
        for (int i = 0; i < D; i += 8) {
          const uint4 x = *reinterpret_cast<const uint4 *>(v + i), m = not_finite8(x);
          if ((m.x | m.y | m.z | m.w) == 0) continue;
#pragma unroll 1
          for (int e = i; e < i + 8; ++e) {
            const float f = __bfloat162float(v[e]);
            if (fabsf(f) <= FLT_MAX) continue;
            if (w.whole())
              out[e] = __float2bfloat16(__bfloat162float(out[e]) + f);
            else
              part[e] += f;
          }
        }
      }
    }
  }
}

// One walk of a CTA through its segments, every warp in its role. The groups, steps and
// segments that a role has come past, and with them the barriers' phases, go on from the
// first walk to the second.
struct Past {
  int grp, j, seg;
};

template <int D, bool kSecond>
__device__ __forceinline__ void walk(const TreeParams &p, Ctl *c, uint8_t *smem, uint32_t tmem,
                                     Past &past) {
  using C = Cfg<D>;
  constexpr int kSlots = C::kSlots;
  const uint32_t sbase = smem_u32(smem);
  volatile int *abort = &c->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int grp = past.grp, j = past.j, seg = past.seg;
  Walk w;
  w.start(p, c);

  if (warp >= kProducerWarp) {
    // -------------------------------------------------------------- producers
    const int tid = threadIdx.x - kProducerWarp * 32;
    constexpr int kVecs = D / 8;             // 16-byte vectors of a row
    constexpr int kPer = 32 / kVecs;         // rows that a warp copies at a time
    const int vec = lane % kVecs, sub = lane / kVecs;
    const int col = (vec / 8) * (kKeys * 128);  // block of 64 elements within a slot
    bool ok = true;
    // row of the cache (of head g) that holds the key `pos`, ~0 for none
    auto find_row = [&](int page, int pos) -> uint32_t {
      const int pg = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
      return (static_cast<uint32_t>(page) * p.hkv + w.g) * p.page_size + (pos - pg * p.page_size);
    };
    auto find_page = [&](int pos) -> int {
      const int pg = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
      return pos < w.s.lk ? __ldg(p.table + static_cast<int64_t>(w.b) * p.max_pages + pg) : -1;
    };
    // K and V of one step, row by row side by side
    auto copy = [&](uint32_t row) -> bool {
      const int ks = grp % kSlots, vs = (grp + 1) % kSlots;
      if (grp >= kSlots &&
          !mbar_wait_warp(&c->empty[ks], ((grp / kSlots) - 1) & 1, abort, &g_tree_error))
        return false;
      if (grp + 1 >= kSlots &&
          !mbar_wait_warp(&c->empty[vs], (((grp + 1) / kSlots) - 1) & 1, abort, &g_tree_error))
        return false;
      const int r0 = (warp - kProducerWarp) * 32 + sub;
      const uint32_t ring = sbase + C::kOffRing + col + r0 * 128;
      const uint32_t kdst = ring + ks * C::kSlotBytes, vdst = ring + vs * C::kSlotBytes;
#pragma unroll 8
      for (int i = 0; i < 32; i += kPer) {
        const uint32_t at = __shfl_sync(0xffffffffu, row, i + sub);
        const uint32_t n = at == ~0u ? 0u : 16u;
        const size_t off = static_cast<size_t>(at == ~0u ? 0 : at) * D + vec * 8;
        const uint32_t to = i * 128 + (((vec & 7) ^ ((r0 + i) & 7)) << 4);
        cp_async_16(kdst + to, p.k + off, n);
        cp_async_16(vdst + to, p.v + off, n);
      }
      cp_async_mbar_arrive_noinc(&c->full[ks]);
      cp_async_mbar_arrive_noinc(&c->full[vs]);
      grp += 2;
      return true;
    };
    // Q of the segment, once the last Q K^T of the one before has read its own
    auto load_q = [&]() {
      if (seg > 0 && !mbar_wait_warp(&c->q_empty, (seg - 1) & 1, abort, &g_tree_error)) return false;
      const int rows = w.s.lq * p.group;
      // rows tid / kVecs, + kProducers / kVecs, ..: (token, head) without a division for each
      constexpr int kStep = kProducers / kVecs;
      const int qv = tid % kVecs, qcol = (qv / 8) * (kRows * 128);
      int r = tid / kVecs;
      int tok = (w.rt * kRows + r) / p.group, hh = w.rt * kRows + r - tok * p.group;
      const int up_tok = kStep / p.group, up_h = kStep - up_tok * p.group;
#pragma unroll 4
      for (int i = 0; i < kRows / kStep; ++i, r += kStep) {
        const bool there = w.rt * kRows + r < rows;
        const size_t src = (static_cast<size_t>(w.s.first + tok) * p.hq + w.g * p.group + hh) * D +
                           qv * 8;
        cp_async_16(sbase + qcol + r * 128 + (((qv & 7) ^ (r & 7)) << 4), p.q + (there ? src : 0),
                    there ? 16u : 0u);
        tok += up_tok, hh += up_h;
        if (hh >= p.group) hh -= p.group, ++tok;
      }
      cp_async_mbar_arrive_noinc(&c->q_full);
      return true;
    };
    for (; ok && w.on; w.next(p), ++seg) {
      const int base = w.s.lo + w.t0 * kKeys + tid;
      const int n = w.t1 - w.t0;
      int page = find_page(base);
#pragma unroll 1
      for (int t = 0; ok && t < n; ++t) {
        const int pos = base + t * kKeys;
        uint32_t row = ~0u;
        if (pos < w.s.lk) {
          if (page >= 0 && page < p.num_pages)
            row = find_row(page, pos);
          else
            atomicExch(&g_tree_error, kErrBadPage);
        }
        if (t + 1 < n) page = find_page(pos + kKeys);
        __syncwarp();
        ok = copy(row);
        // behind the first two tiles, whose slots become free without this Q
        if (ok && t == min(n, 2) - 1) ok = load_q();
      }
    }
    cp_async_wait<0>();  // nothing is in flight when the CTA ends
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------ Q K^T issuer
    // Step J's S is issued once P V of step J - 2, whose P lies in the same buffer, has
    // completed. cp.async writes through the generic proxy: a fence follows each wait
    // for them before the tensor core reads. (One warp for both products took 1.9 k cycles
    // a step, most of it the issue of one after the other.)
    const uint64_t qdesc = sdesc_sw128(sbase);
    const uint64_t rdesc = sdesc_sw128(sbase + C::kOffRing);
    constexpr uint64_t kSlotDesc = C::kSlotBytes >> 4;
    bool ok = true;
    for (; ok && w.on; w.next(p), ++seg) {
      ok = mbar_wait_warp(&c->q_full, seg & 1, abort, &g_tree_error);
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++j) {
        const int buf = j & 1, grp = 2 * j, slot = grp % kSlots;
        ok = mbar_wait_warp(&c->full[slot], (grp / kSlots) & 1, abort, &g_tree_error) &&
             (j < 2 || mbar_wait_warp(&c->pv_done[buf], ((j - 2) >> 1) & 1, abort, &g_tree_error));
        if (!ok) break;
        fence_proxy_async();
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)  // 16 dims: block ks / 4, 32-byte step ks % 4
          umma_ss_elect(tmem + buf * kKeys, qdesc + (ks >> 2) * (kRows * 128 >> 4) + 2 * (ks & 3),
                        rdesc + slot * kSlotDesc + (ks >> 2) * (kKeys * 128 >> 4) + 2 * (ks & 3),
                        kIdescQK, ks > 0 ? 1u : 0u);
        umma_commit_elect(&c->s_full[buf]);
        umma_commit_elect(&c->empty[slot]);
      }
      if (ok) umma_commit_elect(&c->q_empty);
    }
    // every product issued has finished before TMEM is released
    umma_commit_elect(&c->drain[0]);
    mbar_wait_warp(&c->drain[0], kSecond, abort, &g_tree_error, true);
  } else if (warp == kPvWarp) {
    // -------------------------------------------------------------- P V issuer
    const uint64_t rdesc = sdesc_sw128(sbase + C::kOffRing);
    constexpr uint64_t kSlotDesc = C::kSlotBytes >> 4;
    bool ok = true;
    for (; ok && w.on; w.next(p), ++seg) {
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++j) {
        const int buf = j & 1, grp = 2 * j + 1, slot = grp % kSlots;
        ok = mbar_wait_warp(&c->full[slot], (grp / kSlots) & 1, abort, &g_tree_error);
        if (!ok) break;
        if (kSecond && mixed(w.s, w.s.lo + t * kKeys, p.window))
          clear_values<D>(smem + C::kOffRing + slot * C::kSlotBytes);
        ok = (t > w.t0 || seg == 0 ||
              mbar_wait_warp(&c->o_free, (seg - 1) & 1, abort, &g_tree_error)) &&
             mbar_wait_warp(&c->p_full[buf], (j >> 1) & 1, abort, &g_tree_error);
        if (!ok) break;
        fence_proxy_async();
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half)  // the halves of P
#pragma unroll
          for (int hb = 0; hb < D / 64; ++hb)
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              umma_ts_elect(tmem + C::kTmemO + hb * 64,
                            tmem + buf * kKeys + half * (kKeys / 2) + kk * 8,
                            rdesc + slot * kSlotDesc + hb * (kKeys * 128 >> 4) + kk * (16 * 128 / 16),
                            kIdescPV, (t > w.t0 || half > 0 || kk > 0) ? 1u : 0u);
        umma_commit_elect(&c->pv_done[buf]);
        umma_commit_elect(&c->empty[slot]);
      }
      // A value that is not finite leaves no row of its column finite, whoever sees it: this
      // warp's 32 rows tell, and it has the time of the epilogue for them.
      if (ok && !kSecond && (mixed(w.s, w.s.lo + w.t0 * kKeys, p.window) ||
                             mixed(w.s, w.s.lo + (w.t1 - 1) * kKeys, p.window))) {
        ok = mbar_wait_warp(&c->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort, &g_tree_error);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          tmem_ld32f(tmem + C::kTmemO + i * 32, o);
          tmem_wait_ld();
          if (any_not_finite(o)) c->odd = 1;
        }
        __syncwarp();
      }
    }
    umma_commit_elect(&c->drain[1]);
    mbar_wait_warp(&c->drain[1], kSecond, abort, &g_tree_error, true);
  } else {
    // ---------------------------------------------------------------- softmax
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t o_addr = lane_addr + C::kTmemO;
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    bool ok = p.stall_ns == 0 ||
              __all_sync(0xffffffffu,
                         mbar_wait(&c->never, 0, abort, &g_tree_error, false, p.stall_ns));
    Header head{0, 0, 0, 0};
    for (; ok && w.on; w.next(p)) {
      const int at = w.rt * kRows + threadIdx.x;  // row of the item: (drafted token, head)
      const int rows = w.s.lq * p.group;
      const bool mine = at < rows;
      const bool warp_on = w.rt * kRows + warp * 32 < rows;  // some row of this warp is one
      const int tok = at / p.group, h = w.g * p.group + (at - tok * p.group);
      const int context = w.s.lk - w.s.lq;
      const int32_t *parents = p.parents != nullptr ? p.parents + w.s.first : nullptr;
      const int lo = mine ? first_key(parents, tok, context, p.window) : 0;
      float m = -INFINITY, d = 0.f;
      if (w.t0 == 0 && p.sinks != nullptr && mine) {
        const float sink = p.sinks[h];
        m = fminf(fmaxf(sink * kLog2e, -FLT_MAX), FLT_MAX);
        d = sink == sink ? 1.f : sink;  // a NaN stays one in d, whatever the maximum
      }
      const int n = w.t1 - w.t0;
      for (int t = 0; t < n; ++t, ++j) {
        const int buf = j & 1;
        const uint32_t s_addr = lane_addr + buf * kKeys;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&c->s_full[buf], (j >> 1) & 1, abort, &g_tree_error))) {
          ok = false;
          break;
        }
        const int key0 = w.s.lo + (w.t0 + t) * kKeys;
        const bool tail = key0 + kKeys > context;
        if (!warp_on) {  // rows that are none: their P is not read by any other
          arrive(&c->p_full[buf]);
          continue;
        }
        tc_fence_after();
        uint64_t vis = ~0ull;
        if (tail || __any_sync(0xffffffffu, key0 < lo)) {
          vis = mine ? visible_keys(parents, tok, lo, context, key0, p.window) : 0;
          __syncwarp();
        }
        const bool hide = __any_sync(0xffffffffu, vis != ~0ull);
        float s0[32], s1[32];
        tmem_ld32f(s_addr, s0);
        tmem_ld32f(s_addr + 32, s1);
        tmem_wait_ld();
        if (hide) {
          hide32(s0, static_cast<uint32_t>(vis));
          hide32(s1, static_cast<uint32_t>(vis >> 32));
        }
        const float m_new = fmaxf(m, fmaxf(max32(s0), max32(s1)) * p.scale_log2);
        float alpha = 1.f;
        if (m_new > m + kRescaleThreshold) {
          alpha = fast_exp2(m - m_new);
          d *= alpha;
          m = m_new;
        }
        const float base = m == -INFINITY ? 0.f : m;
        const float2 nb2 = make_float2(-base, -base);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // P's halves replace S: hi in columns [0, 32), lo in [32, 64)
        uint32_t hi[16], lw[16];
        exp32(s0, c2, nb2, acc, hi, lw);
        tmem_st16(s_addr, hi);
        tmem_st16(s_addr + kKeys / 2, lw);
        exp32(s1, c2, nb2, acc, hi, lw);
        tmem_st16(s_addr + 16, hi);
        tmem_st16(s_addr + kKeys / 2 + 16, lw);
        const float2 sum = __fadd2_rn(acc[0], acc[1]);
        d += sum.x + sum.y;
        tmem_wait_st();
        // O holds the products up to step j - 1, which must be complete before it is rescaled.
        // S of step j was issued after P V of step j - 2 had completed, so the wait's
        // phase is the present one or the next.
        if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!__all_sync(0xffffffffu, mbar_wait(&c->pv_done[buf ^ 1], ((j - 1) >> 1) & 1, abort,
                                                 &g_tree_error))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(o_addr + i * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(o_addr + i * 32, o);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        arrive(&c->p_full[buf]);
      }
      if (!ok) break;
      // ------------------------------------------------------------- epilogue
      if (!__all_sync(0xffffffffu, mbar_wait(&c->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort,
                                             &g_tree_error))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (w.whole()) {
        if (warp_on) {
          const float inv = d == 0.f ? 0.f : 1.f / d;
          const size_t row = static_cast<size_t>(w.s.first + tok) * p.hq + h;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(o_addr + i * 32, o);
            tmem_wait_ld();
            if (mine) {
              uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * D + i * 32);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float *f = reinterpret_cast<const float *>(&o[8 * e]);
                dst[e] = make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv),
                                    pack_bf16x2(f[2] * inv, f[3] * inv),
                                    pack_bf16x2(f[4] * inv, f[5] * inv),
                                    pack_bf16x2(f[6] * inv, f[7] * inv));
              }
            }
          }
          if (mine && p.lse != nullptr) {
            float lse = d == 0.f ? -INFINITY : (m + fast_log2(d)) * kLn2;
            // a sink beyond log2 units: it alone counts
            if (fabsf(m) == FLT_MAX && d == d) lse = p.sinks[h];
            p.lse[row] = lse;
          }
        }
      } else {
        const int part = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
        if (w.t0 == 0 && threadIdx.x == 0) {  // the item goes on in the shares behind this one
          const int64_t first = c->end - w.left;  // its first tile's place in the line
          head.parts = static_cast<int>((first + w.s.tiles - 1) / c->share - blockIdx.x) + 1;
          head.b = w.b, head.g = w.g, head.rt = w.rt;
        }
        if (warp_on) {
          const size_t row = static_cast<size_t>(part) * kRows + threadIdx.x;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(o_addr + i * 32, o);
            tmem_wait_ld();
            uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + row * D + i * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          p.part_md[row] = make_float2(m, d);
        }
      }
      tc_fence_before();
      arrive(&c->o_free);
    }
    if (p.shared && threadIdx.x == 0) p.headers[blockIdx.x] = head;
  }
  past.grp = grp, past.j = j, past.seg = seg;
}

// (Not inlined: within the kernel's own code it slowed the first walk's loops, 178 -> 183 us
// on 64 sequences of 1k to 8k keys.)
template <int D>
__device__ __noinline__ void second_walk(const TreeParams &p, Ctl *c, uint8_t *smem, uint32_t tmem,
                                         Past past) {
  tc_fence_after();
  walk<D, true>(p, c, smem, tmem, past);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < kRows) put_values<D>(p, c);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) tree_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl *c = reinterpret_cast<Ctl *>(smem + C::kOffCtl);
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&c->full[i], kProducers);
      mbar_init(&c->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->s_full[i], 1);
      mbar_init(&c->p_full[i], kSoftmaxWarps);
      mbar_init(&c->pv_done[i], 1);
    }
    mbar_init(&c->q_full, kProducers);
    mbar_init(&c->q_empty, 1);
    mbar_init(&c->o_free, kSoftmaxWarps);
    mbar_init(&c->drain[0], 1);
    mbar_init(&c->drain[1], 1);
    mbar_init(&c->never, 1);
    c->abort = 0;
    c->odd = 0;
    fence_mbar_init();
  }
  if (warp == kPvWarp) {
    tmem_alloc(&c->tmem, C::kTmemCols);
    tmem_relinquish();
  }
  if (p.shared) {
    find_share(p, c);
  } else if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.batch; b += kThreads) load_seq(p, b, true);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  Past past{0, 0, 0};
  walk<D, false>(p, c, smem, tmem, past);
  tc_fence_before();
  __syncthreads();
  if (c->odd && !c->abort) second_walk<D>(p, c, smem, tmem, past);  // the whole block or none
  if (warp == kPvWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of the item that starts in share blockIdx.x and goes on behind it:
// O = sum_k 2^(m_k - M) O_k over sum_k 2^(m_k - M) d_k. A row's D elements take D / 4
// threads. Reads (4 D + 8) bytes per row and part, from L2 as a rule.
template <int D>
__global__ void __launch_bounds__(512) tree_merge_kernel(const TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kCols = D / 4, kPerBlock = 512 / kCols;
  const Header head = p.headers[blockIdx.x];
  if (head.parts == 0) return;
  const int r = blockIdx.y * kPerBlock + threadIdx.x / kCols, col = threadIdx.x % kCols;
  const Seq s = load_seq(p, head.b, false);
  const int at = head.rt * kRows + r;
  if (at >= s.lq * p.group) return;
  // part k: slot 1 of the first share, slot 0 of those behind it
  const auto row = [&](int k) {
    return (2 * (static_cast<size_t>(blockIdx.x) + k) + (k == 0 ? 1 : 0)) * kRows + r;
  };
  float M = -INFINITY;
#pragma unroll 8
  for (int k = 0; k < head.parts; ++k) M = fmaxf(M, p.part_md[row(k)].x);
  // no part has a maximum: nothing visible, or scores that are all NaN, which stay so
  const float base = M == -INFINITY ? 0.f : M;
  float W = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < head.parts; ++k) {
    const float2 md = p.part_md[row(k)];
    const float4 x = *reinterpret_cast<const float4 *>(p.part_o + row(k) * D + 4 * col);
    const float f = fast_exp2(md.x - base);
    W = fmaf(f, md.y, W);
    o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;
  const int tok = at / p.group, h = head.g * p.group + (at - tok * p.group);
  const size_t to = static_cast<size_t>(s.first + tok) * p.hq + h;
  *reinterpret_cast<uint2 *>(p.out + to * D + 4 * col) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (col == 0 && p.lse != nullptr) {
    float lse = W == 0.f ? -INFINITY : (M + fast_log2(W)) * kLn2;
    if (fabsf(M) == FLT_MAX && W == W) lse = p.sinks[h];
    p.lse[to] = lse;
  }
}

// testing hook (sinkattn_debug_stall_waits): stall_ns of later launches
std::atomic<uint64_t> g_stall_ns{0};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }
size_t headers_bytes(const DecodeTreePlan &plan) { return round256(plan.blocks * sizeof(Header)); }
size_t md_bytes(const DecodeTreePlan &plan) {
  return static_cast<size_t>(plan.blocks) * 2 * kRows * sizeof(float2);
}

}  // namespace

DecodeTreePlan plan_decode_tree(int batch, int max_seqlen_q, int max_seqlen_k, int hq, int hkv,
                                int, int window, int num_splits) {
  const int64_t rows = static_cast<int64_t>(max_seqlen_q) * (hq / hkv);
  const int64_t items = static_cast<int64_t>(batch) * hkv * ((rows + kRows - 1) / kRows);
  int64_t seen = max_seqlen_k;
  if (window > 0 && seen > static_cast<int64_t>(window) - 1 + max_seqlen_q)
    seen = static_cast<int64_t>(window) - 1 + max_seqlen_q;
  const int64_t tiles = seen > kKeys ? (seen + kKeys - 1) / kKeys : 1;
  DecodeTreePlan plan;
  plan.shared = num_splits != 1 && batch <= kMaxShared && tiles > kWholeTiles;
  // of the bound's tiles: shares of a batch far below it are longer than they need be
  const int64_t most = (tiles + kMaxParts - 1) / kMaxParts;
  plan.min_share = static_cast<int>(most > 2 ? most : 2);
  int64_t blocks = items;
  // (more than kBlocks items or tiles: no product needed, which might overflow)
  if (plan.shared && items < kBlocks)
    blocks = (items * tiles + plan.min_share - 1) / plan.min_share;
  plan.blocks = static_cast<int>(blocks < kBlocks ? blocks : kBlocks);
  return plan;
}

size_t decode_tree_workspace_bytes(const DecodeTreePlan &plan, int head_dim) {
  if (!plan.shared) return 0;
  return headers_bytes(plan) + md_bytes(plan) +
         static_cast<size_t>(plan.blocks) * 2 * kRows * head_dim * sizeof(float);
}

cudaError_t launch_decode_tree(const DecodeTreeLaunch &a, cudaStream_t stream) {
  TreeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v);
  if (p.k == nullptr) p.k = p.v = p.q;  // no pages: only zero-filled copies, which read nothing
  p.cu_q = a.cu_q, p.parents = a.parents, p.table = a.block_table, p.seqlens_k = a.seqlens_k;
  p.num_pages = a.num_pages, p.max_pages = a.max_pages, p.page_size = a.page_size;
  p.page_shift = -1;
  if ((a.page_size & (a.page_size - 1)) == 0)
    for (p.page_shift = 0; (1 << p.page_shift) < a.page_size;) ++p.page_shift;
  p.batch = a.batch, p.max_q = a.max_seqlen_q, p.max_k = a.max_seqlen_k;
  p.hq = a.hq, p.hkv = a.hkv, p.group = a.hq / a.hkv, p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.shared = a.plan.shared, p.min_share = a.plan.min_share;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  p.headers = reinterpret_cast<Header *>(ws);
  p.part_md = reinterpret_cast<float2 *>(ws + headers_bytes(a.plan));
  p.part_o = reinterpret_cast<float *>(ws + headers_bytes(a.plan) + md_bytes(a.plan));
  p.stall_ns = g_stall_ns.load(std::memory_order_relaxed);
  const unsigned blocks = static_cast<unsigned>(a.plan.blocks);
  const auto go = [&](auto kernel, auto merge, int smem, int merge_rows) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, kThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !a.plan.shared) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks, kRows / merge_rows);
    cfg.blockDim = dim3(512);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge, p);
  };
  return a.head_dim == 128
             ? go(tree_kernel<128>, tree_merge_kernel<128>, Cfg<128>::kSmemBytes, 512 / 32)
             : go(tree_kernel<64>, tree_merge_kernel<64>, Cfg<64>::kSmemBytes, 512 / 16);
}

cudaError_t decode_tree_read_error(cudaStream_t stream, int *code) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_tree_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(int));
  return e;
}

cudaError_t decode_tree_set_stall(uint64_t ns) {
  g_stall_ns.store(ns, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace sinkattn
