// Split-KV decode over a paged fp8 cache with one scale per (block of tokens,
// KV head): one query token per sequence.
//
// Page "GPT-OSS on day 0": the model is served with FP8; page "Fast embeddings
// on GPUs", section "ROSE": paged decode. With key j of block c(j) standing for
// ks_c * e4m3(k_j) and value j for vs_c * e4m3(v_j):
//
//   x_j = scale * ks_c(j) * <q, code(k_j)>
//   out = sum_j e^{x_j} vs_c(j) code(v_j) / (e^{sink} + sum_j e^{x_j})
//
// The value scale changes from block to block inside one P V product, so it
// multiplies P before P is rounded to fp16: w_j = p_j vs_c(j). The running
// reference of the online softmax is therefore r = max_j (x_j + log2 vs_c(j))
// (log2 units), moved only when a score passes it by 2^8: every w_j = 2^(x_j - r) vs
// is at most 2^8 and the largest is near or above 1, so fp16 keeps 11 bits of the
// weights that matter whatever the scales' spread.
// The denominator sums p_j = 2^(x_j - r) in fp32. As the scales lie in [2^-60, 2^60],
// it stays between 2^-60 and 2^68 times the number of keys, and the weights of small
// values count beside large ones although their references differ by up to 2^120 and
// the scores' own distance: a change of reference multiplies by 2^(g / 2) twice, since
// 2^g alone can pass below fp32's range where its product with a sum does not.
// The sink has no value row, so it takes no part in r; it enters the denominator once, where a
// (sequence, KV head)'s first piece is finished, with a maximum of its own.
//
// The unit of work is a slab of 32 tokens (head_dim 64) or 16 (128): a warp
// streams slabs of K and V codes and their scales through its own shared-memory
// ring (TMA, or cp.async row by row), so no block-wide barrier sits in the loop, and
// serves up to 8 query heads of a KV head from one read of each byte with mma.sync. Bound by
// the HBM traffic of the cache. Three ways to spread the slabs over the GPU:
//
//  pairs    many short spans: one warp per (sequence, KV head), no barrier.
//  cluster  few (sequence, KV head) pairs: the pieces of a pair are the blocks of
//           one thread-block cluster, which merge their states through it, with no
//           scratch memory and no second launch.
//  flat     everything else: the slabs of all pairs in one line, cut into equal
//           ranges, one per resident block, so that no block waits for a longer
//           one and the ring runs on from one pair into the next. Pairs that a
//           range border cuts leave partials, which a second kernel merges.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "launch.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace sinkattn {
namespace {

__device__ int g_decode_block_error;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxGroup = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMinVScale = 8.673617379884035e-19f;  // 2^-60: bound of the reference only
constexpr int64_t kMaxKeys = INT32_MAX - 65536;  // keeps the key arithmetic within int
constexpr int kBlocksPerSm = 4;  // pairs and cluster kernels
constexpr int kMaxCluster = 16;  // blocks of a cluster, at most
// Pieces up to this long (tokens) go to clusters or unsplit blocks: 256 windows of
// 1024 tokens 53 us (flat 57), 8 pairs of 16k tokens in 16 pieces 12.2 us (flat
// 13.5); one 32768-token context in 16 pieces of 2048 18.7 us (flat 16.2), 256
// contexts of 1k-8k unsplit 206 us (flat 198).
constexpr int kClusterChunk = 1280;
constexpr int kMaxFlatBatch = 4096;
constexpr int kSms = 152;
constexpr float kSlack = 8.f;  // log2

// Spans up to this long take one warp per pair. It needs more pairs than there are
// resident blocks: a 128-token window takes 6.9 us with 800 pairs (blocks 8.0), 8.1
// with 1280 (11.2), 9.5 with 2048 (15.3), but with 64 pairs a third more than blocks;
// 512 tokens 20.2 us with 1280 pairs (20.3), 29.2 with 2048 (32.0), but with 800 a
// twelfth more than blocks.
constexpr int pair_max_span(int64_t pairs) {
  return pairs >= 2 * kSms * kBlocksPerSm ? 512 : pairs > kSms * kBlocksPerSm ? 128 : 0;
}

// Shared memory of a block: per warp a ring of stages (K codes, V codes of one
// slab) and as many buffers of scales, the rings' barriers, and in the flat kernel
// buffers of query rows.
template <int D, int kDepth = 3>
struct Cfg {
  static constexpr int kStages = kDepth;
  static constexpr int kSlab = D == 64 ? 32 : 16;  // tokens per warp step
  static constexpr int kMT = kSlab / 16;           // 16-token m-tiles
  static constexpr int kKS = D / 16;               // k-steps of Q K^T, dim tiles of P V
  static constexpr int kGroup = kWarps * kSlab;    // tokens per step of a block
  static constexpr int kAhead = 32 / kMT;          // slabs whose page ids one register holds
  static constexpr int kSlabBytes = kSlab * D;
  static constexpr int kStageBytes = 2 * kSlabBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kScaleBytes = kStages * 64 * 4;  // K scales [32], V scales [32] each
  static constexpr int kQBytes = kMaxGroup * D * 2;
  static constexpr int kScaleOff = kWarps * kRingBytes;
  static constexpr int kBarOff = kScaleOff + kWarps * kScaleBytes;
  static constexpr int kSmemBytes = kBarOff + kWarps * kStages * 8;
  static constexpr int kQOff = (kSmemBytes + 127) / 128 * 128;
  static constexpr int kFlatSmemBytes = kQOff + kStages * kQBytes;
  static constexpr int kState = D * kMaxGroup;  // floats of one warp's o of 8 heads
  static_assert(kStageBytes == 4096, "TMA destinations need 1 KB alignment");
  static_assert(kStageBytes >= kState * 4, "a warp's state fits one stage");
  static_assert(kWarps * kRingBytes >= (kWarps + 1) * (kState + 16) * 4, "combine area");
};

// The flat kernel at head_dim 128 needs more than 128 registers for its two
// cursors: three blocks per SM with three stages there (serving batch of 64 contexts
// 109 us, four blocks of two stages 115 us), four with two at 64 (64 us, three
// stages 66 us, five blocks 67 us).
template <int D>
struct Flat : Cfg<D, D == 64 ? 2 : 3> {
  static constexpr int kBlocks = D == 64 ? 4 : 3;
};

struct Params {
  const __nv_bfloat16 *q;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;  // [num_pages, hkv, scales_per_page]
  const int32_t *block_table, *seqlens_k;
  int num_pages, max_pages, page_size, page_shift;  // shift: log2, or -1
  int scale_block, block_shift, scales_per_page;
  int batch, hq, hkv, group, window, chunk, nht;
  const float *sinks;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
  float *part_o, *part_lse;
  int2 *cuts;
  // Testing hook (0: off): each warp that loads by TMA first waits, for at most
  // stall_ns, on a barrier that nothing completes, and so takes its timeout path.
  uint64_t stall_ns;
};


__device__ __forceinline__ int page_index(const Params &p, int j) {
  return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
}
__device__ __forceinline__ int page_slot(const Params &p, int j) {
  return p.page_shift >= 0 ? j & (p.page_size - 1) : j % p.page_size;
}
__device__ __forceinline__ int scale_index(const Params &p, int slot) {
  return p.block_shift >= 0 ? slot >> p.block_shift : slot / p.scale_block;
}
// A page id is checked where it is read: one outside [0, num_pages) is recorded
// and its rows count as zeros.
__device__ __forceinline__ int check_page(const Params &p, int page) {
  if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return page;
  atomicExch(&g_decode_block_error, kErrBadPage);
  return -1;
}

// The visible keys [lo, len) of a sequence, and where its slabs start. A length
// that the block table cannot address is cut to what it can.
struct Span {
  int lo, start, len;
};
template <bool kTile>
__device__ __forceinline__ Span span_of(const Params &p, int b) {
  const int64_t cap = min(static_cast<int64_t>(p.max_pages) * p.page_size, kMaxKeys);
  const int raw = p.seqlens_k[b];
  Span s;
  s.len = raw < 0 ? 0 : raw > cap ? static_cast<int>(cap) : raw;
  if (s.len != raw) atomicExch(&g_decode_block_error, kErrBadLength);
  s.lo = p.window > 0 ? max(0, s.len - p.window) : 0;
  s.start = kTile ? s.lo & ~15 : s.lo;
  return s;
}

// Rows of codes: 16-byte chunks XOR-swizzled by row / 2 (four chunks, head_dim 64)
// or row (eight), free of bank conflicts for the fragment loads.
template <int D>
__device__ __forceinline__ int swz8(int row, int chunk) {
  return row * D + ((chunk ^ (D == 64 ? ((row >> 1) & 3) : (row & 7))) << 4);
}

// kTile: pages and scale blocks are multiples of 16 tokens and slabs start at
// multiples of 16, so each 16-token m-tile lies in one page and one scale block:
// a page id, a pair of scales and one TMA box per K and V serve the whole tile.
// Otherwise every row looks up its own page and scales.
//
// The testing hook's wait (a call: its code stays out of the kernels' own).
__device__ __noinline__ bool stall(uint64_t ns, uint64_t *never, volatile int *abort) {
  if ((threadIdx.x & 31) == 0) {
    mbar_init(never, 1);
    fence_mbar_init();
  }
  __syncwarp();
  return mbar_wait_warp(never, 0, abort, &g_decode_block_error, false, ns);
}

// Feed (kTile): a warp's loads. Lane l holds the page of tile l of the current
// kAhead slabs (slab t0 + l / kMT, tile l % kMT), and the raw id of the tile that
// is 32 further, read while the current ones are used; the scales of those tiles
// go to one of the scale buffers when the batch begins.
template <class C, int D>
struct Feed {
  static constexpr int kStages = C::kStages, kMT = C::kMT;
  uint8_t *ring;    // this warp's stages
  float *scales;    // [kStages][2][32]
  uint64_t *bars;   // [kStages]
  int pages, next, t0, buf;
  unsigned dirty;   // stages last written through the generic proxy

  __device__ __forceinline__ void init(uint8_t *smem, int warp, int lane) {
    ring = smem + warp * C::kRingBytes;
    scales = reinterpret_cast<float *>(smem + C::kScaleOff + warp * C::kScaleBytes);
    bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff) + warp * kStages;
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) mbar_init(bars + i, 1);
      fence_mbar_init();
    }
    __syncwarp();
    pages = next = -1;
    t0 = 0;
    buf = kStages - 1;
    dirty = 0u;
  }

  // Starts the copy of slab t of a piece into `stage`; its tokens start at slab0,
  // slab t + 1 is `stride` tokens further, and [lo, hi) are visible. fresh: the
  // first slab loaded of its sequence.
  __device__ __forceinline__ void load(const Params &p, const CUtensorMap *tk,
                                       const CUtensorMap *tv, int stage, bool fresh,
                                       const int32_t *table, int t, int slab0, int stride, int g,
                                       int lo, int hi, int lane) {
    if (fresh || t == t0 + C::kAhead) {
      auto ids = [&](int ahead) {
        const int j = slab0 + (ahead + lane / kMT) * stride + 16 * (lane % kMT);
        return j >= 0 && j < hi ? __ldg(table + page_index(p, j)) : 0;
      };
      const int j = slab0 + lane / kMT * stride + 16 * (lane % kMT);
      const int id = fresh ? ids(0) : next;
      next = ids(C::kAhead);
      pages = j >= 0 && j < hi ? check_page(p, id) : -1;
      t0 = t;
      buf = buf + 1 == kStages ? 0 : buf + 1;
      const bool ok = pages >= 0;
      const int64_t at =
          ok ? (static_cast<int64_t>(pages) * p.hkv + g) * p.scales_per_page +
                   scale_index(p, page_slot(p, j))
             : 0;
      const uint32_t dst = smem_u32(scales + buf * 64 + lane);
      cp_async_4(dst, p.k_scale + at, ok ? 4u : 0u);
      cp_async_4(dst + 128, p.v_scale + at, ok ? 4u : 0u);
    }
    const uint32_t kdst = smem_u32(ring) + stage * C::kStageBytes;
    const uint32_t vdst = kdst + C::kSlabBytes;
    const bool whole = slab0 >= lo && slab0 + C::kSlab <= hi;
    int page[kMT];
    bool plain = whole;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      page[mt] = __shfl_sync(0xffffffffu, pages, (t - t0) * kMT + mt);
      plain = plain && page[mt] >= 0;
    }
    if (plain) {
      if (dirty >> stage & 1u) {  // order the earlier copies' writes before the TMA's
        fence_proxy_async();
        __syncwarp();
        dirty &= ~(1u << stage);
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(bars + stage, C::kStageBytes);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          const int row = (page[mt] * p.hkv + g) * p.page_size + page_slot(p, slab0 + 16 * mt);
          tma_load_2d(kdst + mt * 16 * D, tk, bars + stage, 0, row);
          tma_load_2d(vdst + mt * 16 * D, tv, bars + stage, 0, row);
        }
      }
      return;
    }
    if (lane == 0) mbar_arrive_expect_tx(bars + stage, 0);
    if (slab0 >= hi) return;  // nothing there; not computed either
    // a slab with masked rows or a bad page: rows copied one by one or zeroed
    dirty |= 1u << stage;
    constexpr int kCols = D / 16;  // 16-byte chunks per row
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      const int j0 = slab0 + 16 * mt;
      const int64_t off = ((static_cast<int64_t>(max(page[mt], 0)) * p.hkv + g) * p.page_size +
                           page_slot(p, j0)) * D + lane * 16;
#pragma unroll
      for (int r = 0; r < 16 * kCols / 32; ++r) {
        const int row = (r * 32 + lane) / kCols;
        const bool ok = page[mt] >= 0 && j0 + row >= lo && j0 + row < hi;
        const uint32_t at = swz8<D>(16 * mt + row, lane % kCols);
        cp_async_16(kdst + at, p.k + (ok ? off + r * 512 : 0), ok ? 16u : 0u);
        cp_async_16(vdst + at, p.v + (ok ? off + r * 512 : 0), ok ? 16u : 0u);
      }
    }
  }

  // Waits for the copies of the stage (bounded; false after a timeout). The
  // cp.async part is the caller's group.
  __device__ __forceinline__ bool wait(int stage, uint32_t parity, volatile int *abort) const {
    bool ok = false;
    for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bars + stage, parity);
    if (!__all_sync(0xffffffffu, ok))
      return mbar_wait_warp(bars + stage, parity, abort, &g_decode_block_error);
    return true;
  }
  // After a timeout: waits for the copies still in flight, `issued` slabs in all.
  __device__ __forceinline__ void drain(int issued, volatile int *abort) const {
    for (int s = 0; s < kStages && s < issued; ++s)
      mbar_wait_warp(bars + s, (issued - 1 - s) / kStages & 1, abort, &g_decode_block_error, true);
  }
};

// Row-by-row copy of a slab: lane l finds row l's place in the cache, once, and the
// lanes that copy its chunks get it by shuffles; the page id of the row that is
// `stride` tokens further is read meanwhile (next). The scales go to scales [2][32].
template <int D>
__device__ __forceinline__ void load_rows(const Params &p, uint32_t kdst, uint32_t scales,
                                          bool fresh, const int32_t *table, int slab0, int stride,
                                          int g, int hi, int lane, int &next) {
  using C = Cfg<D>;
  constexpr int kCols = D / 16;
  const uint32_t vdst = kdst + C::kSlabBytes;
  auto id_of = [&](int j) {
    return lane < C::kSlab && j >= 0 && j < hi ? __ldg(table + page_index(p, j)) : 0;
  };
  const int j = slab0 + lane;
  const int id = fresh ? id_of(j) : next;
  next = id_of(j + stride);
  const int page = lane < C::kSlab && j < hi ? check_page(p, id) : -1;
  const int slot = page_slot(p, j);
  const int64_t head = static_cast<int64_t>(max(page, 0)) * p.hkv + g;
  const int64_t my_row = page >= 0 ? head * p.page_size + slot : -1;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int idx = r * 32 + lane;
    const int row = idx / kCols, col = idx % kCols;
    const int64_t at = __shfl_sync(0xffffffffu, my_row, row);
    const int64_t off = at >= 0 ? at * D + col * 16 : 0;
    cp_async_16(kdst + swz8<D>(row, col), p.k + off, at >= 0 ? 16u : 0u);
    cp_async_16(vdst + swz8<D>(row, col), p.v + off, at >= 0 ? 16u : 0u);
  }
  if (lane < C::kSlab) {
    const int64_t off = page >= 0 ? head * p.scales_per_page + scale_index(p, slot) : 0;
    cp_async_4(scales + lane * 4, p.k_scale + off, page >= 0 ? 4u : 0u);
    cp_async_4(scales + (32 + lane) * 4, p.v_scale + off, page >= 0 ? 4u : 0u);
  }
}

// Q^T as the B operand of S^T = K Q^T: lane
// (lr, lc) holds head lr; k positions 2lc, 2lc+1 / 2lc+8, 2lc+9 of k-step ks
// stand for dims f, f+1 / f+2, f+3 with f = 16 (lc + 4 (ks / 4)) + 4 (ks % 4),
// so that one 16-byte load of a K row holds the A bytes of four k-steps.
// qrow: the lane's head's row; rows past the group's heads count as zeros.
// A head's elements are taken relative to a power of two that brings the largest to
// [2^14, 2^15): as fp16 they keep their bits down to 2^-28 of it whatever their size,
// and elements that are not finite stay so. Returns the softmax scale times that power
// for heads 2lc and 2lc + 1, whose scores the lane computes.
template <int D>
__device__ __forceinline__ float2 load_q(const __nv_bfloat16 *qrow, bool valid, int lc,
                                         float scale_log2, uint32_t (&qf)[D / 16][2]) {
  uint32_t m = 0u;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int f = 16 * (lc + 4 * (ks >> 2)) + 4 * (ks & 3) + 2 * i;
      qf[ks][i] = valid ? *reinterpret_cast<const uint32_t *>(qrow + f) : 0u;
      m = __vmaxu2(m, qf[ks][i] & 0x7fff7fffu);
    }
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const int e = min(max(static_cast<int>(max(m & 0xffffu, m >> 16) >> 7) - 127, -100), 127);
  const float to = __int_as_float((14 - e + 127) << 23);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      qf[ks][i] = pack_f16x2(bf16_lo(qf[ks][i]) * to, bf16_hi(qf[ks][i]) * to);
  const float from = __int_as_float((e - 14 + 127) << 23) * scale_log2;
  return make_float2(__shfl_sync(0xffffffffu, from, 8 * lc),
                     __shfl_sync(0xffffffffu, from, 8 * lc + 4));
}

// Online-softmax state of a warp: heads 2lc and 2lc + 1 of its 8.
template <int D>
struct Softmax {
  float m0, m1, d0, d1, o[D / 16][4];
  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    d0 = d1 = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  }
  // d is summed over the 8 lane rows once, at the end
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      d0 += __shfl_xor_sync(0xffffffffu, d0, off);
      d1 += __shfl_xor_sync(0xffffffffu, d1, off);
    }
  }
  // m, d [8] (md) and o [8][D] (so) to shared memory
  __device__ __forceinline__ void put(float *md, float *so, int lr, int lc) const {
    if (lr == 0) {
      md[2 * lc] = m0;
      md[2 * lc + 1] = m1;
      md[8 + 2 * lc] = d0;
      md[8 + 2 * lc + 1] = d1;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      float *x = so + 2 * lc * D + (D / 8) * lr + 2 * dt;
      *reinterpret_cast<float2 *>(x) = make_float2(o[dt][0], o[dt][2]);
      *reinterpret_cast<float2 *>(x + D) = make_float2(o[dt][1], o[dt][3]);
    }
  }
};

// One slab: scores, softmax step, P V. Keys outside [lo, hi) are masked. ksc, vsc:
// the scales of its tiles (kTile) or of its rows.
template <int D, bool kTile>
__device__ __forceinline__ void slab_step(const uint8_t *k8, const float *ksc, const float *vsc,
                                          int slab0, int lo, int hi, float2 scale_log2,
                                          const uint32_t (&qf)[D / 16][2], int lr, int lc,
                                          Softmax<D> &st) {
  using C = Cfg<D>;
  constexpr int kMT = C::kMT, kKS = C::kKS;
  const uint8_t *v8 = k8 + C::kSlabBytes;
  // scores in log2 units (s[mt][0]: row lr, s[mt][1]: row lr + 8; x, y: the two
  // heads), and the reference x + log2(vs)
  const bool whole = slab0 >= lo && slab0 + C::kSlab <= hi;
  float2 s[kMT][2];
  float vs[kMT][2];
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt) {
    // Two sums of every other k-step, joined once: a product waits for the one two before it,
    // not for its neighbour (64 sequences of 1k to 8k at head_dim 128 109.4 -> 108.6 us, a
    // single split's chain of slabs 176.8 -> 168.5 us).
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
    const int r0 = mt * 16 + lr, r1 = r0 + 8;
    uint4 kx0, kx1;  // rows r0 / r1: 16 bytes = four k-steps' words
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      if ((ks & 3) == 0) {
        kx0 = *reinterpret_cast<const uint4 *>(k8 + swz8<D>(r0, lc + 4 * (ks >> 2)));
        kx1 = *reinterpret_cast<const uint4 *>(k8 + swz8<D>(r1, lc + 4 * (ks >> 2)));
      }
      const int q = ks & 3;
      const uint32_t x0 = q == 0 ? kx0.x : q == 1 ? kx0.y : q == 2 ? kx0.z : kx0.w;
      const uint32_t x1 = q == 0 ? kx1.x : q == 1 ? kx1.y : q == 2 ? kx1.z : kx1.w;
      uint32_t a[4];
      e4m3x4_to_f16x4(x0, a[0], a[2]);
      e4m3x4_to_f16x4(x1, a[1], a[3]);
      mma_f16_16816(ks & 1 ? acc2 : acc, a, qf[ks][0], qf[ks][1]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += acc2[e];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!kTile || i == 0) vs[mt][i] = vsc[kTile ? mt : i == 0 ? r0 : r1];
      if (kTile && i == 1) vs[mt][1] = vs[mt][0];
      const float f = ksc[kTile ? mt : i == 0 ? r0 : r1];
      s[mt][i] = __fmul2_rn(__fmul2_rn(make_float2(acc[2 * i], acc[2 * i + 1]),
                                       make_float2(f, f)), scale_log2);
    }
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = slab0 + (i == 0 ? r0 : r1);
        if (j < lo || j >= hi) s[mt][i] = make_float2(-INFINITY, -INFINITY);
      }
    }
    const float l0 = fast_log2(fmaxf(fabsf(vs[mt][0]), kMinVScale));
    if (kTile) {
      mx0 = fmaxf(mx0, fmaxf(s[mt][0].x, s[mt][1].x) + l0);
      mx1 = fmaxf(mx1, fmaxf(s[mt][0].y, s[mt][1].y) + l0);
    } else {
      const float l1 = fast_log2(fmaxf(fabsf(vs[mt][1]), kMinVScale));
      mx0 = fmaxf(mx0, fmaxf(s[mt][0].x + l0, s[mt][1].x + l1));
      mx1 = fmaxf(mx1, fmaxf(s[mt][0].y + l0, s[mt][1].y + l1));
    }
  }
  // The reference moves only when a score passes it by more than 2^kSlack (the
  // weights then stay below 2^kSlack, well inside fp16): most slabs need neither
  // the maximum over the lanes nor a rescaling of O and d.
  if (__any_sync(0xffffffffu, mx0 > st.m0 + kSlack || mx1 > st.m1 + kSlack)) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    const float mn0 = fmaxf(st.m0, mx0), mn1 = fmaxf(st.m1, mx1);
    const float h0 = fast_exp2(0.5f * (st.m0 - (mn0 == -INFINITY ? 0.f : mn0)));
    const float h1 = fast_exp2(0.5f * (st.m1 - (mn1 == -INFINITY ? 0.f : mn1)));
    st.m0 = mn0;
    st.m1 = mn1;
    st.d0 = st.d0 * h0 * h0;
    st.d1 = st.d1 * h1 * h1;
    // O holds weights of at most 2^kSlack: what the product loses is nothing beside them
    const float al0 = h0 * h0, al1 = h1 * h1;
#pragma unroll
    for (int dt = 0; dt < kKS; ++dt) {
      st.o[dt][0] *= al0;
      st.o[dt][1] *= al1;
      st.o[dt][2] *= al0;
      st.o[dt][3] *= al1;
    }
  }
  const float2 nbase = make_float2(st.m0 == -INFINITY ? 0.f : -st.m0,
                                   st.m1 == -INFINITY ? 0.f : -st.m1);
  float2 sum = make_float2(st.d0, st.d1);
  uint32_t pb[kMT][2];  // w = p * vs as fp16 (11 bits), the B fragments of P^T
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = __fadd2_rn(s[mt][i], nbase);
      const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      sum = __fadd2_rn(sum, e);
      const float2 w = __fmul2_rn(e, make_float2(vs[mt][i], vs[mt][i]));
      pb[mt][i] = movmatrix_trans(pack_f16x2(w.x, w.y));
    }
  st.d0 = sum.x;
  st.d1 = sum.y;
  // O^T += V^T W^T: MMA rows lr / lr + 8 of dim tile dt stand for dims
  // (D / 8) lr + 2 dt and + 1: one (D / 8)-byte load per token holds the lane's
  // bytes of every dim tile, paired across tokens by a byte permute
  constexpr int kW = D / 32;  // 32-bit words per token load
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt) {
    const int t = mt * 16 + 2 * lc;
    const int byte0 = (D / 8) * lr;
    const int ch = byte0 >> 4, within = byte0 & 15;
    uint32_t w[4][kW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = t + (i & 1) + 8 * (i >> 1);
      const uint8_t *src = v8 + swz8<D>(tok, ch) + within;
      if constexpr (kW == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(src);
        w[i][0] = x.x;
        w[i][1] = x.y;
      } else {
        const uint4 x = *reinterpret_cast<const uint4 *>(src);
        w[i][0] = x.x;
        w[i][1] = x.y;
        w[i][2] = x.z;
        w[i][3] = x.w;
      }
    }
#pragma unroll
    for (int dt = 0; dt < kKS; ++dt) {
      uint32_t a[4];
      const unsigned sel = (dt & 1) ? 0x7362u : 0x5140u;
      e4m3x4_to_f16x4(__byte_perm(w[0][dt >> 1], w[1][dt >> 1], sel), a[0], a[1]);
      e4m3x4_to_f16x4(__byte_perm(w[2][dt >> 1], w[3][dt >> 1], sel), a[2], a[3]);
      mma_f16_16816(st.o[dt], a, pb[mt][0], pb[mt][1]);
    }
  }
}

// kPer dims of one head from several states with maxima: the sums, in units of
// 2^base, and the maximum.
template <int kPer>
struct Merged {
  float M, base, W, r[kPer];
  __device__ __forceinline__ void begin(float max_m) {
    M = max_m;
    base = max_m == -INFINITY ? 0.f : max_m;
    W = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) r[e] = 0.f;
  }
  template <class Load4>
  __device__ __forceinline__ void add(float m, float d, const Load4 &load4) {
    // twice: see the denominator, above; the infinite base of a huge sink is its own
    const float h = m == base ? 1.f : fast_exp2(0.5f * (m - base));
    W += d * h * h;
#pragma unroll
    for (int e = 0; e < kPer; e += 4) {
      const float4 x = load4(e);
      r[e] += x.x * h * h;
      r[e + 1] += x.y * h * h;
      r[e + 2] += x.z * h * h;
      r[e + 3] += x.w * h * h;
    }
  }
  // W = 0: nothing visible and no sink. A NaN (of a sink, say) stays one.
  __device__ __forceinline__ float inv() const { return W == 0.f ? 0.f : 1.f / W; }
  // Natural log. Infinite: nothing but the sink counts, which may be a number that
  // overflows in log2 units only.
  __device__ __forceinline__ float lse(const Params &p, int head) const {
    const float l = W == 0.f ? -INFINITY : (M + fast_log2(W)) * kLn2;
    return fabsf(l) == INFINITY && p.sinks != nullptr ? p.sinks[head] : l;
  }
  // bf16 output and lse of a sequence's query head, dims c0..
  __device__ __forceinline__ void store(const Params &p, int b, int head, int D, int c0) const {
    const size_t row_h = static_cast<size_t>(b) * p.hq + head;
    const float mul = inv();
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
      *reinterpret_cast<uint2 *>(p.out + row_h * D + c0 + e) =
          make_uint2(pack_bf16x2(r[e] * mul, r[e + 1] * mul),
                     pack_bf16x2(r[e + 2] * mul, r[e + 3] * mul));
    if (p.lse != nullptr && c0 == 0) p.lse[row_h] = lse(p, head);
  }
};

// States of kStates warps (md 16 floats apart, o `stride` floats apart) and the
// sink (log2, -inf: none).
template <int D, int kStates, int kPer>
__device__ __forceinline__ Merged<kPer> combine(const float *md, const float *so, int stride,
                                                float sink, int hh, int c0) {
  float M = sink;
#pragma unroll
  for (int w = 0; w < kStates; ++w) M = fmaxf(M, md[16 * w + hh]);
  Merged<kPer> x;
  x.begin(M);
  x.W = sink == x.base ? 1.f : fast_exp2(sink - x.base);
#pragma unroll
  for (int w = 0; w < kStates; ++w)
    x.add(md[16 * w + hh], md[16 * w + 8 + hh], [&](int e) {
      return *reinterpret_cast<const float4 *>(so + w * stride + hh * D + c0 + e);
    });
  return x;
}

// ---- pairs and cluster --------------------------------------------------------

template <int D, bool kPair, bool kTile>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    decode_block_kernel(const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const Params p) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages, kSlab = C::kSlab;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int s_abort[kWarps];
  __shared__ uint64_t s_never[kWarps];
  __shared__ __align__(16) float s_md[(kWarps + 1) * 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lr = lane >> 2, lc = lane & 3;  // mma fragment row / column group
  int split = 0, b, gh;  // gh: KV head and tile of up to 8 of its query heads
  if (kPair) {
    const int pair = static_cast<int>(blockIdx.x) * kWarps + warp;
    if (pair >= p.batch * p.hkv * p.nht) return;  // no block barrier follows
    b = pair / (p.hkv * p.nht);
    gh = pair - b * p.hkv * p.nht;
  } else {
    split = blockIdx.x;
    gh = blockIdx.y;
    b = blockIdx.z;
  }
  const int g = gh / p.nht, ht = gh - g * p.nht;
  const int hbase = g * p.group + ht * kMaxGroup;
  const int gt = min(kMaxGroup, p.group - ht * kMaxGroup);
  const Span sp = span_of<kTile>(p, b);
  const int nkv = sp.len - sp.start;
  // A span longer than the host's bound gets longer pieces, not more of them.
  int chunk = kPair ? max(nkv, 1) : p.chunk;
  if (!kPair && nkv > static_cast<int64_t>(chunk) * gridDim.x)
    chunk = ((nkv + gridDim.x - 1) / gridDim.x + C::kGroup - 1) / C::kGroup * C::kGroup;
  const int nsplit = max(1, nkv / chunk + (nkv % chunk != 0));
  if (split >= nsplit) return;  // exited blocks do not count in the cluster's barrier
  const int t0 = sp.start + split * chunk;
  const int t1 = sp.len - t0 < chunk ? sp.len : t0 + chunk;
  const int nslab = (max(0, t1 - t0) + kSlab - 1) / kSlab;
  const int32_t *table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  const int stride = kPair ? kSlab : C::kGroup, first = t0 + (kPair ? 0 : warp * kSlab);
  const int my_slabs = kPair ? nslab : (warp < nslab ? (nslab - warp + kWarps - 1) / kWarps : 0);

  Feed<C, D> feed;
  feed.init(smem, warp, lane);
  volatile int *abort = s_abort + warp;
  if (lane == 0) *abort = 0;
  __syncwarp();
  auto load_slab = [&](int i) {
    const int slab0 = first + i * stride, stage = i % kStages;
    if constexpr (kTile)
      feed.load(p, &tk, &tv, stage, i == 0, table, i, slab0, stride, g, sp.lo, t1, lane);
    else
      load_rows<D>(p, smem_u32(feed.ring) + stage * C::kStageBytes,
                   smem_u32(feed.scales + stage * 64), i == 0, table, slab0, stride, g, t1, lane,
                   feed.next);
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < my_slabs) load_slab(i);
    cp_async_commit();
  }
  uint32_t qf[C::kKS][2];
  const float2 scale_log2 =
      load_q<D>(p.q + (static_cast<size_t>(b) * p.hq + hbase + (lr < gt ? lr : 0)) * D, lr < gt,
                lc, p.scale_log2, qf);
  Softmax<D> st;
  st.reset();
  bool live = !kTile || p.stall_ns == 0 || stall(p.stall_ns, s_never + warp, abort);
  int issued = min(kStages - 1, my_slabs);
  for (int it = 0; it < my_slabs; ++it) {
    const int stage = it % kStages;
    cp_async_wait<kStages - 2>();
    if (kTile && live) live = feed.wait(stage, it / kStages & 1, abort);
    __syncwarp();
    if (live && issued < my_slabs) load_slab(issued++);
    cp_async_commit();
    const float *sc = feed.scales + (kTile ? it / C::kAhead % kStages : stage) * 64 +
                      (kTile ? it % C::kAhead * C::kMT : 0);
    slab_step<D, kTile>(feed.ring + stage * C::kStageBytes, sc, sc + 32, first + it * stride,
                        sp.lo, t1, scale_log2, qf, lr, lc, st);
  }
  cp_async_wait<0>();
  if (kTile && !live) feed.drain(issued, abort);
  st.finish();

  // the states go to shared memory: a warp's own ring, or one after the other
  auto sync = [&] {
    if (kPair)
      __syncwarp();
    else
      __syncthreads();
  };
  sync();  // everyone concerned is done with the ring
  float *so = reinterpret_cast<float *>(kPair ? feed.ring : smem);
  float *md = s_md + (kPair ? 16 * warp : 0);
  st.put(s_md + 16 * warp, kPair ? so : so + warp * C::kState, lr, lc);
  sync();
  constexpr int kLanes = kPair ? 4 : 16, kPer = D / kLanes;  // lanes per head, dims per lane
  const int tid = kPair ? lane : static_cast<int>(threadIdx.x);
  const int hh = tid / kLanes, sub = tid % kLanes, c0 = sub * kPer;
  const bool head_ok = hh < gt;
  const float sink = p.sinks != nullptr && split == 0 && head_ok ? p.sinks[hbase + hh] * kLog2e
                                                                 : -INFINITY;
  const Merged<kPer> mine =
      combine<D, kPair ? 1 : kWarps, kPer>(md, so, C::kState, sink, hh, c0);
  if (nsplit == 1) {
    if (head_ok) mine.store(p, b, hbase + hh, D, c0);
    return;
  }
  if constexpr (!kPair) {
    // the block's state behind its warps'; the blocks share the heads out
    float *cmd = s_md + kWarps * 16, *cso = so + kWarps * C::kState;
    if (sub == 0) {
      cmd[hh] = mine.M;
      cmd[8 + hh] = mine.W;
    }
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
      *reinterpret_cast<float4 *>(cso + hh * D + c0 + e) =
          make_float4(mine.r[e], mine.r[e + 1], mine.r[e + 2], mine.r[e + 3]);
    cluster_sync();
    if (head_ok && hh % nsplit == split) {
      const uint32_t at_md = smem_u32(cmd + hh), at_o = smem_u32(cso + hh * D + c0);
      float M = -INFINITY;
      for (int k = 0; k < nsplit; ++k) M = fmaxf(M, cluster_ld(cluster_map(at_md, k)));
      Merged<kPer> x;
      x.begin(M);
#pragma unroll 4
      for (int k = 0; k < nsplit; ++k) {
        const uint32_t omd = cluster_map(at_md, k), oo = cluster_map(at_o, k);
        x.add(cluster_ld(omd), cluster_ld(omd + 32), [&](int e) { return cluster_ld4(oo + 4 * e); });
      }
      x.store(p, b, hbase + hh, D, c0);
    }
    cluster_sync();  // no block leaves while its state may be read
  }
}

// ---- flat -----------------------------------------------------------------------

// A worker's partial rows: [worker][head tile][which][8], and for each worker the
// sequence that its range's end cuts, if it holds that sequence's first group, and
// the last worker of that sequence. A worker is the first of at most one cut
// sequence: that piece is its second partial.
__device__ __forceinline__ size_t partial_row(int w, int heads, int gh, bool is_first, int h) {
  return ((static_cast<size_t>(w) * heads + gh) * 2 + (is_first ? 1 : 0)) * kMaxGroup + h;
}

// Merges the partials of cut sequences: block (worker, head tile). Launched with
// the decode kernel still running; the wait makes its partials visible. Warp k
// sums partials first + k, first + k + 4, .. (lane: a head, a quarter of its
// dims), so that many loads are in flight, and the four sums are combined; the
// order is fixed.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) merge_flat_kernel(const Params p) {
  constexpr int kState = D * kMaxGroup, kQ = D / 4, kPer = D / 16;
  __shared__ __align__(16) float s_md[kWarps * 16];
  __shared__ __align__(16) float s_o[kWarps * kState];
  const int heads = p.hkv * p.nht;
  const int first = blockIdx.x / heads, gh = blockIdx.x - first * heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 cut = __ldcg(p.cuts + first);  // (sequence, last worker)
  if (cut.x < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = lane >> 2, at = (lane & 3) * kQ;
  auto row = [&](int w) { return partial_row(w, heads, gh, w == first, h); };
  float M = -INFINITY;
#pragma unroll 4
  for (int w = first + warp + kWarps * (lane & 3); w <= cut.y; w += 4 * kWarps)
    M = fmaxf(M, __ldcg(p.part_lse + row(w)));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
  Merged<kQ> y;
  y.begin(M);
#pragma unroll 4
  for (int w = first + warp; w <= cut.y; w += kWarps)
    y.add(__ldcg(p.part_lse + row(w)), 1.f, [&](int e) {
      return __ldcg(reinterpret_cast<const float4 *>(p.part_o + row(w) * D + at + e));
    });
  if ((lane & 3) == 0) {
    s_md[16 * warp + h] = M;
    s_md[16 * warp + 8 + h] = y.W;
  }
#pragma unroll
  for (int e = 0; e < kQ; e += 4)
    *reinterpret_cast<float4 *>(s_o + warp * kState + h * D + at + e) =
        make_float4(y.r[e], y.r[e + 1], y.r[e + 2], y.r[e + 3]);
  __syncthreads();
  const int hh = threadIdx.x / 16, c0 = threadIdx.x % 16 * kPer;
  const int g = gh / p.nht, ht = gh - g * p.nht;
  const Merged<kPer> z = combine<D, kWarps, kPer>(s_md, s_o, kState, -INFINITY, hh, c0);
  if (hh < min(kMaxGroup, p.group - ht * kMaxGroup))
    z.store(p, cut.x, g * p.group + ht * kMaxGroup + hh, D, c0);
}

// A sequence has max(1, ceil(keys / kGroup)) groups of one slab per warp; the
// groups of all sequences stand in a line. Worker w of W takes the groups
// [total * w / W, total * (w + 1) / W), and there is one block for each (worker,
// KV head and head tile): the blocks of a worker walk the same keys in step, so
// that the heads of a page, which lie side by side in memory, are read together
// (256 contexts of 1k-32k: 699 us with the heads one after the other in the line, 665 us so).
template <int D, bool kTile>
__global__ void __launch_bounds__(kThreads, Flat<D>::kBlocks)
    decode_flat_kernel(const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const Params p) {
  using C = Flat<D>;
  constexpr int kStages = C::kStages, kSlab = C::kSlab;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int s_b, s_at, s_abort[kWarps];
  __shared__ uint64_t s_never[kWarps];
  __shared__ __align__(16) float s_md[kWarps * 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lr = lane >> 2, lc = lane & 3;
  const int heads = p.hkv * p.nht;
  asm volatile("griddepcontrol.launch_dependents;");
  auto groups_of = [](const Span &s) {
    return max(1, (s.len - s.start + C::kGroup - 1) / C::kGroup);
  };

  // Find the range's first pair: each thread sums a run of sequences, the block
  // scans the sums, and the thread whose run holds the place walks it.
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b_first = threadIdx.x * per, b_end = min(p.batch, b_first + per);
  int64_t mine = 0;
  for (int b = b_first; b < b_end; ++b) mine += groups_of(span_of<kTile>(p, b));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  // at least four groups per worker, so that short calls are not all merging
  const int me = blockIdx.x / heads, gh = blockIdx.x - me * heads;
  const int W = static_cast<int>(
      min(static_cast<int64_t>(gridDim.x) / heads, max(total / 4, int64_t(1))));
  if (me >= W) {
    if (gh == 0 && threadIdx.x == 0) p.cuts[me] = make_int2(-1, -1);
    return;
  }
  int2 cut = make_int2(-1, -1);
  const int64_t begin = total * me / W;
  const int count = static_cast<int>(total * (me + 1) / W - begin);
  {
    int64_t ex = before + incl - mine;
    if (begin >= ex && begin < ex + mine)
      for (int b = b_first; b < b_end; ++b) {
        const int n = groups_of(span_of<kTile>(p, b));
        if (begin < ex + n) {
          s_b = b;
          s_at = static_cast<int>(begin - ex);
          break;
        }
        ex += n;
      }
  }
  __syncthreads();
  const int g = gh / p.nht, ht = gh - g * p.nht;
  const int hbase = g * p.group + ht * kMaxGroup;
  const int gt = min(kMaxGroup, p.group - ht * kMaxGroup);

  // A cursor walks the groups of the range: sequence b, group t of n.
  struct Cursor {
    int b, t, n;
    Span s;
  };
  auto next = [&](Cursor &c) {
    if (++c.t < c.n) return;
    c.t = 0;
    if (++c.b >= p.batch) return;  // the end of the line
    c.s = span_of<kTile>(p, c.b);
    c.n = groups_of(c.s);
  };
  Cursor cur;  // computing
  cur.b = s_b;
  cur.t = s_at;
  cur.s = span_of<kTile>(p, cur.b);
  cur.n = groups_of(cur.s);
  Cursor ld = cur;  // loading, up to kStages - 1 groups ahead

  Feed<C, D> feed;
  feed.init(smem, warp, lane);
  volatile int *abort = s_abort + warp;
  if (lane == 0) *abort = 0;
  __syncwarp();
  // The query rows of a piece are copied with its first slab, a quarter by each
  // warp, into one of kStages buffers; the barrier at the end of the piece before
  // it publishes them.
  int q_ld = 0;
  bool ld_fresh = true;
  auto load_slab = [&](int stage) {
    const int slab0 = ld.s.start + (ld.t * kWarps + warp) * kSlab;
    const int32_t *table = p.block_table + static_cast<size_t>(ld.b) * p.max_pages;
    if (ld_fresh) {
      constexpr int kChunks = C::kQBytes / 16 / kWarps, kCols = D / 8;
      if (lane < kChunks) {
        const int c = warp * kChunks + lane, h = c / kCols;
        const bool ok = h < gt;
        cp_async_16(smem_u32(smem) + C::kQOff + q_ld * C::kQBytes + c * 16,
                    p.q + (ok ? (static_cast<size_t>(ld.b) * p.hq + hbase + h) * D + c % kCols * 8
                              : 0),
                    ok ? 16u : 0u);
      }
      q_ld = q_ld + 1 == kStages ? 0 : q_ld + 1;
    }
    if constexpr (kTile) {
      feed.load(p, &tk, &tv, stage, ld_fresh, table, ld.t, slab0, C::kGroup, g, ld.s.lo, ld.s.len,
                lane);
    } else if (slab0 < ld.s.len) {
      load_rows<D>(p, smem_u32(feed.ring) + stage * C::kStageBytes,
                   smem_u32(feed.scales + stage * 64), ld_fresh, table, slab0, C::kGroup, g,
                   ld.s.len, lane, feed.next);
    }
    ld_fresh = ld.t + 1 == ld.n;
    next(ld);
  };

  int loaded = 0;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (loaded < count) {
      load_slab(i);
      ++loaded;
    }
    cp_async_commit();
  }
  cp_async_wait<kStages - 2>();
  __syncthreads();  // the first piece's query rows are there
  uint32_t qf[C::kKS][2];
  float2 scale_log2 = make_float2(0.f, 0.f);  // set with qf
  Softmax<D> st;
  int stage = 0, t_first = 0;  // t_first: the piece's first group of its pair
  int q_cur = 0, batch_t = 0, batch = kStages - 1;  // query buffer; scale batch and buffer
  uint32_t parity = 0;
  bool fresh = true, live = !kTile || p.stall_ns == 0 || stall(p.stall_ns, s_never + warp, abort);
  for (int i = 0; i < count; ++i) {
    if (fresh) {
      scale_log2 = load_q<D>(
          reinterpret_cast<const __nv_bfloat16 *>(smem + C::kQOff + q_cur * C::kQBytes) + lr * D,
          true, lc, p.scale_log2, qf);
      q_cur = q_cur + 1 == kStages ? 0 : q_cur + 1;
      st.reset();
      t_first = cur.t;
    }
    if (fresh || cur.t == batch_t + C::kAhead) {
      batch_t = cur.t;
      batch = batch + 1 == kStages ? 0 : batch + 1;
    }
    fresh = false;
    cp_async_wait<kStages - 2>();
    if (kTile && live) live = feed.wait(stage, parity, abort);
    __syncwarp();
    if (live && loaded < count) {
      load_slab(stage == 0 ? kStages - 1 : stage - 1);
      ++loaded;
    }
    cp_async_commit();
    const int slab0 = cur.s.start + (cur.t * kWarps + warp) * kSlab;
    if (slab0 < cur.s.len) {
      const float *sc = feed.scales + (kTile ? batch : stage) * 64 +
                        (kTile ? (cur.t - batch_t) * C::kMT : 0);
      slab_step<D, kTile>(feed.ring + stage * C::kStageBytes, sc, sc + 32, slab0, cur.s.lo,
                          cur.s.len, scale_log2, qf, lr, lc, st);
    }
    if (cur.t + 1 == cur.n || i + 1 == count) {  // the piece ends here
      // each warp's state takes the stage that it has just read, which the next
      // copy reaches only after the barrier below
      st.finish();
      __syncwarp();
      st.put(s_md + 16 * warp, reinterpret_cast<float *>(feed.ring + stage * C::kStageBytes), lr,
             lc);
      __syncthreads();
      constexpr int kLanes = 16, kPer = D / kLanes;
      const int hh = threadIdx.x / kLanes, sub = threadIdx.x % kLanes, c0 = sub * kPer;
      const bool head_ok = hh < gt;
      const float sink = p.sinks != nullptr && t_first == 0 && head_ok
                             ? p.sinks[hbase + hh] * kLog2e
                             : -INFINITY;
      const Merged<kPer> x = combine<D, kWarps, kPer>(
          s_md, reinterpret_cast<const float *>(smem + stage * C::kStageBytes),
          C::kRingBytes / 4, sink, hh, c0);
      if (t_first == 0 && cur.t + 1 == cur.n) {
        if (head_ok) x.store(p, cur.b, hbase + hh, D, c0);
      } else {
        const int64_t p0 = begin + i - cur.t;  // the sequence's first group in the line
        const bool is_first = p0 >= begin;
        const size_t row = partial_row(me, heads, gh, is_first, hh);
        const float inv = x.inv();
#pragma unroll
        for (int e = 0; e < kPer; e += 4)
          *reinterpret_cast<float4 *>(p.part_o + row * D + c0 + e) = make_float4(
              x.r[e] * inv, x.r[e + 1] * inv, x.r[e + 2] * inv, x.r[e + 3] * inv);
        if (sub == 0) p.part_lse[row] = x.W == 0.f ? -INFINITY : x.M + fast_log2(x.W);
        if (is_first) cut = make_int2(cur.b, static_cast<int>(((p0 + cur.n) * W - 1) / total));
      }
      // The states are read (their stages may be refilled, by TMA too) and the next
      // piece's query rows, copied with its first slab, are there.
      if (kTile) fence_proxy_async();
      cp_async_wait<kStages - 2>();
      __syncthreads();
      fresh = true;
    }
    next(cur);
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1u;
    }
  }
  cp_async_wait<0>();
  if (kTile && !live) feed.drain(loaded, abort);
  if (gh == 0 && threadIdx.x == 0) p.cuts[me] = cut;
}

// [rows, d] codes; a box is 16 rows, swizzled as swz8 does.
bool encode_code_tiles(EncodeTiledFn fn, CUtensorMap *map, const void *base, int64_t rows, int d) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(d), 16};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// testing hook (sinkattn_debug_stall_waits): stall_ns of later launches
std::atomic<uint64_t> g_stall_ns{0};

int log2_or_minus1(int x) {
  if (x <= 0 || (x & (x - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace

DecodeBlockPlan plan_decode_block(int batch, int hq, int hkv, int head_dim, int max_seqlen_k,
                                  int window, int num_splits) {
  const int unit = head_dim == 64 ? Cfg<64>::kGroup : Cfg<128>::kGroup;
  // a window's first slab starts up to 15 tokens before it
  const int seen = window > 0 && window < max_seqlen_k ? window : max_seqlen_k;
  const int64_t span = window > 0 && window + int64_t(15) < max_seqlen_k ? window + int64_t(15)
                       : max_seqlen_k > 0 ? std::min<int64_t>(max_seqlen_k, kMaxKeys)
                                          : 1;
  const int64_t pairs = static_cast<int64_t>(batch) * hkv * decode_head_tiles(hq, hkv);
  DecodeBlockPlan plan;
  plan.blocks = 0;
  auto cut = [&](int64_t s) {  // pieces of whole groups
    plan.chunk = static_cast<int>(((span + s - 1) / s + unit - 1) / unit * unit);
    plan.splits = static_cast<int>((span + plan.chunk - 1) / plan.chunk);
  };
  plan.kind = DecodeBlockPlan::kCluster;
  if (num_splits > 0 && num_splits <= kMaxCluster) {
    cut(num_splits);
    return plan;
  }
  cut(1);
  if (num_splits == 0 && seen <= pair_max_span(pairs)) {
    plan.kind = DecodeBlockPlan::kPairs;
    return plan;
  }
  // Locating a flat block's range reads every length: not for thousands of
  // sequences, which fill the GPU unsplit.
  if (batch > kMaxFlatBatch) return plan;
  if (num_splits == 0) {
    // Clusters while all blocks are resident at once and the pieces are short
    // (flat pays about 5 us more for its search and its merge).
    cut(std::clamp<int64_t>(kSms * kBlocksPerSm / pairs, 1, kMaxCluster));
    if (plan.chunk <= kClusterChunk) return plan;
  }
  const int heads = hkv * decode_head_tiles(hq, hkv);
  const int slots = kSms * (head_dim == 64 ? Flat<64>::kBlocks : Flat<128>::kBlocks);
  if (slots / heads < 2) {  // a single worker: nothing to share out
    cut(1);
    return plan;
  }
  plan.kind = DecodeBlockPlan::kFlat;
  plan.blocks = slots / heads * heads;
  return plan;
}

size_t decode_block_workspace_bytes(const DecodeBlockPlan &plan, int head_dim) {
  if (plan.kind != DecodeBlockPlan::kFlat) return 0;
  const size_t rows = static_cast<size_t>(plan.blocks) * 2 * kMaxGroup;
  return rows * head_dim * 4 + rows * 4 + plan.blocks * sizeof(int2);
}

cudaError_t launch_decode_block(const DecodeBlockLaunch &a, cudaStream_t stream) {
  Params p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k = static_cast<const uint8_t *>(a.k);
  p.v = static_cast<const uint8_t *>(a.v);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_table = a.block_table;
  p.seqlens_k = a.seqlens_k;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.page_size = a.page_size;
  p.page_shift = log2_or_minus1(a.page_size);
  p.scale_block = a.scale_block;
  p.block_shift = log2_or_minus1(a.scale_block);
  p.scales_per_page = a.page_size / a.scale_block;
  p.batch = a.batch;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = a.hq / a.hkv;
  p.nht = decode_head_tiles(a.hq, a.hkv);
  p.window = a.window;
  p.chunk = a.plan.chunk;
  p.sinks = a.sinks;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  const size_t rows = static_cast<size_t>(a.plan.blocks) * 2 * kMaxGroup;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  p.part_o = reinterpret_cast<float *>(ws);
  p.part_lse = reinterpret_cast<float *>(ws + rows * a.head_dim * 4);
  p.cuts = reinterpret_cast<int2 *>(ws + rows * a.head_dim * 4 + rows * 4);
  p.stall_ns = g_stall_ns.load();

  const int64_t pairs = static_cast<int64_t>(a.batch) * a.hkv * p.nht;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  const int64_t code_rows = static_cast<int64_t>(a.num_pages) * a.hkv * a.page_size;
  // max_pages 0: no table, no keys, and the caches may be null. TMA coordinates are 32-bit.
  const bool tile = a.page_size % 16 == 0 && a.scale_block % 16 == 0 && a.max_pages > 0 &&
                    code_rows > 0 && code_rows <= INT32_MAX;
  CUtensorMap tk = {}, tv = {};
  if (tile) {
    const EncodeTiledFn fn = get_encode_fn();
    if (fn == nullptr || !encode_code_tiles(fn, &tk, a.k, code_rows, a.head_dim) ||
        !encode_code_tiles(fn, &tv, a.v, code_rows, a.head_dim))
      return cudaErrorInvalidValue;
  }
  auto go = [&](auto kernel, int smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && cfg.numAttrs == 1 && a.plan.splits > 8)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    e = cudaLaunchKernelEx(&cfg, kernel, tk, tv, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  };
  auto pick = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    constexpr int smem = Cfg<D>::kSmemBytes, flat_smem = Flat<D>::kFlatSmemBytes;
    if (a.plan.kind == DecodeBlockPlan::kPairs) {
      cfg.gridDim = dim3(static_cast<unsigned>((pairs + kWarps - 1) / kWarps));
      return tile ? go(decode_block_kernel<D, true, true>, smem)
                  : go(decode_block_kernel<D, true, false>, smem);
    }
    if (a.plan.kind == DecodeBlockPlan::kCluster) {
      cfg.gridDim = dim3(a.plan.splits, a.hkv * p.nht, a.batch);
      if (a.plan.splits > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(a.plan.splits);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
      }
      return tile ? go(decode_block_kernel<D, false, true>, smem)
                  : go(decode_block_kernel<D, false, false>, smem);
    }
    cfg.gridDim = dim3(a.plan.blocks);
    cudaError_t e = tile ? go(decode_flat_kernel<D, true>, flat_smem)
                         : go(decode_flat_kernel<D, false>, flat_smem);
    if (e != cudaSuccess) return e;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, merge_flat_kernel<D>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  };
  return a.head_dim == 128 ? pick(std::integral_constant<int, 128>())
                           : pick(std::integral_constant<int, 64>());
}

cudaError_t decode_block_set_stall(uint64_t ns) {
  g_stall_ns.store(ns);
  return cudaSuccess;
}

cudaError_t decode_block_read_error(cudaStream_t stream, int *code) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_decode_block_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_decode_block_error, &zero, sizeof(int));
  return e;
}

}  // namespace sinkattn
