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
// (log2 units): every w_j = 2^(x_j - r) vs is at most 1 and the largest is 1, so
// fp16 keeps 11 bits of the weights that matter whatever the scales' spread.
// The denominator sums p_j = 2^(x_j - r) in fp32, where the offset between the
// two maxima (the scales lie in [2^-60, 2^60]) is harmless. The sink has no
// value row, so it takes no part in r; it enters the denominator once, at the
// end of split 0, with a maximum of its own.
//
// Block = (split s, KV head g, sequence b), 4 warps, each streaming 32-token
// (head_dim 64) or 16-token (128) slabs of K and V codes and their scales
// through its own shared-memory ring with cp.async, as the decode over an
// unscaled cache does; bound by the HBM traffic of the cache.
#include <math.h>

#include <type_traits>

#include "launch.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

__device__ int g_decode_block_error;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxGroup = 8;
// Visible spans up to this many tokens take one warp per (sequence, KV head).
constexpr int kPairMaxSpan = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMinVScale = 8.673617379884035e-19f;  // 2^-60: bound of the reference only
constexpr int kMaxCluster = 16;  // splits merged through a thread-block cluster
constexpr int kMaxBlockPages = 1024;  // page ids staged in shared memory per block
constexpr int64_t kMaxKeys = INT32_MAX - 65536;  // keeps the key arithmetic within int
constexpr int kStages = 3;
constexpr int kBlocksPerSm = 4;

template <int D>
struct Cfg {
  static constexpr int kSlab = D == 64 ? 32 : 16;  // tokens per warp step
  static constexpr int kMT = kSlab / 16;           // 16-token m-tiles
  static constexpr int kKS = D / 16;               // k-steps of Q K^T, dim tiles of P V
  static constexpr int kSlabBytes = kSlab * D;
  static constexpr int kScaleOff = 2 * kSlabBytes;            // K scales, then V scales
  static constexpr int kStageBytes = kScaleOff + 2 * kSlab * 4;
  static constexpr int kSmemBytes = kWarps * kStages * kStageBytes;
  static_assert(kStageBytes % 128 == 0, "stage alignment");
  static_assert(kStages * kStageBytes >= (2 + D) * kMaxGroup * 4, "one warp's combine area");
  static_assert(kSmemBytes >= (kWarps + 1) * (2 + D) * kMaxGroup * 4, "the block's combine area");
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
  unsigned int *counters;
};

__device__ __forceinline__ int page_index(const Params &p, int j) {
  return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
}
__device__ __forceinline__ int page_slot(const Params &p, int j) {
  return p.page_shift >= 0 ? j & (p.page_size - 1) : j % p.page_size;
}

// 64- or 128-byte rows of codes: 16-byte chunks XOR-swizzled by row / 2 (four
// chunks) or row (eight), free of bank conflicts for the fragment loads.
template <int D>
__device__ __forceinline__ int swz8(int row, int chunk) {
  return row * D + ((chunk ^ (D == 64 ? ((row >> 1) & 3) : (row & 7))) << 4);
}

enum Merge { kPairs, kCluster, kCounter };

// Zeroes the split-merge counters; the decode grid may launch at once and
// waits for this grid before its first counter access.
__global__ void __launch_bounds__(256) zero_counters_kernel(unsigned int *c, int64_t n) {
  asm volatile("griddepcontrol.launch_dependents;");
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    c[i] = 0u;
}

// kPair: short spans; each warp owns one (sequence, KV head, head tile) and no
// barrier spans the block.
// kTile: pages and scale blocks are multiples of 16 tokens. Slabs then start at
// multiples of 16, each 16-token m-tile lies in one page and one scale block, and
// a page lookup, an address and a pair of scales serve the whole tile. Otherwise
// every row looks up its own page and scales.
//
// How the splits of a (sequence, KV head) are merged (kMerge, not kPair):
// kCluster: they are one thread-block cluster; each block leaves its state in its
// shared memory and the blocks share the heads out among them, reading the others'
// states through the cluster (no scratch, no second launch). kCounter: more splits
// than a cluster holds; partials go through global memory and the last block to
// arrive merges them.
template <int D, Merge kMerge, bool kTile>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) decode_block_kernel(const Params p) {
  constexpr bool kPair = kMerge == kPairs;
  using C = Cfg<D>;
  constexpr int kSlab = C::kSlab, kMT = C::kMT, kKS = C::kKS;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lr = lane >> 2, lc = lane & 3;  // mma fragment row / column group
  int split = 0, g, b, ht;
  if (kPair) {
    const int pair = static_cast<int>(blockIdx.x) * kWarps + warp;
    if (pair >= p.batch * p.hkv * p.nht) return;  // no block barrier follows
    b = pair / (p.hkv * p.nht);
    const int gh = pair - b * p.hkv * p.nht;
    g = gh / p.nht;
    ht = gh - g * p.nht;
  } else {
    split = blockIdx.x;
    g = static_cast<int>(blockIdx.y) / p.nht;
    ht = static_cast<int>(blockIdx.y) - g * p.nht;
    b = blockIdx.z;
  }
  const int hbase = g * p.group + ht * kMaxGroup;
  const int gt = min(kMaxGroup, p.group - ht * kMaxGroup);
  const int cidx = (b * p.hkv + g) * p.nht + ht;  // split-merge counter

  // A length that the block table cannot address is cut to what it can.
  const int64_t cap = min(static_cast<int64_t>(p.max_pages) * p.page_size, kMaxKeys);
  const int L_raw = p.seqlens_k[b];
  const int L = L_raw < 0 ? 0 : L_raw > cap ? static_cast<int>(cap) : L_raw;
  if (L != L_raw && lane == 0) atomicExch(&g_decode_block_error, kErrBadLength);
  const int lo = p.window > 0 ? max(0, L - p.window) : 0;
  const int start = kTile ? lo & ~15 : lo;
  const int nkv = L - start;
  // A span longer than the host's bound gets longer blocks, not more of them.
  int chunk = kPair ? max(nkv, 1) : p.chunk;
  if (!kPair && (nkv + chunk - 1) / chunk > static_cast<int>(gridDim.x)) {
    const int unit = kWarps * kSlab;
    chunk = ((nkv + gridDim.x - 1) / gridDim.x + unit - 1) / unit * unit;
  }
  const int nsplit = max(1, (nkv + chunk - 1) / chunk);
  if (split >= nsplit) return;
  const int t0 = start + split * chunk;
  const int t1 = L - t0 < chunk ? L : t0 + chunk;
  const int nslab = (max(0, t1 - t0) + kSlab - 1) / kSlab;

  // Page ids are checked when they are read: one outside [0, num_pages) is
  // recorded and its rows count as zeros.
  const int32_t *table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  auto check_page = [&](int page) {
    if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return page;
    atomicExch(&g_decode_block_error, kErrBadPage);
    return -1;
  };
  __shared__ int s_pages[kPair ? 1 : kMaxBlockPages];
  int pg0 = 0;
  bool staged = false;
  if (!kPair) {
    pg0 = page_index(p, t0);
    const int npg = t1 > t0 ? page_index(p, t1 - 1) - pg0 + 1 : 0;
    staged = npg <= kMaxBlockPages;
    if (staged)
      for (int i = threadIdx.x; i < npg; i += kThreads) s_pages[i] = check_page(table[pg0 + i]);
    __syncthreads();
  }
  const int slab_first = kPair ? 0 : warp, slab_step = kPair ? 1 : kWarps;
  const int my_slabs = kPair ? nslab : (warp < nslab ? (nslab - warp + kWarps - 1) / kWarps : 0);

  // Q^T as the B operand of S^T = K Q^T, in fp16 (clamped to its range): lane
  // (lr, lc) holds head lr; k positions 2lc, 2lc+1 / 2lc+8, 2lc+9 of k-step ks
  // stand for dims f, f+1 / f+2, f+3 with f = 16 (lc + 4 (ks / 4)) + 4 (ks % 4),
  // so that one 16-byte load of a K row holds the A bytes of four k-steps.
  uint32_t qf[kKS][2];
  {
    const bool valid = lr < gt;
    const __nv_bfloat16 *qrow =
        p.q + (static_cast<size_t>(b) * p.hq + hbase + (valid ? lr : 0)) * D;
    auto frag = [&](int at) -> uint32_t {
      if (!valid) return 0u;
      const uint32_t x = *reinterpret_cast<const uint32_t *>(qrow + at);
      const float lim = 65504.f;
      return pack_f16x2(fminf(fmaxf(bf16_lo(x), -lim), lim), fminf(fmaxf(bf16_hi(x), -lim), lim));
    };
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      const int f = 16 * (lc + 4 * (ks >> 2)) + 4 * (ks & 3);
      qf[ks][0] = frag(f);
      qf[ks][1] = frag(f + 2);
    }
  }

  float m0 = -INFINITY, m1 = -INFINITY, d0 = 0.f, d1 = 0.f;  // heads 2lc, 2lc + 1
  float o[kKS][4];
#pragma unroll
  for (int i = 0; i < kKS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  uint8_t *ring = smem + warp * kStages * C::kStageBytes;
  const uint32_t wbase = smem_u32(ring);

  auto page_of = [&](int j) {
    const int pi = page_index(p, j);
    return staged ? s_pages[pi - pg0] : check_page(__ldg(table + pi));
  };
  // kPair, kTile: the pages of the first 32 m-tiles, one per lane, read at once
  int first_pages = -1;
  if (kPair && kTile && t0 + 16 * lane < t1) first_pages = page_of(t0 + 16 * lane);
  auto load_tiles = [&](int i) {
    const int slab0 = t0 + (slab_first + i * slab_step) * kSlab;
    const uint32_t kdst = wbase + (i % kStages) * C::kStageBytes;
    const uint32_t vdst = kdst + C::kSlabBytes;
    constexpr int kCols = D / 16, kPer = 16 * kCols / 32;  // 16-byte chunks per row, per lane
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      const int j0 = slab0 + 16 * mt;
      int page = -1;
      if (kPair) page = __shfl_sync(0xffffffffu, first_pages, ((j0 - t0) >> 4) & 31);
      if (!kPair || j0 - t0 >= 512) page = j0 < t1 ? page_of(j0) : -1;
      const int slot = page_slot(p, j0);
      const size_t head = static_cast<size_t>(page < 0 ? 0 : page) * p.hkv + g;
      const size_t off = page < 0 ? 0 : (head * p.page_size + slot) * D + lane * 16;
      const int row_lo = lo - j0, row_hi = page < 0 ? 0 : t1 - j0;  // rows [row_lo, row_hi) count
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int row = (r * 32 + lane) / kCols, col = (r * 32 + lane) % kCols;
        const uint32_t bytes = row >= row_lo && row < row_hi ? 16u : 0u;
        cp_async_16(kdst + swz8<D>(16 * mt + row, col), p.k + off + r * 512, bytes);
        cp_async_16(vdst + swz8<D>(16 * mt + row, col), p.v + off + r * 512, bytes);
      }
      if (lane < 2) {  // K scale, V scale of the tile
        const size_t at = head * p.scales_per_page +
                          (p.block_shift >= 0 ? slot >> p.block_shift : slot / p.scale_block);
        cp_async_4(kdst + C::kScaleOff + (lane * kSlab + 16 * mt) * 4,
                   (lane == 0 ? p.k_scale : p.v_scale) + (page < 0 ? 0 : at), page < 0 ? 0u : 4u);
      }
    }
  };
  auto load_rows = [&](int i) {
    const int slab0 = t0 + (slab_first + i * slab_step) * kSlab;
    const uint32_t kdst = wbase + (i % kStages) * C::kStageBytes;
    const uint32_t vdst = kdst + C::kSlabBytes;
    constexpr int kCols = D / 16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int idx = r * 32 + lane;
      const int row = idx / kCols, col = idx % kCols;
      const int j = slab0 + row;
      const int page = j < t1 ? page_of(j) : -1;
      const bool ok = page >= 0;
      const size_t off =
          ok ? ((static_cast<size_t>(page) * p.hkv + g) * p.page_size + page_slot(p, j)) * D +
                   col * 16
             : 0;
      cp_async_16(kdst + swz8<D>(row, col), p.k + off, ok ? 16u : 0u);
      cp_async_16(vdst + swz8<D>(row, col), p.v + off, ok ? 16u : 0u);
    }
    if (lane < kSlab) {
      const int j = slab0 + lane;
      const int page = j < t1 ? page_of(j) : -1;
      const bool ok = page >= 0;
      size_t off = 0;
      if (ok) {
        const int slot = page_slot(p, j);
        off = (static_cast<size_t>(page) * p.hkv + g) * p.scales_per_page +
              (p.block_shift >= 0 ? slot >> p.block_shift : slot / p.scale_block);
      }
      cp_async_4(kdst + C::kScaleOff + lane * 4, p.k_scale + off, ok ? 4u : 0u);
      cp_async_4(kdst + C::kScaleOff + (kSlab + lane) * 4, p.v_scale + off, ok ? 4u : 0u);
    }
  };

  auto load_slab = [&](int i) {
    if constexpr (kTile)
      load_tiles(i);
    else
      load_rows(i);
  };

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < my_slabs) load_slab(i);
    cp_async_commit();
  }

  for (int it = 0; it < my_slabs; ++it) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    if (it + kStages - 1 < my_slabs) load_slab(it + kStages - 1);
    cp_async_commit();

    const int slab0 = t0 + (slab_first + it * slab_step) * kSlab;
    const uint8_t *k8 = ring + (it % kStages) * C::kStageBytes;
    const uint8_t *v8 = k8 + C::kSlabBytes;
    const float *ksc = reinterpret_cast<const float *>(k8 + C::kScaleOff);
    const float *vsc = ksc + kSlab;

    // scores in log2 units, and the reference x + log2(vs)
    const bool whole = slab0 >= lo && slab0 + kSlab <= t1;
    float s[kMT][4], vs[kMT][2];
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[mt][e] = 0.f;
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
        mma_f16_16816(s[mt], a, qf[ks][0], qf[ks][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = i == 0 ? r0 : r1;
        const float f = ksc[kTile ? 16 * mt : row] * p.scale_log2;
        vs[mt][i] = vsc[kTile ? 16 * mt : row];
        const float l = fast_log2(fmaxf(fabsf(vs[mt][i]), kMinVScale));
        const bool see = whole || (slab0 + row >= lo && slab0 + row < t1);
        s[mt][2 * i] = see ? s[mt][2 * i] * f : -INFINITY;
        s[mt][2 * i + 1] = see ? s[mt][2 * i + 1] * f : -INFINITY;
        mx0 = fmaxf(mx0, s[mt][2 * i] + l);
        mx1 = fmaxf(mx1, s[mt][2 * i + 1] + l);
      }
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
    const float base0 = mn0 == -INFINITY ? 0.f : mn0;
    const float base1 = mn1 == -INFINITY ? 0.f : mn1;
    const float al0 = fast_exp2(m0 - base0), al1 = fast_exp2(m1 - base1);
    m0 = mn0;
    m1 = mn1;
    float sum0 = 0.f, sum1 = 0.f;
    uint32_t pb[kMT][2];  // w = p * vs as fp16 (11 bits), the B fragments of P^T
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      const float p0 = fast_exp2(s[mt][0] - base0), p1 = fast_exp2(s[mt][1] - base1);
      const float p2 = fast_exp2(s[mt][2] - base0), p3 = fast_exp2(s[mt][3] - base1);
      sum0 += p0 + p2;
      sum1 += p1 + p3;
      pb[mt][0] = movmatrix_trans(pack_f16x2(p0 * vs[mt][0], p1 * vs[mt][0]));
      pb[mt][1] = movmatrix_trans(pack_f16x2(p2 * vs[mt][1], p3 * vs[mt][1]));
    }
    d0 = d0 * al0 + sum0;
    d1 = d1 * al1 + sum1;
#pragma unroll
    for (int dt = 0; dt < kKS; ++dt) {
      o[dt][0] *= al0;
      o[dt][1] *= al1;
      o[dt][2] *= al0;
      o[dt][3] *= al1;
    }
    // O^T += V^T W^T: MMA rows lr / lr + 8 of dim tile dt stand for dims
    // (D / 8) lr + 2 dt and + 1: one (D / 8)-byte load per token holds the
    // lane's bytes of every dim tile, paired across tokens by a byte permute
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
        mma_f16_16816(o[dt], a, pb[mt][0], pb[mt][1]);
      }
    }
  }
  cp_async_wait<0>();

#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    d0 += __shfl_xor_sync(0xffffffffu, d0, off);
    d1 += __shfl_xor_sync(0xffffffffu, d1, off);
  }

  // Stage the state in shared memory: m, d [8] and o [8][D] per warp.
  constexpr int kState = (2 + D) * kMaxGroup;
  if (kPair)
    __syncwarp();  // the ring is this warp's own
  else
    __syncthreads();  // every warp is done with its ring
  float *st = kPair ? reinterpret_cast<float *>(ring)
                    : reinterpret_cast<float *>(smem) + warp * kState;
  if (lr == 0) {
    st[2 * lc] = m0;
    st[2 * lc + 1] = m1;
    st[8 + 2 * lc] = d0;
    st[8 + 2 * lc + 1] = d1;
  }
#pragma unroll
  for (int dt = 0; dt < kKS; ++dt) {
    const int dim = (D / 8) * lr + 2 * dt;
    float *x = st + 16 + 2 * lc * D + dim;
    *reinterpret_cast<float2 *>(x) = make_float2(o[dt][0], o[dt][2]);
    *reinterpret_cast<float2 *>(x + D) = make_float2(o[dt][1], o[dt][3]);
  }
  if (kPair)
    __syncwarp();
  else
    __syncthreads();

  // kLanes threads per head, kPer output dims each
  constexpr int kLanes = kPair ? 4 : 16, kPer = D / kLanes;
  constexpr int kStates = kPair ? 1 : kWarps;
  const int tid = kPair ? lane : static_cast<int>(threadIdx.x);
  const int hh = tid / kLanes, sub = tid % kLanes, c0 = sub * kPer;
  const bool head_ok = hh < gt;
  const float *all = kPair ? st : reinterpret_cast<const float *>(smem);
  const float sink = p.sinks != nullptr && split == 0 && head_ok ? p.sinks[hbase + hh] * kLog2e
                                                                 : -INFINITY;
  float M = sink;
#pragma unroll
  for (int w = 0; w < kStates; ++w) M = fmaxf(M, all[w * kState + hh]);
  const float baseM = M == -INFINITY ? 0.f : M;
  float Dn = fast_exp2(sink - baseM), acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll
  for (int w = 0; w < kStates; ++w) {
    const float *x = all + w * kState;
    const float f = fast_exp2(x[hh] - baseM);
    Dn += f * x[8 + hh];
#pragma unroll
    for (int e = 0; e < kPer; e += 4) {
      const float4 ov = *reinterpret_cast<const float4 *>(x + 16 + hh * D + c0 + e);
      acc[e] += f * ov.x;
      acc[e + 1] += f * ov.y;
      acc[e + 2] += f * ov.z;
      acc[e + 3] += f * ov.w;
    }
  }
  const float inv = Dn > 0.f ? 1.f / Dn : 0.f;
  const float blse = Dn > 0.f ? (M + fast_log2(Dn)) * kLn2 : -INFINITY;
  const size_t row_h = static_cast<size_t>(b) * p.hq + hbase + hh;
  auto store_out = [&](const float *x, float mul) {
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
      *reinterpret_cast<uint2 *>(p.out + row_h * D + c0 + e) =
          make_uint2(pack_bf16x2(x[e] * mul, x[e + 1] * mul),
                     pack_bf16x2(x[e + 2] * mul, x[e + 3] * mul));
  };
  if (nsplit == 1) {
    if (head_ok) {
      store_out(acc, inv);
      if (p.lse != nullptr && sub == 0) p.lse[row_h] = blse;
    }
    return;
  }
  if constexpr (kMerge == kCluster) {
    float *cs = reinterpret_cast<float *>(smem) + kWarps * kState;  // m, d [8] and o [8][D]
    if (sub == 0) {
      cs[hh] = M;
      cs[8 + hh] = Dn;
    }
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
      *reinterpret_cast<float4 *>(cs + 16 + hh * D + c0 + e) =
          make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    cluster_sync();
    if (head_ok && hh % nsplit == split) {
      const uint32_t at = smem_u32(cs);
      float Mx = -INFINITY;
      for (int k = 0; k < nsplit; ++k)
        Mx = fmaxf(Mx, cluster_ld(cluster_map(at + 4 * hh, k)));
      const float base = Mx == -INFINITY ? 0.f : Mx;
      float W = 0.f, r[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) r[e] = 0.f;
#pragma unroll 4
      for (int k = 0; k < nsplit; ++k) {
        const uint32_t other = cluster_map(at, k);
        const float f = fast_exp2(cluster_ld(other + 4 * hh) - base);
        W += f * cluster_ld(other + 4 * (8 + hh));
#pragma unroll
        for (int e = 0; e < kPer; e += 4) {
          const float4 ov = cluster_ld4(other + 4 * (16 + hh * D + c0 + e));
          r[e] += f * ov.x;
          r[e + 1] += f * ov.y;
          r[e + 2] += f * ov.z;
          r[e + 3] += f * ov.w;
        }
      }
      store_out(r, W > 0.f ? 1.f / W : 0.f);
      if (p.lse != nullptr && sub == 0)
        p.lse[row_h] = W > 0.f ? (Mx + fast_log2(W)) * kLn2 : -INFINITY;
    }
    cluster_sync();  // no block leaves while its state may be read
  }
  if constexpr (kMerge == kCounter) {
    const size_t rows_hq = static_cast<size_t>(p.batch) * p.hq;
    if (head_ok) {
#pragma unroll
      for (int e = 0; e < kPer; e += 4)
        *reinterpret_cast<float4 *>(p.part_o + (split * rows_hq + row_h) * D + c0 + e) =
            make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
      if (sub == 0) p.part_lse[split * rows_hq + row_h] = blse;
    }
    __threadfence();
    __syncthreads();
    __shared__ int s_last;
    if (tid == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zeroed
      s_last = atomicAdd(p.counters + cidx, 1u) == static_cast<unsigned>(nsplit - 1);
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the last block merges the partials of this (sequence, KV head), in order;
    // the 16 lanes of a head find the maximum together
    float Mx = -INFINITY;
    for (int k = sub; k < nsplit; k += kLanes)
      if (head_ok) Mx = fmaxf(Mx, __ldcg(p.part_lse + k * rows_hq + row_h));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, o));
    if (!head_ok) return;
    float W = 0.f, r[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) r[e] = 0.f;
    if (Mx != -INFINITY) {
#pragma unroll 8
      for (int k = 0; k < nsplit; ++k) {
        const float w = fast_exp2((__ldcg(p.part_lse + k * rows_hq + row_h) - Mx) * kLog2e);
        W += w;
#pragma unroll
        for (int e = 0; e < kPer; e += 4) {
          const float4 ov = __ldcg(reinterpret_cast<const float4 *>(
              p.part_o + (k * rows_hq + row_h) * D + c0 + e));
          r[e] += w * ov.x;
          r[e + 1] += w * ov.y;
          r[e + 2] += w * ov.z;
          r[e + 3] += w * ov.w;
        }
      }
    }
    store_out(r, W > 0.f ? 1.f / W : 0.f);
    if (p.lse != nullptr && sub == 0)
      p.lse[row_h] = W > 0.f ? Mx + fast_log2(W) * kLn2 : -INFINITY;
  }
}

int log2_or_minus1(int x) {
  if (x <= 0 || (x & (x - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace

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
  const DecodeWorkspace w = decode_workspace_layout(a.batch, a.hq, a.hkv, a.plan, a.head_dim);
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  p.part_o = reinterpret_cast<float *>(ws);
  p.part_lse = reinterpret_cast<float *>(ws + w.off_lse);
  p.counters = reinterpret_cast<unsigned int *>(ws + w.off_counters);

  const bool split = a.plan.max_splits > 1;
  const int64_t pairs = static_cast<int64_t>(a.batch) * a.hkv * p.nht;
  // Clusters win while all of their blocks fit the GPU at once (one 1000-token
  // context 6.7 -> 5.2 us); beyond that the blocks of a cluster wait for slots on
  // one another (64 contexts of 1k-8k: 71 -> 84 us).
  const bool cluster = split && a.plan.max_splits <= kMaxCluster &&
                       pairs * a.plan.max_splits <= 152 * kBlocksPerSm;
  const bool counters = split && !cluster;
  if (counters) {
    const int blocks = static_cast<int>((pairs + 255) / 256 < 1024 ? (pairs + 255) / 256 : 1024);
    zero_counters_kernel<<<blocks, 256, 0, stream>>>(p.counters, pairs);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int span = a.window > 0 && a.window < a.max_seqlen_k ? a.window : a.max_seqlen_k;
  const bool pair = !split && span <= kPairMaxSpan;
  const dim3 grid = pair ? dim3(static_cast<unsigned>((pairs + kWarps - 1) / kWarps))
                         : dim3(a.plan.max_splits, a.hkv * p.nht, a.batch);
  auto go = [&](auto kernel, int smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && cluster && a.plan.max_splits > 8)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (cluster) {
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(a.plan.max_splits);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
    } else {
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = split ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  };
  const bool tile = a.page_size % 16 == 0 && a.scale_block % 16 == 0;
  auto pick = [&](auto dim, auto merge) {
    constexpr int D = decltype(dim)::value;
    constexpr Merge kM = decltype(merge)::value;
    constexpr int smem = Cfg<D>::kSmemBytes;
    return tile ? go(decode_block_kernel<D, kM, true>, smem)
                : go(decode_block_kernel<D, kM, false>, smem);
  };
  auto pick_merge = [&](auto dim) {
    if (pair) return pick(dim, std::integral_constant<Merge, kPairs>());
    if (counters) return pick(dim, std::integral_constant<Merge, kCounter>());
    return pick(dim, std::integral_constant<Merge, kCluster>());
  };
  return a.head_dim == 128 ? pick_merge(std::integral_constant<int, 128>())
                           : pick_merge(std::integral_constant<int, 64>());
}

cudaError_t decode_block_read_error(cudaStream_t stream, int *code) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_decode_block_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_decode_block_error, &zero, sizeof(int));
  return e;
}

}  // namespace sinkattn
