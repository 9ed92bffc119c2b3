// Verification of a tree of drafted tokens against the target's probabilities.
//
// p is the target's distribution after the current node, q the one its children were
// drafted from. A child x is accepted with probability min(1, p_k(x) / q(x)), where p_0 = p
// and, after k rejections, p_k is what is left of the target: max(p_{k-1} - q, 0),
// normalised. With v_k = S_k p_k, S_k = sum v_k (S_0 = 1) the normalisation goes away:
//
//   v_k = max(v_{k-1} - S_{k-1} q, 0) = max(p - A_k q, 0),  A_k = S_0 + .. + S_{k-1}
//
// (clamping first changes nothing, since q only takes more off). So a rejection costs
// one scalar, S_k, a sum over the vocabulary, and only if another child is then tested;
// a test is u S_k q(x) < v_k(x). At the end the next token is the smallest x with
// v(0) + .. + v(x) > u_0 sum(v). Without draft probabilities a drafted token is certain
// (q is 1 at it): v_k is p without the rejected tokens and S_k = S_{k-1} - v_{k-1}(x_k).
//
// The answer is whole numbers that hang on sums over 10^5 terms, so the sums are exact:
// probabilities become multiples of 2^-60 in 64-bit integers (every float32 from 2^-37 up
// without rounding), whose sum is the same in every order, any split over blocks. A is
// their sum too, of up to 1023 siblings' S: it may pass 16, where it takes more than 64
// bits, and A q, rounded down, is cut to 64, far above any p.
//
// A cluster of blocks takes a sequence and walks its tree in step: every block gathers
// the few probabilities that the tests need, takes the same decisions, and sums its
// share of the vocabulary where a sum is needed; totals pass through distributed shared
// memory. Bound by HBM: one row of p and one of q per sequence.
#include <math.h>

#include "launch.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

__device__ int g_verify_error;

// Trees of 8 over 131072 tokens, with 8, 4 and 2 blocks a cluster: one of them 12, 18 and 26 us,
// 64 of them 42, 55 and 87, 200 of them 87, 90 and 117. Over 32768 tokens 8 blocks are
// behind only from about 200 trees on (47, 37 and 39 us). Blocks of 512 threads took 78 us
// where 256 took 60 (64 trees of 16 over 131072): small blocks fill the SMs evenly.
constexpr int kThreads = 256, kWarps = kThreads / 32, kCluster = 8;
constexpr int kNodes = 256;                  // nodes whose data is held at a time
constexpr int kRejected = kVerifyMaxTokens;  // rejected children of a node, at most

struct VerifyParams {
  const float *p, *q;
  const int64_t *tokens;
  const int32_t *parents, *cu;
  const float *u;
  int batch, vocab, max_q;
  int32_t *path, *num;
  int64_t *next;
};

constexpr uint64_t kOne = 1ull << 60;

// x >> n, 0 for n above 63
__device__ __forceinline__ uint64_t shift_down(uint64_t x, uint32_t n) {
  uint64_t y;
  asm("shr.u64 %0, %1, %2;" : "=l"(y) : "l"(x), "r"(n));
  return y;
}
__device__ __forceinline__ uint32_t bits01(float x) {
  return __float_as_uint(fminf(fmaxf(x, 0.f), 1.f));
}
__device__ __forceinline__ uint32_t significand(uint32_t b) { return (b & 0x7fffffu) | 0x800000u; }

// x in [0, 1] as a multiple of 2^-60, rounded down: the 24-bit significand at bit 37
// and shifted down by the exponent. NaN and negative values count as 0, above 1 as 1.
__device__ __forceinline__ uint64_t fixed60(float x) {
  const uint32_t b = bits01(x);
  return shift_down(static_cast<uint64_t>(significand(b) << 5) << 32, 127u - (b >> 23));
}

// A sum of up to 1023 values below 16, in 2^-60: hi 2^64 + lo.
struct Mass {
  uint64_t lo;
  uint32_t hi;
  __device__ __forceinline__ bool is(uint64_t x) const { return hi == 0 && lo == x; }
  __device__ __forceinline__ bool below8() const { return hi == 0 && lo < 8 * kOne; }
  __device__ __forceinline__ void add(uint64_t x) {
    lo += x;
    hi += lo < x ? 1u : 0u;
  }
  __device__ __forceinline__ double value() const {
    return hi * 16.0 + static_cast<double>(lo) * 0x1p-60;
  }
};

// a q in 2^-60, rounded down, for q in [0, 1] (clamped): q's significand times a's 32-bit
// words, shifted down by 23 and then by the exponent. Below 8 the first shift leaves 64
// bits.
__device__ __forceinline__ uint64_t times_below8(uint64_t a, float q) {
  const uint32_t b = bits01(q), m = significand(b);
  const uint64_t t0 = static_cast<uint64_t>(m) * static_cast<uint32_t>(a);
  const uint64_t t1 = static_cast<uint64_t>(m) * static_cast<uint32_t>(a >> 32) + (t0 >> 32);
  return shift_down((t1 << 9) | (static_cast<uint32_t>(t0) >> 23), 127u - (b >> 23));
}
// The same for any a; the largest number where the product takes more than 64 bits.
__device__ __forceinline__ uint64_t times(const Mass &a, float q) {
  const uint32_t b = bits01(q), m = significand(b), n = 127u - (b >> 23);
  const uint64_t t0 = static_cast<uint64_t>(m) * static_cast<uint32_t>(a.lo);
  const uint64_t t1 = static_cast<uint64_t>(m) * static_cast<uint32_t>(a.lo >> 32) + (t0 >> 32);
  const uint64_t t2 = static_cast<uint64_t>(m) * a.hi + (t1 >> 32);  // of 2^64
  const uint64_t low = (t2 << 41) | (static_cast<uint64_t>(static_cast<uint32_t>(t1)) << 9) |
                       (static_cast<uint32_t>(t0) >> 23);
  const uint64_t top = t2 >> 23;
  if (n >= 64) return shift_down(top, n - 64);
  if (shift_down(top, n) != 0) return ~0ull;
  return n == 0 ? low : (top << (64 - n)) | (low >> n);
}

// What is left of the target at one token, by how large A is.
enum class Taken { kNone, kOnce, kBelow8, kAny };
__device__ __forceinline__ Taken how(const Mass &a) {
  return a.is(0) ? Taken::kNone : a.is(kOne) ? Taken::kOnce
                              : a.below8()   ? Taken::kBelow8
                                             : Taken::kAny;
}
template <Taken kHow>
__device__ __forceinline__ uint64_t rest(float p, float q, const Mass &taken) {
  const uint64_t a = fixed60(p);
  if (kHow == Taken::kNone) return a;
  const uint64_t b = kHow == Taken::kOnce     ? fixed60(q)
                     : kHow == Taken::kBelow8 ? times_below8(taken.lo, q)
                                              : times(taken, q);
  return a > b ? a - b : 0;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ uint64_t cluster_ld_u64(uint32_t addr) {
  uint64_t x;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(addr) : "memory");
  return x;
}

struct Shared {
  uint64_t warp_total[kWarps];
  uint64_t block_total[2];  // of the present pass and of the one before it
  float p[kNodes], q[kNodes], u[kNodes];
  int64_t token[kNodes];
  int parent[kNodes];
  int rejected[kRejected];  // tokens of the current node's rejected children (no draft)
};

// Four values of a row from index i of its 16-byte grid on; the row's own elements are
// [a, end) of that grid.
__device__ __forceinline__ float4 load4(const float *grid, int i, int a, int end) {
  if (i >= a && i + 4 <= end) return __ldg(reinterpret_cast<const float4 *>(grid + i));
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i >= a && i < end) x.x = __ldg(grid + i);
  if (i + 1 >= a && i + 1 < end) x.y = __ldg(grid + i + 1);
  if (i + 2 >= a && i + 2 < end) x.z = __ldg(grid + i + 2);
  if (i + 3 >= a && i + 3 < end) x.w = __ldg(grid + i + 3);
  return x;
}

// Sum of what is left over a warp's share [seg, seg_end) of a row's grid, this lane's part.
template <Taken kHow>
__device__ __forceinline__ uint64_t share_sum(const float *pg, const float *qg, int seg, int a,
                                              int end, int seg_end, const Mass &taken) {
  uint64_t s = 0;
  constexpr int kU = 2;
  for (int i0 = seg + 4 * static_cast<int>(threadIdx.x & 31); i0 < seg_end; i0 += 128 * kU) {
    float4 x[kU], y[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int i = i0 + 128 * j;
      x[j] = y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < seg_end) {
        x[j] = load4(pg, i, a, end);
        if (kHow != Taken::kNone) y[j] = load4(qg, i, a, end);
      }
    }
#pragma unroll
    for (int j = 0; j < kU; ++j)
      s += rest<kHow>(x[j].x, y[j].x, taken) + rest<kHow>(x[j].y, y[j].y, taken) +
           rest<kHow>(x[j].z, y[j].z, taken) + rest<kHow>(x[j].w, y[j].w, taken);
  }
  return s;
}

__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyParams g, int cluster) {
  __shared__ Shared sm;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const int64_t first = g.cu[b];
  int n = g.cu[b + 1] - g.cu[b];
  if (n > g.max_q || n < 0) {
    if (threadIdx.x == 0 && rank == 0) atomicExch(&g_verify_error, kErrBadLength);
    n = min(max(n, 0), g.max_q);
  }
  int32_t *path = g.path + static_cast<int64_t>(b) * g.max_q;
  if (n == 0) {  // the same in every block of the cluster
    if (rank == 0) {
      for (int i = threadIdx.x; i < g.max_q; i += kThreads) path[i] = -1;
      if (threadIdx.x == 0) g.num[b] = 0, g.next[b] = -1;
    }
    return;
  }
  // replaced where a token is found, behind the first pass's cluster barrier
  if (rank == 0 && threadIdx.x == 0) g.next[b] = -1;

  // this warp's share of a row: [seg, seg_end) of the grid that starts at the row's last
  // 16-byte boundary at or before its first element
  const int seg_len = ((g.vocab + 3 + cluster * kWarps - 1) / (cluster * kWarps) + 127) / 128 * 128;
  const int64_t seg64 = static_cast<int64_t>(rank * kWarps + wid) * seg_len;
  const int seg = static_cast<int>(min(seg64, static_cast<int64_t>(g.vocab) + 3));

  int num_rejected = 0;
  int passes = 0;
  // Sum over the vocabulary of what is left at node `cur`: warp_total, block_total, the sum.
  auto total = [&](int cur, const Mass &taken) -> uint64_t {
    const int64_t row = (first + cur) * g.vocab;
    const int a = static_cast<int>(row & 3), end = a + g.vocab;
    const float *pg = g.p + (row - a), *qg = g.q != nullptr ? g.q + (row - a) : nullptr;
    const int seg_end = min(seg + seg_len, end);
    const Taken mode = qg != nullptr ? how(taken) : Taken::kNone;
    uint64_t s;
    if (mode == Taken::kNone)
      s = share_sum<Taken::kNone>(pg, qg, seg, a, end, seg_end, taken);
    else if (mode == Taken::kOnce)
      s = share_sum<Taken::kOnce>(pg, qg, seg, a, end, seg_end, taken);
    else if (mode == Taken::kBelow8)
      s = share_sum<Taken::kBelow8>(pg, qg, seg, a, end, seg_end, taken);
    else
      s = share_sum<Taken::kAny>(pg, qg, seg, a, end, seg_end, taken);
    s = warp_sum(s);
    for (int k = 0; k < num_rejected; ++k) {
      const int i = sm.rejected[k] + a;
      if (i >= seg && i < seg_end) s -= fixed60(__ldg(pg + i));
    }
    __syncthreads();  // the last pass's warp_total has been read
    if (lane == 0) sm.warp_total[wid] = s;
    __syncthreads();
    const int slot = passes & 1;
    ++passes;
    if (threadIdx.x == 0) {
      uint64_t t = 0;
      for (int w = 0; w < kWarps; ++w) t += sm.warp_total[w];
      sm.block_total[slot] = t;
    }
    cluster_sync();
    uint64_t sum = 0;
    for (int r = 0; r < cluster; ++r)
      sum += cluster_ld_u64(cluster_map(smem_u32(&sm.block_total[slot]), r));
    return sum;
  };

  // ------------------------------------------------------------------ the walk
  int cur = 0, accepted = 1;
  Mass taken{0, 0};   // A, and as a double
  double off = 0.0;
  double left = 1.0;  // S
  uint64_t left60 = kOne;
  bool stale = false;  // S has to be summed before the next test
  for (int base = 0; base < n; base += kNodes) {
    const int cnt = min(kNodes, n - base);
    __syncthreads();
    for (int i = threadIdx.x; i < cnt; i += kThreads) {
      const int t = base + i;
      int parent = t - 1;
      if (g.parents != nullptr) {
        parent = g.parents[first + t];
        if (parent >= t || parent < -1) {
          if (rank == 0) atomicExch(&g_verify_error, kErrBadPage);
          parent = -1;
        }
      }
      const int64_t token = g.tokens[first + t];
      if (t > 0 && (token < 0 || token >= g.vocab)) {
        if (rank == 0) atomicExch(&g_verify_error, kErrBadPage);
        parent = -1;
      }
      if (t == 0) parent = -1;
      sm.parent[i] = parent;
      if (parent >= 0) {
        const int64_t at = (first + parent) * g.vocab + token;
        sm.token[i] = token;
        sm.p[i] = __ldg(g.p + at);
        sm.q[i] = g.q != nullptr ? __ldg(g.q + at) : 1.f;
        sm.u[i] = g.u[first + t];
      }
    }
    __syncthreads();
    // every warp of every block takes the same decisions
    for (int s = 0; s < cnt; s += 32) {
      const int mine = s + lane < cnt ? sm.parent[s + lane] : -1;
      unsigned todo = __ballot_sync(0xffffffffu, mine == cur);
      while (todo != 0) {
        const int j = __ffs(todo) - 1, i = s + j;
        if (stale) {
          left60 = total(cur, taken);
          left = static_cast<double>(left60) * 0x1p-60;
          stale = false;
        }
        const double p = fminf(fmaxf(sm.p[i], 0.f), 1.f);
        double q = 1.0, v = p;
        if (g.q != nullptr) {
          q = fminf(fmaxf(sm.q[i], 0.f), 1.f);
          v = fmax(__dsub_rn(p, __dmul_rn(off, q)), 0.0);
        } else {
          for (int k = 0; k < num_rejected; ++k)
            if (sm.rejected[k] == sm.token[i]) v = 0.0;
        }
        const bool ok = static_cast<double>(sm.u[i]) * left * q < v;
        if (ok) {
          cur = base + i;
          if (rank == 0 && threadIdx.x == 0) path[accepted] = cur;
          ++accepted;
          taken = Mass{0, 0}, off = 0.0, left = 1.0, left60 = kOne, stale = false;
          num_rejected = 0;
          todo = __ballot_sync(0xffffffffu, mine == cur) & ~((2u << j) - 1u);
        } else {
          if (g.q != nullptr) {
            taken.add(left60);
            off = taken.value();
            stale = true;
          } else {
            left = __dsub_rn(left, v);
            if (v > 0.0) {
              __syncthreads();
              if (threadIdx.x == 0) sm.rejected[num_rejected] = static_cast<int>(sm.token[i]);
              __syncthreads();
              ++num_rejected;
            }
          }
          todo &= todo - 1;
        }
      }
    }
  }
  if (rank == 0) {
    for (int i = accepted + threadIdx.x; i < g.max_q; i += kThreads) path[i] = -1;
    if (threadIdx.x == 0) path[0] = 0, g.num[b] = accepted;
  }

  // ------------------------------------------------------------- the next token
  uint64_t sum = total(cur, taken);
  if (sum == 0 && (!taken.is(0) || num_rejected > 0)) {
    taken = Mass{0, 0};  // nothing is left (sums that are not 1): the target itself
    num_rejected = 0;
    sum = total(cur, taken);
  }
  if (sum == 0) {
    if (rank == 0 && threadIdx.x == 0) atomicExch(&g_verify_error, kErrBadValue);
  } else {
    const float u0 = g.u[first];
    const float uc = u0 >= 0.f ? fminf(u0, 1.f - 0x1p-24f) : 0.f;
    // the running sum is whole: it exceeds u sum where it exceeds that rounded down
    uint64_t aim = times(Mass{sum, 0}, uc);
    const int slot = (passes - 1) & 1;
    bool here = true;
    for (int r = 0; r < rank; ++r) {
      const uint64_t t = cluster_ld_u64(cluster_map(smem_u32(&sm.block_total[slot]), r));
      if (aim < t) {  // in an earlier block
        here = false;
        break;
      }
      aim -= t;
    }
    here = here && aim < sm.block_total[slot];
    if (here) {
      for (int w = 0; w < wid; ++w) {
        if (aim < sm.warp_total[w]) {
          here = false;
          break;
        }
        aim -= sm.warp_total[w];
      }
      here = here && aim < sm.warp_total[wid];
    }
    if (here) {  // this warp's share holds the token
      const int64_t row = (first + cur) * g.vocab;
      const int a = static_cast<int>(row & 3), end = a + g.vocab;
      const float *pg = g.p + (row - a), *qg = g.q != nullptr ? g.q + (row - a) : nullptr;
      const bool with_q = qg != nullptr && !taken.is(0);
      const Taken mode = with_q ? how(taken) : Taken::kNone;
      const auto left_at = [&](float p, float q) {
        return mode == Taken::kNone   ? rest<Taken::kNone>(p, q, taken)
               : mode == Taken::kOnce ? rest<Taken::kOnce>(p, q, taken)
                                      : rest<Taken::kAny>(p, q, taken);
      };
      const int seg_end = min(seg + seg_len, end);
      for (int i0 = seg; i0 < seg_end; i0 += 128) {
        const int i = i0 + 4 * lane;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (i < seg_end) {
          x = load4(pg, i, a, end);
          if (with_q) y = load4(qg, i, a, end);
        }
        uint64_t v[4] = {left_at(x.x, y.x), left_at(x.y, y.y), left_at(x.z, y.z),
                         left_at(x.w, y.w)};
        for (int k = 0; k < num_rejected; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (sm.rejected[k] + a == i + e) v[e] = 0;
        const uint64_t own = v[0] + v[1] + v[2] + v[3];
        uint64_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t below = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += below;
        }
        const unsigned over = __ballot_sync(0xffffffffu, upto > aim);
        if (over != 0) {
          if (lane == __ffs(over) - 1) {
            uint64_t at = upto - own + v[0];
            int e = 0;
            if (at <= aim) e = 1, at += v[1];
            if (e == 1 && at <= aim) e = 2, at += v[2];
            if (e == 2 && at <= aim) e = 3;
            g.next[b] = i + e - a;
          }
          break;
        }
        aim -= __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  cluster_sync();  // no block ends while another reads its totals
}

}  // namespace

cudaError_t launch_verify(const VerifyLaunch &a, cudaStream_t stream) {
  VerifyParams p;
  p.p = a.target_probs, p.q = a.draft_probs;
  p.tokens = a.tokens, p.parents = a.parents, p.cu = a.cu_q, p.u = a.uniforms;
  p.batch = a.batch, p.vocab = a.vocab, p.max_q = a.max_seqlen_q;
  p.path = a.path, p.num = a.num_path, p.next = a.next_tokens;
  const int cluster = kCluster;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel, p, cluster);
}

cudaError_t verify_read_error(cudaStream_t stream, int *code) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_verify_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_verify_error, &zero, sizeof(int));
  return e;
}

}  // namespace sinkattn
