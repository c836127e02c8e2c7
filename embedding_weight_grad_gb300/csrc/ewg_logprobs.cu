// Token log probabilities, entropies and best alternatives of rows of logits, and the
// gradient of the first two.
//
// Per row z[0..V) with token t and scale s > 0: m = max z, x_v = s (z_v - m),
//
//     1 + R = sum_v exp(x_v)          (R leaves out one occurrence of the maximum)
//     log_sum = log1p(R)
//     log p_v = x_v - log_sum
//     entropy = log_sum - (sum_v exp(x_v) x_v) / (1 + R)
//
// and for the gradients G of log p_t and E of the entropy
//
//     dz_v = s (G ([v = t] - p_v) - E p_v (log p_v + entropy)).
//
// Keeping the maximum's own term (exactly 1) out of the sum keeps the digits of the other
// terms where a row is all but sure of one token: log p_t and the entropy of such a row are
// about -R, and 1 + R in 32 bits would round R away.
//
// Both kernels are bound by the one read of the logits (and the one write of the gradient):
// 8192 x 129280 bf16 without padding takes 311 us (6.8 TB/s; 348 with 8 alternatives, whose logits
// are mostly gone from L2 when they are read again), its gradient 608 us (7.0 TB/s).
#include <cfloat>

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "ewg.h"
#include "ewg_internal.cuh"
#include "ewg_ops.cuh"
#include "ewg_ptx.cuh"

namespace cg = cooperative_groups;

namespace ewg {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Exponents (base 2) are clamped here: 2^-200 is 0 in 32 bits, and 0 * -200 is 0 where
// 0 * -inf (a masked logit) would be NaN.
constexpr float kLowestExponent = -200.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max that returns NaN if either is NaN (a NaN logit must reach the sums)
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// 16 bytes of a row of T: kE elements.
template <typename T>
struct Vec;

template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kE = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ float2 pair(uint4 v, int i) {
    const uint32_t u = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 elementwise_max(uint4 a, uint4 b) {
    return make_uint4(max2(a.x, b.x), max2(a.y, b.y), max2(a.z, b.z), max2(a.w, b.w));
  }
  static __device__ __forceinline__ float max_of(uint4 a) {
    const uint32_t u = max2(max2(a.x, a.y), max2(a.z, a.w));
    return fmaxf(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint4 pack(const float2* g) {
    uint4 o;
    uint32_t* w = &o.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(g[i].y), "f"(g[i].x));
    return o;
  }
  static __device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

template <>
struct Vec<float> {
  static constexpr int kE = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float2 pair(uint4 v, int i) {
    return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                  : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 elementwise_max(uint4 a, uint4 b) {
    return make_uint4(max1(a.x, b.x), max1(a.y, b.y), max1(a.z, b.z), max1(a.w, b.w));
  }
  static __device__ __forceinline__ float max_of(uint4 a) {
    return __uint_as_float(max1(max1(a.x, a.y), max1(a.z, a.w)));
  }
  static __device__ __forceinline__ uint32_t max1(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ uint4 pack(const float2* g) {
    return make_uint4(__float_as_uint(g[0].x), __float_as_uint(g[0].y), __float_as_uint(g[1].x),
                      __float_as_uint(g[1].y));
  }
  static __device__ __forceinline__ float load1(const float* p) { return *p; }
  static __device__ __forceinline__ void store1(float* p, float v) { *p = v; }
};

// Streaming 16-byte load: every logit is read once by the main loops.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Unsigned numbers in the order of the floats (-0 is first made +0).
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

__device__ __forceinline__ long long target_of(const void* targets, int is64, long long row) {
  return is64 ? static_cast<const long long*>(targets)[row] : static_cast<const int*>(targets)[row];
}

// Whether one of the targets i, i + step, i + 2 step, ... is V or more.
__device__ __forceinline__ bool bad_target(const void* targets, int is64, int n, int V, long long i, long long step) {
  bool bad = false;
  constexpr int kU = 8;
  for (; i < n; i += step * kU) {
    long long t[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) t[u] = i + u * step < n ? target_of(targets, is64, i + u * step) : -1;
#pragma unroll
    for (int u = 0; u < kU; ++u) bad |= t[u] >= V;
  }
  return bad;
}

// Writes the call's device status: EWG_ERR_ID_OUT_OF_RANGE if a target is V or more.
// Run by all `threads` threads of one block.
__device__ void report_targets(const void* targets, int is64, int n, int V, int* status, int threads) {
  const bool bad = __syncthreads_or(bad_target(targets, is64, n, V, threadIdx.x, threads));
  if (threadIdx.x == 0) *status = bad ? kStatusBadId : kStatusOk;
}

// The same by a whole grid, to a status that is kStatusOk before.
__global__ void __launch_bounds__(256) targets_kernel(const void* targets, int is64, int n, int V, int* status) {
  const long long at = blockIdx.x * 256LL + threadIdx.x;
  if (bad_target(targets, is64, n, V, at, gridDim.x * 256LL)) *status = kStatusBadId;
}

// A row's (or a slice's) statistics: maximum, the sum of the other terms relative to it (-1
// where there is no finite logit: the terms then add up to 1 + R = 0), and the sum of
// term * exponent (base 2).
struct Stats {
  float m, R, T;
};

// Keys order candidates by logit, then by lower id; 0 is "none".  A list of best candidates
// is a warp's: lane l holds the l-th best key.
using Key = unsigned long long;

__device__ __forceinline__ Key key_of(float z, uint32_t id) {
  return (static_cast<Key>(order_of(z)) << 32) | (~id);
}

// Compare-exchange with the lane `distance` away: the larger key stays where `larger`.
__device__ __forceinline__ Key exchange(Key k, int distance, bool larger) {
  const Key o = __shfl_xor_sync(kAll, k, distance);
  return (o > k) == larger ? o : k;
}

// The lanes' keys as a list, best first (bitonic network).
__device__ __forceinline__ Key sort_keys(Key k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d; d /= 2) k = exchange(k, d, ((lane & d) == 0) == ((lane & size) == 0 || size == 32));
  return k;
}

// The best 32 of two lists, as a list.
__device__ __forceinline__ Key merge_lists(Key a, Key b, int lane) {
  const Key r = __shfl_sync(kAll, b, 31 - lane);
  Key k = a > r ? a : r;
#pragma unroll
  for (int d = 16; d; d /= 2) k = exchange(k, d, (lane & d) == 0);
  return k;
}

// Inserts the lanes' keys (0: nothing) into a list, one after the other, while they belong
// among its best `top`; `worst` is the list's top-th key.
__device__ __forceinline__ void insert_keys(Key& list, Key& worst, Key key, int top, int lane) {
  unsigned mask = __ballot_sync(kAll, key > worst);
  while (mask) {
    const int src = __ffs(mask) - 1;
    mask &= mask - 1;
    const Key k = __shfl_sync(kAll, key, src);
    if (k <= worst) continue;                       // the list has improved meanwhile
    const int pos = __popc(__ballot_sync(kAll, list > k));
    const Key above = __shfl_up_sync(kAll, list, 1);
    list = lane < pos ? list : lane == pos ? k : above;
    worst = __shfl_sync(kAll, list, top - 1);
  }
}

constexpr int kBatch = 4;            // vectors a thread has in flight
constexpr int kMaxCluster = 8;       // blocks that share a row, at most

template <int kT>
struct GroupSmem {
  static constexpr int kWarps = kT / 32;
  static constexpr int kSets = kT < 64 ? kT : 64;    // sets of neighbouring threads
  static constexpr int kCandidates = kT == 512 ? 256 : 64;
  alignas(16) uint32_t maxima[kSets];   // order_of the sets' maxima
  uint32_t tau;
  int num_tasks, num_candidates;
  uint16_t tasks[kT];
  Key candidates[kCandidates];
  Key lists[kWarps][32];
  uint32_t warp_max[kWarps];
  float warp_s[kWarps], warp_t[kWarps], warp_own[kWarps];
  int warp_holds[kWarps];            // whether the warp has the maximum
  int warp_owner[kWarps];            // the thread held out, -1: an edge element or none
  float own_again;
  // what the other blocks of the cluster read
  Stats stats;
  Key best[32];
};

// Forward kernel.  kT threads take a row (kT = 32: a warp, eight rows to a block; else one
// block), or with a cluster of C blocks each block takes 1/C of it and block 0 joins the
// results through distributed shared memory.
//
// One pass over the row: each thread keeps a running maximum, the sum of exponentials and
// the sum of exponential * exponent over its vectors, rescaled once per batch of kBatch
// vectors.  The alternatives cost the pass nothing: afterwards the top-th largest of the
// maxima of 64 sets of threads bounds the row's top-th largest logit from below (tau), and only
// threads whose maximum reaches it (about `top` of them) can hold one; their vectors are
// read again (from L2), the logits that reach tau collected (about 1.3 top of them) and sorted.
// Where ties make them too many to collect, they are inserted into lists one by one.  In the
// same way the vectors of the thread that holds the maximum are summed again without it
// where its own term would drown the others (R < 8).
//
// 1536 threads on an SM (40 registers each; 2048 take 135 us instead of 126 at 8192 x 50257, 1280
// take 130), 2048 for bf16 rows of 512 threads: 32 registers and 96 bytes of spills each, 395 us at
// 4096 x 310000 (1536: 390), 114 at 2048 x 129280 with 8 alternatives (115), 369 at 4096 x 256000 with
// 8 (362).
constexpr int threads_of(int kT) { return kT == 32 ? 256 : kT; }
template <typename T>
constexpr int blocks_per_sm(int kT) { return (sizeof(T) == 2 && kT == 512 ? 2048 : 1536) / threads_of(kT); }

//
// kLong: a thread's sums run over more than kLongBatches batches, and a batch is summed by
// itself first: fewer terms in a row to round (17 x 140 000 000 bf16: log_sum off by 1.1e-5 without).
// It takes 5 % longer.
constexpr int kLongBatches = 64;

template <typename T, int kT, bool kLong = false>
__global__ void __launch_bounds__(threads_of(kT), blocks_per_sm<T>(kT)) logprobs_kernel(const LogprobsArgs a) {
  using V = Vec<T>;
  constexpr int kE = V::kE;
  constexpr int kGroups = kT == 32 ? 8 : 1;
  constexpr int kWarps = kT / 32;
  __shared__ GroupSmem<kT> smem_all[kGroups];
  const int group = kT == 32 ? threadIdx.x / 32 : 0;
  GroupSmem<kT>& sm = smem_all[group];
  const int tid = kT == 32 ? threadIdx.x % 32 : threadIdx.x;
  const int lane = tid % 32, warp = tid / 32;
  auto sync = [] {
    if constexpr (kT == 32) __syncwarp(); else __syncthreads();
  };
  int C = 1, rank = 0;
  if constexpr (kT == 512) {
    C = cg::this_cluster().num_blocks();
    rank = cg::this_cluster().block_rank();
  }

  long long row = static_cast<long long>(blockIdx.x / C) * kGroups + group;
  if (a.status && blockIdx.x == 0) report_targets(a.targets, a.targets_int64, a.n, a.V, a.status, blockDim.x);
  if (row >= a.n) return;
  const int top = a.top;
  const T* z = static_cast<const T*>(a.logits) + row * a.row_stride;
  // The row is `head` elements up to the first 16-byte boundary, nv whole vectors, and a
  // tail; the up to 2 (kE - 1) elements outside the vectors go to the lanes of warp 0.
  const int head = min(static_cast<int>((16 - reinterpret_cast<uintptr_t>(z) % 16) % 16 / sizeof(T)), a.V);
  const int nv = (a.V - head) / kE;
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);
  const int per = (nv + C - 1) / C;
  const int v0 = min(rank * per, nv), v1 = min(v0 + per, nv);
  uint4 r[kBatch];
  auto load_batch = [&](int v) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      r[u] = v + u * kT < v1 ? load16(zv + v + u * kT)
                             : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
  };
  // Short rows: on its way while the target comes.  (8192 x 50257 with 256 threads a row
  // takes 126 us without, 132 with.)
  constexpr bool kAhead = kT <= 128;
  if constexpr (kAhead) load_batch(v0 + tid);
  const long long target = target_of(a.targets, a.targets_int64, row);
  if (target < 0) {                  // padding: the row does not matter
    if (rank == 0) {
      if (tid == 0) {
        a.logprobs[row] = 0.0f;
        a.entropy[row] = 0.0f;
        a.row_max[row] = 0.0f;
        a.log_sum[row] = 0.0f;
      }
      if (tid < top) {
        a.top_logprobs[row * top + tid] = -INFINITY;
        a.top_ids[row * top + tid] = -1;
      }
    }
    return;
  }
  float z_target = NAN;              // of a target outside [0, V)
  if (rank == 0 && warp == 0 && target < a.V) z_target = V::load1(z + target);

  const int edges = rank == 0 ? a.V - nv * kE : 0;
  int edge_id = 0;
  float edge = -INFINITY;
  if (warp == 0 && lane < edges) {
    edge_id = lane < head ? lane : nv * kE + lane;
    edge = V::load1(z + edge_id);
  }

  const float c = a.scale_log2;
  const float2 c2 = make_float2(c, c);
  float m = -FLT_MAX;
  float2 S2 = make_float2(0.f, 0.f), T2 = make_float2(0.f, 0.f);
  for (int v = v0 + tid; v < v1; v += kT * kBatch) {
    if (!kAhead || v != v0 + tid) load_batch(v);
    uint4 mx = r[0];
#pragma unroll
    for (int u = 1; u < kBatch; ++u) mx = V::elementwise_max(mx, r[u]);
    const float m_new = fmaxf(m, V::max_of(mx));
    const float d = fmaxf((m - m_new) * c, -1000.0f);
    const float f = ex2(d);
    m = m_new;
    T2 = ptx::mul2(make_float2(f, f), ptx::fma2(make_float2(d, d), S2, T2));
    S2 = ptx::mul2(make_float2(f, f), S2);
    const float2 minus_m = make_float2(-m, -m);
    float2 bs = make_float2(0.f, 0.f), bt = bs;      // kLong: the batch's own
    float2& s2 = kLong ? bs : S2;
    float2& t2 = kLong ? bt : T2;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) {
        float2 t = ptx::mul2(ptx::add2(V::pair(r[u], i), minus_m), c2);
        t.x = max_nan(t.x, kLowestExponent);
        t.y = max_nan(t.y, kLowestExponent);
        const float2 e = make_float2(ex2(t.x), ex2(t.y));
        s2 = ptx::add2(s2, e);
        t2 = ptx::fma2(e, t, t2);
      }
    }
    if constexpr (kLong) {
      S2 = ptx::add2(S2, bs);
      T2 = ptx::add2(T2, bt);
    }
  }

  // ---- the group's maximum
  uint32_t om = __reduce_max_sync(kAll, order_of(warp == 0 ? fmaxf(m, edge) : m));
  if (top) {
    constexpr int kSet = kT / GroupSmem<kT>::kSets;
    float set = m;
#pragma unroll
    for (int d = kSet / 2; d; d /= 2) set = fmaxf(set, __shfl_xor_sync(kAll, set, d));
    if (tid % kSet == 0) sm.maxima[tid / kSet] = order_of(set);
  }
  if (tid == 0) sm.num_tasks = sm.num_candidates = 0;
  if constexpr (kWarps > 1) {
    if (lane == 0) sm.warp_max[warp] = om;
    sync();
    om = __reduce_max_sync(kAll, lane < kWarps ? sm.warp_max[lane] : 0u);
  } else {
    sync();
  }
  const float M = fmaxf(float_of(om), -FLT_MAX);

  // ---- its sums.  Each warp that has the maximum holds one occurrence out: an edge
  // element's whole term, or 1 off the sum of its first thread that has it.
  float s, t;
  {
    const float d = fmaxf((m - M) * c, -1000.0f);
    const float f = ex2(d);
    const float S = S2.x + S2.y;
    s = S * f;
    t = f * (T2.x + T2.y + d * S);
  }
  const unsigned edge_has = __ballot_sync(kAll, warp == 0 && edge == M);
  const unsigned has = __ballot_sync(kAll, m == M);
  const int owner = has && !edge_has ? __ffs(has) - 1 : -1;     // lane of the thread held out
  float own = owner >= 0 ? __shfl_sync(kAll, s, owner) - 1.0f : 0.0f;
  if (lane == owner) s = 0.0f;
  if (warp == 0 && lane < edges) {
    const float x = max_nan((edge - M) * c, kLowestExponent);
    const float e = ex2(x);
    s += edge_has && lane == __ffs(edge_has) - 1 ? e - 1.0f : e;    // e is 1, or NaN for an infinite maximum
    t += e * x;
  }
  s = warp_sum(s);
  t = warp_sum(t);
  int owner_tid = owner >= 0 ? warp * 32 + owner : -1;
  if constexpr (kWarps > 1) {
    if (lane == 0) {
      sm.warp_s[warp] = s;
      sm.warp_t[warp] = t;
      sm.warp_own[warp] = own;
      sm.warp_holds[warp] = has || edge_has;
      sm.warp_owner[warp] = owner_tid;
    }
    sync();
    // the first warp that has the maximum holds it out; the other warps' occurrences count
    const bool in = lane < kWarps;
    const int first = __ffs(__ballot_sync(kAll, in && sm.warp_holds[lane])) - 1;
    s = warp_sum(in ? sm.warp_s[lane] + (sm.warp_holds[lane] && lane != first ? 1.0f + sm.warp_own[lane] : 0.0f)
                    : 0.0f);
    t = warp_sum(in ? sm.warp_t[lane] : 0.0f);
    own = sm.warp_own[first];
    owner_tid = sm.warp_owner[first];
  }
  if (s + own < 8.0f && owner_tid >= 0) {   // the same in every thread of the group
    if (warp == owner_tid / 32) {
      float r = 0.0f, equal = 0.0f;
      for (int v = v0 + owner_tid + lane * kT; v < v1; v += 32 * kT) {
        const uint4 raw = load16(zv + v);
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
          const float2 p = V::pair(raw, i);
          if (p.x == M) equal += 1.0f; else r += ex2(max_nan((p.x - M) * c, kLowestExponent));
          if (p.y == M) equal += 1.0f; else r += ex2(max_nan((p.y - M) * c, kLowestExponent));
        }
      }
      own = warp_sum(r) + (warp_sum(equal) - 1.0f);
      if (lane == 0) sm.own_again = own;
    }
    if constexpr (kWarps > 1) {
      sync();
      own = sm.own_again;
    }
  }
  Stats st{M, s + own, t};

  // ---- the group's best candidates
  Key list = 0;
  if (top) {
    // tau: the top-th largest of the sets' maxima (there are `top` sets or more)
    constexpr int kSets = GroupSmem<kT>::kSets, kCandidates = GroupSmem<kT>::kCandidates;
    if (tid < kSets) {
      const uint32_t mine = sm.maxima[tid];
      int above = 0, not_below = 0;
      const uint4* all = reinterpret_cast<const uint4*>(sm.maxima);
#pragma unroll 4
      for (int i = 0; i < kSets / 4; ++i) {
        const uint4 w = all[i];
        above += (w.x > mine) + (w.y > mine) + (w.z > mine) + (w.w > mine);
        not_below += (w.x >= mine) + (w.y >= mine) + (w.z >= mine) + (w.w >= mine);
      }
      if (above < top && top <= not_below) sm.tau = mine;       // equal ones write the same
    }
    sync();
    const uint32_t tau = sm.tau;
    const float tau_f = float_of(tau);
    if (order_of(m) >= tau) sm.tasks[atomicAdd(&sm.num_tasks, 1)] = static_cast<uint16_t>(tid);
    sync();
    const int tasks = sm.num_tasks;
    auto offer = [&](float x, uint32_t id) {
      if (!(x >= tau_f)) return;
      const int at = atomicAdd(&sm.num_candidates, 1);
      if (at < kCandidates) sm.candidates[at] = key_of(x, id);
    };
    auto offer_vector = [&](uint4 raw, int v) {
      if (V::max_of(raw) < tau_f) return;
      const uint32_t id = head + v * kE;
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        const float2 p = V::pair(raw, e);
        offer(p.x, id + 2 * e);
        offer(p.y, id + 2 * e + 1);
      }
    };
    const int length = (v1 - v0 + kT - 1) / kT;
    if constexpr (kT == 256) {
      // Up to 128 vectors of a thread: all over the block, thread i vector i % 2^shift of task
      // i / 2^shift, kB in flight (4 for bf16 cost the main loop registers: 4 %).
      constexpr int kB = kE == 8 ? 2 : 4;
      int shift = 0;
      while ((1 << shift) < length) ++shift;
      for (int i = tid; i < tasks << shift; i += kT * kB) {
        uint4 raw[kB];
        int at[kB];
#pragma unroll
        for (int u = 0; u < kB; ++u) {
          const int iu = i + u * kT;
          at[u] = iu < tasks << shift ? v0 + sm.tasks[iu >> shift] + (iu & ((1 << shift) - 1)) * kT : v1;
          raw[u] = at[u] < v1 ? load16(zv + at[u]) : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
        }
#pragma unroll
        for (int u = 0; u < kB; ++u) offer_vector(raw[u], at[u]);
      }
    } else {
      // a warp takes as many threads' vectors at once as it has lanes for
      int width = 1;
      while (width < 32 && width < length) width *= 2;
      for (int i = (warp * 32 + lane) / width; i < tasks; i += kT / width)
        for (int v = v0 + sm.tasks[i] + lane % width * kT; v < v1; v += width * kT) offer_vector(load16(zv + v), v);
    }
    if (warp == 0 && lane < edges) offer(edge, edge_id);
    sync();
    const int found = sm.num_candidates;
    if (found <= kCandidates) {
      if (warp * 32 < found || warp == 0) {
        const int at = warp * 32 + lane;
        list = sort_keys(at < found ? sm.candidates[at] : 0, lane);
      }
      if (found > 32) {
        if constexpr (kWarps > 1) {
          if (warp * 32 < found) sm.lists[warp][lane] = list;
          sync();
          if (warp == 0)
            for (int w = 1; w * 32 < found && w < kWarps; ++w) list = merge_lists(list, sm.lists[w][lane], lane);
        } else {
          for (int at = 32; at < found; at += 32)
            list = merge_lists(list, sort_keys(at + lane < found ? sm.candidates[at + lane] : 0, lane), lane);
        }
      }
    } else {
      Key worst = 0;
      for (int i = warp; i < tasks; i += kWarps) {
        for (int vb = v0 + sm.tasks[i]; vb < v1; vb += 32 * kT) {
          const int v = vb + lane * kT;
          const uint4 raw = v < v1 ? load16(zv + v) : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
          const uint32_t id = head + v * kE;
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const float2 p = V::pair(raw, e / 2);
            const float x = e % 2 ? p.y : p.x;
            insert_keys(list, worst, x >= tau_f ? key_of(x, id + e) : 0, top, lane);
          }
        }
      }
      if (warp == 0) insert_keys(list, worst, edge >= tau_f ? key_of(edge, edge_id) : 0, top, lane);
      if constexpr (kWarps > 1) {
        sm.lists[warp][lane] = lane < top ? list : 0;
        sync();
        if (warp == 0) {
          list = lane < top ? list : 0;
          for (int w = 1; w < kWarps; ++w) list = merge_lists(list, sm.lists[w][lane], lane);
        }
      }
    }
  }

  // ---- the cluster's blocks joined, in the order of their slices
  if constexpr (kT == 512) {
    if (C > 1) {
      cg::cluster_group cluster = cg::this_cluster();
      if (tid == 0) sm.stats = st;
      if (warp == 0) sm.best[lane] = list;
      cluster.sync();
      if (rank == 0 && warp == 0) {
        Stats other{-FLT_MAX, -1.0f, 0.0f};
        if (lane < C) other = *cluster.map_shared_rank(&sm.stats, lane);
        const float Mg = float_of(__reduce_max_sync(kAll, order_of(other.m)));
        const int first = __ffs(__ballot_sync(kAll, other.m == Mg)) - 1;
        const float d = fmaxf((other.m - Mg) * c, -1000.0f);
        const float f = ex2(d);
        const float r = warp_sum(lane == first ? other.R : f * (1.0f + other.R));
        const float tt = warp_sum(f * (other.T + d * (1.0f + other.R)));
        st = Stats{Mg, r, tt};
        if (top) {
          Key theirs[kMaxCluster];
#pragma unroll
          for (int q = 1; q < kMaxCluster; ++q) theirs[q] = q < C ? cluster.map_shared_rank(&sm.best[0], q)[lane] : 0;
#pragma unroll
          for (int q = 1; q < kMaxCluster; ++q)
            if (q < C) list = merge_lists(list, theirs[q], lane);
        }
      }
      cluster.sync();                // the blocks' shared memory stays until it has been read
      if (rank != 0) return;
    }
  }

  // ---- outputs
  if (warp != 0) return;
  const bool empty = st.R == -1.0f;  // no finite logit
  const float log_sum = empty ? 0.0f : log1pf(st.R);
  if (lane == 0) {
    a.logprobs[row] = target >= a.V ? NAN : empty ? -INFINITY : (z_target - st.m) * a.scale - log_sum;
    a.entropy[row] = empty ? 0.0f : log_sum - st.T * kLn2 / (1.0f + st.R);
    a.row_max[row] = empty ? -INFINITY : st.m;
    a.log_sum[row] = log_sum;
  }
  if (lane < top) {
    a.top_logprobs[row * top + lane] =
        list ? (float_of(static_cast<uint32_t>(list >> 32)) - st.m) * a.scale - log_sum : -INFINITY;
    a.top_ids[row * top + lane] = list ? static_cast<long long>(~static_cast<uint32_t>(list)) : -1;
  }
}

// Forward kernel of short rows without alternatives: kG lanes hold a row of up to kHeld kG
// vectors in registers, a warp 32 / kG rows.  Such rows are bound by the instructions that each
// costs a warp, most of them in the reductions, which here serve several rows at once; and with
// the whole row at hand the maximum comes first and nothing is rescaled.  131072 x 1024 bf16
// takes 46.5 us (5.8 TB/s; 52 where the rows are all but sure of a token), a warp a row 61.7
// (76); 262144 x 512 45.3 and 120; 65536 x 2048 45.8 and 48.8.
constexpr int kHeld = 8;

template <typename T, int kG>
__global__ void __launch_bounds__(256, 4) logprobs_short_kernel(const LogprobsArgs a) {
  using V = Vec<T>;
  constexpr int kE = V::kE;
  constexpr int kEdges = (2 * (kE - 1) + kG - 1) / kG;
  if (a.status && blockIdx.x == 0) report_targets(a.targets, a.targets_int64, a.n, a.V, a.status, blockDim.x);
  const int lane = threadIdx.x % kG;
  const long long mine = static_cast<long long>(blockIdx.x) * (256 / kG) + threadIdx.x / kG;
  const long long row = min(mine, static_cast<long long>(a.n) - 1);    // all lanes stay for the reductions
  const T* z = static_cast<const T*>(a.logits) + row * a.row_stride;
  const int head = min(static_cast<int>((16 - reinterpret_cast<uintptr_t>(z) % 16) % 16 / sizeof(T)), a.V);
  const int nv = (a.V - head) / kE, edges = a.V - nv * kE;
  const int most = a.V / kE;         // of any row
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);
  uint4 r[kHeld];
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    r[u] = lane + u * kG < nv ? load16(zv + lane + u * kG) : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
  float edge[kEdges];
#pragma unroll
  for (int u = 0; u < kEdges; ++u) {
    const int e = lane + u * kG;
    edge[u] = e < edges ? V::load1(z + (e < head ? e : nv * kE + e)) : -INFINITY;
  }
  const long long target = target_of(a.targets, a.targets_int64, row);
  float z_target = 0.0f;
  if (lane == 0 && target >= 0 && target < a.V) z_target = V::load1(z + target);

  uint4 mx = r[0];
#pragma unroll
  for (int u = 1; u < kHeld; ++u) mx = V::elementwise_max(mx, r[u]);
  const float held = fmaxf(V::max_of(mx), -FLT_MAX);          // the lane's vectors' maximum
  float M = held;
#pragma unroll
  for (int u = 0; u < kEdges; ++u) M = fmaxf(M, edge[u]);
#pragma unroll
  for (int d = kG / 2; d; d /= 2) M = fmaxf(M, __shfl_xor_sync(kAll, M, d));

  const float c = a.scale_log2;
  const float2 c2 = make_float2(c, c), minus_m = make_float2(-M, -M);
  float2 S2 = make_float2(0.f, 0.f), T2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    if (u * kG >= most) break;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      float2 t = ptx::mul2(ptx::add2(V::pair(r[u], i), minus_m), c2);
      t.x = max_nan(t.x, kLowestExponent);
      t.y = max_nan(t.y, kLowestExponent);
      const float2 e = make_float2(ex2(t.x), ex2(t.y));
      S2 = ptx::add2(S2, e);
      T2 = ptx::fma2(e, t, T2);
    }
  }
  // One occurrence of the maximum is held out: an edge element's whole term, or 1 off the sum of
  // the first lane that holds it.
  float S = S2.x + S2.y, Tt = T2.x + T2.y, S_edge = 0.0f;
  bool edge_has = false;
#pragma unroll
  for (int u = 0; u < kEdges; ++u) {
    const float x = max_nan((edge[u] - M) * c, kLowestExponent);
    const float e = ex2(x);
    const bool held_out = edge[u] == M && !edge_has;
    edge_has |= held_out;
    S_edge += held_out ? e - 1.0f : e;                        // e is 1, or NaN for an infinite maximum
    Tt = fmaf(e, x, Tt);
  }
  const int first_lane = threadIdx.x % 32 - lane;             // of the group, in the warp
  const unsigned group = (kG == 32 ? kAll : (1u << kG % 32) - 1u) << first_lane;
  const unsigned edges_have = __ballot_sync(kAll, edge_has) & group;
  const unsigned lanes_have = __ballot_sync(kAll, held == M) & group;
  const int owner = edges_have || !lanes_have ? -1 : __ffs(lanes_have) - 1 - first_lane;
  if (edge_has && __ffs(edges_have) - 1 != static_cast<int>(threadIdx.x % 32)) S_edge += 1.0f;   // not the first
  float own = S - 1.0f;
  S = (lane == owner ? 0.0f : S) + S_edge;
#pragma unroll
  for (int d = kG / 2; d; d /= 2) {
    S += __shfl_xor_sync(kAll, S, d);
    Tt += __shfl_xor_sync(kAll, Tt, d);
  }
  own = __shfl_sync(kAll, own, max(owner, 0), kG);
  own = owner < 0 ? 0.0f : own;
  const bool again = owner >= 0 && S + own < 8.0f;
  if (__any_sync(kAll, again)) {     // the owner's other terms, which that 1 drowned, a lane to each vector
    float rest = 0.0f, equal = 0.0f;
    if (again) {
      for (int v = owner + lane * kG; v < nv; v += kG * kG) {
        const uint4 raw = load16(zv + v);
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
          const float2 p = V::pair(raw, i);
          if (p.x == M) equal += 1.0f; else rest += ex2(max_nan((p.x - M) * c, kLowestExponent));
          if (p.y == M) equal += 1.0f; else rest += ex2(max_nan((p.y - M) * c, kLowestExponent));
        }
      }
    }
#pragma unroll
    for (int d = kG / 2; d; d /= 2) {
      rest += __shfl_xor_sync(kAll, rest, d);
      equal += __shfl_xor_sync(kAll, equal, d);
    }
    if (again) own = rest + (equal - 1.0f);
  }
  const float R = S + own;
  if (lane != 0 || mine >= a.n) return;
  const bool padding = target < 0, empty = R == -1.0f;
  const float log_sum = empty || padding ? 0.0f : log1pf(R);
  a.logprobs[row] = padding ? 0.0f : target >= a.V ? NAN : empty ? -INFINITY : (z_target - M) * a.scale - log_sum;
  a.entropy[row] = empty || padding ? 0.0f : log_sum - Tt * kLn2 / (1.0f + R);
  a.row_max[row] = padding ? 0.0f : empty ? -INFINITY : M;
  a.log_sum[row] = log_sum;
}

// Gradient kernel: kT threads take kBatch * kT vectors of a row, 256 / kT such items to a block.
// Items of one row are neighbours.  The vectors are the 16-byte ones of
// the gradient's row; a logits row of another alignment is read as two vectors each, put
// together in registers.
//
// With y = log2 p_v, dz_v = p_v (A + B y), A = -s (G + E entropy), B = -s E ln 2; the row's
// token itself takes G (-expm1(log p)) for G (1 - p).
//
// Six blocks on an SM (40 registers a thread) and four vectors in flight each: 8192 x 50257 takes
// 253 us, with four blocks 290, with two vectors 301.  The forms of few threads a row spill (bf16, 4
// threads: 80 bytes stored and 268 loaded a thread; 8: 32 and 168): 1000000 x 100 takes 126 us so, with
// four blocks and no spills 124 (fp32 176 and 192); 262144 x 256 64 and 67 (98 and 104).
template <typename T, int kT>
__global__ void __launch_bounds__(256, 6) logprobs_grad_kernel(const LogprobsGradArgs a, int items_per_row) {
  using V = Vec<T>;
  constexpr int kE = V::kE;
  constexpr int kGroups = 256 / kT;
  if (a.status && blockIdx.x == 0) report_targets(a.targets, a.targets_int64, a.n, a.V, a.status, blockDim.x);
  const long long item = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / kT;
  const int tid = threadIdx.x % kT;
  const long long row = items_per_row == 1 ? item : item / items_per_row;
  if (row >= a.n) return;
  const int part = static_cast<int>(item - row * items_per_row);

  T* g = static_cast<T*>(a.grad) + row * a.grad_stride;
  const T* z = static_cast<const T*>(a.logits) + row * a.row_stride;
  const int head = min(static_cast<int>((16 - reinterpret_cast<uintptr_t>(g) % 16) % 16 / sizeof(T)), a.V);
  const int nv = (a.V - head) / kE;
  uint4* gv = reinterpret_cast<uint4*>(g + head);
  const int v_begin = part * kT * kBatch + tid;
  const T* zb = z + head;
  const unsigned shift = reinterpret_cast<uintptr_t>(zb) % 16;
  uint4 r[kBatch];
  auto load_aligned = [&] {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (v_begin + u * kT < nv) r[u] = load16(reinterpret_cast<const uint4*>(zb) + v_begin + u * kT);
  };
  // Short rows: on their way while the row's numbers come (a row of padding is read in
  // vain, which costs long rows more than the wait).
  if (kT <= 32 && shift == 0) load_aligned();

  const long long target = target_of(a.targets, a.targets_int64, row);
  const float m = a.row_max[row];
  const bool zero = target < 0 || target >= a.V || m == -INFINITY;
  const float log_sum = a.log_sum[row];
  const float G = a.grad_logprobs[row];
  const float E = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
  const float H = a.grad_entropy ? a.entropy[row] : 0.0f;
  const float c = a.scale_log2;
  const float minus_ls2 = -log_sum * kLog2e;
  const float A = -a.scale * (G + E * H), B = -a.scale * E * kLn2;

  auto one = [&](float x, int id) {  // the gradient of one element
    const float y = max_nan(fmaf(x - m, c, minus_ls2), kLowestExponent);
    const float p = ex2(y);
    if (id != static_cast<int>(target)) return p * fmaf(B, y, A);
    const float lp = (x - m) * a.scale - log_sum;
    return a.scale * (-G * expm1f(lp)) - (E != 0.0f ? a.scale * E * p * (fmaxf(lp, -1e30f) + H) : 0.0f);
  };

  if (part == 0) {                   // the elements outside the vectors
    const int edges = a.V - nv * kE;
#pragma unroll
    for (int u = 0; u < (2 * (kE - 1) + kT - 1) / kT; ++u) {
      const int e = tid + u * kT;
      if (e >= edges) break;
      const int id = e < head ? e : nv * kE + e;
      V::store1(g + id, zero ? 0.0f : one(V::load1(z + id), id));
    }
  }
  if (zero) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (v_begin + u * kT < nv) gv[v_begin + u * kT] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (shift == 0) {
    if (kT > 32) load_aligned();
  } else {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int v = v_begin + u * kT;
      if (v >= nv) continue;
      if (v == 0 || v == nv - 1) {   // the aligned vectors around these may leave the row
        float2 x[kE / 2];
#pragma unroll
        for (int i = 0; i < kE / 2; ++i)
          x[i] = make_float2(V::load1(zb + v * kE + 2 * i), V::load1(zb + v * kE + 2 * i + 1));
        r[u] = V::pack(x);           // exact: the values are of type T
      } else {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(zb + static_cast<long long>(v) * kE) - shift);
        const uint4 lo = p[0], hi = p[1];
        uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (shift & 8) {
#pragma unroll
          for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (shift & 4) {
#pragma unroll
          for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const unsigned bits = (shift & 3) * 8;
        r[u] = make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
      }
    }
  }
  const float2 minus_m = make_float2(-m, -m), c2 = make_float2(c, c), ls2 = make_float2(minus_ls2, minus_ls2);
  const float2 A2 = make_float2(A, A), B2 = make_float2(B, B);
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int v = v_begin + u * kT;
    if (v >= nv) continue;
    float2 out[kE / 2];
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      float2 y = ptx::fma2(ptx::add2(V::pair(r[u], i), minus_m), c2, ls2);
      y.x = max_nan(y.x, kLowestExponent);
      y.y = max_nan(y.y, kLowestExponent);
      out[i] = ptx::mul2(make_float2(ex2(y.x), ex2(y.y)), ptx::fma2(B2, y, A2));
    }
    const long long e = target - head - static_cast<long long>(v) * kE;
    if (e >= 0 && e < kE) {          // the vector that holds the token
      float* o = &out[0].x;
      const float x = V::load1(zb + static_cast<long long>(v) * kE + e);
      const float val = one(x, static_cast<int>(target));
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (i == e) o[i] = val;
    }
    gv[v] = V::pack(out);
  }
}

template <typename T, int kT, bool kLong = false>
cudaError_t launch_forward(const LogprobsArgs& a, int cluster, cudaStream_t stream) {
  constexpr int kGroups = kT == 32 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(a.n) * cluster + kGroups - 1) / kGroups));
  cfg.blockDim = dim3(kT * kGroups);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  if (cluster > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kT, kLong>, a);
}

template <typename T, int kG>
cudaError_t launch_short(const LogprobsArgs& a, cudaStream_t stream) {
  logprobs_short_kernel<T, kG><<<static_cast<unsigned>((a.n + 256LL / kG - 1) / (256 / kG)), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_forward_of(const LogprobsArgs& a, int num_sms, cudaStream_t stream) {
  // Threads of a row by its vectors and by whether there are rows enough to fill the device
  // (bf16 in us, without | with 8 alternatives, by threads a row):
  //                  32         128        256        512
  //   65536 x  4097  85 | 132  121 |  -
  //   32768 x  8192  84 | 130   94 | 148  125 | 209
  //     512 x  8192  7.1| 12.6  4.0| 6.1             7.2| 10.2
  //    8192 x 32000 103 | 240   83 | 103   83 | 102  100 | 130
  //     160 x 64000             14 |  18  7.9 | 10.3
  //    8192 x 50257            129 | 165  126 | 148  144 | 174
  //    8192 x 80000            197 | 270  187 | 214  211 | 231
  //    8192 x129280            312 | 437  294 | 345  327 | 349  (with 20: 425 and 383)
  //    2048 x129280             99 | 131   85 | 101   82 |  92
  // Short rows pay for what a row costs besides its read, which more threads raise; in long
  // ones few threads leave each with more vectors to read again for the alternatives.  How many
  // alternatives turn it round (256 | 512 threads, bf16, the same logits without padding):
  //   8192 x 102400    8: 299 | 302   16: 339 | 316      4096 x 256000    2: 336 | 335    4: 350 | 340
  //   8192 x 129280    5: 352 | 354    8: 372 | 360      fp32
  //   4096 x 160000    3: 224 | 228    4: 229 | 228      4096 x  65536    5: 183 | 191    8: 193 | 193
  //   4096 x 200000    3: 275 | 277    4: 282 | 279      4096 x 129280    4: 341 | 343    5: 347 | 344
  // at 64000 to 200000 alternatives times vectors of a row; the rule's 131072 costs 4 % at most between.
  const int nv = a.V / Vec<T>::kE;
  const bool many = a.n >= 16 * num_sms;
  // (kHeld vectors a lane are what 64 registers a thread hold)
  if (!a.top && nv <= 32 * kHeld)
    return nv <= 4 * kHeld    ? launch_short<T, 4>(a, stream)
           : nv <= 8 * kHeld  ? launch_short<T, 8>(a, stream)
           : nv <= 16 * kHeld ? launch_short<T, 16>(a, stream)
                              : launch_short<T, 32>(a, stream);
  if (nv <= 128 || (nv <= 1024 && many)) return launch_forward<T, 32>(a, 1, stream);
  if (nv <= 1024 || (nv < 4096 && a.n >= num_sms)) return launch_forward<T, 128>(a, 1, stream);
  if (a.n >= num_sms && (nv <= 12288 || (many && nv <= 32768 && a.top * nv <= 131072))) return launch_forward<T, 256>(a, 1, stream);
  // Few rows: up to 8 blocks a row, one on an SM, of 1024 vectors at least.  Joining them
  // costs 1.2 us, which a row of 4000 vectors does not win back (64 x 32000 bf16 with 8
  // alternatives: 6.6 us, in two blocks 8.9; 1 x 129280: 8.0 in eight, 10.4 in one).
  int cluster = 1;
  while (cluster < kMaxCluster && 2LL * cluster * a.n <= num_sms && nv > 4096 && nv / (2 * cluster) >= 1024) cluster *= 2;
  if (nv / cluster > 512 * kBatch * kLongBatches) return launch_forward<T, 512, true>(a, cluster, stream);
  return launch_forward<T, 512>(a, cluster, stream);
}

template <typename T, int kT>
cudaError_t launch_grad(const LogprobsGradArgs& a, int nv, cudaStream_t stream) {
  constexpr int kGroups = 256 / kT;
  const int items = (nv + kT * kBatch - 1) / (kT * kBatch);
  const long long blocks = (static_cast<long long>(a.n) * items + kGroups - 1) / kGroups;
  logprobs_grad_kernel<T, kT><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a, items);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_grad_of(const LogprobsGradArgs& a, cudaStream_t stream) {
  // as many threads an item as a short row fills (262144 x 256 bf16: 56 us with 8, 87 with 32;
  // 1000000 x 100: 118 with 4, 354 with 32)
  const int nv = a.V >= Vec<T>::kE ? a.V / Vec<T>::kE : 1;   // an item takes the row's edges
  return nv <= 4 * kBatch     ? launch_grad<T, 4>(a, nv, stream)
         : nv <= 8 * kBatch   ? launch_grad<T, 8>(a, nv, stream)
         : nv <= 16 * kBatch  ? launch_grad<T, 16>(a, nv, stream)
         : nv <= 128 * kBatch ? launch_grad<T, 32>(a, nv, stream)
                              : launch_grad<T, 256>(a, nv, stream);
}

// The status of a call that moves `row_bytes` for a row: by the first block of its kernel, which reads
// all targets before the others are through where rows are long; else by a grid ahead of the kernel
// (args.status is then null).  In us, forward and backward, bf16:
//
//                   no status      one block      a grid ahead
//   1000000 x 100   74.3  119      229   335      79.5  126
//    262144 x 256   27.5   58       47    91      31.4   64
//    262144 x 512   47.0   98.4     51.0  98.8    51.9
template <typename Args>
cudaError_t report_apart(Args& a, long long row_bytes, cudaStream_t stream) {
  if (!a.status || a.n <= 65536 || row_bytes > 1024) return cudaSuccess;
  static_assert(kStatusOk == 0, "the word's bytes");
  cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int), stream);
  if (e != cudaSuccess) return e;
  targets_kernel<<<static_cast<unsigned>((a.n + 2047LL) / 2048), 256, 0, stream>>>(a.targets, a.targets_int64, a.n, a.V, a.status);
  a.status = nullptr;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& args, bool bf16, int num_sms, cudaStream_t stream) {
  LogprobsArgs a = args;
  const cudaError_t e = report_apart(a, a.V * (bf16 ? 2LL : 4LL), stream);
  if (e != cudaSuccess) return e;
  return bf16 ? launch_forward_of<__nv_bfloat16>(a, num_sms, stream) : launch_forward_of<float>(a, num_sms, stream);
}

cudaError_t launch_logprobs_grad(const LogprobsGradArgs& args, bool bf16, cudaStream_t stream) {
  LogprobsGradArgs a = args;
  const cudaError_t e = report_apart(a, 2 * a.V * (bf16 ? 2LL : 4LL), stream);
  if (e != cudaSuccess) return e;
  return bf16 ? launch_grad_of<__nv_bfloat16>(a, stream) : launch_grad_of<float>(a, stream);
}

}  // namespace ewg
