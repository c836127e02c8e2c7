// Layer norm of rows, and its gradient.
//
// Per row x[0..H), avg over the row:
//
//     mean = avg(x)     rstd = 1 / sqrt(avg((x - mean)^2) + eps)     out = (x - mean) rstd w + b
//
// and with n = (x - mean) rstd, u = g w:
//
//     dx = rstd (u - avg(u) - n avg(u n))     dw_j = sum over rows of g n     db_j = sum over rows of g
//
// Both are bound by memory: forward each element is read and written once, for its gradient two are read and
// one written (131072 x 8192 bf16: 616 us, 7.0 TB/s, and 966 us, 6.7 TB/s; 8192 x 7168: 42 and 60 us, where a copy of
// the forward pass's bytes takes 36).  What stands in the way are the sums over a row: a barrier and a chain of
// shuffles, during which a team computes nothing else.  So a thread has many elements of a row (sixteen, which
// spreads the shuffles), several rows go through a sum together, and the rows after them are being copied to
// shared memory meanwhile.  A block stays on its SM and keeps what belongs to columns, the weights and the
// sums for dw and db, in registers.
//
// Rows that do not begin at 16 bytes repeat their places in them after at most eight rows.  A group takes rows of
// one place, so that its accesses are whole ones too, and the few elements beside them go by themselves
// (65536 x 1001 fp32: 93 and 124 us, bf16 53 and 78).  Where the arrays' rows begin differently they move element by
// element (fp32 110 and 167 us, bf16 87 and 155).
//
// Tried and slower: every thread's next row in registers instead of shared memory (8192 x 7168 backward 96 us),
// 1024 threads of eight columns (85 us), deviations from the average of a row's first 32 elements,
// which saves one of the forward pass's two barriers (48 us), twice the rows in a batch, read again from shared memory
// for each sum (45 us, and 65536 x 1024 46 instead of 44), a cluster's sums by asynchronous stores that an mbarrier counts
// (4096 x 16384 backward 81 us instead of 87 in bf16, but 163 instead of 139 in fp32).
#include <atomic>
#include <cfloat>

#include <cuda_bf16.h>

#include "ewg_ptx.cuh"
#include "ewg_train.cuh"

namespace ewg {
namespace {

constexpr unsigned kAll = 0xffffffffu;

using ptx::add2;
using ptx::fma2;
using ptx::mul2;
using ptx::sub2;

__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 from_bf16x2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t to_bf16x2(float2 f) {
  uint32_t u;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(f.y), "f"(f.x));
  return u;
}

// kE neighbouring elements of a row, which one access moves: 16 bytes, or a single element where rows' alignments
// do not allow that.  Arithmetic goes by pairs, two 32-bit operations an instruction.
template <typename T, int kE>
struct Access;

template <>
struct Access<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(Raw v, float2* f) {
    f[0] = from_bf16x2(v.x), f[1] = from_bf16x2(v.y), f[2] = from_bf16x2(v.z), f[3] = from_bf16x2(v.w);
  }
  static __device__ __forceinline__ Raw pack(const float2* f) {
    return make_uint4(to_bf16x2(f[0]), to_bf16x2(f[1]), to_bf16x2(f[2]), to_bf16x2(f[3]));
  }
};
template <>
struct Access<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void unpack(Raw v, float2* f) {
    f[0] = make_float2(v.x, v.y), f[1] = make_float2(v.z, v.w);
  }
  static __device__ __forceinline__ Raw pack(const float2* f) { return make_float4(f[0].x, f[0].y, f[1].x, f[1].y); }
};

// Element j of a vector of bf16 or fp32.
__device__ __forceinline__ float element(const void* p, int bf16, int j) {
  return bf16 ? load(static_cast<const __nv_bfloat16*>(p) + j) : load(static_cast<const float*>(p) + j);
}

// kE elements of a weight or bias vector of W, as pairs; for one element, in x.
template <typename W, int kE>
__device__ __forceinline__ void vector_part(const W* p, float2* f) {
  if constexpr (kE == 1) {
    if constexpr (sizeof(W) == 2) f->x = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
    else f->x = __ldg(p);
  } else if constexpr (sizeof(W) == 2) {
    alignas(16) uint32_t u[kE / 2];
    if constexpr (kE == 8) *reinterpret_cast<uint4*>(u) = __ldg(reinterpret_cast<const uint4*>(p));
    else *reinterpret_cast<uint2*>(u) = __ldg(reinterpret_cast<const uint2*>(p));
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) f[i] = from_bf16x2(u[i]);
  } else if constexpr (kE == 8) {
    asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y), "=f"(f[2].x), "=f"(f[2].y), "=f"(f[3].x), "=f"(f[3].y)
        : "l"(p));
  } else {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = make_float2(v.x, v.y);
    f[1] = make_float2(v.z, v.w);
  }
}

// Of 2 kPairs elements that a thread has of a row, in accesses of kE: the pairs' values from where
// access k lies at `at + k plane`, and back to where it goes to `to + k pitch`.
template <typename T, int kE, int kPairs>
__device__ __forceinline__ void read_pairs(const char* at, int plane, float2 (&f)[kPairs]) {
#pragma unroll
  for (int k = 0; k < 2 * kPairs / kE; ++k) {
    if constexpr (kE == 1) {
      const float v = load(reinterpret_cast<const T*>(at + k * plane));
      if (k % 2) f[k / 2].y = v;
      else f[k / 2].x = v;
    } else {
      using A = Access<T, kE>;
      A::unpack(*reinterpret_cast<const typename A::Raw*>(at + k * plane), f + k * kE / 2);
    }
  }
}

template <typename T, int kE, int kPairs>
__device__ __forceinline__ void write_pairs(T* to, int pitch, int count, const float2 (&f)[kPairs]) {
#pragma unroll
  for (int k = 0; k < 2 * kPairs / kE; ++k) {
    if (k >= count) continue;
    if constexpr (kE == 1) {
      store(to + k * pitch, k % 2 ? f[k / 2].y : f[k / 2].x);
    } else {
      using A = Access<T, kE>;
      *reinterpret_cast<typename A::Raw*>(to + k * pitch) = A::pack(f + k * kE / 2);
    }
  }
}

// The same of a vector of W from the thread's first column on.
template <typename W, int kE, int kPairs>
__device__ __forceinline__ void read_vector(const W* p, int pitch, int count, float2 (&f)[kPairs]) {
#pragma unroll
  for (int k = 0; k < 2 * kPairs / kE; ++k) {
    if (k >= count) continue;
    if constexpr (kE == 1) {
      float2 v;
      vector_part<W, 1>(p + k * pitch, &v);
      if (k % 2) f[k / 2].y = v.x;
      else f[k / 2].x = v.x;
    } else {
      vector_part<W, kE>(p + k * pitch, f + k * kE / 2);
    }
  }
}
// Where there is no vector, its elements are `none`.
template <int kE, int kPairs>
__device__ __forceinline__ void vector_columns(const void* p, int bf16, int column, int pitch, int count, float none,
                                            float2 (&f)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) f[i] = both(none);
  if (!p) return;
  if (bf16) read_vector<__nv_bfloat16, kE, kPairs>(static_cast<const __nv_bfloat16*>(p) + column, pitch, count, f);
  else read_vector<float, kE, kPairs>(static_cast<const float*>(p) + column, pitch, count, f);
}

// A number near a row's mean from which deviations are taken.  bf16 elements less a number of more than
// bf16's digits would all be rounded the same way, and their sum be off by as much; less one of bf16 they
// are exact, and their squares' mean is at least twice the square of theirs.
template <typename T>
__device__ __forceinline__ float centre_of(float mean) {
  return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(mean)) : mean;
}

// 1 / standard deviation from the averages of the deviations from some centre and of their squares; NaN where
// an element is not finite.
__device__ __forceinline__ float rstd_of(float rest, float square, float eps) {
  const float var = fmaxf(fmaf(-rest, rest, square), 0.0f);
  return square <= FLT_MAX ? 1.0f / sqrtf(var + eps) : square - square;
}

// Sum of pairs, by halves.
template <int kN>
__device__ __forceinline__ float pairs_sum(const float2* f) {
  float2 s[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) s[i] = f[i];
#pragma unroll
  for (int n = kN / 2; n; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = add2(s[i], s[i + n]);
  return s[0].x + s[0].y;
}

// Sums of kM numbers over a warp at once: the first steps leave half of the numbers to each half of the
// lanes; in the end kM groups of neighbouring lanes have one number's sum each.
template <int kM>
__device__ __forceinline__ float warp_fold(float (&v)[kM]) {
#pragma unroll
  for (int m = kM / 2, d = 16; m; m /= 2, d /= 2) {
    const bool upper = threadIdx.x & d;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float keep = upper ? v[m + i] : v[i], send = upper ? v[i] : v[m + i];
      v[i] = keep + __shfl_xor_sync(kAll, send, d);
    }
  }
#pragma unroll
  for (int d = 16 / kM; d; d /= 2) v[0] += __shfl_xor_sync(kAll, v[0], d);
  return v[0];
}

// Sums of kM numbers over a team, in each of its threads.  kTeam: its threads, or 0 where they are
// several warps (`threads` of them), which meet in `slots` [kM][32], zeros where there is no warp.
template <int kM, int kTeam>
__device__ __forceinline__ void team_sum(float (&v)[kM], float* slots, int team, int threads) {
  const int lane = threadIdx.x % 32;
  if constexpr (kTeam && kTeam < 32) {
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int d = kTeam / 2; d; d /= 2) v[i] += __shfl_xor_sync(kAll, v[i], d);
  } else {
    constexpr int kGroup = 32 / kM;
    float s = warp_fold<kM>(v);
    if constexpr (kTeam == 0) {
      if (lane % kGroup == 0) slots[lane / kGroup * 32 + threadIdx.x % threads / 32] = s;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
      const float* mine = slots + lane / kGroup * 32 + lane % kGroup * kM;
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < kM; ++i) s += mine[i];
#pragma unroll
      for (int d = kGroup / 2; d; d /= 2) s += __shfl_xor_sync(kAll, s, d);
    }
#pragma unroll
    for (int i = 0; i < kM; ++i) v[i] = __shfl_sync(kAll, s, i * kGroup);
  }
}

// Sums of kM numbers over the blocks of a cluster, all threads of each having its own: they leave in cluster_send and
// arrive in cluster_take.  `box` [2][kMostBlocks][kM] is in every block's shared memory, its halves taken in
// turn, so that one barrier is enough: who sends into a half has seen all threads arrive that read it before.
constexpr int kMostBlocks = 8;          // of a cluster, as many as any device runs

template <int kM>
__device__ __forceinline__ void cluster_send(const float (&v)[kM], float (&box)[kMostBlocks][kM], int blocks, int rank) {
  if (threadIdx.x < blocks) {
    const uint32_t to = ptx::map_to_rank(ptx::smem_u32(&box[rank][0]), threadIdx.x);
#pragma unroll
    for (int i = 0; i < kM; ++i) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * i), "f"(v[i]) : "memory");
  }
  ptx::cluster_arrive();
}
template <int kM>
__device__ __forceinline__ void cluster_take(float (&v)[kM], const float (&box)[kMostBlocks][kM], int blocks) {
  ptx::cluster_wait();
#pragma unroll
  for (int i = 0; i < kM; ++i) v[i] = 0.0f;
  for (int b = 0; b < blocks; ++b)
#pragma unroll
    for (int i = 0; i < kM; ++i) v[i] += box[b][i];
}

// ---- rows that a block holds (or, for the gradient of those of more than 8192 elements, a cluster of up to
// eight), copied ahead into shared memory

constexpr int kStreamThreads = 512;                        // of a block, at most; it is the only one of its SM
constexpr int kStreamHidden = 8192;
static_assert(kStreamHidden * kMostBlocks == kNormHeld);

// Of an array of rows: its first element, and the bytes from a row to the next one and from a team's batch
// to its next one.
struct Rows {
  const char* p;
  long long pitch, advance;
};

// What the two kernels below have in common.  A team of threads takes kR neighbouring rows at a
// time, and of the batches after that one kStages - 1 are on their way: every thread copies what it will read
// itself (kArrays arrays' rows), so that the copies need no barrier.  Where an element is too
// small for an asynchronous copy (single elements of bf16), kStages is 1 and a batch is read when its turn comes.
// A cluster's blocks are one team, each with the columns from `lead` on.
//
// kShift: rows that begin anywhere, all arrays' alike.  Their places in 16 bytes repeat every `period` rows; a
// group takes rows of one place only, so that columns stay with their threads.  Accesses begin at the first 16 bytes
// within the row; the elements before them and behind the last whole one, less than two accesses' together, are
// the team's first threads' extra ones, one each, in four bytes of their own behind the ring.
template <typename T, int kE, int kColumns, int kR, int kArrays, int kStages, int kTeam, bool kShift>
struct Stream {
  static constexpr int kPairs = kColumns / 2;
  static constexpr int kK = kColumns / kE, kBytes = kE * static_cast<int>(sizeof(T));
  static_assert(!kShift || kBytes == 16);
  int threads, teams, team, thread, lead, group;      // (group: which of the grid's blocks or clusters)
  int count;                         // of the thread's kK accesses to a row those that lie in it
  int period, place_of, head;        // kShift: which of the period's rows are the group's; their elements before the accesses
  int extra = -1, extra_half = 0;    // the column of the thread's extra element; whether it is the upper one of its four bytes
  uint32_t n, row, step;             // rows; the first row of the team's next batch to be copied; rows of all teams' batches
  const char* from[kArrays];         // of `row`, the thread's first access
  char* ring;
  int stage = 0;

  __device__ __forceinline__ Stream(int team_threads, int rows, int H, int blocks, int period_, const Rows& like, char* shared) {
    const int rank = blocks > 1 ? static_cast<int>(ptx::cluster_rank()) : 0;
    group = blockIdx.x / blocks;
    int groups = gridDim.x / blocks, mine = group, accesses = H / kE;       // (without kShift H is a multiple of kE)
    period = 1, place_of = head = 0, n = rows;
    if constexpr (kShift) {
      period = period_;
      place_of = group % period;
      groups /= period, mine /= period;
      n = rows > place_of ? (rows - place_of + period - 1) / period : 0;
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(like.p + place_of * like.pitch) % 16) / static_cast<int>(sizeof(T));
      head = (kE - off) % kE < H ? (kE - off) % kE : H;
      accesses = (H - head) / kE;
    }
    const int share = (accesses + blocks - 1) / blocks;     // accesses of a block
    lead = rank * share * kE;
    threads = kTeam ? kTeam : team_threads;
    teams = blockDim.x / threads;
    team = threadIdx.x / threads;
    thread = threadIdx.x % threads;
    const int end = accesses - rank * share;
    const int left = (end < share ? end : share) - thread;
    count = left > 0 ? (left + threads - 1) / threads : 0;
    if constexpr (kShift) {
      const int behind = head + accesses * kE;               // (the first column behind the accesses)
      if (thread < head) extra = thread;
      else if (thread < head + H - behind) extra = behind + thread - head;
      if (sizeof(T) == 2) extra_half = reinterpret_cast<uintptr_t>(extra_of(like, 0)) / 2 % 2;
    }
    ring = shared + threadIdx.x * kBytes;
    step = groups * teams * kR;
    row = (mine * teams + team) * kR;
  }
  __device__ __forceinline__ int column(int k) const { return lead + head + (k * threads + thread) * kE; }
  __device__ __forceinline__ int pitch() const { return threads * kE; }
  // Which of the arrays' rows is the group's `r`th.
  __device__ __forceinline__ uint32_t index(uint32_t r) const { return kShift ? place_of + period * r : r; }
  __device__ __forceinline__ long long bytes_to(const Rows& rows, int r) const { return kShift ? r * (rows.pitch * period) : r * rows.pitch; }
  // The thread's first access to the team's first row.
  __device__ __forceinline__ const char* begin(const Rows& rows) const {
    return rows.p + index(row) * rows.pitch + column(0) * static_cast<int>(sizeof(T));
  }
  // The first row of the first team of the thread's warp: teams that share a warp go on together.
  __device__ __forceinline__ uint32_t first() const {
    return row - (kTeam ? team % (32 / (kTeam ? kTeam : 32)) : 0) * kR;
  }
  __device__ __forceinline__ char* place(int st, int r, int array) const {
    return ring + ((st * kR + r) * kArrays + array) * kK * static_cast<int>(blockDim.x) * kBytes;
  }
  __device__ __forceinline__ char* extra_place(int st, int r, int array) const {
    return ring - threadIdx.x * kBytes + kStages * kR * kArrays * kK * static_cast<int>(blockDim.x) * kBytes +
           (((st * kR + r) * kArrays + array) * static_cast<int>(blockDim.x) + threadIdx.x) * 4;
  }
  // Begins the copy of the next batch; what is not there becomes zeros.
  __device__ __forceinline__ void copy(int st, const Rows (&rows)[kArrays]) {
#pragma unroll
    for (int array = 0; array < kArrays; ++array) {
      const char* none = rows[array].p;
      if constexpr (kShift) none -= reinterpret_cast<uintptr_t>(none) % 16;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const char* p = from[array] + bytes_to(rows[array], r);
        char* to = place(st, r, array);
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const bool there = k < count && row + r < n;
          // (where nothing is there nothing is read: the address is an aligned one all the same)
          const char* src = there ? p + k * threads * kBytes : none;
          char* at = to + k * static_cast<int>(blockDim.x) * kBytes;
          const int bytes = there ? kBytes : 0;
          if constexpr (kBytes == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(at)), "l"(src), "r"(bytes) : "memory");
          else if constexpr (kBytes == 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(at)), "l"(src), "r"(bytes) : "memory");
          else
            *reinterpret_cast<T*>(at) = there ? *reinterpret_cast<const T*>(src) : T(0.0f);
        }
      }
      if constexpr (kShift) {
        if (extra >= 0) {
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            // the upper element of four bytes comes with the one before it, but for the array's first
            const T* p = extra_of(rows[array], row + r);
            char* to = extra_place(st, r, array);
            const int bytes = row + r < n ? sizeof(T) == 2 && !extra_half ? 2 : 4 : 0;
            const void* src = bytes ? static_cast<const void*>(p - extra_half) : static_cast<const void*>(none);
            if (bytes && src < static_cast<const void*>(rows[array].p)) *reinterpret_cast<T*>(to + 2) = *p;
            else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(to)), "l"(src), "r"(bytes) : "memory");
          }
        }
      }
      from[array] += rows[array].advance;
    }
    row += step;
    if constexpr (kBytes > 2) ptx::cp_async_commit();
  }
  // Begins the copies of the first batches.
  __device__ __forceinline__ void start(const Rows (&rows)[kArrays]) {
#pragma unroll
    for (int array = 0; array < kArrays; ++array) from[array] = begin(rows[array]);
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) copy(st, rows);
  }
  // Begins one more copy, waits for the oldest and returns its stage.
  __device__ __forceinline__ int next(const Rows (&rows)[kArrays]) {
    const int now = stage;
    copy(now == 0 ? kStages - 1 : now - 1, rows);
    if constexpr (kBytes > 2) ptx::cp_async_wait<kStages - 1>();
    stage = now == kStages - 1 ? 0 : now + 1;
    return now;
  }
  // Waits for all copies but those of the last kStages - 2 batches (where two batches are in use).
  __device__ __forceinline__ void wait_for_next() const {
    if constexpr (kBytes > 2) ptx::cp_async_wait<kStages - 2>();
  }
  __device__ __forceinline__ void read(int st, int r, int array, float2 (&f)[kPairs]) const {
    read_pairs<T, kE, kPairs>(place(st, r, array), blockDim.x * kBytes, f);
  }
  // The address of the thread's extra element of the group's row r; and that element of a batch, 0 where there is none.
  __device__ __forceinline__ T* extra_of(const Rows& rows, uint32_t r) const {
    return reinterpret_cast<T*>(const_cast<char*>(rows.p) + index(r) * rows.pitch) + extra;
  }
  __device__ __forceinline__ float read_extra(int st, int r, int array) const {
    return extra >= 0 ? load(reinterpret_cast<const T*>(extra_place(st, r, array)) + extra_half) : 0.0f;
  }
  // Whether the thread's element c is in the row.
  __device__ __forceinline__ bool in_row(int c) const { return c / kE < count; }
  __device__ __forceinline__ void write(char* to, const float2 (&f)[kPairs]) const {
    write_pairs<T, kE, kPairs>(reinterpret_cast<T*>(to), pitch(), count, f);
  }
  // The thread's columns of a vector, `none` each where there is no vector.
  __device__ __forceinline__ void read_vector(const void* p, int bf16, float none, float2 (&f)[kPairs]) const {
    if constexpr (kShift) {
#pragma unroll
      for (int c = 0; c < kColumns; ++c) {
        float v = none;
        if (p && in_row(c)) v = element(p, bf16, column(c / kE) + c % kE);
        if (c % 2) f[c / 2].y = v;
        else f[c / 2].x = v;
      }
    } else {
      vector_columns<kE, kPairs>(p, bf16, column(0), pitch(), count, none, f);
    }
  }
};

struct NormStream {
  Rows x[1];
  Rows out;
  const void* weight;
  const void* bias;
  float* mean;
  float* rstd;
  int weight_bf16, n, H, team_threads;
  int period;                // rows whose places in 16 bytes differ
  float eps, inv_h;
};

// Floats for each of a batch's rows, of a team of several warps.
__host__ __device__ constexpr int norm_slots(bool ahead) { return (ahead ? 2 * 4 : 3) * 32; }

// A batch takes two sums over its rows, one after the other: the elements', then the deviations' and their squares'.
// kAhead: the second one goes together with the next batch's first, for one barrier a batch instead of two, and
// every batch is read from shared memory twice.
template <typename T, int kE, int kColumns, int kR, int kStages, int kTeam, bool kShift, bool kAhead>
__global__ void __launch_bounds__(kStreamThreads) norm_stream_kernel(const NormStream a) {
  extern __shared__ float4 shared[];
  constexpr int kSums = (kAhead ? 4 : 2) * kR;             // (with kAhead 3 kR, filled up to a power of two)
  // slots of the sums for every team (with kAhead of two batches, which take turns), then the ring
  constexpr int kSlots = kTeam ? 0 : norm_slots(kAhead) * kR, kPairs = kColumns / 2;
  const int teams = blockDim.x / (kTeam ? kTeam : a.team_threads);
  float* slots = reinterpret_cast<float*>(shared);
  Stream<T, kE, kColumns, kR, 1, kStages, kTeam, kShift> s(a.team_threads, a.n, a.H, 1, a.period, a.x[0],
                                                           reinterpret_cast<char*>(slots + teams * kSlots));
  uint32_t row = s.row, turn = s.first();
  char* to = const_cast<char*>(s.begin(a.out));
  s.start(a.x);
  if constexpr (kSlots > 0) {
    for (int i = threadIdx.x; i < teams * kSlots; i += blockDim.x) slots[i] = 0.0f;
    __syncthreads();
    slots += s.team * kSlots;
  }
  float2 w[kPairs], b[kPairs];
  s.read_vector(a.weight, a.weight_bf16, 1.0f, w);
  s.read_vector(a.bias, a.weight_bf16, 0.0f, b);
  const float extra_w = kShift && s.extra >= 0 && a.weight ? element(a.weight, a.weight_bf16, s.extra) : 1.0f;
  const float extra_b = kShift && s.extra >= 0 && a.bias ? element(a.bias, a.weight_bf16, s.extra) : 0.0f;
  int stage = 0, flip = 0;
  // A row of the batch, and the thread's part of its sum.
  const auto read = [&](int r, float2 (&x)[kPairs], float& more) {
    s.read(stage, r, 0, x);
    float sum = pairs_sum<kPairs>(x);
    if constexpr (kShift) {
      more = s.read_extra(stage, r, 0);
      sum += more;
    }
    return sum;
  };
  // The next batch's rows' sums alone, into the last ones.
  const auto next_sums = [&](float (&sums)[kSums]) {
    stage = s.next(a.x);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float2 x[kPairs];
      float more;
      sums[kSums / 2 + r] = read(r, x, more);
    }
  };
  float centre[kR], extra[kR];
  if constexpr (kAhead) {
    float sums[kSums] = {};
    next_sums(sums);
    team_sum<kSums, kTeam>(sums, slots, s.team, s.threads);
#pragma unroll
    for (int r = 0; r < kR; ++r) centre[r] = sums[kSums / 2 + r];
  }
  for (; turn < s.n; turn += s.step, row += s.step, to += a.out.advance) {
    float2 d[kR][kPairs];
    float sums[kSums];
    if constexpr (kAhead) {
#pragma unroll
      for (int r = 0; r < kR; ++r) read(r, d[r], extra[r]);
    } else {
      stage = s.next(a.x);
#pragma unroll
      for (int r = 0; r < kR; ++r) centre[r] = read(r, d[r], extra[r]);
      team_sum<kR, kTeam>(centre, slots + kSums * 32, s.team, s.threads);
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      centre[r] = centre_of<T>(centre[r] * a.inv_h);
      float2 squares[kPairs];
      // (what is not in the row stays 0)
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        d[r][i] = sub2(d[r][i], make_float2(2 * i / kE < s.count ? centre[r] : 0.0f, (2 * i + 1) / kE < s.count ? centre[r] : 0.0f));
#pragma unroll
      for (int i = 0; i < kPairs; ++i) squares[i] = mul2(d[r][i], d[r][i]);
      sums[r] = pairs_sum<kPairs>(d[r]);
      sums[kR + r] = pairs_sum<kPairs>(squares);
      if constexpr (kShift) {
        extra[r] = s.extra >= 0 ? extra[r] - centre[r] : 0.0f;
        sums[r] += extra[r];
        sums[kR + r] = fmaf(extra[r], extra[r], sums[kR + r]);
      }
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int r = 0; r < kR; ++r) sums[3 * kR + r] = 0.0f;
      next_sums(sums);                     // (the batch itself is in registers)
      flip ^= 1;
    }
    team_sum<kSums, kTeam>(sums, slots + flip * kSums * 32, s.team, s.threads);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      // what the centre is off the mean, the deviations' own mean shows
      const float rest = sums[r] * a.inv_h, rstd = rstd_of(rest, sums[kR + r] * a.inv_h, a.eps);
      if (row + r >= s.n) break;
      if (s.thread == 0 && a.mean) {
        a.mean[s.index(row + r)] = centre[r] + rest;
        a.rstd[s.index(row + r)] = rstd;
      }
      const float shift = -rest * rstd;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) d[r][i] = fma2(fma2(d[r][i], both(rstd), both(shift)), w[i], b[i]);
      s.write(to + s.bytes_to(a.out, r), d[r]);
      if constexpr (kShift)
        if (s.extra >= 0) store(s.extra_of(a.out, row + r), fmaf(fmaf(extra[r], rstd, shift), extra_w, extra_b));
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int r = 0; r < kR; ++r) centre[r] = sums[kSums / 2 + r];
    }
  }
}

// A block takes a row at a time, 32 elements a thread in registers; several blocks of an SM hide one another's sums.
// kStages: a block stays on its SM and the rows that it takes after this one are being copied ahead; 0: it takes one.
constexpr int kBlockThreads = 1024, kBlockPairs = 16;
constexpr int kBlockHidden = kBlockThreads * 2 * kBlockPairs, kBlockStages = 2;

template <typename T, int kE, int kStages>
__global__ void __launch_bounds__(kBlockThreads) norm_block_kernel(const NormStream a) {
  extern __shared__ float4 shared[];
  __shared__ float slots[2][2 * 32];
  const int threads = blockDim.x, thread = threadIdx.x;
  using S = Stream<T, kE, 2 * kBlockPairs, 1, 1, kStages ? kStages : 1, 0, false>;
  S s(threads, a.n, a.H, 1, 1, a.x[0], reinterpret_cast<char*>(shared));
  const int count = s.count;
  uint32_t row = s.row;
  char* to = const_cast<char*>(s.begin(a.out));
  if constexpr (kStages > 0) s.start(a.x);
  if (thread < 2 * 32) slots[0][thread] = slots[1][thread] = 0.0f;
  __syncthreads();
  for (; row < a.n; row += gridDim.x, to += a.out.advance) {
    float2 d[kBlockPairs];
    if constexpr (kStages > 0) {
      s.read(s.next(a.x), 0, 0, d);
    } else {
      const T* x = reinterpret_cast<const T*>(s.begin(a.x[0]));
#pragma unroll
      for (int i = 0; i < kBlockPairs; ++i) d[i] = both(0.0f);
#pragma unroll
      for (int k = 0; k < 2 * kBlockPairs / kE; ++k) {
        if (k >= count) continue;
        if constexpr (kE == 1) (k % 2 ? d[k / 2].y : d[k / 2].x) = load(x + k * threads);
        else Access<T, kE>::unpack(*reinterpret_cast<const typename Access<T, kE>::Raw*>(x + k * threads * kE), d + k * kE / 2);
      }
    }
    float centre[1] = {pairs_sum<kBlockPairs>(d)}, sums[2];
    team_sum<1, 0>(centre, slots[0], 0, threads);
    centre[0] = centre_of<T>(centre[0] * a.inv_h);
    float2 squares = both(0.0f);
#pragma unroll
    for (int i = 0; i < kBlockPairs; ++i) {
      d[i] = sub2(d[i], make_float2(2 * i / kE < count ? centre[0] : 0.0f, (2 * i + 1) / kE < count ? centre[0] : 0.0f));
      squares = fma2(d[i], d[i], squares);
    }
    sums[0] = pairs_sum<kBlockPairs>(d);
    sums[1] = squares.x + squares.y;
    team_sum<2, 0>(sums, slots[1], 0, threads);
    const float rest = sums[0] * a.inv_h, rstd = rstd_of(rest, sums[1] * a.inv_h, a.eps), shift = -rest * rstd;
    if (thread == 0 && a.mean) {
      a.mean[row] = centre[0] + rest;
      a.rstd[row] = rstd;
    }
    T* out = reinterpret_cast<T*>(to);
#pragma unroll
    for (int k = 0; k < 2 * kBlockPairs / kE; ++k) {
      if (k >= count) continue;
      constexpr int kP = kE > 1 ? kE / 2 : 1;
      float2 w[kP], b[kP], y[kP];
#pragma unroll
      for (int i = 0; i < kP; ++i) w[i] = both(1.0f), b[i] = both(0.0f);
      const int j = (k * threads + thread) * kE;
      if (a.weight && a.weight_bf16) vector_part<__nv_bfloat16, kE>(static_cast<const __nv_bfloat16*>(a.weight) + j, w);
      else if (a.weight) vector_part<float, kE>(static_cast<const float*>(a.weight) + j, w);
      if (a.bias && a.weight_bf16) vector_part<__nv_bfloat16, kE>(static_cast<const __nv_bfloat16*>(a.bias) + j, b);
      else if (a.bias) vector_part<float, kE>(static_cast<const float*>(a.bias) + j, b);
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const float2 v = kE > 1 ? d[k * kP + i] : both(k % 2 ? d[k / 2].y : d[k / 2].x);
        y[i] = fma2(fma2(v, both(rstd), both(shift)), w[i], b[i]);
      }
      if constexpr (kE == 1) store(out + k * threads, y[0].x);
      else *reinterpret_cast<typename Access<T, kE>::Raw*>(out + k * threads * kE) = Access<T, kE>::pack(y);
    }
    if constexpr (kStages == 0) break;
  }
}

// main_grad[j] += v, in 32 bits; nothing without a main_grad.
__device__ __forceinline__ void add_to_main_grad(void* to, int bf16, int j, float v) {
  if (!to) return;
  if (bf16) store(static_cast<__nv_bfloat16*>(to) + j, element(to, 1, j) + v);
  else static_cast<float*>(to)[j] += v;
}

struct NormGradStream {
  Rows in[2];                // x, grad
  Rows grad_x;
  const void* weight;
  const float* mean;
  const float* rstd;
  float* partial;            // null: no sums
  void* main_grads[2];       // where the only group adds its sums by itself
  int main_grad_bf16, alone;
  int weight_bf16, n, H, team_threads;
  int blocks;                // of a cluster
  int period;                // rows whose places in 16 bytes differ
  float inv_h;
};

// A block's teams take batches in turn, a thread the same columns of every row: their weights and the sums
// for the main_grads stay in its registers.
template <typename T, int kE, int kColumns, int kR, int kStages, int kTeam, bool kShift, bool kCluster>
__global__ void __launch_bounds__(kStreamThreads) norm_grad_stream_kernel(const NormGradStream a) {
  extern __shared__ float4 shared[];
  const int blocks = kCluster ? a.blocks : 1;
  ptx::pdl_launch_dependents();
  // two batches' slots for every team, then the ring
  constexpr int kSlots = kTeam ? 0 : 2 * 2 * kR * 32, kPairs = kColumns / 2;
  using S = Stream<T, kE, kColumns, kR, 2, kStages, kTeam, kShift>;
  const int teams = blockDim.x / (kTeam ? kTeam : a.team_threads);
  float* slots = reinterpret_cast<float*>(shared);
  S s(a.team_threads, a.n, a.H, blocks, a.period, a.in[0], reinterpret_cast<char*>(slots + teams * kSlots));
  uint32_t row = s.row, turn = s.first();
  char* to = const_cast<char*>(s.begin(a.grad_x));
  s.start(a.in);
  float means[kR], rstds[kR];
  auto moments = [&](uint32_t at) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      means[r] = at + r < s.n ? __ldg(a.mean + s.index(at + r)) : 0.0f;
      rstds[r] = at + r < s.n ? __ldg(a.rstd + s.index(at + r)) : 0.0f;
    }
  };
  moments(row);
  if constexpr (kCluster) ptx::cluster_sync_all();         // (all blocks are there before their memory is written)
  if constexpr (kSlots > 0) {
    for (int i = threadIdx.x; i < teams * kSlots; i += blockDim.x) slots[i] = 0.0f;
    __syncthreads();
    slots += s.team * kSlots;
  }
  float2 w[kPairs], dw[kPairs], db[kPairs];
  s.read_vector(a.weight, a.weight_bf16, 1.0f, w);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) dw[i] = db[i] = both(0.0f);
  const float extra_w = kShift && s.extra >= 0 && a.weight ? element(a.weight, a.weight_bf16, s.extra) : 1.0f;
  float extra_dw = 0.0f, extra_db = 0.0f;
  int flip = 0;
  // A batch's sums over the thread's columns, and what it adds to the columns' own.
  const auto add_up = [&](int stage, const float (&mean)[kR], const float (&rstd)[kR], float (&sums)[2 * kR]) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float2 x[kPairs], g[kPairs], s1 = both(0.0f), s2 = both(0.0f);
      s.read(stage, r, 0, x);
      s.read(stage, r, 1, g);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 n = mul2(sub2(x[i], both(mean[r])), both(rstd[r])), u = mul2(g[i], w[i]);
        dw[i] = fma2(g[i], n, dw[i]);
        db[i] = add2(db[i], g[i]);
        s1 = add2(s1, u);
        s2 = fma2(u, n, s2);
      }
      sums[r] = s1.x + s1.y;
      sums[kR + r] = s2.x + s2.y;
      if constexpr (kShift) {
        const float n = (s.read_extra(stage, r, 0) - mean[r]) * rstd[r], extra_g = s.read_extra(stage, r, 1);
        extra_dw = fmaf(extra_g, n, extra_dw);
        extra_db += extra_g;
        sums[r] = fmaf(extra_g, extra_w, sums[r]);
        sums[kR + r] = fmaf(extra_g * extra_w, n, sums[kR + r]);
      }
    }
    team_sum<2 * kR, kTeam>(sums, slots + flip * 2 * kR * 32, s.team, s.threads);
    flip ^= 1;
  };
  // Its gradient, from the sums over its rows.  The rows are read again rather than kept: registers hold the
  // columns' sums.
  const auto write = [&](int stage, const float (&mean)[kR], const float (&rstd)[kR], const float (&sums)[2 * kR]) {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (row + r >= s.n) break;
      float2 x[kPairs], g[kPairs];
      s.read(stage, r, 0, x);
      s.read(stage, r, 1, g);
      // rstd (u - avg(u) - n avg(u n))
      const float c1 = -sums[r] * a.inv_h * rstd[r], c2 = -sums[kR + r] * a.inv_h * rstd[r];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 n = mul2(sub2(x[i], both(mean[r])), both(rstd[r])), u = mul2(g[i], w[i]);
        x[i] = fma2(n, both(c2), fma2(u, both(rstd[r]), both(c1)));
      }
      s.write(to + s.bytes_to(a.grad_x, r), x);
      if constexpr (kShift)
        if (s.extra >= 0) {
          const float n = (s.read_extra(stage, r, 0) - mean[r]) * rstd[r], u = s.read_extra(stage, r, 1) * extra_w;
          store(s.extra_of(a.grad_x, row + r), fmaf(n, c2, fmaf(u, rstd[r], c1)));
        }
    }
  };
  float mean[kR], rstd[kR], sums[2 * kR];
  const auto take_moments = [&](uint32_t next) {
#pragma unroll
    for (int r = 0; r < kR; ++r) mean[r] = means[r], rstd[r] = rstds[r];
    moments(next);
  };
  if constexpr (!kCluster) {
    for (; turn < s.n; turn += s.step, row += s.step, to += a.grad_x.advance) {
      const int stage = s.next(a.in);
      take_moments(row + s.step);
      add_up(stage, mean, rstd, sums);
      write(stage, mean, rstd, sums);
    }
  } else if (row < s.n) {
    // A cluster's sums take their time: the next batch's are sent before a batch is written (4096 x 16384 bf16: 87 us
    // instead of 89, fp32 139 instead of 160; 1024 x 65536 bf16: 113 instead of 122).  Two batches are in use then,
    // and the copies of one or two more on their way.
    __shared__ float box[2][kMostBlocks][2 * kR];
    const int rank = static_cast<int>(ptx::cluster_rank());
    int stage = 0;
    s.wait_for_next();
    take_moments(row + s.step);
    add_up(stage, mean, rstd, sums);
    cluster_send(sums, box[0], blocks, rank);
    s.copy(kStages - 1, a.in);
    for (int half = 0;; half ^= 1) {
      float total[2 * kR], mean_now[kR], rstd_now[kR];
      cluster_take(total, box[half], blocks);
#pragma unroll
      for (int r = 0; r < kR; ++r) mean_now[r] = mean[r], rstd_now[r] = rstd[r];
      const bool more = row + s.step < s.n;
      const int next = stage == kStages - 1 ? 0 : stage + 1;
      if (more) {
        s.wait_for_next();
        take_moments(row + 2 * s.step);
        add_up(next, mean, rstd, sums);
        cluster_send(sums, box[half ^ 1], blocks, rank);
      }
      write(stage, mean_now, rstd_now, total);
      if (!more) break;
      s.copy(stage, a.in);
      stage = next;
      row += s.step;
      to += a.grad_x.advance;
    }
  }
  if (!a.partial) return;
  // the teams' sums, in their order, to the block's share, or where there is no other, to the main_grads
  float* out = a.partial + static_cast<long long>(s.group) * 2 * a.H;
  float* meet = reinterpret_cast<float*>(shared);
  if constexpr (S::kBytes > 2) ptx::cp_async_wait<0>();        // (the ring is about to be used for them)
  constexpr int kMine = kColumns + kShift;           // the extra element's sums are the last
  auto column = [&](int c) { return c == kColumns ? s.extra : s.column(c / kE) + c % kE; };
  auto in_row = [&](int c) { return c == kColumns ? s.extra >= 0 : s.in_row(c); };
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float mine[kMine];
#pragma unroll
    for (int c = 0; c < kColumns; ++c) {
      const float2 v = half ? db[c / 2] : dw[c / 2];
      mine[c] = c % 2 ? v.y : v.x;
    }
    if constexpr (kShift) mine[kColumns] = half ? extra_db : extra_dw;
    if (teams > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kMine; ++c) meet[(s.team * kMine + c) * s.threads + s.thread] = mine[c];
      __syncthreads();
      for (int c = s.team; c < kMine; c += teams) {
        float v = 0.0f;
        for (int t = 0; t < teams; ++t) v += meet[(t * kMine + c) * s.threads + s.thread];
        if (!in_row(c)) continue;
        if (a.alone) add_to_main_grad(a.main_grads[half], a.main_grad_bf16, column(c), v);
        else out[half * a.H + column(c)] = v;
      }
    } else if (a.alone) {
      void* to = a.main_grads[half];
      if (!to) continue;
      float before[kMine];                         // all read before the first is written
#pragma unroll
      for (int c = 0; c < kMine; ++c) before[c] = in_row(c) ? element(to, a.main_grad_bf16, column(c)) : 0.0f;
#pragma unroll
      for (int c = 0; c < kMine; ++c) {
        if (!in_row(c)) continue;
        if (a.main_grad_bf16) store(static_cast<__nv_bfloat16*>(to) + column(c), before[c] + mine[c]);
        else static_cast<float*>(to)[column(c)] = before[c] + mine[c];
      }
    } else {
#pragma unroll
      for (int c = 0; c < kMine; c += kE < 4 || kShift ? 1 : 4) {
        if (!in_row(c)) continue;
        // (rows whose vectors move whole have a multiple of four elements, and shares lie at 256 bytes)
        if constexpr (kE >= 4 && !kShift)
          *reinterpret_cast<float4*>(out + half * a.H + column(c)) = make_float4(mine[c], mine[c + 1], mine[c + 2], mine[c + 3]);
        else
          out[half * a.H + column(c)] = mine[c];
      }
    }
  }
}

// Sum of both parts over a block of kThreads, in every thread.
template <int kThreads>
__device__ __forceinline__ float2 block_sum(float2 v) {
  __shared__ float2 warps[kThreads / 32];
#pragma unroll
  for (int d = 16; d; d /= 2) {
    v.x += __shfl_xor_sync(kAll, v.x, d);
    v.y += __shfl_xor_sync(kAll, v.y, d);
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = v;
  __syncthreads();
  v = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    v.x += warps[i].x;
    v.y += warps[i].y;
  }
  return v;
}

constexpr int kRowThreads = 256;

// ---- rows that no block holds: gone through from memory

// Pairs of sums over a row, in every thread of its block; add(j, s) adds column j's numbers to s.  A thread has up to
// 65536 columns: it adds up 32 at a time, then 32 of these sums at a time, then those, so that a sum is off by at most
// 129 roundings there and 13 where the threads' meet, however wide the row is (one after the other equal numbers of a
// row of 2^24 come out 6e-4 off).  32 loads at once make up for the shorter loops: 2048 x 65536 bf16 forward 379
// us, one after the other 369; 8 loads at once 391.
template <typename F>
__device__ __forceinline__ float2 row_sum(int H, F add) {
  constexpr int kAtOnce = 32;
  float2 total = make_float2(0.0f, 0.0f), some = total;
  int j = threadIdx.x;
  for (int parts = 1; j < H; ++parts) {
    float2 s = make_float2(0.0f, 0.0f);
    if (j + (kAtOnce - 1) * kRowThreads < H) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) add(j + k * kRowThreads, s);
      j += kAtOnce * kRowThreads;
    } else {
      for (; j < H; j += kRowThreads) add(j, s);
    }
    some = add2(some, s);
    if (parts % kAtOnce == 0) {
      total = add2(total, some);
      some = make_float2(0.0f, 0.0f);
    }
  }
  return block_sum<kRowThreads>(add2(total, some));
}

// A block goes through one row three times.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) norm_kernel(NormArgs a) {
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  T* out = static_cast<T*>(a.out) + row * a.out_stride;
  float2 s = row_sum(a.H, [&](int j, float2& t) { t.x += load(x + j); });
  const float near = centre_of<T>(s.x * a.inv_h);
  s = row_sum(a.H, [&](int j, float2& t) {
    const float d = load(x + j) - near;
    t.x += d;
    t.y = fmaf(d, d, t.y);
  });
  // what `near` is off the mean, the deviations' own mean shows
  const float rest = s.x * a.inv_h;
  const float rstd = rstd_of(rest, s.y * a.inv_h, a.eps);
  if (threadIdx.x == 0 && a.mean) {
    a.mean[row] = near + rest;
    a.rstd[row] = rstd;
  }
  for (int j = threadIdx.x; j < a.H; j += kRowThreads) {
    float y = ((load(x + j) - near) - rest) * rstd;
    if (a.weight) y *= element(a.weight, a.weight_bf16, j);
    if (a.bias) y += element(a.bias, a.weight_bf16, j);
    store(out + j, y);
  }
}

// avg(u) and avg(u n) of a row, a block for each.  (All of an SM's threads are wanted: with six blocks instead of eight
// 1024 x 131072 bf16 takes 567 us instead of 517 with what follows.)
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 2048 / kRowThreads) norm_grad_rows_kernel(NormGradArgs a) {
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* g = static_cast<const T*>(a.grad) + row * a.grad_stride;
  const float mean = a.mean[row], rstd = a.rstd[row];
  const float2 s = row_sum(a.H, [&](int j, float2& t) {
    const float u = load(g + j) * (a.weight ? element(a.weight, a.weight_bf16, j) : 1.0f);
    t.x += u;
    t.y = fmaf(u, (load(x + j) - mean) * rstd, t.y);
  });
  if (threadIdx.x == 0) a.row_sums[row] = make_float2(s.x * a.inv_h, s.y * a.inv_h);
}

// A thread takes a column of one share of the rows: dx, and the share of the column's sums.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) norm_grad_columns_kernel(NormGradArgs a) {
  const int j = blockIdx.x * kRowThreads + threadIdx.x, part = blockIdx.y;
  if (j >= a.H) return;
  const int first = static_cast<int>(static_cast<long long>(a.n) * part / a.parts);
  const int end = static_cast<int>(static_cast<long long>(a.n) * (part + 1) / a.parts);
  const float w = a.weight ? element(a.weight, a.weight_bf16, j) : 1.0f;
  float dw = 0.0f, db = 0.0f;
  for (long long row = first; row < end; ++row) {
    const float g = load(static_cast<const T*>(a.grad) + row * a.grad_stride + j);
    const float x = load(static_cast<const T*>(a.x) + row * a.x_stride + j);
    const float rstd = a.rstd[row], n = (x - a.mean[row]) * rstd;
    const float2 avg = a.row_sums[row];
    dw = fmaf(g, n, dw);
    db += g;
    store(static_cast<T*>(a.grad_x) + row * a.grad_x_stride + j, (g * w - avg.x - n * avg.y) * rstd);
  }
  float* p = a.partial + static_cast<long long>(part) * 2 * a.H;
  p[j] = dw;
  p[a.H + j] = db;
}

// The blocks' shares of a column's sums, joined by sixteen threads a column in an order that depends on their
// number alone, and added to the main_grad.
constexpr int kJoinGroups = 16;

__global__ void __launch_bounds__(32 * kJoinGroups) norm_grad_join_kernel(const NormGradArgs a) {
  __shared__ float sums[kJoinGroups][33];
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
  const int j = blockIdx.x * 32 + lane;
  void* to = blockIdx.y == 0 ? a.weight_main_grad : a.bias_main_grad;
  if (!to) return;
  ptx::pdl_wait_prior_grid();
  constexpr int kMost = (kNormParts + kJoinGroups - 1) / kJoinGroups;
  float v[kMost];
  const float* p = a.partial + static_cast<long long>(blockIdx.y) * a.H + j;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int part = group + i * kJoinGroups;
    v[i] = j < a.H && part < a.parts ? p[static_cast<long long>(part) * 2 * a.H] : 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kMost; ++i) s += v[i];
  sums[group][lane] = s;
  __syncthreads();
  if (group || j >= a.H) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinGroups; ++i) s += sums[i][lane];
  add_to_main_grad(to, a.main_grad_bf16, j, s);
}

cudaError_t launch_join(const NormGradArgs& a, cudaStream_t stream) {
  if (!a.weight_main_grad && !a.bias_main_grad) return cudaGetLastError();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.H + 31) / 32, 2);
  cfg.blockDim = dim3(32 * kJoinGroups);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_grad_join_kernel, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// A launch of one of the two: threads of a team, teams of a block, blocks, shared memory.
struct StreamShape {
  int threads, teams, blocks, groups;     // blocks: of a cluster; groups: clusters, or blocks by themselves
  size_t bytes;
};

// team: its threads, or 0 for as many warps as it takes; rows: of a batch; slots: floats for each of a batch's
// rows of a team of several warps; unit: bytes of the ring for a thread.
StreamShape make_stream_shape(int H, int access, int team, int columns, int rows, int slots, int unit) {
  StreamShape s{};
  s.blocks = 1;
  while (s.blocks < kMostBlocks && H > s.blocks * kStreamHidden) s.blocks *= 2;
  const int mine = (H / access + s.blocks - 1) / s.blocks * access;
  s.threads = team ? team : ((mine + columns - 1) / columns + 31) / 32 * 32;
  s.teams = s.blocks > 1 ? 1 : kStreamThreads / s.threads;
  if (!team && s.teams > 15) s.teams = 15;                 // named barriers 1 to 15
  s.bytes = static_cast<size_t>(s.teams) * ((team ? 0 : slots * rows * sizeof(float)) + static_cast<size_t>(s.threads) * unit);
  return s;
}

// No more groups than rows for all their teams; as many for each of `period` places.
void set_groups(StreamShape& s, int n, int rows, int most, int period) {
  const long long each = (static_cast<long long>(n) + period - 1) / period;
  const long long want = (each + rows * s.teams - 1) / (rows * s.teams);
  s.groups = static_cast<int>(want < most / period ? want : most / period) * period;
}

Rows make_rows(const void* p, long long stride, size_t size, const StreamShape& s, int rows) {
  const long long pitch = stride * static_cast<long long>(size);
  return {static_cast<const char*>(p), pitch, pitch * s.groups * s.teams * rows};
}

constexpr int kMaxDevices = 64;

// A kernel's set-up on each device: whether it may have all of an SM's shared memory, and how many of its clusters
// of 2, 4 and 8 blocks run at once.
struct StreamSetUp {
  std::atomic<bool> ready[kMaxDevices];
  std::atomic<int> clusters[kMaxDevices][4];
};

template <typename K>
cudaError_t set_up(K kernel, StreamSetUp& state, int dev) {
  if (state.ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024);
  if (e == cudaSuccess) state.ready[dev].store(true, std::memory_order_release);
  return e;
}

cudaLaunchConfig_t stream_config(const StreamShape& s, cudaLaunchAttribute* attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(s.groups * s.blocks);
  cfg.blockDim = dim3(s.teams * s.threads);
  cfg.dynamicSmemBytes = s.bytes;
  cfg.stream = stream;
  if (s.blocks > 1) {
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = s.blocks;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cfg;
}

// Groups that run at once, `sms` of single blocks.
template <typename K>
cudaError_t groups_at_once(K kernel, StreamSetUp& state, StreamShape s, int dev, int sms, int* groups) {
  *groups = sms;
  if (s.blocks == 1) return cudaSuccess;
  std::atomic<int>& known = state.clusters[dev][s.blocks / 4];
  if ((*groups = known.load()) > 0) return cudaSuccess;
  s.groups = 1;
  s.bytes = 200 * 1024;                                    // (the same for all sizes: one block an SM)
  cudaLaunchAttribute attr{};
  const cudaLaunchConfig_t cfg = stream_config(s, &attr, nullptr);
  const cudaError_t e = cudaOccupancyMaxActiveClusters(groups, kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (*groups < 1) return cudaErrorInvalidConfiguration;
  known.store(*groups);
  return cudaSuccess;
}

// Rows of a batch, 64 bytes of each array a thread, and stages, by what fits into registers and shared memory.
template <typename T, int kColumns>
constexpr int batch_rows() { return 64 / (kColumns * static_cast<int>(sizeof(T))); }
template <typename T, int kE>
constexpr int stages(int arrays, bool cluster) { return kE * sizeof(T) == 2 ? 1 + cluster : sizeof(T) == 4 && arrays == 1 ? 4 : 3; }

NormStream norm_stream(const NormArgs& a, size_t size, const StreamShape& s, int rows) {
  NormStream k{};
  k.x[0] = make_rows(a.x, a.x_stride, size, s, rows);
  k.out = make_rows(a.out, a.out_stride, size, s, rows);
  k.weight = a.weight;
  k.bias = a.bias;
  k.mean = a.mean;
  k.rstd = a.rstd;
  k.weight_bf16 = a.weight_bf16;
  k.n = a.n;
  k.H = a.H;
  k.team_threads = s.threads;
  k.period = a.period;
  k.eps = a.eps;
  k.inv_h = a.inv_h;
  return k;
}

template <typename T, int kE, int kColumns, int kTeam, bool kShift, bool kAhead>
cudaError_t launch_stream(const NormArgs& a, cudaStream_t stream) {
  constexpr int kR = batch_rows<T, kColumns>(), kStages = stages<T, kE>(1, false);
  static StreamSetUp state;
  const auto kernel = norm_stream_kernel<T, kE, kColumns, kR, kStages, kTeam, kShift, kAhead>;
  const cudaError_t e = set_up(kernel, state, a.dev);
  if (e != cudaSuccess) return e;
  StreamShape s = make_stream_shape(a.H, kE, kTeam, kColumns, kR, norm_slots(kAhead), kStages * kR * (kColumns * static_cast<int>(sizeof(T)) + 4 * kShift));
  set_groups(s, a.n, kR, a.num_sms, a.period);
  kernel<<<s.groups, s.teams * s.threads, s.bytes, stream>>>(norm_stream(a, sizeof(T), s, kR));
  return cudaGetLastError();
}

template <typename T, int kE, int kColumns, int kTeam, bool kShift>
cudaError_t launch_stream(const NormArgs& a, cudaStream_t stream) {
  // Of up to three teams an SM none may be left to work while the others wait for their sums: taken with the next
  // batch's these take 616 us instead of 672 for 131072 x 8192 bf16, 42.3 instead of 44.4 for 8192 x 7168, 52.0 instead of
  // 53.7 for 32768 x 2304; four teams of 2048 columns 44.2 instead of 42.5, fp32 rows of 8192 92 instead of 82.  The first
  // batch's sums come alone, which few rows do not make up for: 1216 x 7168 takes 11.0 us so, 10.5 without.
  if constexpr (sizeof(T) == 2 && kE == 8 && kColumns == 16 && kTeam == 0)
    if (a.H > 2048 && a.n > 16 * a.num_sms) return launch_stream<T, kE, kColumns, kTeam, kShift, true>(a, stream);
  return launch_stream<T, kE, kColumns, kTeam, kShift, false>(a, stream);
}

int block_threads(int H) { return ((H + 2 * kBlockPairs - 1) / (2 * kBlockPairs) + 31) / 32 * 32; }

template <typename T, int kE, int kStages>
cudaError_t launch_block(const NormArgs& a, cudaStream_t stream) {
  static StreamSetUp state;
  const auto kernel = norm_block_kernel<T, kE, kStages>;
  StreamShape s{block_threads(a.H), 1, 1, a.n, 0};
  if constexpr (kStages > 0) {
    s.bytes = static_cast<size_t>(s.threads) * kStages * 2 * kBlockPairs * sizeof(T);
    const cudaError_t e = set_up(kernel, state, a.dev);
    if (e != cudaSuccess) return e;
    const int most = a.num_sms * (kBlockThreads / s.threads);
    if (s.groups > most) s.groups = most;
  }
  kernel<<<s.groups, s.threads, s.bytes, stream>>>(norm_stream(a, sizeof(T), s, 1));
  return cudaGetLastError();
}

template <typename T, int kE, int kColumns, int kTeam, bool kShift, bool kCluster = false>
cudaError_t launch_stream(NormGradArgs a, cudaStream_t stream) {
  // (the extra elements of four rows do not fit)
  constexpr int kR = batch_rows<T, kColumns>() / (kShift && kColumns == 8 && sizeof(T) == 2 ? 2 : 1), kStages = stages<T, kE>(2, kCluster);
  static StreamSetUp state;
  const auto kernel = norm_grad_stream_kernel<T, kE, kColumns, kR, kStages, kTeam, kShift, kCluster>;
  StreamShape s = make_stream_shape(a.H, kE, kTeam, kColumns, kR, 4 * 32, kStages * kR * 2 * (kColumns * static_cast<int>(sizeof(T)) + 4 * kShift));
  const size_t meet = static_cast<size_t>(s.teams) * s.threads * (kColumns + 1) * sizeof(float);
  if (s.bytes < meet) s.bytes = meet;
  int most = 0;
  cudaError_t e = set_up(kernel, state, a.dev);
  if (e != cudaSuccess || (e = groups_at_once(kernel, state, s, a.dev, a.num_sms, &most)) != cudaSuccess) return e;
  set_groups(s, a.n, kR, most < a.parts ? most : a.parts, a.period);
  a.parts = s.groups;
  NormGradStream k{};
  k.in[0] = make_rows(a.x, a.x_stride, sizeof(T), s, kR);
  k.in[1] = make_rows(a.grad, a.grad_stride, sizeof(T), s, kR);
  k.grad_x = make_rows(a.grad_x, a.grad_x_stride, sizeof(T), s, kR);
  k.weight = a.weight;
  k.mean = a.mean;
  k.rstd = a.rstd;
  k.partial = a.weight_main_grad || a.bias_main_grad ? a.partial : nullptr;
  k.main_grads[0] = a.weight_main_grad;
  k.main_grads[1] = a.bias_main_grad;
  k.main_grad_bf16 = a.main_grad_bf16;
  k.alone = s.groups == 1;
  k.weight_bf16 = a.weight_bf16;
  k.n = a.n;
  k.H = a.H;
  k.team_threads = s.threads;
  k.blocks = s.blocks;
  k.period = a.period;
  k.inv_h = a.inv_h;
  cudaLaunchAttribute attr{};
  const cudaLaunchConfig_t cfg = stream_config(s, &attr, stream);
  if ((e = cudaLaunchKernelEx(&cfg, kernel, k)) != cudaSuccess) return e;
  return k.alone ? cudaGetLastError() : launch_join(a, stream);
}

template <typename T, int kE, int kColumns, bool kShift, typename Args>
cudaError_t by_team(const Args& a, cudaStream_t stream) {
  const int H = a.H;
  // (extra elements, up to two accesses' less two, are a thread's each)
  if constexpr (!kShift)
    if (H <= 4 * kColumns) return launch_stream<T, kE, kColumns, 4, kShift>(a, stream);
  if constexpr (!kShift || kE <= 4)
    if (H <= 8 * kColumns) return launch_stream<T, kE, kColumns, 8, kShift>(a, stream);
  if (H <= 16 * kColumns) return launch_stream<T, kE, kColumns, 16, kShift>(a, stream);
  if (H <= 32 * kColumns) return launch_stream<T, kE, kColumns, 32, kShift>(a, stream);
  return launch_stream<T, kE, kColumns, 0, kShift>(a, stream);
}

// One of the kernels by a row's elements.  A thread has sixteen of them, which spreads a sum's shuffles
// over the most (65536 x 1024 bf16 forward: 44 us, with eight 51), but for short rows of fp32,
// of which a batch would be one (65536 x 1024 forward: 93 us, with eight 80), and short rows'
// gradient, where the columns' sums take the registers (65536 x 256 bf16: 33 us, with eight 23).
template <typename T, int kE, bool kShift>
cudaError_t stream_rows(const NormArgs& a, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    return by_team<T, kE, 16, kShift>(a, stream);
  } else {
    return a.H <= 1024 ? by_team<T, kE, 8, kShift>(a, stream) : launch_stream<T, kE, 16, 0, kShift>(a, stream);
  }
}
template <typename T, int kE, bool kShift>
cudaError_t stream_rows(const NormGradArgs& a, cudaStream_t stream) {
  // (rows of bf16 with extra elements have batches of two either way: 65536 x 1001 97 us with eight, 78 with sixteen)
  if (a.H <= (kShift && sizeof(T) == 2 ? 768 : 1024)) return by_team<T, kE, 8, kShift>(a, stream);
  return launch_stream<T, kE, 16, 0, kShift>(a, stream);
}

template <typename T>
cudaError_t grad_loops(const NormGradArgs& a, cudaStream_t stream) {
  const unsigned columns = (a.H + kRowThreads - 1) / kRowThreads;
  norm_grad_rows_kernel<T><<<a.n, kRowThreads, 0, stream>>>(a);
  norm_grad_columns_kernel<T><<<dim3(columns, a.parts), kRowThreads, 0, stream>>>(a);
  return launch_join(a, stream);
}

// The places of some arrays' rows in 16 bytes.
struct Places {
  bool alike = true;         // the same for all arrays, row by row
  bool whole = true;         // every row begins at 16 bytes
  int period = 1;            // rows after which they repeat
  uintptr_t begin = 0, step = 0;

  void add(const void* p, long long stride, int rows, size_t size, bool first) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p) % 16, d = rows > 1 ? static_cast<uintptr_t>(stride) * size % 16 : 0;
    if (first) begin = b, step = d;
    alike &= b == begin && d == step;
    whole &= b == 0 && d == 0;
    for (period = 1; step * period % 16; ++period) {}
  }
};

// Whether a vector's kE elements from a multiple of them on are one access.
bool vector_aligned(const void* p, int bf16, int elements) {
  return reinterpret_cast<uintptr_t>(p) % (elements * (bf16 ? 2 : 4)) == 0;
}

// The form that suits rows: whole accesses, whole accesses after a shift, or single elements.
enum Form { kWholeRows, kShiftedRows, kElements };

template <int kE>
Form form_of(const Places& places, int H, bool vectors) {
  if (places.whole && H % kE == 0 && vectors) return kWholeRows;
  return places.alike && H <= kStreamHidden ? kShiftedRows : kElements;
}

template <typename T>
cudaError_t forward(NormArgs a, cudaStream_t stream) {
  constexpr int kE = 16 / sizeof(T);
  Places places;
  places.add(a.x, a.x_stride, a.n, sizeof(T), true);
  places.add(a.out, a.out_stride, a.n, sizeof(T), false);
  const Form form = form_of<kE>(places, a.H, vector_aligned(a.weight, a.weight_bf16, kE) && vector_aligned(a.bias, a.weight_bf16, kE));
  a.period = form == kShiftedRows ? places.period : 1;
  if (a.H > kBlockHidden) {
    norm_kernel<T><<<a.n, kRowThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  if (a.H > kStreamHidden) {
    if (form != kWholeRows) return launch_block<T, 1, 0>(a, stream);
    // bf16 rows are copied ahead where the weights and biases still fit into the L1 cache beside the rings (4096 x
    // 12288: 47 us instead of 51; 16384 with fp32 vectors, which do not, 61 instead of 59), and where the
    // SM has no other block (2048 x 24576: 53 instead of 64, 32768: 69 instead of 79).
    if constexpr (sizeof(T) == 2) {
      const int blocks = kBlockThreads / block_threads(a.H);
      const size_t rings = static_cast<size_t>(blocks) * a.H * sizeof(T) * kBlockStages;
      const size_t vectors = static_cast<size_t>((a.weight != nullptr) + (a.bias != nullptr)) * a.H * (a.weight_bf16 ? 2 : 4);
      if (blocks == 1 || rings + vectors <= 216 * 1024) return launch_block<T, kE, kBlockStages>(a, stream);
    }
    return launch_block<T, kE, 0>(a, stream);
  }
  return form == kWholeRows     ? stream_rows<T, kE, false>(a, stream)
         : form == kShiftedRows ? stream_rows<T, kE, true>(a, stream)
                                : stream_rows<T, 1, false>(a, stream);
}

template <typename T>
cudaError_t grad(NormGradArgs a, cudaStream_t stream) {
  constexpr int kE = 16 / sizeof(T);
  Places places;
  places.add(a.x, a.x_stride, a.n, sizeof(T), true);
  places.add(a.grad, a.grad_stride, a.n, sizeof(T), false);
  places.add(a.grad_x, a.grad_x_stride, a.n, sizeof(T), false);
  Form form = form_of<kE>(places, a.H, vector_aligned(a.weight, a.weight_bf16, kE));
  if (form == kShiftedRows && a.parts < places.period) form = kElements;       // (too few rows for a share of each place)
  a.period = form == kShiftedRows ? places.period : 1;
  if (a.H > kNormHeld) return grad_loops<T>(a, stream);
  if (a.H > kStreamHidden)
    return form == kWholeRows ? launch_stream<T, kE, 16, 0, false, true>(a, stream) : launch_stream<T, 1, 16, 0, false, true>(a, stream);
  return form == kWholeRows     ? stream_rows<T, kE, false>(a, stream)
         : form == kShiftedRows ? stream_rows<T, kE, true>(a, stream)
                                : stream_rows<T, 1, false>(a, stream);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? forward<__nv_bfloat16>(a, stream) : forward<float>(a, stream);
}

cudaError_t launch_norm_grad(const NormGradArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? grad<__nv_bfloat16>(a, stream) : grad<float>(a, stream);
}

}  // namespace ewg
