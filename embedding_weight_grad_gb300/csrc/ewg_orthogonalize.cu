// Newton-Schulz orthogonalisation of an update.
//
// With X0 = G / |G|_F (its transpose where G has more rows than columns, so that X is r x c
// with r <= c) a step is
//
//     A = X X^T,    B = b A + c A^2,    X <- a X + B X,
//
// an odd polynomial of the singular values of X that drives them towards 1.  A and A^2 are
// symmetric: only the blocks on and below the diagonal are computed and mirrored, so a step
// is 3 r^2 c + r^3 floating-point operations instead of 4 r^2 c + 2 r^3.
//
// Precision.  The products run on the tensor cores with fp16 operands (11 significant bits) and
// fp32 accumulators.  What keeps the result near its bf16 rounding:
//   * X itself is kept to 22 bits: beside the fp16 numbers that feed the products, a second
//     fp16 number each holds what their rounding left; a X is taken from the sum.  Directions with small singular values, which the steps enlarge by up
//     to a^5 = 485, then carry no noise from the rounding of the large ones: B is small on
//     them.  Without it a matrix of low effective rank loses ten times the precision.
//   * What rounding left of the diagonals of A and B, their largest entries, is kept apart in
//     fp32: (b A + c A^2)_ii takes it in, and B X = fp16(B) X + rest(diag(B)) X.  (Taking the
//     whole diagonal out of the fp16 matrices would serve full-rank updates better, 1.8e-3
//     instead of 2.1e-3 with the bf16 rounding's 1.66e-3, and others worse, up to 3.9e-3: in
//     directions on which B vanishes its diagonal and the rest of it cancel, but not their
//     products with differently rounded X.)
//   * X is stored times s ~ sqrt(r c), a power of two, so that its entries are about 1 at first
//     and at most 1.2 s; A and B need no scale.
//
// Layout.  Every buffer is [., ld] fp16 with the r index inside: X^T (two, alternating), the
// rest of X^T, A and B.  The accumulator of a product has its row index across the lanes of a
// warp, so all stores of X^T and of the mirrored blocks are contiguous.  As an operand of X
// X^T, X^T has the product's rows inside (MN-major); for B X it has the inner index inside
// (K-major), as A and B have by symmetry.
#include <algorithm>
#include <cmath>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ewg.h"
#include "ewg_internal.cuh"
#include "ewg_ops.cuh"
#include "ewg_ptx.cuh"

namespace ewg {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- norm and first X

struct OrthoIn {
  const void* grad;
  int bf16, tall;
  long long batch_stride, row_stride;
  int rows, cols;
  int ld;
  long long x_batch;                 // elements between matrices of X^T
  float s;                           // X is stored times s
  double* norm;                      // [batch][norm_blocks] sums of squares
  int norm_blocks;
  __half* xt;
  __half* xl;
  Header* header;
  int* counters;                     // of the steps kernel, `num_counters` for each matrix
  int num_counters;
};

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ float grad_at(const OrthoIn& a, long long i) {
  return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.grad)[i])
                : static_cast<const float*>(a.grad)[i];
}

// The sum of the squares of a lane's kLaneElems elements, to about 2^-45 of it: each square
// and each addition with its rounding error (an fma, and Knuth's two-sum), the errors
// summed beside.  The norm then rounds to the same fp32 factor whatever the order of the
// elements (strides, alignment, a transposed matrix).  The elements are first scaled by the power
// of two that brings the largest near 1, which is exact, so that neither large nor small
// gradients leave fp32's range.  64-bit arithmetic would bound the kernel.
constexpr int kLaneElems = 32;

__device__ __forceinline__ double sum_of_squares(const float (&g)[kLaneElems]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kLaneElems; ++i) m = fmaxf(m, fabsf(g[i]));
  const int e = min(static_cast<int>(__float_as_uint(m) >> 23), 253);
  const float scale = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);          // 2^(127 - e)
  float sum = 0.0f, err = 0.0f;
#pragma unroll
  for (int i = 0; i < kLaneElems; ++i) {
    const float x = __fmul_rn(g[i], scale);
    const float p = __fmul_rn(x, x);
    const float t = __fadd_rn(sum, p);
    const float b = __fsub_rn(t, sum);
    const float lost = __fadd_rn(__fsub_rn(sum, __fsub_rn(t, b)), __fsub_rn(p, b));
    err = __fadd_rn(err, __fadd_rn(lost, __fmaf_rn(x, x, -p)));
    sum = t;
  }
  const double back = __longlong_as_double(static_cast<long long>(1023 + 2 * (e - 127)) << 52);
  // (an infinite or NaN sum has no error term)
  return (static_cast<double>(sum) + (isfinite(sum) ? static_cast<double>(err) : 0.0)) * back;
}

// Sums of squares of one matrix per blockIdx.y, a warp to 1024 neighbouring elements of a row
// (a matrix without gaps is one long row).  Bound by the read of G.
__global__ void __launch_bounds__(256) ortho_norm_kernel(const OrthoIn a) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.header->status = kStatusOk;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.num_counters; i += 256)
      a.counters[static_cast<long long>(blockIdx.y) * a.num_counters + i] = 0;
  constexpr int kChunk = 32 * kLaneElems;
  const bool whole = a.row_stride == a.cols;
  const long long cols = whole ? static_cast<long long>(a.rows) * a.cols : a.cols;
  const int chunks_per_row = static_cast<int>((cols + kChunk - 1) / kChunk);
  const long long chunks = static_cast<long long>(chunks_per_row) * (whole ? 1 : a.rows);
  const int lane = threadIdx.x % 32;
  double sum = 0.0;
  for (long long q = blockIdx.x * 8 + threadIdx.x / 32; q < chunks; q += gridDim.x * 8) {
    const long long row = whole ? 0 : q / chunks_per_row;
    const long long col = (q - row * chunks_per_row) * kChunk;
    const long long at = blockIdx.y * a.batch_stride + row * a.row_stride + col;
    const int n = static_cast<int>(min(cols - col, static_cast<long long>(kChunk)));
    float g[kLaneElems];
    const char* p = static_cast<const char*>(a.grad) + at * (a.bf16 ? 2 : 4);
    if (n == kChunk && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      const uint4* v = reinterpret_cast<const uint4*>(p) + lane;
      if (a.bf16) {
        uint4 r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = v[32 * i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            g[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
            g[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
          }
        }
      } else {
        uint4 r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = v[32 * i];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g[4 * i] = __uint_as_float(r[i].x);
          g[4 * i + 1] = __uint_as_float(r[i].y);
          g[4 * i + 2] = __uint_as_float(r[i].z);
          g[4 * i + 3] = __uint_as_float(r[i].w);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i) g[i] = lane + 32 * i < n ? grad_at(a, at + lane + 32 * i) : 0.0f;
    }
    sum += sum_of_squares(g);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  __shared__ double part[8];
  if (lane == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += part[w];
    a.norm[blockIdx.y * a.norm_blocks + blockIdx.x] = sum;
  }
}

// X^T times s / |G|, split into two fp16 numbers, by 64 x 64 tiles of G.  Bound by the read of G
// and the two writes.
__global__ void __launch_bounds__(256) ortho_scale_kernel(const OrthoIn a) {
  __shared__ float tile[64][65];
  __shared__ double factor;
  const int tid = threadIdx.x;
  const int row0 = blockIdx.y * 64, col0 = blockIdx.x * 64;
  // 16 bytes of G a thread, all of its part of the tile before the wait for the norm
  const int per = a.bf16 ? 8 : 4;                    // elements of a vector
  const int line = 64 / per, rows = 256 / line;      // threads to a row, rows at once
  const int cx = tid % line * per, ry = tid / line;
  const int es = a.bf16 ? 2 : 4;
  const char* base = static_cast<const char*>(a.grad) +
                     (blockIdx.z * a.batch_stride + static_cast<long long>(row0) * a.row_stride + col0) * es;
#pragma unroll 4
  for (int k = ry; k < 64; k += rows) {
    if (row0 + k >= a.rows) break;
    const char* p = base + (k * a.row_stride + cx) * es;
    const int n = a.cols - col0 - cx;
    if (n >= per && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (a.bf16) {
          tile[k][cx + 2 * q] = __uint_as_float(w[q] << 16);
          tile[k][cx + 2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        } else {
          tile[k][cx + q] = __uint_as_float(w[q]);
        }
      }
    } else {
      for (int q = 0; q < per && q < n; ++q)
        tile[k][cx + q] = a.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[q])
                                 : reinterpret_cast<const float*>(p)[q];
    }
  }
  if (tid < 32) {
    double sum = 0.0;
    for (int i = tid; i < a.norm_blocks; i += 32) sum += a.norm[blockIdx.z * a.norm_blocks + i];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    if (tid == 0) factor = sum == 0.0 ? 0.0 : a.s / sqrt(sum);   // a zero matrix stays zero
  }
  __syncthreads();
  // factor = f1 f2 with f1 a power of two, so that neither product leaves fp32's range
  int e;
  const float f2 = static_cast<float>(frexp(factor, &e));
  const int e1 = min(max(e, -120), 120);
  const float f1 = ldexpf(1.0f, e1);
  const float f3 = ldexpf(f2, min(max(e - e1, -126), 126));
  // the r index is G's column where G is tall, else its row
  const int outer0 = a.tall ? row0 : col0, inner0 = a.tall ? col0 : row0;
  const int outers = a.tall ? a.rows : a.cols, inners = a.tall ? a.cols : a.rows;
  const int x = tid % 8 * 8;
  if (inner0 + x >= a.ld) return;
#pragma unroll
  for (int k = tid / 8; k < 64; k += 32) {
    if (outer0 + k >= outers) break;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int in = x + 2 * q + h;
        v[h] = inner0 + in < inners ? (a.tall ? tile[k][in] : tile[in][k]) * f1 * f3 : 0.0f;
      }
      hi[q] = pack_half(v[0], v[1]);
      const float2 kept = unpack_half(hi[q]);
      lo[q] = pack_half(v[0] - kept.x, v[1] - kept.y);
    }
    const long long at = blockIdx.z * a.x_batch + static_cast<long long>(outer0 + k) * a.ld + inner0 + x;
    *reinterpret_cast<uint4*>(a.xt + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(a.xl + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ---------------------------------------------------------------- the products

constexpr int kBlock = 256;          // a pair of CTAs computes 256 x 256; each CTA 128 rows
constexpr int kStepK = 64;           // inner elements of a stage: one 128-byte swizzled row
constexpr int kStages = 6;
constexpr int kOperandBytes = 128 * kStepK * 2;       // one CTA's half of an operand's stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kBoxBytes = 64 * kStepK * 2;            // one tensor copy: 64 rows of 128 bytes
constexpr int kFirstEpilogueWarp = 4;
constexpr int kEpilogueWarps = 8;
constexpr int kWarpCols = 4 * kBlock / kEpilogueWarps;   // columns of an epilogue warp (all take 32 rows)
constexpr int kGemmThreads = 32 * (kFirstEpilogueWarp + kEpilogueWarps);
// The epilogue takes an accumulator in pieces of 32 rows x kPiece columns a warp, turned
// through shared memory: kPiece rows of 32 fp32 numbers, 16 bytes between rows (which puts a
// quarter-warp's 16-byte reads on different banks).
constexpr int kPiece = 16;
constexpr int kPieces = kWarpCols / kPiece;
constexpr int kTurnPitch = 36;                        // floats
constexpr int kTurnFloats = kPiece * kTurnPitch;
constexpr size_t kGemmSmem = static_cast<size_t>(kStages) * kStageBytes + kEpilogueWarps * kTurnFloats * 4 + 1024;
static_assert(kGemmSmem + 512 <= 227 * 1024, "stages and turning buffers fit in shared memory");
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr uint32_t kReadyLimit = 1u << 22;

enum Phase { kGram = 0, kPoly = 1, kUpdate = 2 };

struct OrthoMaps {
  CUtensorMap xt[2], a[2], b;        // boxes of 64 x 64, swizzled
};

struct OrthoArgs {
  int batch, r, c, ld;
  int steps;
  float ca, cb, cc;                  // the polynomial's coefficients
  float s;                           // X is stored times s
  __half* xt[2];
  __half* xl;
  __half* a[2];                      // of even and odd steps
  __half* b;
  float* diag_a[2];                  // [batch][ld]: what rounding left of the diagonals
  float* diag_b;
  int split[2];                      // parts of the inner dimension of X X^T and A A
  float* partial;                    // split products: [batch][block][part][CTA][warp][column][row]
  __nv_bfloat16* out;
  long long out_batch, out_row;
  int tall;
  Header* header;
  int* ready;                        // [phase][batch][block row]: warps done, over all steps
  int* arrived;                      // [phase][batch][block][CTA][warp]: parts done, over all steps
};

struct GemmSmem {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
  uint32_t tmem;
  int abort;
};

// Shared-memory operand descriptor: 128-byte swizzle; `lead` and `stride` in bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

__device__ __forceinline__ int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// A unit of work of a pair: block (I, J) of matrix z, part `part` of its inner dimension.  A
// and B: blocks on and below the diagonal only.
struct Unit {
  int z, I, J, part;
};

__device__ __forceinline__ int units_of(const OrthoArgs& a, int phase) {
  const int nr = blocks_of(a.r);
  return a.batch * (phase == kUpdate ? nr * blocks_of(a.c) : nr * (nr + 1) / 2 * a.split[phase]);
}

// Unit t of a phase.  The orders let a phase start before the one before it has ended: the
// update goes by rows, which is what A's blocks by rows need; B's blocks go by columns, whose
// first ones complete B's first rows, which the update's first rows need.
__device__ __forceinline__ Unit unit_at(const OrthoArgs& a, int phase, int t) {
  const int nr = blocks_of(a.r);
  Unit x;
  if (phase == kUpdate) {
    const int nc = blocks_of(a.c);
    x.z = t / (nr * nc);
    t -= x.z * nr * nc;
    x.I = t / nc;
    x.J = t - x.I * nc;
    x.part = 0;
    return x;
  }
  const int blocks = nr * (nr + 1) / 2, parts = a.split[phase];
  x.z = t / (blocks * parts);
  t -= x.z * blocks * parts;
  x.part = t % parts;
  t /= parts;
  if (phase == kPoly) t = blocks - 1 - t;
  int row = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
  while ((row + 1) * (row + 2) / 2 <= t) ++row;
  while (row * (row + 1) / 2 > t) --row;
  const int col = t - row * (row + 1) / 2;
  x.I = phase == kPoly ? nr - 1 - col : row;
  x.J = phase == kPoly ? nr - 1 - row : col;
  return x;
}

// The inner blocks [first, last) of a unit.
__device__ __forceinline__ void inner_of(const OrthoArgs& a, int phase, const Unit& x, int& first, int& last) {
  const int blocks = ((phase == kGram ? a.c : a.r) + kStepK - 1) / kStepK;
  const int per = phase == kUpdate ? blocks : (blocks + a.split[phase] - 1) / a.split[phase];
  first = x.part * per;
  last = min(first + per, blocks);
}

// ---- what a unit waits for.  ready[phase][z][I] counts the epilogue warps (16 a block) that
// have stored their part of block row I of X, A or B, over all steps.  (Nothing else is
// needed: a complete row of B needs all of A, which needs all of X of the step before, so
// that no buffer is written while an earlier phase still reads it, with two A in turn.)
constexpr int kWarpsOfBlock = 2 * kEpilogueWarps;

__device__ __forceinline__ int* ready_at(const OrthoArgs& a, int phase, int z, int I) {
  const int nr = blocks_of(a.r);
  return a.ready + (static_cast<long long>(z) * 3 + phase) * nr + I;
}

__device__ bool wait_ready(const OrthoArgs& a, const int* p, int want, volatile int* abort) {
  for (uint32_t n = 0; n < kReadyLimit; ++n) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= want) return true;
    if ((n & 255u) == 255u &&
        (*abort || *reinterpret_cast<volatile int*>(&a.header->status) == kStatusTimeout))
      return false;
  }
  return false;
}

// Waits until what unit x reads is there.
__device__ bool wait_inputs(const OrthoArgs& a, int phase, int step, const Unit& x, volatile int* abort) {
  const int nr = blocks_of(a.r), nc = blocks_of(a.c);
  if (phase == kGram) {              // X's rows I and J of the step before
    if (step == 0) return true;
    const int want = step * nc * kWarpsOfBlock;
    return wait_ready(a, ready_at(a, kUpdate, x.z, x.I), want, abort) &&
           (x.I == x.J || wait_ready(a, ready_at(a, kUpdate, x.z, x.J), want, abort));
  }
  const int want = (step + 1) * nr * kWarpsOfBlock;
  if (phase == kPoly)
    return wait_ready(a, ready_at(a, kGram, x.z, x.I), want, abort) &&
           (x.I == x.J || wait_ready(a, ready_at(a, kGram, x.z, x.J), want, abort));
  return wait_ready(a, ready_at(a, kPoly, x.z, x.I), want, abort);
}

// The warp has stored its part of unit x.
__device__ __forceinline__ void signal_ready(const OrthoArgs& a, int phase, const Unit& x) {
  ptx::fence_proxy_async();          // tensor copies read it next
  __syncwarp();
  if (threadIdx.x % 32 == 0) {
    ptx::red_release_add(ready_at(a, phase, x.z, x.I), 1);
    if (phase != kUpdate && x.I != x.J) ptx::red_release_add(ready_at(a, phase, x.z, x.J), 1);
  }
}

// Waits for the phase of `bar` with the given parity; false if it gave up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
    if ((i & 63u) == 63u && *abort) return false;
  }
  return false;
}

__device__ void gave_up(const OrthoArgs& a, volatile int* abort) {
  *abort = 1;
  atomicExch(&a.header->status, kStatusTimeout);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// 16 neighbouring fp16 numbers, 32-byte aligned.
struct Half16 {
  uint32_t w[8];
};
__device__ __forceinline__ Half16 load_half16(const __half* p) {
  Half16 h;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(h.w[0]), "=r"(h.w[1]), "=r"(h.w[2]), "=r"(h.w[3]), "=r"(h.w[4]), "=r"(h.w[5]), "=r"(h.w[6]),
                 "=r"(h.w[7])
               : "l"(p)
               : "memory");
  return h;
}
__device__ __forceinline__ void store_half16(__half* p, const float (&v)[kPiece]) {
  uint32_t w[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) w[q] = pack_half(v[2 * q], v[2 * q + 1]);
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A piece of 32 rows x 16 columns turned through shared memory: in, lane l holds row l; out, lane
// l holds rows 8 (l % 4) .. + 7 of columns l / 4 and l / 4 + 8.
__device__ __forceinline__ void turn(float* buf, int lane, const float (&v)[kPiece], float (&t)[2][8]) {
#pragma unroll
  for (int q = 0; q < kPiece; ++q) buf[q * kTurnPitch + lane] = v[q];
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4* p = reinterpret_cast<const float4*>(buf + (lane / 4 + 8 * h) * kTurnPitch + lane % 4 * 8);
    const float4 x = p[0], y = p[1];
    t[h][0] = x.x, t[h][1] = x.y, t[h][2] = x.z, t[h][3] = x.w;
    t[h][4] = y.x, t[h][5] = y.y, t[h][6] = y.z, t[h][7] = y.w;
  }
  __syncwarp();
}
__device__ __forceinline__ void turn_back(float* buf, int lane, const float (&t)[2][8], float (&v)[kPiece]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float4* p = reinterpret_cast<float4*>(buf + (lane / 4 + 8 * h) * kTurnPitch + lane % 4 * 8);
    p[0] = make_float4(t[h][0], t[h][1], t[h][2], t[h][3]);
    p[1] = make_float4(t[h][4], t[h][5], t[h][6], t[h][7]);
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < kPiece; ++q) v[q] = buf[q * kTurnPitch + lane];
  __syncwarp();
}

// The last update's piece, to the caller's matrix: lane = row i, columns j0 .. + 15 of X.
__device__ __forceinline__ void store_out(const OrthoArgs& a, int z, int i, int j0, const float (&v)[kPiece]) {
  const int n = min(a.c - j0, kPiece);
  if (i >= a.r) return;
  __nv_bfloat16* out = a.out + z * a.out_batch;
  const float unscale = 1.0f / a.s;
  if (a.tall) {                      // out is [c, r]: neighbouring lanes, neighbouring elements
    __nv_bfloat16* p = out + j0 * a.out_row + i;
#pragma unroll
    for (int q = 0; q < kPiece; ++q)
      if (q < n) p[q * a.out_row] = __float2bfloat16_rn(v[q] * unscale);
    return;
  }
  __nv_bfloat16* p = out + i * a.out_row + j0;
  if (n == kPiece && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    uint32_t w[kPiece / 2];
#pragma unroll
    for (int q = 0; q < kPiece / 2; ++q) w[q] = pack_bf16(v[2 * q] * unscale, v[2 * q + 1] * unscale);
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int q = 0; q < kPiece; ++q)
      if (q < n) p[q] = __float2bfloat16_rn(v[q] * unscale);
  }
}

// The warp has read its part of the accumulator.
__device__ __forceinline__ void release_acc(uint32_t acc_empty) {
  ptx::tmem_fence_before();
  __syncwarp();
  if (threadIdx.x % 32 == 0) ptx::mbar_arrive_cluster(acc_empty);
}

// What an epilogue warp keeps through the kernel.
struct EpilogueWarp {
  float* buf;                        // its turning buffer
  volatile int* abort;
  int rank, index;                   // its CTA of the pair, and which of the CTA's epilogue warps it is
};

__device__ __forceinline__ uint4 load_v4(const __half* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// wait_inputs for a warp that reads them itself.
__device__ __forceinline__ bool warp_ready(const OrthoArgs& a, int phase, int step, const Unit& x,
                                           volatile int* abort) {
  const bool ok = threadIdx.x % 32 != 0 || wait_inputs(a, phase, step, x, abort);
  return __all_sync(kAll, ok);
}

// One warp's part of a finished block of an update: 32 rows from i0, kWarpCols columns from j.  The
// products are turned, so that X's two parts are read and written 16 bytes a lane; they are
// read a piece ahead, the first before the products are done.
__device__ __forceinline__ bool epilogue_update(const OrthoArgs& a, int step, const Unit& x, int i0, int j,
                                                uint32_t from, uint64_t* acc_full, uint32_t parity,
                                                uint32_t acc_empty, const EpilogueWarp& w) {
  const int lane = threadIdx.x % 32;
  const int pieces = i0 < a.r ? min(max((a.c - j + kPiece - 1) / kPiece, 0), kPieces) : 0;
  const bool last = step == a.steps - 1;
  const int ld = a.ld;
  const int i = i0 + lane % 4 * 8;                    // this lane's rows i .. i + 7 (inside ld) ...
  // ... and columns: piece u, h: jl + kPiece u + 8 h
  const int jl = j + lane / 4, cols = i < a.r ? a.c - jl : 0;
  const long long base = (static_cast<long long>(x.z) * a.c + jl) * ld + i;
  const __half* hi_in = a.xt[step & 1] + base;
  __half* hi_out = a.xt[(step & 1) ^ 1] + base;
  __half* lo = a.xl + base;
  uint4 hi[2] = {}, rest[2] = {};
  auto load = [&](int u) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (u * kPiece + 8 * h < cols) {
        hi[h] = load_v4(hi_in + (u * kPiece + 8 * h) * static_cast<long long>(ld));
        rest[h] = load_v4(lo + (u * kPiece + 8 * h) * static_cast<long long>(ld));
      }
  };
  if (!warp_ready(a, kUpdate, step, x, w.abort)) return false;
  load(0);
  float own[8];                                       // a + what is left of B_ii
#pragma unroll
  for (int q = 0; q < 8; ++q) own[q] = i + q < a.r ? a.ca + a.diag_b[x.z * static_cast<long long>(ld) + i + q] : 0.0f;
  if (!__all_sync(kAll, wait_bar(acc_full, parity, w.abort))) return false;
  ptx::tmem_fence_after();
  uint32_t acc[kPiece];
  if (pieces > 0) ptx::tmem_load16(acc, from);
  else release_acc(acc_empty);
#pragma unroll 1
  for (int u = 0; u < pieces; ++u) {
    ptx::tmem_wait_load();
    float v[kPiece], t[2][8];
#pragma unroll
    for (int q = 0; q < kPiece; ++q) v[q] = __uint_as_float(acc[q]);
    turn(w.buf, lane, v, t);
    if (u + 1 < pieces) ptx::tmem_load16(acc, from + (u + 1) * kPiece);
    else release_acc(acc_empty);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t hw[4] = {hi[h].x, hi[h].y, hi[h].z, hi[h].w};
      const uint32_t lw[4] = {rest[h].x, rest[h].y, rest[h].z, rest[h].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 b = unpack_half(hw[q]), r = unpack_half(lw[q]);
        t[h][2 * q] = fmaf(own[2 * q], b.x + r.x, t[h][2 * q]);
        t[h][2 * q + 1] = fmaf(own[2 * q + 1], b.y + r.y, t[h][2 * q + 1]);
      }
    }
    if (u + 1 < pieces) load(u + 1);
    if (last) {
      turn_back(w.buf, lane, t, v);
      store_out(a, x.z, i0 + lane, j + u * kPiece, v);
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t hw[4], lw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        hw[q] = pack_half(t[h][2 * q], t[h][2 * q + 1]);
        const float2 b = unpack_half(hw[q]);
        lw[q] = pack_half(t[h][2 * q] - b.x, t[h][2 * q + 1] - b.y);
      }
      if (u * kPiece + 8 * h < cols) {
        const long long at = (u * kPiece + 8 * h) * static_cast<long long>(ld);
        *reinterpret_cast<uint4*>(hi_out + at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(lo + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
    }
  }
  if (!last) signal_ready(a, kUpdate, x);
  return true;
}

// The same for A = X X^T or B = b A + c A^2: 32 rows from i0, kWarpCols columns from j of a block on
// or below the diagonal, and its mirror.
//
// Where the inner dimension is split, each part's warp stores its sums, and the one that comes
// last adds the parts up in their order (so the result does not depend on which that is).
template <int kPhase>
__device__ __forceinline__ bool epilogue_square(const OrthoArgs& a, int step, const Unit& x, int i0, int j,
                                                uint32_t from, uint64_t* acc_full, uint32_t parity,
                                                uint32_t acc_empty, const EpilogueWarp& w) {
  const int lane = threadIdx.x % 32;
  const int i = i0 + lane;
  const int pieces = i0 < a.r ? min(max((a.r - j + kPiece - 1) / kPiece, 0), kPieces) : 0;
  const int ld = a.ld;
  const long long matrix = static_cast<long long>(x.z) * a.r * ld;
  const bool row = i < a.r;
  const __half* o_row = a.a[step & 1] + matrix + static_cast<long long>(i) * ld + j;    // A_ij = A_ji, along the row
  Half16 o = {};
  float rest_a = 0.0f;               // what rounding left of A_ii
  if (kPhase == kPoly) {
    if (!warp_ready(a, kPoly, step, x, w.abort)) return false;
    if (row && pieces > 0) {
      o = load_half16(o_row);
      rest_a = a.diag_a[step & 1][x.z * static_cast<long long>(ld) + i];
    }
  }
  if (!__all_sync(kAll, wait_bar(acc_full, parity, w.abort))) return false;
  ptx::tmem_fence_after();
  const int parts = a.split[kPhase];
  const float* sums = nullptr;       // the first part's
  constexpr int kPartStride = kBlock * kBlock;
  if (parts > 1) {
    const int nr = blocks_of(a.r), blocks = nr * (nr + 1) / 2;
    const long long block = static_cast<long long>(x.z) * blocks + x.I * (x.I + 1) / 2 + x.J;
    const int place = w.rank * kEpilogueWarps + w.index;
    float* first = a.partial + block * parts * kPartStride + place * (32 * kWarpCols) + lane;
    float* mine = first + static_cast<long long>(x.part) * kPartStride;
#pragma unroll 1
    for (int u = 0; u < pieces; ++u) {
      uint32_t acc[kPiece];
      ptx::tmem_load16(acc, from + u * kPiece);
      ptx::tmem_wait_load();
#pragma unroll
      for (int q = 0; q < kPiece; ++q) mine[(u * kPiece + q) * 32] = __uint_as_float(acc[q]);
    }
    release_acc(acc_empty);
    int before = 0;
    if (lane == 0)
      before = ptx::add_acq_rel(a.arrived + ((static_cast<long long>(x.z) * 2 + kPhase) * blocks +
                                             (block - static_cast<long long>(x.z) * blocks)) * kWarpsOfBlock + place, 1);
    before = __shfl_sync(kAll, before, 0);
    if (before % parts != parts - 1) return true;      // not the last part
    sums = first;
  }
  const float f = kPhase == kGram ? 1.0f / (a.s * a.s) : a.cc;
  __half* m = (kPhase == kGram ? a.a[step & 1] : a.b) + matrix;
  __half* m_row = m + static_cast<long long>(i) * ld + j;
  const int ti = i0 + lane % 4 * 8;                   // after the turn: rows ti .. ti + 7 of ...
  const int cols = ti < a.r ? a.r - j - lane / 4 : 0; // ... columns j + lane / 4 + kPiece u + 8 h
  __half* m_col = m + static_cast<long long>(j + lane / 4) * ld + ti;
  uint32_t acc[kPiece];
  if (parts == 1) {
    if (pieces > 0) ptx::tmem_load16(acc, from);
    else release_acc(acc_empty);
  }
#pragma unroll 1
  for (int u = 0; u < pieces; ++u) {
    const int j0 = j + u * kPiece;
    float v[kPiece];
    if (parts == 1) {
      ptx::tmem_wait_load();
#pragma unroll
      for (int q = 0; q < kPiece; ++q) v[q] = __uint_as_float(acc[q]) * f;
      if (u + 1 < pieces) ptx::tmem_load16(acc, from + (u + 1) * kPiece);
      else release_acc(acc_empty);
    } else {
      const float* p = sums + u * kPiece * 32;
#pragma unroll
      for (int q = 0; q < kPiece; ++q) v[q] = p[q * 32];
#pragma unroll 1
      for (int k = 1; k < parts; ++k) {
        p += kPartStride;
#pragma unroll
        for (int q = 0; q < kPiece; ++q) v[q] += p[q * 32];
      }
#pragma unroll
      for (int q = 0; q < kPiece; ++q) v[q] *= f;
    }
    if constexpr (kPhase == kPoly) {
#pragma unroll
      for (int q = 0; q < kPiece / 2; ++q) {
        const float2 p = unpack_half(o.w[q]);
        v[2 * q] = fmaf(a.cb, p.x, v[2 * q]);
        v[2 * q + 1] = fmaf(a.cb, p.y, v[2 * q + 1]);
      }
    }
    if (j0 < i0 + 32 && i0 < j0 + kPiece) {           // the diagonal passes through the piece
      float left = 0.0f;
#pragma unroll
      for (int q = 0; q < kPiece; ++q) {
        if (j0 + q != i) continue;
        if constexpr (kPhase == kPoly) {              // rest_a to first order
          const float2 p = unpack_half(o.w[q / 2]);
          v[q] = fmaf(rest_a, fmaf(2.0f * a.cc, q % 2 ? p.y : p.x, a.cb), v[q]);
        }
        left = v[q] - __half2float(__float2half_rn(v[q]));
      }
      if (i >= j0 && i < j0 + kPiece && row)
        (kPhase == kGram ? a.diag_a[step & 1] : a.diag_b)[x.z * static_cast<long long>(ld) + i] = left;
    }
    if (kPhase == kPoly && row && u + 1 < pieces) o = load_half16(o_row + (u + 1) * kPiece);
    if (x.I != x.J && row) store_half16(m_row + u * kPiece, v);
    float t[2][8];
    turn(w.buf, lane, v, t);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (u * kPiece + 8 * h < cols)
        *reinterpret_cast<uint4*>(m_col + (u * kPiece + 8 * h) * static_cast<long long>(ld)) =
            make_uint4(pack_half(t[h][0], t[h][1]), pack_half(t[h][2], t[h][3]), pack_half(t[h][4], t[h][5]),
                       pack_half(t[h][6], t[h][7]));
    }
  }
  signal_ready(a, kPhase, x);
  return true;
}

// All phases of all steps, one cooperative launch of CTA pairs.  The units of all phases in
// order go round the pairs; a unit waits for the block rows that it reads, which units before
// it in the order store, so the earliest unfinished unit never waits and the phases (and
// the matrices of a batch) overlap without a barrier over the grid.  Per CTA: warp 0 copies
// operands (TMA), warp 1 of the pair's first CTA issues the products, the epilogue warps take
// finished accumulators (two in tensor memory, so that the products of the next unit run
// meanwhile).
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    ortho_steps_kernel(const __grid_constant__ OrthoMaps maps, const OrthoArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ GemmSmem sm;
  const uint32_t stages = (ptx::smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = ptx::cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&sm.full[i], 1);
      ptx::mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.acc_full[i], 1);
      ptx::mbar_init(&sm.acc_empty[i], 2 * kEpilogueWarps);
    }
    ptx::mbar_init(&sm.drained, 1);
    sm.abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensor_map(&maps.xt[0]);
    ptx::prefetch_tensor_map(&maps.xt[1]);
    ptx::prefetch_tensor_map(&maps.a[0]);
    ptx::prefetch_tensor_map(&maps.a[1]);
    ptx::prefetch_tensor_map(&maps.b);
  }
  if (warp == 1) ptx::tmem_alloc_pair(&sm.tmem);
  ptx::tmem_fence_before();
  __syncthreads();
  ptx::cluster_sync_all();
  ptx::tmem_fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int* abort = &sm.abort;

  uint32_t stage = 0, stage_phase = 0;      // producer's or issuer's place in the ring
  uint32_t acc = 0, acc_phase = 0;          // issuer's or epilogue's accumulator
  auto next_stage = [&] {
    if (++stage == kStages) {
      stage = 0;
      stage_phase ^= 1u;
    }
  };
  auto next_acc = [&] {
    if (++acc == 2) {
      acc = 0;
      acc_phase ^= 1u;
    }
  };
  // body(phase, step, unit) for this pair's units in order, until one gives up
  auto for_units = [&](auto&& body) {
    int offset = 0;                  // units of the phases so far, modulo the pairs
    for (int p = 0; p < 3 * a.steps; ++p) {
      const int phase = p % 3, step = p / 3;
      const int units = units_of(a, phase);
      for (int t = pair >= offset ? pair - offset : pair - offset + pairs; t < units; t += pairs) {
        if (*abort) return;
        if (!body(phase, step, unit_at(a, phase, t))) {
          gave_up(a, abort);
          return;
        }
      }
      offset = (offset + units) % pairs;
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      for_units([&](int phase, int step, const Unit& x) {
        const int cur = step & 1;
        const CUtensorMap* ma = phase == kGram ? &maps.xt[cur] : phase == kPoly ? &maps.a[cur] : &maps.b;
        const CUtensorMap* mb = phase == kPoly ? &maps.a[cur] : &maps.xt[cur];
        const int ra = x.I * kBlock + rank * 128, rb = x.J * kBlock + rank * 128;
        int k0, k1;
        inner_of(a, phase, x, k0, k1);
        if (!wait_inputs(a, phase, step, x, abort)) return false;
        ptx::fence_proxy_async();    // the acquires above before the tensor copies
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait_bar(&sm.empty[stage], stage_phase ^ 1u, abort)) return false;
          if (rank == 0) ptx::mbar_arrive_expect_tx(&sm.full[stage], 2 * kStageBytes);
          const uint32_t bar = ptx::map_to_rank(ptx::smem_u32(&sm.full[stage]), 0);
          const uint32_t dst = stages + stage * kStageBytes;
          const int k = kb * kStepK;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int da = ra + 64 * h, db = rb + 64 * h;
            ptx::tma_load_3d_pair(dst + h * kBoxBytes, ma, phase == kGram ? da : k, phase == kGram ? k : da, x.z, bar);
            ptx::tma_load_3d_pair(dst + kOperandBytes + h * kBoxBytes, mb, phase == kGram ? db : k,
                                  phase == kGram ? k : db, x.z, bar);
          }
          next_stage();
        }
        return true;
      });
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    if (lane == 0) {
      for_units([&](int phase, int, const Unit& x) {
        // fp32 accumulator, fp16 operands, 256 x 256; X X^T has both operands MN-major
        const uint32_t idesc = 1u << 4 | (kBlock >> 3) << 17 | (kBlock >> 4) << 24 | (phase == kGram ? 3u << 15 : 0u);
        // K-major: 8-row groups 1024 bytes apart, 16 inner elements = 32 bytes.  MN-major:
        // groups of 64 rows a box apart, groups of 8 inner elements 1024 bytes apart.
        const uint32_t lead = phase == kGram ? kBoxBytes : 16;
        const uint32_t k_bytes = phase == kGram ? 2048 : 32;
        int k0, k1;
        inner_of(a, phase, x, k0, k1);
        if (!wait_bar(&sm.acc_empty[acc], acc_phase ^ 1u, abort)) return false;
        ptx::tmem_fence_after();
        const uint32_t d = tmem + acc * kBlock;
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait_bar(&sm.full[stage], stage_phase, abort)) return false;
          ptx::tmem_fence_after();
          const uint32_t at = stages + stage * kStageBytes;
#pragma unroll
          for (int k = 0; k < kStepK / 16; ++k)
            ptx::mma_f16_pair(d, operand_desc(at + k * k_bytes, lead, 1024),
                              operand_desc(at + kOperandBytes + k * k_bytes, lead, 1024), idesc, kb > k0 || k > 0);
          ptx::mma_commit_pair(&sm.empty[stage]);
          next_stage();
        }
        ptx::mma_commit_pair(&sm.acc_full[acc]);
        next_acc();
        return true;
      });
    }
    __syncwarp();
  } else if (warp >= kFirstEpilogueWarp) {
    const int quarter = warp % 4, part = (warp - kFirstEpilogueWarp) / 4;
    const EpilogueWarp ew{reinterpret_cast<float*>(raw + (stages - ptx::smem_u32(raw)) + kStages * kStageBytes) +
                              (warp - kFirstEpilogueWarp) * kTurnFloats,
                          abort, static_cast<int>(rank), warp - kFirstEpilogueWarp};
    for_units([&](int phase, int step, const Unit& x) {
      const uint32_t from = tmem + acc * kBlock + part * kWarpCols + (static_cast<uint32_t>(quarter) << 21);
      const int i0 = x.I * kBlock + rank * 128 + quarter * 32;
      const int j = x.J * kBlock + part * kWarpCols;
      uint64_t* full = &sm.acc_full[acc];
      const uint32_t empty = ptx::map_to_rank(ptx::smem_u32(&sm.acc_empty[acc]), 0);
      const bool ok = phase == kGram ? epilogue_square<kGram>(a, step, x, i0, j, from, full, acc_phase, empty, ew)
                      : phase == kPoly ? epilogue_square<kPoly>(a, step, x, i0, j, from, full, acc_phase, empty, ew)
                                       : epilogue_update(a, step, x, i0, j, from, full, acc_phase, empty, ew);
      next_acc();
      return ok;
    });
  }

  // ---- end: nothing of the pair may be in flight when it leaves
  if (__syncthreads_or(*abort)) {
    if (warp == 1 && rank == 0 && lane == 0) {
      ptx::mma_commit_pair(&sm.drained);
      for (uint32_t n = 0; n < kWaitLimit && !ptx::mbar_try_wait_cluster(&sm.drained, 0); ++n) {}
    }
    // copies already issued land within microseconds; which of them a barrier of the pair
    // still counts is not known after a give-up, so they get a millisecond
    if (warp == 0)
      for (int n = 0; n < 1000; ++n) __nanosleep(1000);
  }
  ptx::tmem_fence_before();
  __syncthreads();
  ptx::cluster_sync_all();
  if (warp == 1) ptx::tmem_dealloc_pair(tmem);
}

// ---------------------------------------------------------------- host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;
int g_pairs[64] = {};                // per device: pairs resident at once

// [batch][outer][ld] fp16 with r columns used, in swizzled boxes of 64 x 64.
cudaError_t encode(CUtensorMap* map, void* p, const OrthoShape& sh, int64_t outer) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(sh.r), static_cast<cuuint64_t>(outer),
                              static_cast<cuuint64_t>(sh.batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(sh.ld * 2), static_cast<cuuint64_t>(sh.ld * outer * 2)};
  const cuuint32_t box[3] = {64, 64, 1}, step[3] = {1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

float power_of_two_below(double x) { return static_cast<float>(std::exp2(std::floor(std::log2(x)))); }

}  // namespace

// Called once per device, under the library's lock.
cudaError_t prepare_orthogonalize() {
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeTiled>(fn);
  }
  cudaError_t e = cudaFuncSetAttribute(ortho_steps_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kGemmSmem));
  if (e != cudaSuccess) return e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(&g_pairs[dev], ortho_steps_kernel, &cfg);
}

cudaError_t launch_orthogonalize(const OrthoCall& q, cudaStream_t stream) {
  const OrthoShape& sh = q.shape;
  const OrthoLayout L = make_ortho_layout(sh);
  char* ws = static_cast<char*>(q.workspace);
  const double s = std::fmin(std::sqrt(static_cast<double>(sh.r) * sh.c), 32768.0);

  OrthoIn in{};
  in.grad = q.grad;
  in.bf16 = q.grad_bf16;
  in.tall = sh.tall;
  in.batch_stride = q.grad_batch_stride;
  in.row_stride = q.grad_row_stride;
  in.rows = static_cast<int>(sh.rows);
  in.cols = static_cast<int>(sh.cols);
  in.ld = static_cast<int>(sh.ld);
  in.x_batch = sh.c * sh.ld;
  in.s = power_of_two_below(s);
  in.norm = reinterpret_cast<double*>(ws + L.norm);
  in.norm_blocks = sh.norm_blocks;
  in.xt = reinterpret_cast<__half*>(ws + L.xt[0]);
  in.xl = reinterpret_cast<__half*>(ws + L.xl);
  in.header = reinterpret_cast<Header*>(ws + L.header);
  const int64_t nr = sh.blocks_r, nc = sh.blocks_c;
  in.counters = reinterpret_cast<int*>(ws + L.counters);
  in.num_counters = static_cast<int>(sh.counters());

  OrthoMaps maps;
  cudaError_t e = cudaSuccess;
  auto add = [&](CUtensorMap* map, size_t at, int64_t outer) {
    if (e == cudaSuccess) e = encode(map, ws + at, sh, outer);
  };
  add(&maps.xt[0], L.xt[0], sh.c);
  add(&maps.xt[1], L.xt[1], sh.c);
  add(&maps.a[0], L.a[0], sh.r);
  add(&maps.a[1], L.a[1], sh.r);
  add(&maps.b, L.b, sh.r);
  if (e != cudaSuccess) return e;

  OrthoArgs a{};
  a.batch = static_cast<int>(sh.batch);
  a.r = static_cast<int>(sh.r);
  a.c = static_cast<int>(sh.c);
  a.ld = static_cast<int>(sh.ld);
  a.steps = q.steps;
  a.ca = q.a;
  a.cb = q.b;
  a.cc = q.c;
  a.s = in.s;
  a.xt[0] = in.xt;
  a.xt[1] = reinterpret_cast<__half*>(ws + L.xt[1]);
  a.xl = in.xl;
  a.b = reinterpret_cast<__half*>(ws + L.b);
  for (int i = 0; i < 2; ++i) {
    a.a[i] = reinterpret_cast<__half*>(ws + L.a[i]);
    a.diag_a[i] = reinterpret_cast<float*>(ws + L.diag_a[i]);
  }
  a.diag_b = reinterpret_cast<float*>(ws + L.diag_b);
  a.out = static_cast<__nv_bfloat16*>(q.out);
  a.out_batch = q.out_batch_stride;
  a.out_row = q.out_row_stride;
  a.tall = sh.tall;
  a.header = in.header;
  a.ready = in.counters;
  a.arrived = in.counters + sh.batch * 3 * nr;
  a.partial = reinterpret_cast<float*>(ws + L.partial);
  a.split[kGram] = sh.split_gram;
  a.split[kPoly] = sh.split_poly;

  const unsigned batch = static_cast<unsigned>(sh.batch);
  ortho_norm_kernel<<<dim3(sh.norm_blocks, batch), 256, 0, stream>>>(in);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  ortho_scale_kernel<<<dim3((in.cols + 63) / 64, (in.rows + 63) / 64, batch), 256, 0, stream>>>(in);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  const int64_t most = sh.batch * std::max(nr * nc, nr * (nr + 1) / 2 * std::max(sh.split_gram, sh.split_poly));
  const int pairs = static_cast<int>(std::min<int64_t>(most, g_pairs[dev]));
  if (pairs < 1) return cudaErrorLaunchOutOfResources;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ortho_steps_kernel, maps, a);
}

}  // namespace ewg
