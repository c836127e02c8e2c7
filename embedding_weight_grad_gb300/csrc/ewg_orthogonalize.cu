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
//   * The diagonals of A and B, their largest entries, are kept apart in fp32 and the fp16
//     matrices have zeros there: with A = D + O, A^2 = O O + D O + O D + D^2, and
//     B X = offdiag(B) X + diag(B) X with the 22-bit X.
//   * Everything stored in fp16 is scaled by powers of two or by the norm: X by
//     s ~ sqrt(r c), so its entries are about 1 at first and at most 1.2 s, and A, B by
//     rho ~ r / 16.
//
// Layout.  Every buffer is [., ld] fp16 with the r index inside: X^T (two, alternating), the
// rest of X^T, A and B.  The accumulator of a product has its row index across the lanes of a
// warp, so all stores of X^T and of the mirrored blocks are contiguous.  As an operand of X
// X^T, X^T has the product's rows inside (MN-major); for B X it has the inner index inside
// (K-major), as A and B have by symmetry.
#include <cfloat>
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
  int* barrier;
};

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half(w & 0xffffu)); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half(w >> 16)); }

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
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    a.header->status = kStatusOk;
    *a.barrier = 0;
  }
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
      lo[q] = pack_half(v[0] - half_lo(hi[q]), v[1] - half_hi(hi[q]));
    }
    const long long at = blockIdx.z * a.x_batch + static_cast<long long>(outer0 + k) * a.ld + inner0 + x;
    *reinterpret_cast<uint4*>(a.xt + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(a.xl + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ---------------------------------------------------------------- the products

constexpr int kBlock = 256;          // a pair of CTAs computes 256 x 256; each CTA 128 rows
constexpr int kStepK = 64;           // inner elements of a stage: one 128-byte swizzled row
constexpr int kStages = 5;
constexpr int kOperandBytes = 128 * kStepK * 2;       // one CTA's half of an operand's stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kBoxBytes = 64 * kStepK * 2;            // one tensor copy: 64 rows of 128 bytes
constexpr int kEpilogueWarps = 8;
constexpr int kGemmThreads = 128 + 32 * kEpilogueWarps;
// Epilogue staging of one warp: a ring of buffers for pieces of 32 rows x kPiece columns, two
// fp16 numbers an element.  A piece's results replace its inputs.
constexpr int kPiece = 16;
constexpr int kPieces = 128 / kPiece;                 // of a warp's 128 columns
constexpr int kHalfBytes = 32 * kPiece * 2;
constexpr int kPieceBytes = 2 * kHalfBytes;
constexpr int kRing = 4;
constexpr int kWarpStaging = kRing * kPieceBytes;
constexpr size_t kGemmSmem = static_cast<size_t>(kStages) * kStageBytes + kEpilogueWarps * kWarpStaging + 1024;
static_assert(kGemmSmem + 512 <= 227 * 1024, "stages and staging fit in shared memory");
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr uint32_t kGridWaitLimit = 1u << 22;

enum Phase { kGram = 0, kPoly = 1, kUpdate = 2 };

struct OrthoMaps {
  CUtensorMap xt[2], a, b;                            // operands: boxes of 64 x 64, swizzled
  CUtensorMap xt_piece[2], xl_piece, a_piece, b_piece;  // pieces: 32 of the r index, kPiece of the other
  CUtensorMap a_mirror, b_mirror;                     // mirrored pieces: kPiece, 32
};

struct OrthoArgs {
  int batch, r, c, ld;
  int steps;
  float ca, cb, cc;                  // the polynomial's coefficients
  float s, rho;                      // stored X = s X, stored A, B = rho A, rho B
  float* diag_a;                     // [batch][ld], unscaled
  float* diag_b;
  __nv_bfloat16* out;
  long long out_batch, out_row;
  int tall;
  Header* header;
  int* barrier;
};

struct GemmSmem {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
  uint64_t piece[kEpilogueWarps][kRing];
  uint32_t tmem;
  int abort;
};

// Shared-memory operand descriptor: 128-byte swizzle; `lead` and `stride` in bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

__device__ __forceinline__ int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// Block `t` of a phase: matrix, block row I, block column J.  A and B: on and below the diagonal.
struct Tile {
  int z, I, J;
};

__device__ __forceinline__ int tiles_of(const OrthoArgs& a, int phase) {
  const int nr = blocks_of(a.r);
  return a.batch * (phase == kUpdate ? nr * blocks_of(a.c) : nr * (nr + 1) / 2);
}

__device__ __forceinline__ Tile tile_at(const OrthoArgs& a, int phase, int t) {
  const int nr = blocks_of(a.r);
  Tile x;
  if (phase == kUpdate) {
    const int per = nr * blocks_of(a.c);
    x.z = t / per;
    t -= x.z * per;
    x.J = t / nr;
    x.I = t - x.J * nr;
  } else {
    const int per = nr * (nr + 1) / 2;
    x.z = t / per;
    t -= x.z * per;
    x.I = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while ((x.I + 1) * (x.I + 2) / 2 <= t) ++x.I;
    while (x.I * (x.I + 1) / 2 > t) --x.I;
    x.J = t - x.I * (x.I + 1) / 2;
  }
  return x;
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

// Where a warp of the epilogue is: its staging ring and the pieces taken so far.
struct EpilogueState {
  uint32_t staging;                  // shared-memory address
  uint64_t* bars;                    // one for each buffer: its inputs have come
  uint32_t taken;                    // pieces taken; piece n uses buffer n % kRing
  uint32_t parity;                   // bit b: parity of the next wait on buffer b
};

__device__ __forceinline__ float lds_half(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ void sts_half(uint32_t at, __half v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(__half_as_ushort(v)) : "memory");
}
__device__ __forceinline__ void sts_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// One lane requests the inputs of the warp's piece number n, at row i0 and column j0: X's two
// parts for an update, O for B.
template <int kPhase>
__device__ __forceinline__ void request_piece(const OrthoMaps& maps, const EpilogueState& st, uint32_t n, int cur,
                                              int z, int i0, int j0) {
  const uint32_t b = n % kRing, to = st.staging + b * kPieceBytes;
  ptx::mbar_arrive_expect_tx(&st.bars[b], kPhase == kUpdate ? kPieceBytes : kHalfBytes);
  if constexpr (kPhase == kUpdate) {
    ptx::tma_load_3d(to, &maps.xt_piece[cur], i0, j0, z, &st.bars[b]);
    ptx::tma_load_3d(to + kHalfBytes, &maps.xl_piece, i0, j0, z, &st.bars[b]);
  } else {
    ptx::tma_load_3d(to, &maps.a_piece, i0, j0, z, &st.bars[b]);
  }
}

// The last update's piece, to the caller's matrix.
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

// One warp's part of a finished block: 32 rows from i0, 128 columns from j, in pieces of kPiece
// columns.  A piece's inputs come and its results go by tensor copies through shared memory,
// which also clip what leaves the matrix; the next two pieces' inputs are under way while
// one is computed, and the first two's before the products are done.
template <int kPhase>
__device__ __forceinline__ bool epilogue(const OrthoMaps& maps, const OrthoArgs& a, int step, const Tile& x, int i0,
                                         int j, uint32_t from, uint64_t* acc_full, uint32_t parity,
                                         volatile int* abort, EpilogueState& st) {
  const int lane = threadIdx.x % 32;
  const int i = i0 + lane;
  const int cols = kPhase == kUpdate ? a.c : a.r;
  const int pieces = i0 < a.r ? min(max((cols - j + kPiece - 1) / kPiece, 0), kPieces) : 0;
  const long long ld = a.ld;
  const int cur = step & 1;
  const bool last = kPhase == kUpdate && step == a.steps - 1;
  if (kPhase != kGram && lane == 0) {
    for (int u = 0; u < 2 && u < pieces; ++u)
      request_piece<kPhase>(maps, st, st.taken + u, cur, x.z, i0, j + u * kPiece);
  }
  float own = 0.0f, dj4[4] = {};
  if (kPhase == kUpdate && i < a.r) own = a.ca + a.diag_b[x.z * ld + i];
  if (kPhase == kPoly) {
    if (i < a.r) own = a.diag_a[x.z * ld + i];
#pragma unroll
    for (int q = 0; q < 4; ++q) dj4[q] = j + 32 * q + lane < a.r ? a.diag_a[x.z * ld + j + 32 * q + lane] : 0.0f;
  }
  if (!__all_sync(kAll, wait_bar(acc_full, parity, abort))) return false;
  ptx::tmem_fence_after();
  const float f = kPhase == kUpdate ? 1.0f / a.rho : kPhase == kGram ? a.rho / (a.s * a.s) : a.cc / a.rho;
#pragma unroll 1
  for (int u = 0; u < pieces; ++u) {
    const int j0 = j + u * kPiece;
    const uint32_t b = st.taken % kRing;
    const uint32_t buf = st.staging + b * kPieceBytes, at = buf + lane * 2;
    uint32_t acc[kPiece];
    float v[kPiece];
    ptx::tmem_load16(acc, from + u * kPiece);
    if (kPhase != kGram) {
      if (!__all_sync(kAll, wait_bar(&st.bars[b], (st.parity >> b) & 1u, abort))) return false;
      st.parity ^= 1u << b;
    }
    if constexpr (kPhase == kUpdate) {
#pragma unroll
      for (int q = 0; q < kPiece; ++q) v[q] = lds_half(at + q * 64) + lds_half(at + kHalfBytes + q * 64);
      ptx::tmem_wait_load();
#pragma unroll
      for (int q = 0; q < kPiece; ++q) v[q] = fmaf(own, v[q], __uint_as_float(acc[q]) * f);
    } else {
      const float dj_lane = u < 4 ? (u < 2 ? dj4[0] : dj4[1]) : (u < 6 ? dj4[2] : dj4[3]);
      if constexpr (kPhase == kPoly) {
#pragma unroll
        for (int q = 0; q < kPiece; ++q) v[q] = lds_half(at + q * 64);
      }
      ptx::tmem_wait_load();
      float diag = 0.0f;             // the product on the diagonal
#pragma unroll
      for (int q = 0; q < kPiece; ++q) {
        const float p = __uint_as_float(acc[q]);
        const bool on = j0 + q == i;
        if (on) diag = p;
        if constexpr (kPhase == kGram) {
          v[q] = p * f;
        } else {
          const float dj = __shfl_sync(kAll, dj_lane, (u & 1) * kPiece + q);
          v[q] = fmaf(f, p, v[q] * fmaf(a.cc, own + dj, a.cb));
        }
        if (on) v[q] = 0.0f;
      }
      if (i >= j0 && i < j0 + kPiece && i < a.r) {
        if constexpr (kPhase == kGram) a.diag_a[x.z * ld + i] = diag / (a.s * a.s);
        else a.diag_b[x.z * ld + i] = fmaf(a.cb, own, a.cc * fmaf(own, own, diag / (a.rho * a.rho)));
      }
    }
    if (last) {
      store_out(a, x.z, i, j0, v);
    } else {
#pragma unroll
      for (int q = 0; q < kPiece; ++q) {
        const __half hi = __float2half_rn(v[q]);
        sts_half(at + q * 64, hi);
        if constexpr (kPhase == kUpdate) sts_half(at + kHalfBytes + q * 64, __float2half_rn(v[q] - __half2float(hi)));
      }
      if (kPhase != kUpdate && x.I != x.J) {          // mirrored, [row][column]
        uint32_t w[kPiece / 2];
#pragma unroll
        for (int q = 0; q < kPiece / 2; ++q) w[q] = pack_half(v[2 * q], v[2 * q + 1]);
        const uint32_t m = buf + kHalfBytes + lane * kPiece * 2;
        sts_v4(m, w[0], w[1], w[2], w[3]);
        sts_v4(m + 16, w[4], w[5], w[6], w[7]);
      }
      ptx::fence_proxy_async_shared();
    }
    __syncwarp();
    if (lane == 0) {
      if (!last) {
        if constexpr (kPhase == kUpdate) {
          ptx::tma_store_3d(&maps.xt_piece[cur ^ 1], i0, j0, x.z, buf);
          ptx::tma_store_3d(&maps.xl_piece, i0, j0, x.z, buf + kHalfBytes);
        } else {
          ptx::tma_store_3d(kPhase == kGram ? &maps.a_piece : &maps.b_piece, i0, j0, x.z, buf);
          if (x.I != x.J)
            ptx::tma_store_3d(kPhase == kGram ? &maps.a_mirror : &maps.b_mirror, j0, i0, x.z, buf + kHalfBytes);
        }
        ptx::bulk_commit();
        ptx::bulk_wait_read<kRing - 2>();   // the buffer of the piece after the next is free
      }
      if (kPhase != kGram && u + 2 < pieces)
        request_piece<kPhase>(maps, st, st.taken + 2, cur, x.z, i0, j0 + 2 * kPiece);
    }
    __syncwarp();
    ++st.taken;
  }
  return true;
}

// All phases of all steps, one cooperative launch of CTA pairs: a pair takes blocks of 256 x
// 256, and a barrier over the grid ends each phase.  Per CTA: warp 0 copies operands (TMA),
// warp 1 of the pair's first CTA issues the products, warps 4-11 take finished
// accumulators (two in tensor memory, so that the products of the next block run meanwhile).
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
    for (int i = 0; i < kRing * kEpilogueWarps; ++i) ptx::mbar_init(&sm.piece[0][0] + i, 1);
    sm.abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensor_map(&maps.xt[0]);
    ptx::prefetch_tensor_map(&maps.xt[1]);
    ptx::prefetch_tensor_map(&maps.a);
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
  EpilogueState st{};
  if (warp >= 4) {
    st.staging = stages + kStages * kStageBytes + (warp - 4) * kWarpStaging;
    st.bars = sm.piece[warp - 4];
  }

  for (int p = 0; p < 3 * a.steps; ++p) {
    const int phase = p % 3, step = p / 3, cur = step & 1;
    const int tiles = tiles_of(a, phase);
    const int blocks_k = ((phase == kGram ? a.c : a.r) + kStepK - 1) / kStepK;
    if (warp == 0) {
      if (lane == 0) {
        const CUtensorMap* ma = phase == kGram ? &maps.xt[cur] : phase == kPoly ? &maps.a : &maps.b;
        const CUtensorMap* mb = phase == kPoly ? &maps.a : &maps.xt[cur];
        for (int t = pair; t < tiles && !*abort; t += pairs) {
          const Tile x = tile_at(a, phase, t);
          const int ra = x.I * kBlock + rank * 128, rb = x.J * kBlock + rank * 128;
          for (int kb = 0; kb < blocks_k; ++kb) {
            if (!wait_bar(&sm.empty[stage], stage_phase ^ 1u, abort)) {
              gave_up(a, abort);
              break;
            }
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
            if (++stage == kStages) {
              stage = 0;
              stage_phase ^= 1u;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == 1 && rank == 0) {
      if (lane == 0) {
        // fp32 accumulator, fp16 operands, 256 x 256; X X^T has both operands MN-major
        const uint32_t idesc = 1u << 4 | (kBlock >> 3) << 17 | (kBlock >> 4) << 24 | (phase == kGram ? 3u << 15 : 0u);
        // K-major: 8-row groups 1024 bytes apart, 16 inner elements = 32 bytes.  MN-major:
        // groups of 64 rows a box apart, groups of 8 inner elements 1024 bytes apart.
        const uint32_t lead = phase == kGram ? kBoxBytes : 16;
        const uint32_t k_bytes = phase == kGram ? 2048 : 32;
        for (int t = pair; t < tiles && !*abort; t += pairs) {
          if (!wait_bar(&sm.acc_empty[acc], acc_phase ^ 1u, abort)) {
            gave_up(a, abort);
            break;
          }
          ptx::tmem_fence_after();
          const uint32_t d = tmem + acc * kBlock;
          for (int kb = 0; kb < blocks_k; ++kb) {
            if (!wait_bar(&sm.full[stage], stage_phase, abort)) {
              gave_up(a, abort);
              break;
            }
            ptx::tmem_fence_after();
            const uint32_t at = stages + stage * kStageBytes;
#pragma unroll
            for (int k = 0; k < kStepK / 16; ++k)
              ptx::mma_f16_pair(d, operand_desc(at + k * k_bytes, lead, 1024),
                                operand_desc(at + kOperandBytes + k * k_bytes, lead, 1024), idesc, kb > 0 || k > 0);
            ptx::mma_commit_pair(&sm.empty[stage]);
            if (++stage == kStages) {
              stage = 0;
              stage_phase ^= 1u;
            }
          }
          ptx::mma_commit_pair(&sm.acc_full[acc]);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      __syncwarp();
    } else if (warp >= 4) {
      const int quarter = warp % 4, half = (warp - 4) / 4;
      for (int t = pair; t < tiles && !*abort; t += pairs) {
        const Tile x = tile_at(a, phase, t);
        const uint32_t from = tmem + acc * kBlock + half * 128 + (static_cast<uint32_t>(quarter) << 21);
        const int i0 = x.I * kBlock + rank * 128 + quarter * 32;
        const int j = x.J * kBlock + half * 128;
        uint64_t* full = &sm.acc_full[acc];
        const bool ok = phase == kGram ? epilogue<kGram>(maps, a, step, x, i0, j, from, full, acc_phase, abort, st)
                        : phase == kPoly ? epilogue<kPoly>(maps, a, step, x, i0, j, from, full, acc_phase, abort, st)
                                         : epilogue<kUpdate>(maps, a, step, x, i0, j, from, full, acc_phase, abort, st);
        if (!ok) {
          gave_up(a, abort);
          break;
        }
        ptx::tmem_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(&sm.acc_empty[acc]), 0));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (lane == 0) {               // what was stored is there for the next phase
        ptx::bulk_wait<0>();
        ptx::fence_proxy_async();
      }
    }
    if (p + 1 == 3 * a.steps) break;
    // ---- barrier over the grid
    if (__syncthreads_or(*abort)) break;
    if (threadIdx.x == 0) {
      ptx::red_release_add(a.barrier, 1);
      const int want = (p + 1) * static_cast<int>(gridDim.x);
      bool there = false;
      for (uint32_t n = 0; n < kGridWaitLimit && !there; ++n) {
        int v;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a.barrier) : "memory");
        there = v >= want;
        if (!there && (n & 255u) == 255u && *reinterpret_cast<volatile int*>(&a.header->status) == kStatusTimeout) break;
      }
      if (!there) gave_up(a, abort);
    }
    if (__syncthreads_or(*abort)) break;
    if (lane == 0) ptx::fence_proxy_async();   // the acquire before the next tensor copies
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

// [batch][outer][ld] fp16 with r columns used, in boxes of box_x x box_y.
cudaError_t encode(CUtensorMap* map, void* p, const OrthoShape& sh, int64_t outer, int box_x, int box_y,
                   bool swizzle) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(sh.r), static_cast<cuuint64_t>(outer),
                              static_cast<cuuint64_t>(sh.batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(sh.ld * 2), static_cast<cuuint64_t>(sh.ld * outer * 2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_y), 1}, step[3] = {1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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
  in.barrier = reinterpret_cast<int*>(ws + L.barrier);

  OrthoMaps maps;
  cudaError_t e = cudaSuccess;
  auto add = [&](CUtensorMap* map, size_t at, int64_t outer, int x, int y, bool swizzle) {
    if (e == cudaSuccess) e = encode(map, ws + at, sh, outer, x, y, swizzle);
  };
  for (int i = 0; i < 2; ++i) {
    add(&maps.xt[i], L.xt[i], sh.c, 64, 64, true);
    add(&maps.xt_piece[i], L.xt[i], sh.c, 32, kPiece, false);
  }
  add(&maps.xl_piece, L.xl, sh.c, 32, kPiece, false);
  add(&maps.a, L.a, sh.r, 64, 64, true);
  add(&maps.a_piece, L.a, sh.r, 32, kPiece, false);
  add(&maps.a_mirror, L.a, sh.r, kPiece, 32, false);
  add(&maps.b, L.b, sh.r, 64, 64, true);
  add(&maps.b_piece, L.b, sh.r, 32, kPiece, false);
  add(&maps.b_mirror, L.b, sh.r, kPiece, 32, false);
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
  a.rho = power_of_two_below(std::fmax(1.0, static_cast<double>(sh.r) / 16));
  a.diag_a = reinterpret_cast<float*>(ws + L.diag_a);
  a.diag_b = reinterpret_cast<float*>(ws + L.diag_b);
  a.out = static_cast<__nv_bfloat16*>(q.out);
  a.out_batch = q.out_batch_stride;
  a.out_row = q.out_row_stride;
  a.tall = sh.tall;
  a.header = in.header;
  a.barrier = in.barrier;

  const unsigned batch = static_cast<unsigned>(sh.batch);
  ortho_norm_kernel<<<dim3(sh.norm_blocks, batch), 256, 0, stream>>>(in);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  ortho_scale_kernel<<<dim3((in.cols + 63) / 64, (in.rows + 63) / 64, batch), 256, 0, stream>>>(in);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  const int64_t nr = (sh.r + kBlock - 1) / kBlock, nc = (sh.c + kBlock - 1) / kBlock;
  const int64_t most = sh.batch * nr * nc;          // blocks of the largest phase
  const int pairs = static_cast<int>(most < g_pairs[dev] ? most : g_pairs[dev]);
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
