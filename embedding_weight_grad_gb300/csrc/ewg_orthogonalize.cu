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
//     fp16 number each holds what their rounding left; a X is taken from the sum.  Directions
//     with small singular values, which the steps enlarge by up to a^5 = 485, then carry no
//     noise from the rounding of the large ones: B is small on them.  Without it a matrix of
//     low effective rank loses ten times the precision.
//   * What rounding left of the diagonals of A and B, their largest entries, is kept apart in
//     fp32: (b A + c A^2)_ii takes it in, and B X = fp16(B) X + rest(diag(B)) X.  (Taking the
//     whole diagonal out of the fp16 matrices would serve full-rank updates better, 1.8e-3
//     instead of 2.1e-3 with the bf16 rounding's 1.66e-3, and others worse, up to 3.9e-3: in
//     directions on which B vanishes its diagonal and the rest of it cancel, but not their
//     products with differently rounded X.)
//     The operands' roundings average out over a product's terms where those are many and unlike.  Where
//     all singular values are equal they do not, least of all for the identity: 7e-3.
//   * X is stored times s ~ sqrt(r c), a power of two, so that its entries are about 1 at first
//     and at most 1.2 s; A and B need no scale.
//
// Layout.  Every buffer is [., ld] fp16 with the r index inside: X^T (two, alternating), the
// rest of X^T, A (two, alternating) and B; of A and B only the blocks on and below the
// diagonal.  A block above it is read as the transpose of its mirror: the tensor cores take
// an operand with its inner index inside (K-major) or outside (MN-major), so an operand's
// row of blocks changes from one to the other at the diagonal.  X^T is MN-major in X X^T.  The
// update computes X^T's blocks, so that every accumulator lane holds neighbours of one row
// of what it reads and writes.
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
constexpr int kScaleBlocks = 4;      // blocks of the scaling kernel on an SM

// ---------------------------------------------------------------- norm and first X

struct OrthoIn {
  const void* grad;
  int bf16, tall;
  int tiles_of_block;                // of the scaling kernel
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

// A lane's sum of squares, to about 2^-45 of it: each square and each addition with its
// rounding error (an fma, and Knuth's two-sum), the errors summed beside.  The norm then
// rounds to the same fp32 factor whatever the order of the elements (strides, alignment, a
// transposed matrix).  The elements are first scaled by the power of two that brings the
// largest so far near 1, which is exact, so that neither large nor small gradients leave
// fp32's range.  64-bit arithmetic, two elements a cycle on an SM, would bound the kernel: it
// takes over once in kFlush times.
constexpr int kLaneElems = 32;
constexpr int kNormWarps = 8;
constexpr int kFlush = 8;

struct Squares {
  float2 sum, err;
  int e;                             // they are times 2^(2 (127 - e))

  __device__ __forceinline__ void clear() {
    sum = err = make_float2(0.0f, 0.0f);
    e = 0;
  }
  __device__ __forceinline__ void add(const float (&g)[kLaneElems]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kLaneElems; ++i) m = fmaxf(m, fabsf(g[i]));
    const int em = min(static_cast<int>(__float_as_uint(m) >> 23), 253);
    if (em > e) {
      const float f = __uint_as_float(static_cast<uint32_t>(max(127 + e - em, 1)) << 23);   // 2^(e - em)
      sum = make_float2(sum.x * f * f, sum.y * f * f);
      err = make_float2(err.x * f * f, err.y * f * f);
      e = em;
    }
    const float scale = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);              // 2^(127 - e)
    const float2 by = make_float2(scale, scale);
#pragma unroll
    for (int i = 0; i < kLaneElems; i += 2) {         // two at a time
      const float2 x = ptx::mul2(make_float2(g[i], g[i + 1]), by);
      const float2 p = ptx::mul2(x, x);
      const float2 t = ptx::add2(sum, p);
      const float2 b = ptx::sub2(t, sum);
      const float2 lost = ptx::add2(ptx::sub2(sum, ptx::sub2(t, b)), ptx::sub2(p, b));
      err = ptx::add2(err, ptx::add2(lost, ptx::fma2(x, x, make_float2(-p.x, -p.y))));
      sum = t;
    }
  }
  __device__ __forceinline__ double value() const {
    const double back = __longlong_as_double(static_cast<long long>(1023 + 2 * (e - 127)) << 52);
    const double all = static_cast<double>(sum.x) + static_cast<double>(sum.y);
    // (an infinite or NaN sum has no error term)
    return (all + (isfinite(all) ? static_cast<double>(err.x) + static_cast<double>(err.y) : 0.0)) * back;
  }
};

// Sums of squares of one matrix per blockIdx.y, a warp to 1024 neighbouring elements of a row
// (a matrix without gaps is one long row), the next ones' loads under way meanwhile.  Bound by
// the read of G: 13.2 us at 2048 x 7168 fp32, 4.4 TB/s with start and end.
__global__ void __launch_bounds__(32 * kNormWarps, 2) ortho_norm_kernel(const OrthoIn a) {
  ptx::pdl_launch_dependents();      // the scaling kernel's reads of G
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.header->status = kStatusOk;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.num_counters; i += 32 * kNormWarps)
      a.counters[static_cast<long long>(blockIdx.y) * a.num_counters + i] = 0;
  constexpr int kChunk = 32 * kLaneElems;
  const bool whole = a.row_stride == a.cols;
  const long long cols = whole ? static_cast<long long>(a.rows) * a.cols : a.cols;
  const int chunks_per_row = static_cast<int>((cols + kChunk - 1) / kChunk);
  const long long chunks = static_cast<long long>(chunks_per_row) * (whole ? 1 : a.rows);
  const int lane = threadIdx.x % 32;
  // whole and aligned chunks come in vectors of 16 bytes: 8 of fp32, 4 of bf16; `vec` tells
  uint32_t w[kLaneElems];
  bool vec = false;
  auto load = [&](long long q) {
    const long long row = whole ? 0 : q / chunks_per_row;
    const long long col = (q - row * chunks_per_row) * kChunk;
    const long long at = blockIdx.y * a.batch_stride + row * a.row_stride + col;
    const int n = static_cast<int>(min(cols - col, static_cast<long long>(kChunk)));
    const char* p = static_cast<const char*>(a.grad) + at * (a.bf16 ? 2 : 4);
    vec = n == kChunk && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    if (vec) {
      const uint4* v = reinterpret_cast<const uint4*>(p) + lane;
#pragma unroll
      for (int i = 0; i < kLaneElems / 4; ++i) {
        if (a.bf16 && i >= kLaneElems / 8) break;
        const uint4 r = v[32 * i];
        w[4 * i] = r.x;
        w[4 * i + 1] = r.y;
        w[4 * i + 2] = r.z;
        w[4 * i + 3] = r.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i)
        w[i] = __float_as_uint(lane + 32 * i < n ? grad_at(a, at + lane + 32 * i) : 0.0f);
    }
  };
  double sum = 0.0;
  Squares squares;
  squares.clear();
  const long long step = gridDim.x * kNormWarps;
  long long q = blockIdx.x * kNormWarps + threadIdx.x / 32;
  if (q < chunks) load(q);
  for (int n = 1; q < chunks; ++n) {
    float g[kLaneElems];
    if (vec && a.bf16) {
#pragma unroll
      for (int i = 0; i < kLaneElems / 2; ++i) {
        g[2 * i] = __uint_as_float(w[i] << 16);
        g[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i) g[i] = __uint_as_float(w[i]);
    }
    q += step;
    if (q < chunks) load(q);
    squares.add(g);
    if (n % kFlush == 0) {
      sum += squares.value();
      squares.clear();
    }
  }
  sum += squares.value();
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  __shared__ double part[kNormWarps];
  if (lane == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNormWarps; ++w) sum += part[w];
    a.norm[blockIdx.y * a.norm_blocks + blockIdx.x] = sum;
  }
}

// X^T times s / |G|, split into two fp16 numbers, by 64 x 64 tiles of G, a.tiles_of_block
// neighbouring ones to a block, the next tile's loads under way while one is written.  Bound by
// the read of G and the two writes: 19.9 us at 2048 x 7168 fp32, 5.9 TB/s (a tile a block, each
// with its own sum of the norm's parts: 25.5 us).
__global__ void __launch_bounds__(256, kScaleBlocks) ortho_scale_kernel(const OrthoIn a) {
  __shared__ float tile[64][65];
  __shared__ double factor;
  const int tid = threadIdx.x;
  const int es = a.bf16 ? 2 : 4;
  const int z = blockIdx.y;
  const int across = (a.cols + 63) / 64, share = a.tiles_of_block;
  int t = blockIdx.x * share;
  const int end = min(t + share, across * ((a.rows + 63) / 64));
  if (t >= end) return;
  int row0 = t / across * 64, col0 = t % across * 64;
  const long long row_bytes = a.row_stride * es;

  // A tile whole and aligned comes in vectors of 16 bytes: 4 rows of 64 numbers at once in a
  // warp for bf16, 2 for fp32.  Any other: thread = column, every fourth row.
  uint32_t w[16];
  const int per = a.bf16 ? 8 : 4;                    // numbers of a vector
  const int line = 64 / per, rows_at_once = 256 / line;
  auto load = [&]() -> bool {
    const char* base = static_cast<const char*>(a.grad) +
                       (blockIdx.y * a.batch_stride + static_cast<long long>(row0) * a.row_stride + col0) * es;
    const bool whole = row0 + 64 <= a.rows && col0 + 64 <= a.cols &&
                       (reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(row_bytes)) % 16 == 0;
    if (whole) {
      const char* p = base + tid / line * row_bytes + tid % line * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (a.bf16 && k >= 2) break;
        const uint4 v = *reinterpret_cast<const uint4*>(p + k * rows_at_once * row_bytes);
        w[4 * k] = v.x;
        w[4 * k + 1] = v.y;
        w[4 * k + 2] = v.z;
        w[4 * k + 3] = v.w;
      }
    } else {
      const int cx = tid % 64, ry = tid / 64;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const bool in = row0 + ry + 4 * k < a.rows && col0 + cx < a.cols;
        const char* p = base + (ry + 4 * k) * row_bytes + cx * es;
        w[k] = !in ? 0u : a.bf16 ? static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16
                                 : *reinterpret_cast<const uint32_t*>(p);
      }
    }
    return whole;
  };
  bool whole = load();
  ptx::pdl_wait_prior_grid();        // the norm kernel has ended
  float f1 = 0.0f, f3 = 0.0f;
  for (bool first = true;; first = false) {
    if (whole) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (a.bf16 && k >= 2) break;
        float* to = &tile[tid / line + k * rows_at_once][tid % line * per];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (a.bf16) {
            to[2 * q] = __uint_as_float(w[4 * k + q] << 16);
            to[2 * q + 1] = __uint_as_float(w[4 * k + q] & 0xffff0000u);
          } else {
            to[q] = __uint_as_float(w[4 * k + q]);
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) tile[tid / 64 + 4 * k][tid % 64] = __uint_as_float(w[k]);
    }
    if (first && tid < 32) {
      double sum = 0.0;
      for (int i = tid; i < a.norm_blocks; i += 32) sum += a.norm[z * a.norm_blocks + i];
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
      if (tid == 0) factor = sum == 0.0 ? 0.0 : a.s / sqrt(sum);   // a zero matrix stays zero
    }
    __syncthreads();
    if (first) {
      // factor = f1 f2 with f1 a power of two, so that neither product leaves fp32's range
      int e;
      const float f2 = static_cast<float>(frexp(factor, &e));
      const int e1 = min(max(e, -120), 120);
      f1 = ldexpf(1.0f, e1);
      f3 = ldexpf(f2, min(max(e - e1, -126), 126));
    }
    // the r index is G's column where G is tall, else its row
    const int outer0 = a.tall ? row0 : col0, inner0 = a.tall ? col0 : row0;
    if (++t < end) {
      if ((col0 += 64) >= a.cols) {
        col0 = 0;
        row0 += 64;
      }
      whole = load();
    }
    const int outers = a.tall ? a.rows : a.cols, inners = a.tall ? a.cols : a.rows;
    const int x = tid % 8 * 8;
    if (inner0 + x < a.ld) {
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
        const long long to = z * a.x_batch + static_cast<long long>(outer0 + k) * a.ld + inner0 + x;
        *reinterpret_cast<uint4*>(a.xt + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(a.xl + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    if (t >= end) break;
    __syncthreads();                 // the tile has been read
  }
}

// ---------------------------------------------------------------- the products

constexpr int kBlock = 256;          // a pair of CTAs computes 256 x 256; each CTA 128 rows
constexpr int kStepK = 64;           // inner elements of a stage: one 128-byte swizzled row
constexpr int kStages = 5;
constexpr int kOperandBytes = 128 * kStepK * 2;       // one CTA's half of an operand's stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kBoxBytes = 64 * kStepK * 2;            // one tensor copy: 64 rows of 128 bytes
constexpr int kFirstEpilogueWarp = 4;
constexpr int kEpilogueWarps = 8;
constexpr int kWarpsOfBlock = 2 * kEpilogueWarps;     // of the pair
constexpr int kWarpCols = 4 * kBlock / kEpilogueWarps;   // columns of an epilogue warp (all take 32 rows)
// The epilogue takes a warp's 32 rows of A or B in pieces of 64 columns, of X in strips of 32
// columns, which come and go by tensor copies through a slot of the warp: two pieces, or two
// strips of both parts of X.
// (Copies by the threads themselves, of 32 or 64 bytes a row, took two to three times as long:
// the path to L2 carries requests, not bytes.)
constexpr int kPiece = 64;
constexpr int kPieces = kWarpCols / kPiece;
constexpr int kPieceBytes = 32 * kPiece * 2;
constexpr int kStrip = 32;
constexpr int kStripBytes = 32 * kStrip * 2;          // of one part of X
constexpr int kSlotBytes = 2 * kPieceBytes;
static_assert(kSlotBytes == 4 * kStripBytes, "a slot holds two strips of both parts");
// The halves of the slots lie so that the epilogue's 128 x 256 numbers of A form an operand of the
// tensor cores, 128 rows of 128 bytes for each 64 columns: half h of warp w (rows 32 (w % 4),
// columns 128 (w / 4) + 64 h) comes 4 (2 (w / 4) + h) + w % 4 pieces in.
constexpr int kHalfStride = 4 * kPieceBytes;          // between a warp's halves
static_assert(kHalfStride == kOperandBytes, "64 columns of the CTA's rows");
__host__ __device__ constexpr int slot_offset(int w) { return (8 * (w / 4) + w % 4) * kPieceBytes; }
constexpr int kGemmThreads = 32 * (kFirstEpilogueWarp + kEpilogueWarps);
constexpr int kOwnBytes = kBlock * 4;                 // a + what is left of B_ii for a unit's columns
constexpr size_t kGemmSmem =
    static_cast<size_t>(kStages) * kStageBytes + kEpilogueWarps * kSlotBytes + kOwnBytes + 1024;
static_assert(kWarpCols == 128 && kPieces == 2, "a warp's columns, as the epilogue takes them");
static_assert(kWarpsOfBlock == kOrthoWarps && kBlock == kOrthoBlock, "as the workspace is laid out for");
static_assert(kGemmSmem + 512 <= 227 * 1024, "stages and slots fit in shared memory");
#ifndef EWG_ORTHO_WAIT_LIMIT                                  // (a test of the limit has a shorter one)
#define EWG_ORTHO_WAIT_LIMIT 4000000000ull
#endif
constexpr unsigned long long kWaitLimit = EWG_ORTHO_WAIT_LIMIT;       // of a wait, in ns
constexpr uint32_t kPollLimit = 1u << 30;

enum Phase { kGram = 0, kPoly = 1, kUpdate = 2 };

struct OrthoMaps {
  CUtensorMap xt[2], a[2], b;        // operands: boxes of 64 x 64
  CUtensorMap x_strip[2];                    // 32 of the r index x 32, of X^T and of its rest
  CUtensorMap a_piece[2], b_piece;           // 64 x 32
};

struct OrthoArgs {
  int batch, r, c, ld;
  int steps;
  float ca, cb, cc;                  // the polynomial's coefficients
  float s;                           // X is stored times s
  __half* a[2];                      // A of even and odd steps
  __half* b;
  float* diag_a[2];                  // [batch][ld]: what rounding left of the diagonals
  float* diag_b;
  int fused;                         // matrices of one block: A stays with the pair that computed it
  int split;                         // parts of the inner dimension of X X^T
  float* partial;                    // a split product: [batch][block][part][CTA][warp][column][row]
  __nv_bfloat16* out;
  long long out_batch, out_row;
  int out_tall;                      // out is [c, r]
  Header* header;
  int* ready;                        // [phase][batch][block row]: warps done, over all steps
  int* arrived;                      // [batch][block][CTA][warp]: parts done, over all steps
};

struct GemmSmem {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
  uint64_t piece[kEpilogueWarps][2], own_full, a_full;
  int units_done[kEpilogueWarps];    // units an epilogue warp is through with its slot for
  int units_ready;                   // units whose inputs are there
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

__device__ __forceinline__ int parts_of(const OrthoArgs& a, int phase) { return phase == kGram ? a.split : 1; }

__device__ __forceinline__ int units_of(const OrthoArgs& a, int phase) {
  const int nr = blocks_of(a.r);
  return a.batch * (phase == kUpdate ? nr * blocks_of(a.c) : nr * (nr + 1) / 2 * parts_of(a, phase));
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
  const int blocks = nr * (nr + 1) / 2, parts = parts_of(a, phase);
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
  const int parts = parts_of(a, phase), per = (blocks + parts - 1) / parts;
  first = x.part * per;
  last = min(first + per, blocks);
}

// ---- what a unit waits for.  ready[phase][z][I] counts the epilogue warps (16 a unit) that
// have stored their part of block row I of X, A or B, over all steps.  (Nothing else is
// needed: a complete row of B needs all of A, which needs all of X of the step before, so
// that no buffer is written while an earlier phase still reads it, with two A in turn.)  What
// other SMs stored plainly is read past L1.

__device__ __forceinline__ int* ready_at(const OrthoArgs& a, int phase, int z, int I) {
  const int nr = blocks_of(a.r);
  return a.ready + (static_cast<long long>(z) * 3 + phase) * nr + I;
}

// Whether a wait is to end without what it waits for: `abort` is set, or it has lasted for
// seconds.  Looked at once in 64 polls.  (The longest wait of a call that goes well is for most of
// a phase: 0.3 s for the largest matrices that memory holds.)
struct Patience {
  unsigned long long since = 0;
  __device__ __forceinline__ bool over(uint32_t poll, volatile int* abort) {
    if ((poll & 63u) != 63u) return false;
    unsigned long long now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    if (since == 0) since = now;
    return *abort || now - since > kWaitLimit;
  }
};

__device__ bool wait_ready(const OrthoArgs& a, const int* p, int want, volatile int* abort) {
  Patience patience;
  for (uint32_t n = 0; n < kPollLimit; ++n) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= want) return true;
    if (want - v > kWarpsOfBlock) __nanosleep(200);  // far from it: polls hold up who counts
    if (patience.over(n, abort) ||
        ((n & 255u) == 255u && *reinterpret_cast<volatile int*>(&a.header->status) == kStatusTimeout))
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
  const int want = (step + 1) * nr * kWarpsOfBlock * (phase == kPoly ? a.split : 1);
  if (phase == kPoly && a.fused) return true;
  if (phase == kPoly)
    return wait_ready(a, ready_at(a, kGram, x.z, x.I), want, abort) &&
           (x.I == x.J || wait_ready(a, ready_at(a, kGram, x.z, x.J), want, abort));
  return wait_ready(a, ready_at(a, kPoly, x.z, x.I), want, abort);
}

// The warp is through with unit x: with its slot, and (`signal`) with what it stored, by tensor
// copies of lane 0 and (diagonals) plainly.
__device__ __forceinline__ void unit_done(const OrthoArgs& a, int phase, const Unit& x, volatile int* units_done,
                                          bool signal) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) {
    ptx::bulk_wait_read();
    __threadfence_block();
    *units_done = *units_done + 1;
    if (signal) {
      ptx::bulk_wait();              // its copies' writes are done, and visible to it
      ptx::fence_acq_rel_gpu();
      ptx::red_relaxed_add(ready_at(a, phase, x.z, x.I), 1);
      if (phase != kUpdate && x.I != x.J) ptx::red_relaxed_add(ready_at(a, phase, x.z, x.J), 1);
    }
  }
  __syncwarp();
}

// Waits for the phase of `bar` with the given parity; false if it gave up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
  Patience patience;
  for (uint32_t i = 0; i < kPollLimit; ++i) {
    if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
    if (patience.over(i, abort)) return false;
  }
  return false;
}

// Waits for a count in shared memory.
__device__ __forceinline__ bool wait_count(volatile int* count, int want, volatile int* abort) {
  Patience patience;
  for (uint32_t i = 0; i < kPollLimit; ++i) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(ptx::smem_u32(const_cast<int*>(count))) : "memory");
    if (v >= want) return true;
    if (patience.over(i, abort)) return false;
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

// The warp has read its part of the accumulator.
__device__ __forceinline__ void release_acc(uint32_t acc_empty) {
  ptx::tmem_fence_before();
  __syncwarp();
  if (threadIdx.x % 32 == 0) ptx::mbar_arrive_cluster(acc_empty);
}

// Where an epilogue warp finds a unit's accumulator, and its slot.
struct Acc {
  uint32_t from;                     // its columns in tensor memory
  uint64_t* full;
  uint32_t parity;
  uint32_t empty;                    // shared::cluster address
  volatile int* abort;
  int place;                         // the warp's place in the pair
  uint32_t slot;                     // shared-memory address
  uint64_t* bars;                    // of the slot's halves: its copies have come
  volatile int* units_done;          // of the warp
  uint32_t own;                      // shared-memory address: a + what is left of B_ii, of the warp's columns
  uint64_t* own_full;
  uint32_t a_full;                   // shared::cluster address
};

// The first row and column of epilogue warp w's part of a unit (it takes the 32 rows of its
// quarter of tensor memory, which is its number in the block modulo 4).
struct Place {
  int row, col;
};
__device__ __forceinline__ Place place_of(int phase, const Unit& x, int rank, int w) {
  static_assert(kFirstEpilogueWarp % 4 == 0, "warp w's quarter is w % 4");
  return {(phase == kUpdate ? x.J : x.I) * kBlock + rank * 128 + w % 4 * 32,
          (phase == kUpdate ? x.I : x.J) * kBlock + w / 4 * kWarpCols};
}

// How many pieces (or strips) of `width` columns a warp's part has that starts at (row, col).
__device__ __forceinline__ int pieces_of(const OrthoArgs& a, int phase, const Place& at, int width) {
  if (at.row >= (phase == kUpdate ? a.c : a.r)) return 0;
  return min(max((a.r - at.col + width - 1) / width, 0), kWarpCols / width);
}

// Requests (one lane) what a warp's part of a unit reads beside the products: piece u of A, or
// strip u of both parts of X, into half u % 2 of the slot.
__device__ __forceinline__ void request_piece(const OrthoMaps& maps, int step, int z, const Place& at, int u,
                                              uint32_t slot, uint64_t* bars) {
  ptx::mbar_arrive_expect_tx(&bars[u], kPieceBytes);
  ptx::tma_load_3d(slot + u * kHalfStride, &maps.a_piece[step & 1], at.col + u * kPiece, at.row, z, &bars[u]);
}
__device__ __forceinline__ void request_strip(const OrthoMaps& maps, int step, int z, const Place& at, int u,
                                              uint32_t slot, uint64_t* bars) {
  const uint32_t to = slot + u % 2 * kHalfStride;
  ptx::mbar_arrive_expect_tx(&bars[u % 2], 2 * kStripBytes);
  ptx::tma_load_4d(to, &maps.x_strip[step & 1], at.col + u * kStrip, at.row, z, 0, &bars[u % 2]);
}

__device__ __forceinline__ uint4 lds_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts_v4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// 16 bytes (8 columns) of this lane's row of a piece, in the copies' 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(uint32_t piece, int chunk) {
  const uint32_t lane = threadIdx.x % 32;
  return piece + lane * 128 + ((chunk ^ (lane & 7)) << 4);
}

// The same of a strip, in the 64-byte swizzle.
__device__ __forceinline__ uint32_t strip_chunk_at(uint32_t strip, int chunk) {
  const uint32_t lane = threadIdx.x % 32;
  return strip + lane * 64 + ((chunk ^ ((lane >> 1) & 3)) << 4);
}

// Waits (a whole warp) for the copies into half h of the slot.
__device__ __forceinline__ bool wait_piece(const Acc& in, int h, uint32_t& parity) {
  if (!__all_sync(kAll, wait_bar(&in.bars[h], (parity >> h) & 1u, in.abort))) return false;
  parity ^= 1u << h;
  return true;
}

// The last update's strip, to the caller's matrix: lane = row j0 + lane of X^T, columns i0 .. + 31,
// packed in bf16; `buf` is free shared memory for 32 x 64 bytes.
__device__ __forceinline__ void store_out(const OrthoArgs& a, int z, int j0, int i0, const uint32_t (&w)[16],
                                          uint32_t buf) {
  const int lane = threadIdx.x % 32, jx = j0 + lane;
  const int n = min(a.r - i0, kStrip);
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + z * a.out_batch;
  if (!a.out_tall) {                 // out is [r, c]: neighbouring lanes, neighbouring elements
    uint16_t* p = out + i0 * a.out_row + jx;
    if (jx >= a.c) return;
#pragma unroll
    for (int q = 0; q < 32; ++q)
      if (q < n) p[q * a.out_row] = static_cast<uint16_t>(q % 2 ? w[q / 2] >> 16 : w[q / 2]);
    return;
  }
  // out is [c, r]: 16 bytes at once, or through shared memory a row at a time where the rows of
  // out are not aligned for that
  const bool vec = reinterpret_cast<uintptr_t>(out + i0) % 16 == 0 && a.out_row % 8 == 0 && n == kStrip;
  if (vec) {
    if (jx >= a.c) return;
    uint4* p = reinterpret_cast<uint4*>(out + jx * a.out_row + i0);
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    sts_v4(strip_chunk_at(buf, k), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
  __syncwarp();
  const int rows = min(a.c - j0, 32);
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {     // lane = column
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];"
                 : "=h"(v) : "r"(buf + r * 64 + (((lane / 8) ^ ((r >> 1) & 3)) << 4) + lane % 8 * 2));
    if (r < rows && lane < n) out[(j0 + r) * a.out_row + i0 + lane] = v;
  }
  ptx::fence_proxy_async_shared();   // the next copies into `buf` come after these plain writes
  __syncwarp();
}

// One warp's part of a finished block of an update: 32 rows of X^T, kWarpCols columns.  X's two
// parts of the first two strips were requested by the loading warp.
__device__ __forceinline__ bool epilogue_update(const OrthoMaps& maps, const OrthoArgs& a, int step, const Unit& x,
                                                const Place& at, const Acc& in, uint32_t& parity) {
  const int lane = threadIdx.x % 32, cur = step & 1;
  const int strips = pieces_of(a, kUpdate, at, kStrip);
  const bool last = step == a.steps - 1;
  if (!__all_sync(kAll, wait_bar(in.full, in.parity, in.abort))) return false;
  ptx::tmem_fence_after();
  if (strips == 0) release_acc(in.empty);
  // (bit 2 of `parity`: of the next wait on own_full)
  if (!__all_sync(kAll, wait_bar(in.own_full, (parity >> 2) & 1u, in.abort))) return false;
  parity ^= 4u;
  const float unscale = 1.0f / a.s;
#pragma unroll 1
  for (int u = 0; u < strips; ++u) {
    const uint32_t strip = in.slot + u % 2 * kHalfStride;
    uint32_t acc[kStrip];
    ptx::tmem_load32(acc, in.from + u * kStrip);
    if (!wait_piece(in, u % 2, parity)) return false;
    uint4 top[4], low[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      top[k] = lds_v4(strip_chunk_at(strip, k));
      low[k] = lds_v4(strip_chunk_at(strip + kStripBytes, k));
    }
    ptx::tmem_wait_load();
    if (u + 1 == strips) release_acc(in.empty);
    uint32_t hw[16], lw[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t tk[4] = {top[k].x, top[k].y, top[k].z, top[k].w};
      const uint32_t lk[4] = {low[k].x, low[k].y, low[k].z, low[k].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // two columns at a time
        const int e = 8 * k + 2 * q;
        const float2 v = ptx::fma2(lds_f2(in.own + (u * kStrip + e) * 4), ptx::add2(unpack_half(tk[q]), unpack_half(lk[q])),
                                   make_float2(__uint_as_float(acc[e]), __uint_as_float(acc[e + 1])));
        if (last) {
          hw[e / 2] = pack_bf16(v.x * unscale, v.y * unscale);
        } else {
          hw[e / 2] = pack_half(v.x, v.y);
          const float2 left = ptx::sub2(v, unpack_half(hw[e / 2]));
          lw[e / 2] = pack_half(left.x, left.y);
        }
      }
    }
    if (last) {
      __syncwarp();                  // the strip has been read
      store_out(a, x.z, at.row, at.col + u * kStrip, hw, strip);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sts_v4(strip_chunk_at(strip, k), make_uint4(hw[4 * k], hw[4 * k + 1], hw[4 * k + 2], hw[4 * k + 3]));
        sts_v4(strip_chunk_at(strip + kStripBytes, k),
               make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]));
      }
      ptx::fence_proxy_async_shared();
    }
    __syncwarp();
    if (lane == 0) {
      if (u >= 1 && u + 1 < strips) {                 // into the half of the strip before this one
        ptx::bulk_wait_read();
        request_strip(maps, step, x.z, at, u + 1, in.slot, in.bars);
      }
      if (!last) {
        ptx::tma_store_4d(&maps.x_strip[cur ^ 1], at.col + u * kStrip, at.row, x.z, 0, strip);
        ptx::bulk_commit();
      }
    }
  }
  unit_done(a, kUpdate, x, in.units_done, !last);
  return true;
}

// Eight columns of a row of A or B from the products v and, for B, A's numbers `o`; `d` is the
// row less the first column, and what rounding leaves of the diagonal goes to diag[diag_at].
template <int kPhase>
__device__ __forceinline__ uint4 finish8(const OrthoArgs& a, int cur, float f, float (&v)[8], uint4 o, int d,
                                         float rest_a, long long diag_at) {
  float on = 0.0f;                   // A_ii as stored
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] *= f;
  if constexpr (kPhase == kPoly) {
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 p = unpack_half(w[q]);
      v[2 * q] = fmaf(a.cb, p.x, v[2 * q]);
      v[2 * q + 1] = fmaf(a.cb, p.y, v[2 * q + 1]);
      if (d == 2 * q) on = p.x;
      if (d == 2 * q + 1) on = p.y;
    }
  }
  if (d >= 0 && d < 8) {             // the diagonal passes through
    const float more = kPhase == kPoly ? rest_a * fmaf(2.0f * a.cc, on, a.cb) : 0.0f;   // to first order
    float left = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q != d) continue;
      v[q] += more;
      left = v[q] - __half2float(__float2half_rn(v[q]));
    }
    if (diag_at >= 0) (kPhase == kGram ? a.diag_a[cur] : a.diag_b)[diag_at] = left;
  }
  return make_uint4(pack_half(v[0], v[1]), pack_half(v[2], v[3]), pack_half(v[4], v[5]), pack_half(v[6], v[7]));
}

// The same for A = X X^T or B = b A + c A^2: 32 rows from i0, kWarpCols columns from j of a block on
// or below the diagonal.
//
// Matrices of one block (a.fused): A is left in the slots, which form an operand, and the
// same pair goes on to B.
//
// Where the inner dimension of X X^T is split, each part's warp stores its sums, waits for the other
// parts' and finishes its share of the columns, in sixteens, from all parts' sums, added
// in their order.  (The units of such a phase are no more than the pairs of the launch, see
// ortho_split, so the parts run at the same time.)
template <int kPhase>
__device__ __forceinline__ bool epilogue_square(const OrthoMaps& maps, const OrthoArgs& a, int step, const Unit& x,
                                                const Place& at, const Acc& in, uint32_t& parity) {
  const int lane = threadIdx.x % 32, cur = step & 1;
  const int i0 = at.row, j = at.col, i = i0 + lane;
  const int pieces = pieces_of(a, kPhase, at, kPiece);
  const bool row = i < a.r;
  const long long diag_at = x.z * static_cast<long long>(a.ld) + i;
  if (!__all_sync(kAll, wait_bar(in.full, in.parity, in.abort))) return false;
  ptx::tmem_fence_after();
  float rest_a = 0.0f;               // what rounding left of A_ii
  if (kPhase == kPoly && row) rest_a = __ldcg(a.diag_a[cur] + diag_at);
  const float f = kPhase == kGram ? 1.0f / (a.s * a.s) : a.cc;
  if (kPhase == kGram && a.split > 1) {
    const int parts = a.split, nr = blocks_of(a.r), blocks = nr * (nr + 1) / 2;
    const long long block = static_cast<long long>(x.z) * blocks + x.I * (x.I + 1) / 2 + x.J;
    constexpr int kPartStride = kBlock * kBlock;
    const float* sums = a.partial + block * parts * kPartStride + in.place * (32 * kWarpCols) + lane;
    float* mine = a.partial + (block * parts + x.part) * kPartStride + in.place * (32 * kWarpCols) + lane;
#pragma unroll 1
    for (int u = 0; u < 2 * pieces; ++u) {
      uint32_t acc[32];
      ptx::tmem_load32(acc, in.from + u * 32);
      ptx::tmem_wait_load();
#pragma unroll
      for (int q = 0; q < 32; ++q) mine[(u * 32 + q) * 32] = __uint_as_float(acc[q]);
    }
    release_acc(in.empty);
    bool ok = true;
    if (lane == 0) {
      int* arrived = a.arrived + block * kWarpsOfBlock + in.place;
      ptx::red_release_add(arrived, 1);
      ok = wait_ready(a, arrived, (step + 1) * parts, in.abort);
    }
    if (!__all_sync(kAll, ok)) return false;
    __half* m = a.a[cur] + (static_cast<long long>(x.z) * a.r + i) * a.ld + j;
    constexpr int kShares = kWarpCols / 16;
#pragma unroll 1
    for (int g = x.part * kShares / parts; g < (x.part + 1) * kShares / parts; ++g) {
      if (j + 16 * g >= a.r) break;
      float v[2][8];
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q / 8][q % 8] = __ldcg(sums + (16 * g + q) * 32);
#pragma unroll 2
      for (int k = 1; k < parts; ++k) {
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q / 8][q % 8] += __ldcg(sums + k * kPartStride + (16 * g + q) * 32);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 16 * g + 8 * e;
        const uint4 w = finish8<kPhase>(a, cur, f, v[e], uint4{}, i - (j + col), rest_a, row ? diag_at : -1);
        if (row) *reinterpret_cast<uint4*>(m + col) = w;      // (the sixteen lie inside ld)
      }
    }
    ptx::fence_proxy_async();        // these plain stores are read by tensor copies
    unit_done(a, kPhase, x, in.units_done, true);
    return true;
  }
  if (pieces == 0) release_acc(in.empty);
#pragma unroll 1
  for (int u = 0; u < pieces; ++u) {
    const uint32_t slot = in.slot + u * kHalfStride;
    if (kPhase == kPoly && !a.fused && !wait_piece(in, u, parity)) return false;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {    // 32 columns at a time
      uint32_t acc[32];
      ptx::tmem_load32(acc, in.from + u * kPiece + 32 * h);
      ptx::tmem_wait_load();
      if (u + 1 == pieces && h == 1) release_acc(in.empty);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t chunk = chunk_at(slot, 4 * h + k);
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(acc[8 * k + q]);
        uint4 o = {};
        if (kPhase == kPoly) o = lds_v4(chunk);
        sts_v4(chunk, finish8<kPhase>(a, cur, f, v, o, i - (j + u * kPiece + 32 * h + 8 * k), rest_a, row ? diag_at : -1));
      }
    }
    ptx::fence_proxy_async_shared();
    if (kPhase == kGram && a.fused) continue;         // A stays
    __syncwarp();
    if (lane == 0) {
      ptx::tma_store_3d(kPhase == kGram ? &maps.a_piece[cur] : &maps.b_piece, j + u * kPiece, i0, x.z, slot);
      ptx::bulk_commit();
    }
  }
  const bool stays = kPhase == kGram && a.fused;
  if (stays) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_release_cluster(in.a_full);
  }
  unit_done(a, kPhase, x, in.units_done, !stays);
  return true;
}

// How the operands of inner block kb of a unit lie: MN-major where a block above the diagonal is
// read from its mirror, and for X in X X^T.
struct Majors {
  bool a, b;
};
__device__ __forceinline__ Majors majors_of(int phase, const Unit& x, int kb) {
  const int k = kb / (kBlock / kStepK);
  if (phase == kGram) return {true, true};
  if (phase == kPoly) return {k > x.I, k > x.J};
  return {false, k > x.I};
}

// The products' instruction descriptor: fp32 accumulator, fp16 operands, 256 x 256.
__device__ __forceinline__ uint32_t idesc_of(Majors mn) {
  return 1u << 4 | (mn.a ? 1u << 15 : 0u) | (mn.b ? 1u << 16 : 0u) | (kBlock >> 3) << 17 | (kBlock >> 4) << 24;
}

// All phases of all steps, one cooperative launch of CTA pairs.  The units of all phases in
// order go round the pairs; a unit waits for the block rows that it reads, which units before
// it in the order store, so the earliest unfinished unit never waits and the phases (and
// the matrices of a batch) overlap without a barrier over the grid.  Per CTA: warp 0 copies
// operands (TMA), warp 1 of the pair's first CTA issues the products, the epilogue warps take
// finished accumulators (two in tensor memory, so that the products of the next unit run
// meanwhile), warp 2 copies in what those read beside the products, warp 3 watches what units
// wait for.
//
// A pair's block of 256 x 256 uses each operand byte it reads for 256 products; a ring of five
// stages of 64 of the inner dimension (with four, 24 x 1024 x 1024 takes 5 % longer) and the
// epilogue's slots fill shared memory.  Whole calls of five steps, each on other inputs: 7168 x 7168
// 5.2 ms (5.0 to 5.5 by the GPU and its power), 1.42 PFLOP/s of the operations that count (3 r^2 c +
// r^3 a step), bound by the tensor cores at the clock that the power limit leaves; 24 x 1024 x 1024
// 549 us (510 on one input over and over), 0.94 PFLOP/s, by the update's epilogues, which take as long
// as its products; 2048 x 7168 494 us, 1.0 PFLOP/s, and smaller ones by the way from a phase's last
// product to the next one's first (5 to 8 us, three times a step).
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
    for (int i = 0; i < 2 * kEpilogueWarps; ++i) ptx::mbar_init(&sm.piece[0][0] + i, 1);
    ptx::mbar_init(&sm.own_full, 1);
    ptx::mbar_init(&sm.a_full, kWarpsOfBlock);
    for (int i = 0; i < kEpilogueWarps; ++i) sm.units_done[i] = 0;
    sm.units_ready = 0;
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
  const uint32_t slots = stages + kStages * kStageBytes;     // of the epilogue warps
  const uint32_t own = slots + kEpilogueWarps * kSlotBytes;

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
  // body(phase, step, unit) for this pair's units in order, until one gives up.  `whole`: by all lanes
  // of a warp, which leave together (bodies return the same in all lanes, by a vote); else by one.
  auto for_units = [&](bool whole, auto&& body) {
    int offset = 0;                  // units so far, modulo the pairs
    for (int p = 0; p < 3 * a.steps; ++p) {
      const int phase = p % 3, step = p / 3;
      const int units = units_of(a, phase);
      if (a.fused && phase == kPoly) continue;        // with the phase before
      for (int t = pair >= offset ? pair - offset : pair - offset + pairs; t < units; t += pairs) {
        if (whole ? __any_sync(kAll, *abort) : *abort) return;
        if (!body(phase, step, unit_at(a, phase, t)) ||
            (a.fused && phase == kGram && !body(kPoly, step, unit_at(a, kPoly, t)))) {
          gave_up(a, abort);
          return;
        }
      }
      offset = (offset + units) % pairs;
    }
  };

  uint32_t a_parity = 0;             // issuer's, of a_full

  if (warp == 0) {
    if (lane == 0) {
      int units = 0;
      for_units(false, [&](int phase, int step, const Unit& x) {
        ++units;
        if (a.fused && phase == kPoly) return true;   // its operands are there
        const int cur = step & 1;
        // X X^T: X, X.  A A: A, A.  Update: X^T (rows J), B (rows I).
        const CUtensorMap* ma = phase == kPoly ? &maps.a[cur] : &maps.xt[cur];
        const CUtensorMap* mb = phase == kGram ? &maps.xt[cur] : phase == kPoly ? &maps.a[cur] : &maps.b;
        const int ra = (phase == kUpdate ? x.J : x.I) * kBlock + rank * 128;
        const int rb = (phase == kUpdate ? x.I : x.J) * kBlock + rank * 128;
        int k0, k1;
        inner_of(a, phase, x, k0, k1);
        if (!wait_count(&sm.units_ready, units, abort)) return false;
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait_bar(&sm.empty[stage], stage_phase ^ 1u, abort)) return false;
          if (rank == 0) ptx::mbar_arrive_expect_tx(&sm.full[stage], 2 * kStageBytes);
          const uint32_t bar = ptx::map_to_rank(ptx::smem_u32(&sm.full[stage]), 0);
          const uint32_t dst = stages + stage * kStageBytes;
          const int k = kb * kStepK;
          const Majors mn = majors_of(phase, x, kb);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int da = ra + 64 * h, db = rb + 64 * h;
            ptx::tma_load_3d_pair(dst + h * kBoxBytes, ma, mn.a ? da : k, mn.a ? k : da, x.z, bar);
            ptx::tma_load_3d_pair(dst + kOperandBytes + h * kBoxBytes, mb, mn.b ? db : k, mn.b ? k : db, x.z, bar);
          }
          next_stage();
        }
        return true;
      });
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    if (lane == 0) {
      for_units(false, [&](int phase, int, const Unit& x) {
        int k0, k1;
        inner_of(a, phase, x, k0, k1);
        if (!wait_bar(&sm.acc_empty[acc], acc_phase ^ 1u, abort)) return false;
        ptx::tmem_fence_after();
        const uint32_t d = tmem + acc * kBlock;
        if (a.fused && phase == kPoly) {              // A as the epilogue left it, both operands
          if (!wait_bar(&sm.a_full, a_parity, abort)) return false;
          a_parity ^= 1u;
          ptx::tmem_fence_after();
          for (int kb = k0; kb < k1; ++kb) {
            const uint32_t at = slots + kb * kOperandBytes;
#pragma unroll
            for (int k = 0; k < kStepK / 16; ++k) {
              const uint64_t desc = operand_desc(at + k * 32, 16, 1024);
              ptx::mma_f16_pair(d, desc, desc, idesc_of({false, false}), kb > k0 || k > 0);
            }
          }
          ptx::mma_commit_pair(&sm.acc_full[acc]);
          next_acc();
          return true;
        }
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait_bar(&sm.full[stage], stage_phase, abort)) return false;
          ptx::tmem_fence_after();
          const uint32_t at = stages + stage * kStageBytes;
          const Majors mn = majors_of(phase, x, kb);
          const uint32_t idesc = idesc_of(mn);
          // K-major: 8-row groups 1024 bytes apart, 16 inner elements = 32 bytes.  MN-major:
          // groups of 64 rows a box apart, groups of 8 inner elements 1024 bytes apart.
          const uint32_t lead_a = mn.a ? kBoxBytes : 16, lead_b = mn.b ? kBoxBytes : 16;
          const uint32_t k_a = mn.a ? 2048 : 32, k_b = mn.b ? 2048 : 32;
#pragma unroll
          for (int k = 0; k < kStepK / 16; ++k)
            ptx::mma_f16_pair(d, operand_desc(at + k * k_a, lead_a, 1024),
                              operand_desc(at + kOperandBytes + k * k_b, lead_b, 1024), idesc, kb > k0 || k > 0);
          ptx::mma_commit_pair(&sm.empty[stage]);
          next_stage();
        }
        ptx::mma_commit_pair(&sm.acc_full[acc]);
        next_acc();
        return true;
      });
    }
    __syncwarp();
  } else if (warp == 2) {
    // Lane w requests what epilogue warp w reads first in a unit, as soon as the block rows are
    // there and the warp is through with its slot for the unit before.  (A count, not the
    // parity of a barrier: units of X X^T need no loads, and the epilogue may run ahead there.)
    const int w = lane < kEpilogueWarps ? lane : 0;
    int units = 0;
    for_units(true, [&](int phase, int step, const Unit& x) {
      bool ok = wait_count(&sm.units_done[w], units++, abort);
      ok = ok && (phase == kGram || wait_count(&sm.units_ready, units, abort));
      if (!__all_sync(kAll, ok)) return false;
      if (phase == kUpdate) {        // a + what is left of B_ii: eight columns a lane
        const int col = x.I * kBlock + 8 * lane;
        if (col < a.r) {             // (then the eight lie inside ld)
          const float4* d = reinterpret_cast<const float4*>(a.diag_b + x.z * static_cast<long long>(a.ld) + col);
          const float4 d0 = __ldcg(d), d1 = __ldcg(d + 1);
          float4* to = reinterpret_cast<float4*>(raw + (own - ptx::smem_u32(raw))) + 2 * lane;
          to[0] = make_float4(a.ca + d0.x, a.ca + d0.y, a.ca + d0.z, a.ca + d0.w);
          to[1] = make_float4(a.ca + d1.x, a.ca + d1.y, a.ca + d1.z, a.ca + d1.w);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.own_full);
      }
      if (phase != kGram && !(a.fused && phase == kPoly) && lane < kEpilogueWarps) {
        const Place at = place_of(phase, x, rank, w);
        const int n = min(pieces_of(a, phase, at, phase == kPoly ? kPiece : kStrip), 2);
        for (int u = 0; u < n; ++u) {
          if (phase == kPoly) request_piece(maps, step, x.z, at, u, slots + slot_offset(w), sm.piece[w]);
          else request_strip(maps, step, x.z, at, u, slots + slot_offset(w), sm.piece[w]);
        }
      }
      __syncwarp();
      return true;
    });
  } else if (warp == 3) {
    // Watches what units wait for, ahead of the copies: a poll of L2 and the fence take 0.7 us, in
    // which the ring of operands would run low at the start of each unit (24 x 1024 x 1024, one input: 516 us
    // so, 548 where warps 0 and 2 poll; 256 x 256, which only waits: 108 and 105).
    if (lane == 0) {
      int units = 0;
      for_units(false, [&](int phase, int step, const Unit& x) {
        if (!wait_inputs(a, phase, step, x, abort)) return false;
        ptx::fence_proxy_async();    // the acquires above before the tensor copies
        asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(ptx::smem_u32(&sm.units_ready)), "r"(++units) : "memory");
        return true;
      });
    }
    __syncwarp();
  } else if (warp >= kFirstEpilogueWarp) {
    const int index = warp - kFirstEpilogueWarp;
    const int quarter = warp % 4, part = index / 4;
    uint32_t parity = 0;             // of the slot's barriers
    for_units(true, [&](int phase, int step, const Unit& x) {
      const Acc in{tmem + acc * kBlock + part * kWarpCols + (static_cast<uint32_t>(quarter) << 21),
                   &sm.acc_full[acc], acc_phase, ptx::map_to_rank(ptx::smem_u32(&sm.acc_empty[acc]), 0), abort,
                   static_cast<int>(rank) * kEpilogueWarps + index, slots + slot_offset(index), sm.piece[index],
                   &sm.units_done[index], own + part * kWarpCols * 4, &sm.own_full,
                   ptx::map_to_rank(ptx::smem_u32(&sm.a_full), 0)};
      const Place at = place_of(phase, x, rank, index);
      next_acc();
      return phase == kGram ? epilogue_square<kGram>(maps, a, step, x, at, in, parity)
             : phase == kPoly ? epilogue_square<kPoly>(maps, a, step, x, at, in, parity)
                              : epilogue_update(maps, a, step, x, at, in, parity);
    });
    if (lane == 0) ptx::bulk_wait();
  }

  // ---- end: nothing of the pair may be in flight when it leaves
  if (__syncthreads_or(*abort)) {
    if (warp == 1 && rank == 0 && lane == 0) {
      ptx::mma_commit_pair(&sm.drained);
      for (uint32_t n = 0; n < (1u << 22) && !ptx::mbar_try_wait_cluster(&sm.drained, 0); ++n) {}
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

// [batch][outer][ld] fp16 with r columns used, in boxes of box_cols x box_rows, swizzled by their
// rows' bytes; with `rest`, of this array and of one `rest` bytes behind it.
cudaError_t encode(CUtensorMap* map, void* p, const OrthoShape& sh, int64_t outer, int box_cols, int box_rows, size_t rest) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(sh.r), static_cast<cuuint64_t>(outer),
                              static_cast<cuuint64_t>(sh.batch), 2};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(sh.ld * 2), static_cast<cuuint64_t>(sh.ld * outer * 2), rest};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1, 2};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rest ? 4 : 3, p, dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
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
  const int64_t nr = sh.blocks_r, nc = sh.blocks_c;
  in.counters = reinterpret_cast<int*>(ws + L.counters);
  in.num_counters = static_cast<int>(sh.counters());

  OrthoMaps maps;
  cudaError_t e = cudaSuccess;
  auto add = [&](CUtensorMap* map, size_t at, int64_t outer, int box_cols, int box_rows, size_t rest = 0) {
    if (e == cudaSuccess) e = encode(map, ws + at, sh, outer, box_cols, box_rows, rest);
  };
  for (int i = 0; i < 2; ++i) {
    add(&maps.xt[i], L.xt[i], sh.c, 64, 64);
    add(&maps.x_strip[i], L.xt[i], sh.c, kStrip, 32, L.xl - L.xt[i]);
    add(&maps.a[i], L.a[i], sh.r, 64, 64);
    add(&maps.a_piece[i], L.a[i], sh.r, kPiece, 32);
  }
  add(&maps.b, L.b, sh.r, 64, 64);
  add(&maps.b_piece, L.b, sh.r, kPiece, 32);
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
  for (int i = 0; i < 2; ++i) {
    a.a[i] = reinterpret_cast<__half*>(ws + L.a[i]);
    a.diag_a[i] = reinterpret_cast<float*>(ws + L.diag_a[i]);
  }
  a.b = reinterpret_cast<__half*>(ws + L.b);
  a.diag_b = reinterpret_cast<float*>(ws + L.diag_b);
  a.out = static_cast<__nv_bfloat16*>(q.out);
  a.out_batch = q.out_batch_stride;
  a.out_row = q.out_row_stride;
  a.out_tall = q.out_tall;
  a.header = in.header;
  a.ready = in.counters;
  a.arrived = in.counters + sh.batch * 3 * nr;
  a.partial = reinterpret_cast<float*>(ws + L.partial);
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (g_pairs[dev] < 1) return cudaErrorLaunchOutOfResources;
  a.split = ortho_split(sh.batch * sh.square_blocks(), sh.c, g_pairs[dev]);

  const unsigned batch = static_cast<unsigned>(sh.batch);
  const int64_t tiles = (sh.cols + 63) / 64 * ((sh.rows + 63) / 64);
  in.tiles_of_block = static_cast<int>((tiles * sh.batch + 2 * kScaleBlocks * g_pairs[dev] - 1) / (2 * kScaleBlocks * g_pairs[dev]));
  ortho_norm_kernel<<<dim3(sh.norm_blocks, batch), 32 * kNormWarps, 0, stream>>>(in);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  {
    // may start while the norm kernel runs; it waits for it before it needs the norm
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((tiles + in.tiles_of_block - 1) / in.tiles_of_block, batch);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, ortho_scale_kernel, in)) != cudaSuccess) return e;
  }

  const int64_t most = sh.batch * std::max(nr * nc, nr * (nr + 1) / 2 * a.split);
  const int pairs = static_cast<int>(std::min<int64_t>(most, g_pairs[dev]));
  a.fused = nr == 1 && a.split == 1;
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
