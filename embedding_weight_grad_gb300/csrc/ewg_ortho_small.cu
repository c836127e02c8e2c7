// Newton-Schulz steps of matrices with a small side (OrthoShape::small).
//
// Steps are polynomials of A0 = X0 X0^T, r x r, so X is only needed at the ends of some of them:
//
//     A0 = X0 X0^T                             (of G, divided by its trace, |G|^2)
//     each step: P = a + b A + c A^2,  M <- P M,  A <- P^2 A          from M = 1
//     X = M X0                                 (M G / |G|)
//
// with everything in fp32: on so few directions the fp16 roundings of the tensor cores' operands
// do not average out (a 4 x 2 matrix was off by 1.2e-2, its rounding to bf16 being 1.7e-3).  A
// has the squares of the singular values, and its roundings, 2^-24 of the largest, are much of
// the square of a small one; so X is formed, and A anew, after every kRound steps, when small
// singular values have grown by a^2 = 12.  (With all steps in one go a singular value of 3e-3
// of the largest, which the steps take to about 1, would come out with an error of 1e-2.)
//
// The kernels: sums of outer products over shares of the long side; the steps of a round in one
// block's shared memory; the product with M, which also sums the next round's outer products.
// Seven launches for five steps, each bound by latency for short matrices, and for long ones by the
// arithmetic of the products with the long side.  8 x 8 takes 16 us (57 by the tensor cores'
// steps), 32 x 32 25 (55), 48 x 48 51 (57), 7168 x 32 62 (103), 16 x 100000 137 (288), 1000
// matrices of 16 x 16 47 (692).  The same for sides of 64 takes 68 us at 64 x 64 (57) and 185 at
// 64 x 7168 (110), and there the roundings average out.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "ewg.h"
#include "ewg_internal.cuh"
#include "ewg_ops.cuh"
#include "ewg_ptx.cuh"

namespace ewg {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTile = 64;            // of the long side
constexpr int kThreads = 256;
constexpr int kRound = 2;

struct SmallArgs {
  const void* grad;                  // G, or X of the rounds before
  int bf16, tall;
  long long batch_stride, row_stride;
  int first;                         // it is G
  int r, c;
  int parts;                         // shares of the long side
  float* gram;                       // [batch][parts][r][r], scaled: times 2^(2 (127 - exponents))
  int* exponents;                    // [batch][parts]
  float* m;                          // [batch][r][r]
  float* factors;                    // [batch][2]: 1 / |G| as a power of two and a number
  int steps;                         // of the round
  float ca, cb, cc;
  __nv_bfloat16* out;
  int out_tall;
  long long out_batch, out_row;
  float* x;                          // [batch][c][r]: X after a round
  Header* header;
};

// Element i of the short side, j of the long one.
__device__ __forceinline__ long long at_of(bool tall, long long row, int i, int j) {
  return tall ? j * row + i : i * row + j;
}

// A thread's elements of a tile of the matrix: kR x 64 elements over 256 threads, neighbours in
// memory to neighbouring threads.
template <int kR>
struct Tile {
  static constexpr int kEach = kR * kTile / kThreads;
  static __device__ __forceinline__ void place(const SmallArgs& a, int u, int& i, int& j) {
    const int e = u * kThreads + threadIdx.x;
    i = a.tall ? e % kR : e / kTile;
    j = a.tall ? e / kR : e % kTile;
  }
  static __device__ __forceinline__ void load(const SmallArgs& a, int j0, float (&v)[kEach]) {
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      int i, j;
      place(a, u, i, j);
      const long long at = blockIdx.y * a.batch_stride + at_of(a.tall, a.row_stride, i, j0 + j);
      v[u] = i >= a.r || j0 + j >= a.c ? 0.0f
             : a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.grad)[at])
                      : static_cast<const float*>(a.grad)[at];
    }
  }
  static __device__ __forceinline__ void store(const SmallArgs& a, const float (&v)[kEach], float by,
                                               float (&tile)[kTile][kR + 1]) {
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      int i, j;
      place(a, u, i, j);
      tile[j][i] = v[u] * by;
    }
  }
};

// acc += the outer products of a tile's columns.
template <int kR>
__device__ __forceinline__ void add_outer(const float (&tile)[kTile][kR + 1], float (&acc)[kR / 16][kR / 16]) {
  constexpr int kP = kR / 16;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll 4
  for (int j = 0; j < kTile; ++j) {
    float x[kP], y[kP];
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      x[p] = tile[j][ty + 16 * p];
      y[p] = tile[j][tx + 16 * p];
    }
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int q = 0; q < kP; ++q) acc[p][q] = fmaf(x[p], y[q], acc[p][q]);
  }
}

// A block's sums, times 2^(2 (127 - e)), as share blockIdx.x of matrix blockIdx.y.
template <int kR>
__device__ __forceinline__ void store_share(const SmallArgs& a, const float (&acc)[kR / 16][kR / 16], int e) {
  constexpr int kP = kR / 16;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const long long share = static_cast<long long>(blockIdx.y) * a.parts + blockIdx.x;
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int q = 0; q < kP; ++q) {
      const int i = ty + 16 * p, j = tx + 16 * q;
      if (i < a.r && j < a.r) a.gram[(share * a.r + i) * a.r + j] = acc[p][q];
    }
  if (threadIdx.x == 0) a.exponents[share] = e;
}

// Share blockIdx.x of matrix blockIdx.y.  Tiles are scaled by the power of two that brings the
// largest element so far near 1, so that no square leaves fp32's range.
template <int kR>
__global__ void __launch_bounds__(kThreads) small_gram_kernel(const SmallArgs a) {
  constexpr int kP = kR / 16;
  __shared__ float tile[kTile][kR + 1];
  __shared__ uint32_t largest[kThreads / 32];
  ptx::pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.header->status = kStatusOk;
  float acc[kP][kP] = {};
  int e = 0;                         // the sums are times 2^(2 (127 - e))
  const int tiles = (a.c + kTile - 1) / kTile;
  float v[Tile<kR>::kEach];
  int t = blockIdx.x;
  if (t < tiles) Tile<kR>::load(a, t * kTile, v);
  for (; t < tiles; t += a.parts) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < Tile<kR>::kEach; ++u) m = max(m, __float_as_uint(v[u]) & 0x7fffffffu);
    m = __reduce_max_sync(kAll, m);
    if (threadIdx.x % 32 == 0) largest[threadIdx.x / 32] = m;
    __syncthreads();                 // (and the tile before has been read)
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, largest[w]);
    const int em = min(static_cast<int>(m >> 23), 253);
    if (em > e) {
      const float f = __uint_as_float(static_cast<uint32_t>(max(127 + e - em, 1)) << 23);   // 2^(e - em)
#pragma unroll
      for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int q = 0; q < kP; ++q) acc[p][q] *= f * f;
      e = em;
    }
    Tile<kR>::store(a, v, __uint_as_float(static_cast<uint32_t>(254 - e) << 23), tile);     // 2^(127 - e)
    __syncthreads();
    if (t + a.parts < tiles) Tile<kR>::load(a, (t + a.parts) * kTile, v);
    add_outer<kR>(tile, acc);
  }
  store_share<kR>(a, acc, e);
}

// In the steps kernel a thread has kP x kP neighbouring elements of each matrix; kP numbers of a
// row come from shared memory at once.
template <int kR>
using Square = float[kR][kR + 4];

template <int kP>
__device__ __forceinline__ void read_row(const float* from, float (&x)[kP]) {
  if constexpr (kP == 2) {
    const float2 v = *reinterpret_cast<const float2*>(from);
    x[0] = v.x;
    x[1] = v.y;
  } else {
#pragma unroll
    for (int p = 0; p < kP; ++p) x[p] = from[p];
  }
}

// acc = X Y of two matrices in shared memory; X is symmetric.
template <int kR>
__device__ __forceinline__ void product(const Square<kR>& x, const Square<kR>& y, float (&acc)[kR / 16][kR / 16]) {
  constexpr int kP = kR / 16;
  const int j0 = threadIdx.x % 16 * kP, i0 = threadIdx.x / 16 * kP;
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int q = 0; q < kP; ++q) acc[p][q] = 0.0f;
#pragma unroll 8
  for (int k = 0; k < kR; ++k) {
    float u[kP], w[kP];
    read_row<kP>(&x[k][i0], u);
    read_row<kP>(&y[k][j0], w);
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int q = 0; q < kP; ++q) acc[p][q] = fmaf(u[p], w[q], acc[p][q]);
  }
}

// The steps of matrix blockIdx.x.
template <int kR>
__global__ void __launch_bounds__(kThreads) small_steps_kernel(const SmallArgs a) {
  constexpr int kP = kR / 16;
  extern __shared__ __align__(16) float raw[];
  Square<kR>& A = reinterpret_cast<Square<kR>*>(raw)[0];
  Square<kR>& P = reinterpret_cast<Square<kR>*>(raw)[1];
  Square<kR>& M = reinterpret_cast<Square<kR>*>(raw)[2];
  __shared__ int most;
  const int j0 = threadIdx.x % 16 * kP, i0 = threadIdx.x / 16 * kP;
  const int z = blockIdx.x;
  ptx::pdl_launch_dependents();      // the next kernel's reads of G
  ptx::pdl_wait_prior_grid();
  const int* exponents = a.exponents + static_cast<long long>(z) * a.parts;
  const float* gram = a.gram + static_cast<long long>(z) * a.parts * a.r * a.r;
  if (threadIdx.x < 32) {
    int e = 0;
    for (int p = threadIdx.x; p < a.parts; p += 32) e = max(e, exponents[p]);
    e = __reduce_max_sync(kAll, e);
    if (threadIdx.x == 0) most = e;
  }
  __syncthreads();
  const int e = most;
  float acc[kP][kP] = {};
#pragma unroll 4
  for (int s = 0; s < a.parts; ++s) {
    const float f = __uint_as_float(static_cast<uint32_t>(max(127 + exponents[s] - e, 1)) << 23);
    const float f2 = f * f;
    const float* part = gram + static_cast<long long>(s) * a.r * a.r;
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const int i = i0 + p, j = j0 + q;
        if (i < a.r && j < a.r) acc[p][q] = fmaf(part[i * a.r + j], f2, acc[p][q]);
      }
  }
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int q = 0; q < kP; ++q) A[i0 + p][j0 + q] = acc[p][q];
  __syncthreads();
  float trace = 0.0f;
  for (int i = threadIdx.x % 32; i < kR; i += 32) trace += A[i][i];
#pragma unroll
  for (int d = 16; d; d /= 2) trace += __shfl_xor_sync(kAll, trace, d);
  if (threadIdx.x == 0) {            // 1 / |G| = f1 f2, f1 a power of two
    int e2 = 0;
    float f2 = a.first ? 0.0f : 1.0f;
    if (a.first && trace > 0.0f && isfinite(trace)) {
      f2 = frexpf(rsqrtf(trace), &e2);
      e2 += 127 - e;
      const int e1 = min(max(e2, -120), 120);
      f2 = ldexpf(f2, e2 - e1);
      e2 = e1;
    }
    a.factors[2 * z] = ldexpf(1.0f, e2);
    a.factors[2 * z + 1] = f2;
  }
  const float by = !a.first ? 1.0f : trace == 0.0f ? 0.0f : 1.0f / trace;      // a zero matrix stays zero
  const float none = isfinite(trace) ? 0.0f : NAN;           // and one with a NaN or an infinity is NaN
  __syncthreads();
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int q = 0; q < kP; ++q) {
      const int i = i0 + p, j = j0 + q;
      A[i][j] = acc[p][q] * by;
    }
  __syncthreads();
  for (int step = 0; step < a.steps; ++step) {
    product<kR>(A, A, acc);
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const int i = i0 + p, j = j0 + q;
        P[i][j] = fmaf(a.cc, acc[p][q], fmaf(a.cb, A[i][j], i == j ? a.ca : 0.0f));
      }
    __syncthreads();
    float next[kP][kP], half[kP][kP];
    if (step > 0) product<kR>(P, M, next);
    const bool more = step + 1 < a.steps;
    if (more) product<kR>(P, A, half);
    __syncthreads();                 // M and A have been read
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        M[i0 + p][j0 + q] = step > 0 ? next[p][q] : P[i0 + p][j0 + q] + none;
        if (more) A[i0 + p][j0 + q] = half[p][q];
      }
    __syncthreads();
    if (more) {
      product<kR>(P, A, acc);
      __syncthreads();
#pragma unroll
      for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int q = 0; q < kP; ++q) A[i0 + p][j0 + q] = acc[p][q];
      __syncthreads();
    }
  }
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int q = 0; q < kP; ++q) {
      const int i = i0 + p, j = j0 + q;
      if (i < a.r && j < a.r) a.m[(static_cast<long long>(z) * a.r + i) * a.r + j] = M[i][j];
    }
}

// X = M G / |G| of tiles blockIdx.x, + gridDim.x, ... of matrix blockIdx.y: rounded to out, or
// (kMid) to a.x, from which it may have come, with its outer products summed on the way.
template <int kR, bool kMid>
__global__ void __launch_bounds__(kThreads) small_apply_kernel(const SmallArgs a) {
  constexpr int kP = kR / 16, kQ = kTile / 16;
  __shared__ float tile[kTile][kR + 1];
  __shared__ float M[kR][kR + 1];
  // the fast index of a warp is out's: along the short side where it is tall (a.x is)
  const bool tall = kMid || a.out_tall;
  const int fast = threadIdx.x % 16, slow = threadIdx.x / 16;
  const int ti = tall ? fast : slow, tj = tall ? slow : fast;
  const int tiles = (a.c + kTile - 1) / kTile;
  int t = blockIdx.x;
  float v[Tile<kR>::kEach];
  ptx::pdl_launch_dependents();
  if (a.first) Tile<kR>::load(a, t * kTile, v);      // (a.x is still being written)
  ptx::pdl_wait_prior_grid();
  if (!a.first) Tile<kR>::load(a, t * kTile, v);
  const float f1 = a.factors[2 * blockIdx.y], f2 = a.factors[2 * blockIdx.y + 1];
  for (int x = threadIdx.x; x < kR * kR; x += kThreads) {
    const int i = x / kR, k = x % kR;
    M[k][i] = i < a.r && k < a.r ? a.m[(static_cast<long long>(blockIdx.y) * a.r + i) * a.r + k] : 0.0f;
  }
  float outer[kP][kP] = {};
  while (true) {
#pragma unroll
    for (int u = 0; u < Tile<kR>::kEach; ++u) v[u] *= f1;
    Tile<kR>::store(a, v, f2, tile);
    __syncthreads();
    const int j0 = t * kTile;
    t += gridDim.x;
    if (t < tiles) Tile<kR>::load(a, t * kTile, v);
    float acc[kP][kQ] = {};
#pragma unroll 4
    for (int k = 0; k < kR; ++k) {
      float m[kP], x[kQ];
#pragma unroll
      for (int p = 0; p < kP; ++p) m[p] = M[k][ti + 16 * p];
#pragma unroll
      for (int q = 0; q < kQ; ++q) x[q] = tile[tj + 16 * q][k];
#pragma unroll
      for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int q = 0; q < kQ; ++q) acc[p][q] = fmaf(m[p], x[q], acc[p][q]);
    }
    if constexpr (kMid) __syncthreads();              // the tile has been read
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const int i = ti + 16 * p, j = j0 + tj + 16 * q;
        if constexpr (kMid) tile[tj + 16 * q][i] = acc[p][q];       // (0 outside the matrix)
        if (i >= a.r || j >= a.c) continue;
        if constexpr (kMid) a.x[(static_cast<long long>(blockIdx.y) * a.c + j) * a.r + i] = acc[p][q];
        else a.out[blockIdx.y * a.out_batch + at_of(tall, a.out_row, i, j)] = __float2bfloat16_rn(acc[p][q]);
      }
    if constexpr (kMid) {
      __syncthreads();
      add_outer<kR>(tile, outer);
    }
    if (t >= tiles) break;
    __syncthreads();                 // the tile has been read
  }
  if constexpr (kMid) store_share<kR>(a, outer, 127);
}

template <int kR>
cudaError_t launch(SmallArgs a, int steps, int batch, int num_sms, cudaStream_t stream) {
  small_gram_kernel<kR><<<dim3(a.parts, batch), kThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;     // its start overlaps the kernel's before
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int tiles = (a.c + kTile - 1) / kTile;
  for (int done = 0; done < steps; done += kRound) {
    const bool last = done + kRound >= steps;
    a.steps = std::min(kRound, steps - done);
    cfg.gridDim = dim3(batch);
    cfg.dynamicSmemBytes = 3 * sizeof(Square<kR>);
    if ((e = cudaLaunchKernelEx(&cfg, small_steps_kernel<kR>, a)) != cudaSuccess) return e;
    cfg.dynamicSmemBytes = 0;
    if (last) {
      cfg.gridDim = dim3(std::min(tiles, std::max(1, 4 * num_sms / batch)), batch);
      return cudaLaunchKernelEx(&cfg, small_apply_kernel<kR, false>, a);
    }
    cfg.gridDim = dim3(a.parts, batch);
    if ((e = cudaLaunchKernelEx(&cfg, small_apply_kernel<kR, true>, a)) != cudaSuccess) return e;
    a.grad = a.x;
    a.bf16 = 0;
    a.tall = 1;
    a.batch_stride = static_cast<long long>(a.c) * a.r;
    a.row_stride = a.r;
    a.first = 0;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_orthogonalize_small(const OrthoCall& q, int num_sms, cudaStream_t stream) {
  const OrthoShape& sh = q.shape;
  const OrthoLayout L = make_ortho_layout(sh);
  char* ws = static_cast<char*>(q.workspace);
  SmallArgs a{};
  a.grad = q.grad;
  a.bf16 = q.grad_bf16;
  a.tall = sh.tall;
  a.batch_stride = q.grad_batch_stride;
  a.row_stride = q.grad_row_stride;
  a.r = static_cast<int>(sh.r);
  a.c = static_cast<int>(sh.c);
  a.parts = sh.small_parts;
  a.gram = reinterpret_cast<float*>(ws + L.small_gram);
  a.exponents = reinterpret_cast<int*>(ws + L.small_exponents);
  a.m = reinterpret_cast<float*>(ws + L.small_m);
  a.factors = reinterpret_cast<float*>(ws + L.small_factors);
  a.ca = q.a;
  a.cb = q.b;
  a.cc = q.c;
  a.first = 1;
  a.out_tall = q.out_tall;
  a.x = reinterpret_cast<float*>(ws + L.small_x);
  a.out = static_cast<__nv_bfloat16*>(q.out);
  a.out_batch = q.out_batch_stride;
  a.out_row = q.out_row_stride;
  a.header = reinterpret_cast<Header*>(ws + L.header);
  const int batch = static_cast<int>(sh.batch);
  return a.r <= 16   ? launch<16>(a, q.steps, batch, num_sms, stream)
         : a.r <= 32 ? launch<32>(a, q.steps, batch, num_sms, stream)
                     : launch<48>(a, q.steps, batch, num_sms, stream);
}

}  // namespace ewg
