// Layer norm of rows, and its gradient.
//
// Per row x[0..H), avg over the row:
//
//     mean = avg(x)     rstd = 1 / sqrt(avg((x - mean)^2) + eps)     out = (x - mean) rstd w + b
//
// and with n = (x - mean) rstd, u = g w:
//
//     dx = rstd (u - avg(u) - n avg(u n))     dw_j = sum over rows of g n     db_j = sum over rows of g
#include <cuda_bf16.h>

#include "ewg_train.cuh"

namespace ewg {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }

// Element j of a vector of bf16 or fp32.
__device__ __forceinline__ float element(const void* p, int bf16, int j) {
  return bf16 ? load(static_cast<const __nv_bfloat16*>(p) + j) : load(static_cast<const float*>(p) + j);
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

// A block goes through one row three times.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) norm_kernel(NormArgs a) {
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  T* out = static_cast<T*>(a.out) + row * a.out_stride;
  float2 s = make_float2(0.0f, 0.0f);
  for (int j = threadIdx.x; j < a.H; j += kRowThreads) s.x += load(x + j);
  const float near = block_sum<kRowThreads>(s).x * a.inv_h;
  s = make_float2(0.0f, 0.0f);
  for (int j = threadIdx.x; j < a.H; j += kRowThreads) {
    const float d = load(x + j) - near;
    s.x += d;
    s.y = fmaf(d, d, s.y);
  }
  s = block_sum<kRowThreads>(s);
  // `near` is the mean but for its rounding, which the deviations' own mean shows
  const float rest = s.x * a.inv_h;
  const float var = fmaxf(fmaf(-rest, rest, s.y * a.inv_h), 0.0f);
  const float rstd = s.y != s.y ? s.y : 1.0f / sqrtf(var + a.eps);
  if (threadIdx.x == 0) {
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

// avg(u) and avg(u n) of a row, a block for each.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) norm_grad_rows_kernel(NormGradArgs a) {
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* g = static_cast<const T*>(a.grad) + row * a.grad_stride;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float2 s = make_float2(0.0f, 0.0f);
  for (int j = threadIdx.x; j < a.H; j += kRowThreads) {
    const float u = load(g + j) * (a.weight ? element(a.weight, a.weight_bf16, j) : 1.0f);
    s.x += u;
    s.y = fmaf(u, (load(x + j) - mean) * rstd, s.y);
  }
  s = block_sum<kRowThreads>(s);
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

// The shares of a column's sums, added up in order and to the main_grad.
__global__ void __launch_bounds__(kRowThreads) norm_grad_join_kernel(NormGradArgs a) {
  const int j = blockIdx.x * kRowThreads + threadIdx.x;
  void* to = blockIdx.y == 0 ? a.weight_main_grad : a.bias_main_grad;
  if (j >= a.H || !to) return;
  float s = 0.0f;
  for (int part = 0; part < a.parts; ++part) s += a.partial[(static_cast<long long>(part) * 2 + blockIdx.y) * a.H + j];
  if (a.main_grad_bf16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(to) + j;
    store(p, load(p) + s);
  } else {
    static_cast<float*>(to)[j] += s;
  }
}

template <typename T>
cudaError_t grad(const NormGradArgs& a, cudaStream_t stream) {
  const unsigned columns = (a.H + kRowThreads - 1) / kRowThreads;
  norm_grad_rows_kernel<T><<<a.n, kRowThreads, 0, stream>>>(a);
  norm_grad_columns_kernel<T><<<dim3(columns, a.parts), kRowThreads, 0, stream>>>(a);
  if (a.weight_main_grad || a.bias_main_grad) norm_grad_join_kernel<<<dim3(columns, 2), kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, bool bf16, cudaStream_t stream) {
  if (bf16) norm_kernel<__nv_bfloat16><<<a.n, kRowThreads, 0, stream>>>(a);
  else norm_kernel<float><<<a.n, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_grad(const NormGradArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? grad<__nv_bfloat16>(a, stream) : grad<float>(a, stream);
}

}  // namespace ewg
