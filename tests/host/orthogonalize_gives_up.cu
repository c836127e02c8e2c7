// The bounded waits of the orthogonalised update's steps kernel, made to run out from the host: the library's
// own source with a wait limit of 50 ms.  Between the kernels that form the first X and the steps
// kernel, one of the counts that units wait for is set to a number far below what it can reach.
//
// Reads lines of
//
//     batch rows cols index
//
// (index of the count) and prints for each
//
//     status ms status_after differing
//
// the device status of the call with that count, how long it took, and of a call with the same workspace
// after it the status and the elements that differ from a call before.
#define EWG_ORTHO_WAIT_LIMIT 50000000ull

#include <cuda_runtime.h>

#include <chrono>
#include <cstdio>
#include <vector>

namespace {
int* g_spoil = nullptr;              // the count to set before the next steps kernel, once

template <typename... Params, typename... Args>
cudaError_t launch_spoilt(const cudaLaunchConfig_t* cfg, void (*kernel)(Params...), Args&&... args) {
  if (cfg->attrs->id == cudaLaunchAttributeCooperative && g_spoil) {
    cudaMemsetAsync(g_spoil, 0x80, sizeof(int), cfg->stream);
    g_spoil = nullptr;
  }
  return cudaLaunchKernelEx(cfg, kernel, static_cast<Args&&>(args)...);
}
}  // namespace

#define cudaLaunchKernelEx launch_spoilt
#include "ewg_orthogonalize.cu"
#undef cudaLaunchKernelEx

int main() {
  long long batch, rows, cols;
  int index;
  if (ewg::prepare_orthogonalize() != cudaSuccess) return 1;
  while (std::scanf("%lld %lld %lld %d", &batch, &rows, &cols, &index) == 4) {
    ewg::OrthoCall q{};
    q.shape = ewg::make_ortho_shape(batch, rows, cols);
    const ewg::OrthoLayout L = ewg::make_ortho_layout(q.shape);
    if (q.shape.small() || index >= batch * q.shape.counters()) return 1;
    const size_t n = batch * rows * cols;
    std::vector<float> g(n);
    uint32_t state = 1;
    for (float& x : g) x = static_cast<int>((state = state * 1664525u + 1013904223u) >> 8) * 0x1p-23f - 1.0f;
    float* grad;
    uint16_t* out;
    char* ws;
    if (cudaMalloc(&grad, n * 4) || cudaMalloc(&out, n * 2) || cudaMalloc(&ws, L.total)) return 1;
    cudaMemcpy(grad, g.data(), n * 4, cudaMemcpyHostToDevice);
    q.grad = grad;
    q.grad_batch_stride = q.out_batch_stride = rows * cols;
    q.grad_row_stride = q.out_row_stride = cols;
    q.out = out;
    q.out_tall = q.shape.tall;
    q.steps = 5;
    q.a = 3.4445f;
    q.b = -4.775f;
    q.c = 2.0315f;
    q.workspace = ws;
    auto call = [&](std::vector<uint16_t>* result, double* ms) {
      const auto start = std::chrono::steady_clock::now();
      if (ewg::launch_orthogonalize(q, nullptr) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return -1;
      if (ms) *ms = std::chrono::duration<double, std::milli>(std::chrono::steady_clock::now() - start).count();
      ewg::Header h;
      if (cudaMemcpy(&h, ws + L.header, sizeof h, cudaMemcpyDeviceToHost) != cudaSuccess) return -1;
      if (result) {
        result->resize(n);
        cudaMemcpy(result->data(), out, n * 2, cudaMemcpyDeviceToHost);
      }
      return static_cast<int>(h.status);
    };
    std::vector<uint16_t> before, after;
    double ms = 0.0;
    if (call(&before, nullptr) != 0) return 1;
    g_spoil = reinterpret_cast<int*>(ws + L.counters) + index;
    const int status = call(nullptr, &ms), status_after = call(&after, nullptr);
    size_t differing = 0;
    for (size_t i = 0; i < n; ++i) differing += before[i] != after[i];
    std::printf("%d %.1f %d %zu\n", status, ms, status_after, differing);
    std::fflush(stdout);
    cudaFree(grad);
    cudaFree(out);
    cudaFree(ws);
  }
  return 0;
}
