// The C entry points on a made-up device on which the set-up of the orthogonalised update fails:
// the library's own entry points, with the runtime's calls and the launchers answered here.  Prints the
// entry points' codes with the set-up failing, then the last one's with it working.
#include <cstdio>

#include "ewg.h"
#include "ewg_internal.cuh"
#include "ewg_ops.cuh"

#ifndef __CUDA_ARCH__      // (the compiler's device pass has some of these already)
namespace {
bool g_fails = true;
}

namespace ewg {
cudaError_t prepare_kernels() { return cudaSuccess; }
cudaError_t prepare_orthogonalize() { return g_fails ? cudaErrorNotSupported : cudaSuccess; }
cudaError_t launch_plan(const PlanArgs&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_apply(const ApplyArgs&, int, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_logprobs(const LogprobsArgs&, bool, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_logprobs_grad(const LogprobsGradArgs&, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_orthogonalize(const OrthoCall&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_orthogonalize_small(const OrthoCall&, int, cudaStream_t) { return cudaSuccess; }
}  // namespace ewg

extern "C" {
cudaError_t cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int) {
  *value = 152;
  return cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* at, const void*) {
  at->type = cudaMemoryTypeDevice;
  at->device = 0;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "error"; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t*, unsigned) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t*, unsigned) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
}  // extern "C"

namespace {
template <typename T = void>
T* at(int i) {                       // addresses 1 GiB apart, which nothing looks behind
  return reinterpret_cast<T*>(static_cast<uintptr_t>(i) << 30);
}

int orthogonalize(int64_t rows, int64_t cols) {
  return ewg_orthogonalize(at(1), EWG_FP32, 1, rows, cols, rows * cols, cols, at(2), rows * cols, cols, 5, 3.4445f, -4.775f,
                           2.0315f, at(3), ewg_orthogonalize_workspace_bytes(1, rows, cols), nullptr);
}
}  // namespace

int main() {
  const int64_t n = 4096, V = 1000, H = 256;
  const int can = ewg_can_accumulate(at(1), EWG_INT64, n, at(2), EWG_BF16, H, at(3), EWG_FP32, V, H, H);
  const int accumulate = ewg_accumulate(at(1), EWG_INT64, n, at(2), EWG_BF16, H, at(3), EWG_FP32, V, H, H, at(4),
                                        ewg_workspace_bytes(n, H), nullptr);
  const int logprobs = ewg_token_logprobs(at(1), EWG_BF16, V, at(2), EWG_INT64, n, V, 1.0f, 0, at<float>(3), at<float>(4),
                                          at<float>(5), at<float>(6), nullptr, nullptr, nullptr, 0, nullptr);
  const int small = orthogonalize(8, 8), large = orthogonalize(300, 300);
  g_fails = false;
  std::printf("%d %d %d %d %d %d\n", can, accumulate, logprobs, small, large, orthogonalize(300, 300));
  return 0;
}
#endif
