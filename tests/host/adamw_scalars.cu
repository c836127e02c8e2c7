// Steps whose numbers lie on the device, on a made-up device: the library's own entry points, with the
// runtime's calls and the launchers answered here.  Addresses are made up too: nothing is read there.
// Prints, for plans in 32 and in 8 bits, a line for each place of a scalar:
//
//     bits array where code
//
// array 0 to 5: param, grad, exp_avg, exp_avg_sq, scales, copy of the last tensor; where: 0 its first bytes,
// 1 its last, 2 just before it, 3 just behind; the code of the call with lr there (step for array 6: its
// 8 bytes across the param's end).
#include <cstdio>
#include <vector>

#include "ewg.h"
#include "ewg_internal.cuh"
#include "ewg_ops.cuh"
#include "ewg_train.cuh"

#ifndef __CUDA_ARCH__      // (the compiler's device pass has some of these already)
namespace ewg {
cudaError_t prepare_kernels() { return cudaSuccess; }
cudaError_t prepare_orthogonalize() { return cudaSuccess; }
cudaError_t launch_plan(const PlanArgs&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_apply(const ApplyArgs&, int, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_norm(const NormArgs&, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_norm_grad(const NormGradArgs&, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_adamw(const AdamwEntry*, int, int, const AdamwHyper&, int, cudaStream_t) { return cudaSuccess; }
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
cudaError_t cudaStreamCreateWithFlags(cudaStream_t*, unsigned) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
}  // extern "C"

namespace {
constexpr int kTensors = 403;
constexpr int64_t kCount = 1000;

// Array k of tensor i: 8192 bytes apart, 64 KiB from tensor to tensor.
char* place(int i, int k) { return reinterpret_cast<char*>(0x700000000000ull + i * 65536ull + 8192 * k); }

void run(int bits) {
  std::vector<ewg_adamw_tensor> tensors(kTensors);
  const int64_t state = bits / 8;
  for (int i = 0; i < kTensors; ++i) {
    tensors[i] = {place(i, 0), place(i, 1), place(i, 2), place(i, 3),
                  bits == 8 ? reinterpret_cast<float*>(place(i, 4)) : nullptr, place(i, 5), kCount, 0.1, EWG_FP32, EWG_FP32};
  }
  std::vector<char> plan(ewg_adamw_plan_bytes(kTensors));
  if (ewg_adamw_plan(tensors.data(), kTensors, bits, plan.data(), plan.size())) std::printf("no plan: %s\n", ewg_last_error());
  const int64_t bytes[6] = {4 * kCount, 4 * kCount, state * kCount, state * kCount, bits == 8 ? 32 : 0, 2 * kCount};
  auto step = [&](const void* step_at, const void* lr_at) {
    return ewg_adamw_step(plan.data(), plan.size(), 1, static_cast<const int64_t*>(step_at), 1e-3, static_cast<const float*>(lr_at),
                          0.9, 0.999, 1e-8, 1.0, nullptr, nullptr);
  };
  for (int k = 0; k < 6; ++k)
    for (int where = 0; where < 4; ++where) {
      char* const p = place(kTensors - 1, k);
      char* const at = where == 0 ? p : where == 1 ? p + bytes[k] - 4 : where == 2 ? p - 4 : p + bytes[k];
      std::printf("%d %d %d %d\n", bits, k, where, step(nullptr, at));
    }
  char* const end = place(0, 0) + 4 * kCount;
  std::printf("%d 6 0 %d\n", bits, step(end - 8, nullptr));
  std::printf("%d 6 3 %d\n", bits, step(end, nullptr));
}
}  // namespace

int main() {
  run(32);
  run(8);
  return 0;
}
#endif
