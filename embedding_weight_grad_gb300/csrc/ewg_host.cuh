// Host-side helpers shared by the entry points: errors, device memory checks, spans.
#pragma once

#include <cstdint>
#include <string>

#include <cuda_runtime.h>

#include "ewg.h"
#include "ewg_internal.cuh"

namespace ewg {
namespace host {

inline int fail(int code, const std::string& msg) {
  set_last_error(msg.c_str());
  return code;
}

inline int cuda_fail(cudaError_t e, const char* what) {
  return fail(EWG_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Index and SM count of the current device; configures the kernels once per device.
int current_device(int* dev, int* num_sms);

// Configures the steps kernel of the orthogonalised update on the current device, `dev`, once.
// (Apart from the rest: what fails here stops no other call.)
int prepare_orthogonalize_on(int dev);

inline bool on_device(const void* p, int dev) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();  // clear the sticky-free error of a foreign pointer
    return false;
  }
  return (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) && at.device == dev;
}

inline size_t elem_size(int dtype) {
  switch (dtype) {
    case EWG_INT32: return 4;
    case EWG_INT64: return 8;
    case EWG_BF16: return 2;
    case EWG_FP32: return 4;
    default: return 0;
  }
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Range {
  uintptr_t lo, hi;
};

inline Range span(const void* p, int64_t rows, int64_t cols, int64_t row_stride, size_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  const uintptr_t bytes = rows > 0 ? (static_cast<uintptr_t>(rows - 1) * row_stride + cols) * es : 0;
  return {lo, lo + bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace host
}  // namespace ewg
