// The host side of the orthogonalised update's launches on a made-up device: the library's own
// source, with the runtime calls that it makes answered here.  Reads lines of
//
//     pairs batch rows cols
//
// (pairs of CTAs that the device holds at once) and prints for each
//
//     code blocks parts units most
//
// the returned code, the steps kernel's blocks, the parts of the inner dimension of X X^T, the
// units of that phase, and the parts that the workspace has room for (blocks .. 0 without a launch).
#include "ewg_orthogonalize.cu"

#include <cstdio>

namespace {
int g_held = 0;
int g_blocks = 0;
ewg::OrthoArgs g_args;
}  // namespace

#ifndef __CUDA_ARCH__      // (the compiler's device pass has some of these already)
namespace {
CUresult encode_nothing(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                        const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                        CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {

cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* found) {
  *fn = reinterpret_cast<void*>(encode_nothing);
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* clusters, const void*, const cudaLaunchConfig_t*) {
  *clusters = g_held;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void** args) {
  if (cfg->attrs->id == cudaLaunchAttributeCooperative) {
    g_blocks = cfg->gridDim.x;
    g_args = *static_cast<const ewg::OrthoArgs*>(args[1]);
  }
  return cudaSuccess;
}

}  // extern "C"
#endif

int main() {
  long long batch, rows, cols;
  while (std::scanf("%d %lld %lld %lld", &g_held, &batch, &rows, &cols) == 4) {
    g_blocks = 0;
    g_args = {};
    if (ewg::prepare_orthogonalize() != cudaSuccess) return 1;
    ewg::OrthoCall q{};
    q.shape = ewg::make_ortho_shape(batch, rows, cols);
    q.steps = 5;
    const int code = ewg::launch_orthogonalize(q, nullptr);
    const int64_t blocks = q.shape.batch * q.shape.square_blocks();
    std::printf("%d %d %d %lld %lld\n", code, g_blocks, g_args.split, static_cast<long long>(blocks) * g_args.split,
                static_cast<long long>(q.shape.split));
    std::fflush(stdout);
  }
  return 0;
}
