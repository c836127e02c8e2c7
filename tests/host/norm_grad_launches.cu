// The host side of layer norm's gradient on a made-up device: the library's own source, with the runtime
// calls that it makes answered here.  Reads lines of
//
//     sms rows hidden bf16 lead
//
// (the device's SMs; rows begin `lead` elements behind 16 bytes) and prints for each
//
//     code blocks parts room
//
// the returned code, the first kernel's blocks, the shares that the joining kernel adds up (0: it is not
// launched), and the shares that the workspace has room for.
#include "ewg_layer_norm.cu"

#include <cstdio>

#ifndef __CUDA_ARCH__      // (the compiler's device pass has some of these already)
namespace {
int g_sms = 0, g_blocks = 0, g_parts = 0;
}

extern "C" {
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* clusters, const void*, const cudaLaunchConfig_t* cfg) {
  *clusters = g_sms / cfg->attrs->val.clusterDim.x;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* kernel, void** args) {
  if (kernel == reinterpret_cast<const void*>(ewg::norm_grad_join_kernel)) g_parts = static_cast<const ewg::NormGradArgs*>(args[0])->parts;
  else g_blocks = cfg->gridDim.x;
  return cudaSuccess;
}
}  // extern "C"

int main() {
  int rows, hidden, bf16, lead, dev = 0;
  while (std::scanf("%d %d %d %d %d", &g_sms, &rows, &hidden, &bf16, &lead) == 5) {
    g_blocks = g_parts = 0;
    ewg::NormGradArgs a{};
    char* const p = reinterpret_cast<char*>(uintptr_t(1) << 40) + lead * (bf16 ? 2 : 4);     // (nothing is read there)
    a.grad = a.x = p;
    a.grad_x = p;
    a.grad_stride = a.x_stride = a.grad_x_stride = a.H = hidden;
    a.weight_main_grad = a.bias_main_grad = p;
    a.partial = reinterpret_cast<float*>(uintptr_t(1) << 41);
    a.n = rows;
    a.parts = ewg::make_norm_grad_layout(rows, hidden).parts;
    a.dev = dev++;                                       // (a device of its own: what it holds is asked once)
    a.num_sms = g_sms;
    const int room = a.parts, code = ewg::launch_norm_grad(a, bf16, nullptr);
    std::printf("%d %d %d %d\n", code, g_blocks, g_parts, room);
    std::fflush(stdout);
  }
  return 0;
}
#endif
