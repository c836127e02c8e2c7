// Arguments and launchers of the operators between the vocabulary's ends and the optimiser:
// layer norm with its gradient, and AdamW over many tensors.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace ewg {

// ---- layer norm

struct NormArgs {
  const void* x;
  long long x_stride;        // elements
  const void* weight;        // [H] of bf16 or fp32, or null
  const void* bias;
  int weight_bf16;
  int n, H;
  float eps;
  float inv_h;               // 1 / H
  void* out;
  long long out_stride;
  float* mean;               // [n] each, or both null
  float* rstd;
  int dev, num_sms;
  int period;                // rows whose places in 16 bytes differ (set by the launcher)
};

struct NormGradArgs {
  const void* grad;
  long long grad_stride;     // elements
  const void* x;
  long long x_stride;
  const float* mean;         // [n] each
  const float* rstd;
  const void* weight;        // [H] of bf16 or fp32, or null
  int weight_bf16;
  int n, H;
  float inv_h;
  void* grad_x;
  long long grad_x_stride;
  void* weight_main_grad;    // [H] of bf16 or fp32, or null
  void* bias_main_grad;
  int main_grad_bf16;
  float2* row_sums;          // [n]: avg(u) and avg(u n), for rows of more than kNormHeld elements
  float* partial;            // [parts][2][H]: shares of the sums over the rows
  int parts;                 // shares of the rows
  int dev, num_sms;
  int period;                // rows whose places in 16 bytes differ (set by the launcher)
};

struct NormGradLayout {
  size_t row_sums, partial, total;
  int parts;
};

constexpr int kNormHeld = 65536;      // elements of a row that the gradient goes through once, at most
constexpr int kNormParts = 152;       // shares of the rows, at most
constexpr int kNormPartRows = 2;     // rows of a share, at least, where that leaves several

inline NormGradLayout make_norm_grad_layout(int64_t n, int64_t H) {
  NormGradLayout L{};
  const int64_t want = (n + kNormPartRows - 1) / kNormPartRows;
  L.parts = static_cast<int>(want < kNormParts ? want : kNormParts);
  L.row_sums = 0;
  L.partial = H > kNormHeld ? (static_cast<size_t>(n) * sizeof(float2) + 255) / 256 * 256 : 0;
  L.total = L.partial + (static_cast<size_t>(L.parts) * 2 * H * sizeof(float) + 255) / 256 * 256;
  return L;
}

cudaError_t launch_norm(const NormArgs& a, bool bf16, cudaStream_t stream);
cudaError_t launch_norm_grad(const NormGradArgs& a, bool bf16, cudaStream_t stream);

// ---- AdamW

constexpr int kAdamwBlock = 256;      // elements that share the scales of 8-bit states: a warp's
constexpr int kAdamwTile = 2048;      // elements that a block of 8 warps takes at a time

struct AdamwEntry {
  void* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  float2* scales;
  void* copy;
  long long count;
  float weight_decay;
  int first_tile;            // of its launch
  int flags;                 // kAdamw...
  int reserved;
};
enum {
  kAdamwParamBf16 = 1,
  kAdamwGradBf16 = 2,
  kAdamwAligned = 4          // every array is aligned to eight of its elements
};

// What a launch carries as its argument: the entries of up to this many tensors, of 32764 bytes that
// an argument may have.
constexpr int kAdamwEntries = 400;
constexpr int kAdamwFew = 48;          // entries of the smaller of two arguments

struct AdamwHyper {
  long long step;
  const long long* step_ptr;           // read in step's place where not null, and so on
  float lr;
  float grad_scale;
  const float* lr_ptr;
  const float* grad_scale_ptr;
  float beta1, rest1, log_beta1;       // rest: 1 - beta
  float beta2, rest2, log_beta2;
  float eps;
};

// A plan: this, then its entries, of which every kAdamwEntries are a launch.
struct AdamwPlan {
  unsigned long long magic;
  int device;
  int state_bits;
  long long entries;                   // tensors that are not empty
  long long bytes;
};
constexpr unsigned long long kAdamwMagic = 0x6577675f6164616dull;

cudaError_t launch_adamw(const AdamwEntry* entries, int num, int state_bits, const AdamwHyper& h, int num_sms,
                         cudaStream_t stream);

}  // namespace ewg
