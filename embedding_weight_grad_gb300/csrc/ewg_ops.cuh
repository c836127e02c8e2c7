// Arguments and launchers of the operators beside the embedding gradient: token log
// probabilities with their gradient, and the orthogonalised update.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace ewg {

struct LogprobsArgs {
  const void* logits;
  long long row_stride;      // elements
  const void* targets;
  int targets_int64;
  int n, V;
  float scale;
  float scale_log2;          // scale * log2(e)
  int top;                   // alternatives per row, 0..kMaxTop
  float* logprobs;           // [n] each
  float* entropy;
  float* row_max;
  float* log_sum;
  float* top_logprobs;       // [n, top]
  long long* top_ids;        // [n, top]
  int* status;               // device status word, or null
};

struct LogprobsGradArgs {
  const void* logits;
  long long row_stride;
  const void* targets;
  int targets_int64;
  int n, V;
  float scale;
  float scale_log2;
  const float* row_max;      // [n] each, as the forward pass left them
  const float* log_sum;
  const float* entropy;      // null without grad_entropy
  const float* grad_logprobs;
  const float* grad_entropy; // or null
  void* grad;                // [n, V], the logits' dtype
  long long grad_stride;
  int* status;
};

constexpr int kMaxTop = 32;  // a warp holds a row's best candidates one to a lane

cudaError_t prepare_logprobs();
cudaError_t launch_logprobs(const LogprobsArgs& a, bool bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_logprobs_grad(const LogprobsGradArgs& a, bool bf16, cudaStream_t stream);

}  // namespace ewg
