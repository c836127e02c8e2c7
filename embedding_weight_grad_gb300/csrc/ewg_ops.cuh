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

cudaError_t launch_logprobs(const LogprobsArgs& a, bool bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_logprobs_grad(const LogprobsGradArgs& a, bool bf16, cudaStream_t stream);

// ---- orthogonalised update

constexpr int kOrthoMaxSide = 16384;      // of the smaller side
constexpr int kOrthoMaxLong = 1 << 20;    // of the larger side
constexpr int kNormBlocks = 304;          // blocks summing the squares of one matrix, at most

// One call's sizes: matrices [rows, cols]; r the smaller side, c the larger; `tall` when the
// rows are more than the columns (the steps then work on the transpose).
struct OrthoShape {
  int64_t batch, rows, cols;
  int64_t r, c, ld;                       // ld: r rounded up to 16, the pitch of every buffer
  int norm_blocks;
  bool tall;
};

struct OrthoLayout {
  size_t header, barrier, norm, diag_a, diag_b, xt[2], xl, a, b, total;
};

inline OrthoShape make_ortho_shape(int64_t batch, int64_t rows, int64_t cols) {
  OrthoShape s{};
  s.batch = batch;
  s.rows = rows;
  s.cols = cols;
  s.tall = rows > cols;
  s.r = s.tall ? cols : rows;
  s.c = s.tall ? rows : cols;
  s.ld = (s.r + 15) / 16 * 16;
  // a block (8 warps of 1024 elements) sums 16384 elements or more
  const int64_t want = (s.r * s.c + 16383) / 16384;
  s.norm_blocks = static_cast<int>(want < kNormBlocks ? want : kNormBlocks);
  return s;
}

inline OrthoLayout make_ortho_layout(const OrthoShape& s) {
  OrthoLayout L{};
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += (static_cast<size_t>(bytes) + 255) / 256 * 256;
    return at;
  };
  L.header = take(256);
  L.barrier = take(256);
  L.norm = take(s.batch * s.norm_blocks * 8);
  L.diag_a = take(s.batch * s.ld * 4);
  L.diag_b = take(s.batch * s.ld * 4);
  L.xt[0] = take(s.batch * s.c * s.ld * 2);
  L.xt[1] = take(s.batch * s.c * s.ld * 2);
  L.xl = take(s.batch * s.c * s.ld * 2);
  L.a = take(s.batch * s.r * s.ld * 2);
  L.b = take(s.batch * s.r * s.ld * 2);
  L.total = off;
  return L;
}

struct OrthoCall {
  OrthoShape shape;
  const void* grad;
  bool grad_bf16;
  int64_t grad_batch_stride, grad_row_stride;   // elements
  void* out;                                    // bf16
  int64_t out_batch_stride, out_row_stride;
  int steps;
  float a, b, c;
  void* workspace;
};

cudaError_t prepare_orthogonalize();   // once per device, before the first launch
cudaError_t launch_orthogonalize(const OrthoCall& call, cudaStream_t stream);

}  // namespace ewg
