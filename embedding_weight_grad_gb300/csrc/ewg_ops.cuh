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
constexpr int kNormBlocks = 304;          // blocks summing squares, at most, if the matrices are not more

// Smaller sides up to the first go without the tensor cores, and up to the second where the larger
// side is not long (48 x 2048: 101 us, with them 111; 48 x 7168: 138 and 111).
constexpr int kOrthoSmall = 32, kOrthoSmallShort = 48, kOrthoShort = 4096;
constexpr int kOrthoBlock = 256;          // side of the blocks the products are computed in
constexpr int kOrthoWarps = 16;           // epilogue warps of a block

// One call's sizes: matrices [rows, cols]; r the smaller side, c the larger; `tall` when the
// rows are more than the columns (the steps then work on the transpose).
struct OrthoShape {
  int64_t batch, rows, cols;
  int64_t r, c, ld;                       // ld: r rounded up to 16, the pitch of every buffer
  int64_t blocks_r, blocks_c;
  int norm_blocks;
  int split;                              // parts of the inner dimension of X X^T
  int small_parts;                        // shares of the larger side, where the smaller one is small
  bool tall;

  bool small() const { return r <= kOrthoSmall || (r <= kOrthoSmallShort && c <= kOrthoShort); }
  int64_t square_blocks() const { return blocks_r * (blocks_r + 1) / 2; }
  // counters of the steps kernel for one matrix
  int64_t counters() const {
    return 3 * blocks_r + (split > 1 ? square_blocks() * kOrthoWarps : 0);
  }
  int64_t partial_floats() const {
    return split > 1 ? batch * square_blocks() * split * kOrthoBlock * kOrthoBlock : 0;
  }
};

struct OrthoLayout {
  size_t header, counters, norm, diag_a[2], diag_b, xt[2], xl, a[2], b, partial, total;
  size_t small_gram, small_exponents, small_m, small_factors, small_x;
};

// Parts of the inner dimension `inner` of X X^T for `units` blocks: as many as leave no more units than
// `pairs`, each of at least kOrthoPartMin; fewer pairs never give more parts.  The workspace is laid
// out for kOrthoPairs, and a launch splits for the pairs that run at once where those are
// fewer: parts wait for one another.  Adding the parts up takes about 8 us, and
// 64 of the inner dimension 0.3 us, so that shorter ones than kOrthoSplitMin stay whole (2048 in
// two parts: 20 us instead of 15; 4097 in four: 15 instead of 23).  (A A has too many blocks for a
// split wherever its inner dimension is that long: 136 of them at 4096.)
constexpr int64_t kOrthoPairs = 76;
constexpr int64_t kOrthoPartMin = 1024;
constexpr int64_t kOrthoSplitMin = 4096;
inline int ortho_split(int64_t units, int64_t inner, int64_t pairs = kOrthoPairs) {
  int64_t parts = (pairs < kOrthoPairs ? pairs : kOrthoPairs) / units;
  if (parts > inner / kOrthoPartMin) parts = inner / kOrthoPartMin;
  if (parts <= 1 || inner < kOrthoSplitMin) return 1;
  // no empty part: `per` inner blocks of 64 each
  const int64_t blocks = (inner + 63) / 64, per = (blocks + parts - 1) / parts;
  return static_cast<int>((blocks + per - 1) / per);
}

inline OrthoShape make_ortho_shape(int64_t batch, int64_t rows, int64_t cols) {
  OrthoShape s{};
  s.batch = batch;
  s.rows = rows;
  s.cols = cols;
  s.tall = rows > cols;
  s.r = s.tall ? cols : rows;
  s.c = s.tall ? rows : cols;
  s.ld = (s.r + 15) / 16 * 16;
  s.blocks_r = (s.r + kOrthoBlock - 1) / kOrthoBlock;
  s.blocks_c = (s.c + kOrthoBlock - 1) / kOrthoBlock;
  // a block (8 warps of 1024 elements) sums 16384 elements or more, and the blocks of all
  // matrices run at once
  const int64_t want = (s.r * s.c + 16383) / 16384;
  const int64_t most = batch < kNormBlocks ? kNormBlocks / batch : 1;
  s.norm_blocks = static_cast<int>(want < most ? want : most);
  // 32 shares of 64 (which one block adds up), and more once they are of 16 times that
  const int64_t tiles = (s.c + 63) / 64, shares = tiles / 16 < 32 ? 32 : tiles / 16 < 152 ? tiles / 16 : 152;
  s.small_parts = static_cast<int>(tiles < shares ? tiles : shares);
  s.split = ortho_split(batch * s.square_blocks(), s.c);
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
  if (s.small()) {
    L.small_gram = take(s.batch * s.small_parts * s.r * s.r * 4);
    L.small_exponents = take(s.batch * s.small_parts * 4);
    L.small_m = take(s.batch * s.r * s.r * 4);
    L.small_factors = take(s.batch * 8);
    L.small_x = take(s.batch * s.c * s.r * 4);
    L.total = off;
    return L;
  }
  L.counters = take(s.batch * s.counters() * 4);
  L.norm = take(s.batch * s.norm_blocks * 8);
  for (int i = 0; i < 2; ++i) L.diag_a[i] = take(s.batch * s.ld * 4);
  L.diag_b = take(s.batch * s.ld * 4);
  for (int i = 0; i < 2; ++i) L.xt[i] = take(s.batch * s.c * s.ld * 2);
  L.xl = take(s.batch * s.c * s.ld * 2);
  for (int i = 0; i < 2; ++i) L.a[i] = take(s.batch * s.r * s.ld * 2);
  L.b = take(s.batch * s.r * s.ld * 2);
  L.partial = take(s.partial_floats() * 4);
  L.total = off;
  return L;
}

struct OrthoCall {
  OrthoShape shape;
  const void* grad;
  bool grad_bf16;
  int64_t grad_batch_stride, grad_row_stride;   // elements
  void* out;                                    // bf16
  bool out_tall;                                // out is [larger side][smaller side]
  int64_t out_batch_stride, out_row_stride;
  int steps;
  float a, b, c;
  void* workspace;
};

cudaError_t prepare_orthogonalize();   // once per device, before the first launch
cudaError_t launch_orthogonalize(const OrthoCall& call, cudaStream_t stream);
cudaError_t launch_orthogonalize_small(const OrthoCall& call, int num_sms, cudaStream_t stream);

}  // namespace ewg
