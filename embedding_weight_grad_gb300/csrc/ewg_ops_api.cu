// C ABI of the operators beside the embedding gradient: argument checks and launches.
// The declarations and their contracts are in include/ewg.h.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "ewg.h"
#include "ewg_host.cuh"
#include "ewg_internal.cuh"
#include "ewg_ops.cuh"

namespace {

using namespace ewg::host;

// An array of an entry point's arguments: its bytes, and its name for messages.
struct Array {
  const char* name;
  const void* p;
  Range r;
};

Array flat(const char* name, const void* p, int64_t count, size_t es) {
  return {name, p, span(p, 1, count, count, es)};
}

// Whether pointers are memory of the current device, asking the runtime once for each 2 MiB
// page: device memory is mapped in pages of that size, which nothing else shares, and a call's
// small arrays mostly come from one.
class DeviceMemory {
 public:
  explicit DeviceMemory(int dev) : dev_(dev) {}
  bool has(const void* p) {
    const uintptr_t page = reinterpret_cast<uintptr_t>(p) >> 21;
    for (int i = 0; i < known_; ++i)
      if (pages_[i] == page) return true;
    if (!on_device(p, dev_)) return false;
    if (known_ < 8) pages_[known_++] = page;
    return true;
  }

 private:
  int dev_, known_ = 0;
  uintptr_t pages_[8];
};

int check_array(const Array& a, size_t align, DeviceMemory& mem) {
  if (!a.p || !aligned(a.p, align))
    return fail(EWG_ERR_UNSUPPORTED, std::string(a.name) + " is null or misaligned");
  if (!mem.has(a.p))
    return fail(EWG_ERR_UNSUPPORTED, std::string(a.name) + " is not memory of the current device");
  return EWG_OK;
}

int check_apart(const Array& a, const Array& b) {
  if (a.p && b.p && overlap(a.r, b.r))
    return fail(EWG_ERR_UNSUPPORTED, std::string(a.name) + " overlaps " + b.name);
  return EWG_OK;
}

constexpr size_t kStatusBytes = sizeof(ewg::Header);

int check_status_workspace(void* ws, size_t bytes, DeviceMemory& mem) {
  if (!ws) return EWG_OK;
  if (!aligned(ws, 256) || bytes < kStatusBytes || !mem.has(ws))
    return fail(EWG_ERR_INVALID, "workspace must be 256 bytes of the current device, 256-byte aligned");
  return EWG_OK;
}

int* status_word(void* ws) { return ws ? &static_cast<ewg::Header*>(ws)->status : nullptr; }

int check_logits(const void* logits, int dtype, int64_t row_stride, const void* targets, int targets_dtype,
                 int64_t n, int64_t V, float scale, DeviceMemory& mem) {
  if (dtype != EWG_BF16 && dtype != EWG_FP32) return fail(EWG_ERR_UNSUPPORTED, "logits must be bf16 or fp32");
  if (targets_dtype != EWG_INT32 && targets_dtype != EWG_INT64)
    return fail(EWG_ERR_UNSUPPORTED, "targets must be int32 or int64");
  if (n < 0 || n > INT32_MAX) return fail(EWG_ERR_UNSUPPORTED, "num_tokens outside [0, 2^31)");
  if (V < 1 || V >= INT32_MAX - 63) return fail(EWG_ERR_UNSUPPORTED, "vocab outside [1, 2^31 - 64)");
  if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(EWG_ERR_UNSUPPORTED, "scale must be finite and positive");
  if (n == 0) return EWG_OK;
  if (n > 1 && row_stride < V) return fail(EWG_ERR_UNSUPPORTED, "logits row stride must be >= vocab");
  // byte offsets stay within 62 bits
  if (row_stride < 0 || row_stride > (int64_t(1) << 62) / (n * 4))
    return fail(EWG_ERR_UNSUPPORTED, "logits row stride is too large");
  int rc = check_array({"logits", logits, {}}, elem_size(dtype), mem);
  if (rc) return rc;
  return check_array({"targets", targets, {}}, elem_size(targets_dtype), mem);
}

bool ortho_sizes_ok(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 1 || batch > 65535 || rows < 1 || cols < 1) return false;
  const int64_t lo = rows < cols ? rows : cols, hi = rows < cols ? cols : rows;
  if (lo > ewg::kOrthoMaxSide || hi > ewg::kOrthoMaxLong) return false;
  return batch * ((lo + 255) / 256) * ((hi + 255) / 256) < (int64_t(1) << 30);   // blocks of a phase
}

// A [batch][rows][cols] array of matrices: its checks and its bytes.
int ortho_array(const char* name, const void* p, size_t es, int64_t batch, int64_t rows, int64_t cols,
                int64_t batch_stride, int64_t row_stride, DeviceMemory& mem, Array* out) {
  const int64_t most = int64_t(1) << 40;
  if ((rows > 1 && row_stride < cols) || row_stride < 0 || row_stride > most || batch_stride < 0 || batch_stride > most)
    return fail(EWG_ERR_UNSUPPORTED, std::string(name) + " row stride must be >= cols, strides below 2^40");
  const int64_t one = (rows - 1) * row_stride + cols;
  if (batch > 1 && batch_stride < one)
    return fail(EWG_ERR_UNSUPPORTED, std::string(name) + " matrices overlap");
  *out = {name, p, span(p, batch, one, batch_stride, es)};
  return check_array(*out, es, mem);
}

// scale log2(e), at most the largest number: above, an exponent of 0 times it would be NaN, and
// any other is clamped by the kernels all the same.
float log2_scale(float scale) {
  return static_cast<float>(std::fmin(static_cast<double>(scale) * 1.4426950408889634074, FLT_MAX));
}

// ewg_orthogonalize, or with `transposed` ewg_orthogonalize_transposed.
int orthogonalize(bool transposed, const void* grad, int grad_dtype, int64_t batch, int64_t rows, int64_t cols,
                  int64_t grad_batch_stride, int64_t grad_row_stride, void* out, int64_t out_batch_stride,
                  int64_t out_row_stride, int steps, float a, float b, float c, void* workspace, size_t workspace_bytes,
                  void* stream) {
  ewg::set_last_error("");
  int dev = 0, sms = 0;
  int rc = current_device(&dev, &sms);
  if (rc) return rc;
  DeviceMemory mem(dev);
  if (grad_dtype != EWG_BF16 && grad_dtype != EWG_FP32) return fail(EWG_ERR_UNSUPPORTED, "grad must be bf16 or fp32");
  if (steps < 1 || steps > EWG_MAX_ORTHO_STEPS)
    return fail(EWG_ERR_UNSUPPORTED, "steps outside [1, EWG_MAX_ORTHO_STEPS]");
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
    return fail(EWG_ERR_UNSUPPORTED, "the coefficients must be finite");
  if (batch == 0 && rows > 0 && cols > 0) return EWG_OK;
  if (!ortho_sizes_ok(batch, rows, cols))
    return fail(EWG_ERR_UNSUPPORTED, "sizes: 0 <= batch <= 65535, 1 <= smaller side <= 16384, larger side <= 2^20, "
                                     "batch * ceil(rows / 256) * ceil(cols / 256) < 2^30");
  const size_t es = elem_size(grad_dtype);
  Array in, res;
  if ((rc = ortho_array("grad", grad, es, batch, rows, cols, grad_batch_stride, grad_row_stride, mem, &in)) ||
      (rc = ortho_array("out", out, 2, batch, transposed ? cols : rows, transposed ? rows : cols, out_batch_stride,
                        out_row_stride, mem, &res)))
    return rc;
  const ewg::OrthoShape shape = ewg::make_ortho_shape(batch, rows, cols);
  const size_t need = ewg::make_ortho_layout(shape).total;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need || !mem.has(workspace))
    return fail(EWG_ERR_INVALID, "workspace null, misaligned, not on the device or smaller than "
                                 "ewg_orthogonalize_workspace_bytes(batch, rows, cols)");
  const Array ws = flat("workspace", workspace, static_cast<int64_t>(need), 1);
  if ((rc = check_apart(res, in)) || (rc = check_apart(ws, in)) || (rc = check_apart(ws, res))) return rc;
  if (!shape.small() && (rc = prepare_orthogonalize_on(dev))) return rc;
  ewg::OrthoCall q{};
  q.shape = shape;
  q.grad = grad;
  q.grad_bf16 = grad_dtype == EWG_BF16;
  q.grad_batch_stride = grad_batch_stride;
  q.grad_row_stride = grad_row_stride;
  q.out = out;
  q.out_tall = shape.tall != transposed;
  q.out_batch_stride = out_batch_stride;
  q.out_row_stride = out_row_stride;
  q.steps = steps;
  q.a = a;
  q.b = b;
  q.c = c;
  q.workspace = workspace;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  cudaError_t e = shape.small() ? ewg::launch_orthogonalize_small(q, sms, on) : ewg::launch_orthogonalize(q, on);
  return e == cudaSuccess ? EWG_OK : cuda_fail(e, "orthogonalisation launch");
}

}  // namespace

extern "C" {

int ewg_token_logprobs(const void* logits, int logits_dtype, int64_t row_stride, const void* targets,
                       int targets_dtype, int64_t num_tokens, int64_t vocab, float scale, int top,
                       float* logprobs, float* entropy, float* row_max, float* log_sum, float* top_logprobs,
                       int64_t* top_ids, void* workspace, size_t workspace_bytes, void* stream) {
  ewg::set_last_error("");
  int dev = 0, sms = 0;
  int rc = current_device(&dev, &sms);
  if (rc) return rc;
  DeviceMemory mem(dev);
  if ((rc = check_logits(logits, logits_dtype, row_stride, targets, targets_dtype, num_tokens, vocab, scale, mem)))
    return rc;
  if (top < 0 || top > EWG_MAX_TOP || top > vocab)
    return fail(EWG_ERR_UNSUPPORTED, "top outside [0, min(vocab, EWG_MAX_TOP)]");
  if ((rc = check_status_workspace(workspace, workspace_bytes, mem))) return rc;
  if (num_tokens == 0) return EWG_OK;
  const int64_t n = num_tokens;
  const Array in[2] = {{"logits", logits, span(logits, n, vocab, row_stride, elem_size(logits_dtype))},
                       flat("targets", targets, n, elem_size(targets_dtype))};
  const Array out[7] = {flat("logprobs", logprobs, n, 4), flat("entropy", entropy, n, 4),
                        flat("row_max", row_max, n, 4), flat("log_sum", log_sum, n, 4),
                        flat("top_logprobs", top ? top_logprobs : nullptr, n * top, 4),
                        flat("top_ids", top ? top_ids : nullptr, n * top, 8),
                        flat("workspace", workspace, kStatusBytes, 1)};
  for (int i = 0; i < 7; ++i) {
    if ((i < 4 || (i < 6 && top)) && (rc = check_array(out[i], i == 5 ? 8 : 4, mem))) return rc;
    for (const Array& a : in)
      if ((rc = check_apart(out[i], a))) return rc;
    for (int j = 0; j < i; ++j)
      if ((rc = check_apart(out[i], out[j]))) return rc;
  }
  ewg::LogprobsArgs a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.targets = targets;
  a.targets_int64 = targets_dtype == EWG_INT64;
  a.n = static_cast<int>(n);
  a.V = static_cast<int>(vocab);
  a.scale = scale;
  a.scale_log2 = log2_scale(scale);
  a.top = top;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.row_max = row_max;
  a.log_sum = log_sum;
  a.top_logprobs = top_logprobs;
  a.top_ids = reinterpret_cast<long long*>(top_ids);
  a.status = status_word(workspace);
  cudaError_t e = ewg::launch_logprobs(a, logits_dtype == EWG_BF16, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EWG_OK : cuda_fail(e, "token log probabilities launch");
}

int ewg_token_logprobs_backward(const void* logits, int logits_dtype, int64_t row_stride, const void* targets,
                                int targets_dtype, int64_t num_tokens, int64_t vocab, float scale,
                                const float* row_max, const float* log_sum, const float* entropy,
                                const float* grad_logprobs, const float* grad_entropy, void* grad_logits,
                                int64_t grad_row_stride, void* workspace, size_t workspace_bytes, void* stream) {
  ewg::set_last_error("");
  int dev = 0, sms = 0;
  int rc = current_device(&dev, &sms);
  if (rc) return rc;
  DeviceMemory mem(dev);
  if ((rc = check_logits(logits, logits_dtype, row_stride, targets, targets_dtype, num_tokens, vocab, scale, mem)))
    return rc;
  if ((rc = check_status_workspace(workspace, workspace_bytes, mem))) return rc;
  if (num_tokens == 0) return EWG_OK;
  const int64_t n = num_tokens;
  const size_t es = elem_size(logits_dtype);
  if ((n > 1 && grad_row_stride < vocab) || grad_row_stride < 0 || grad_row_stride > (int64_t(1) << 62) / (n * 4))
    return fail(EWG_ERR_UNSUPPORTED, "grad_logits row stride must be >= vocab");
  if (n * (vocab / 1024 + 1) >= (int64_t(1) << 31))   // the kernel's items
    return fail(EWG_ERR_UNSUPPORTED, "num_tokens * (vocab / 1024 + 1) must stay below 2^31");
  if (grad_entropy && !entropy) return fail(EWG_ERR_UNSUPPORTED, "grad_entropy needs entropy");
  const Array in[7] = {{"logits", logits, span(logits, n, vocab, row_stride, es)},
                       flat("targets", targets, n, elem_size(targets_dtype)),
                       flat("row_max", row_max, n, 4), flat("log_sum", log_sum, n, 4),
                       flat("grad_logprobs", grad_logprobs, n, 4),
                       flat("entropy", grad_entropy ? entropy : nullptr, n, 4),
                       flat("grad_entropy", grad_entropy, n, 4)};
  const Array out{"grad_logits", grad_logits, span(grad_logits, n, vocab, grad_row_stride, es)};
  const Array ws = flat("workspace", workspace, kStatusBytes, 1);
  if ((rc = check_array(out, es, mem))) return rc;
  for (int i = 0; i < 7; ++i) {
    if (i >= 2 && (i < 5 || grad_entropy) && (rc = check_array(in[i], 4, mem))) return rc;
    const bool in_place = i == 0 && logits == grad_logits && (n == 1 || row_stride == grad_row_stride);
    if (!in_place && (rc = check_apart(out, in[i]))) return rc;
    if ((rc = check_apart(ws, in[i]))) return rc;
  }
  if ((rc = check_apart(ws, out))) return rc;
  ewg::LogprobsGradArgs a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.targets = targets;
  a.targets_int64 = targets_dtype == EWG_INT64;
  a.n = static_cast<int>(n);
  a.V = static_cast<int>(vocab);
  a.scale = scale;
  a.scale_log2 = log2_scale(scale);
  a.row_max = row_max;
  a.log_sum = log_sum;
  a.entropy = entropy;
  a.grad_logprobs = grad_logprobs;
  a.grad_entropy = grad_entropy;
  a.grad = grad_logits;
  a.grad_stride = grad_row_stride;
  a.status = status_word(workspace);
  cudaError_t e = ewg::launch_logprobs_grad(a, logits_dtype == EWG_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EWG_OK : cuda_fail(e, "token log probability gradient launch");
}

size_t ewg_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
  if (!ortho_sizes_ok(batch, rows, cols)) return 0;
  return ewg::make_ortho_layout(ewg::make_ortho_shape(batch, rows, cols)).total;
}

int ewg_orthogonalize(const void* grad, int grad_dtype, int64_t batch, int64_t rows, int64_t cols,
                      int64_t grad_batch_stride, int64_t grad_row_stride, void* out, int64_t out_batch_stride,
                      int64_t out_row_stride, int steps, float a, float b, float c, void* workspace,
                      size_t workspace_bytes, void* stream) {
  return orthogonalize(false, grad, grad_dtype, batch, rows, cols, grad_batch_stride, grad_row_stride, out,
                       out_batch_stride, out_row_stride, steps, a, b, c, workspace, workspace_bytes, stream);
}

int ewg_orthogonalize_transposed(const void* grad, int grad_dtype, int64_t batch, int64_t rows, int64_t cols,
                                 int64_t grad_batch_stride, int64_t grad_row_stride, void* out,
                                 int64_t out_batch_stride, int64_t out_row_stride, int steps, float a, float b, float c,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return orthogonalize(true, grad, grad_dtype, batch, rows, cols, grad_batch_stride, grad_row_stride, out,
                       out_batch_stride, out_row_stride, steps, a, b, c, workspace, workspace_bytes, stream);
}

}  // extern "C"
