// C ABI of layer norm, its gradient and AdamW: argument checks and launches.  The declarations
// and their contracts are in include/ewg.h.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "ewg.h"
#include "ewg_host.cuh"
#include "ewg_internal.cuh"
#include "ewg_train.cuh"

namespace {

using namespace ewg::host;

bool is_float(int dtype) { return dtype == EWG_BF16 || dtype == EWG_FP32; }

// eps is added in fp32, where 1 / eps has to be a number too (a subnormal one counts as 0 in some operations).
int check_eps(double eps) {
  if (eps == 0 || (eps >= 0x1p-126 && eps <= 0x1p126)) return EWG_OK;
  return fail(EWG_ERR_UNSUPPORTED, "eps must be 0 or in [2^-126, 2^126]");
}

int check_norm_sizes(int64_t rows, int64_t hidden) {
  if (rows < 0 || rows > INT32_MAX) return fail(EWG_ERR_UNSUPPORTED, "rows outside [0, 2^31)");
  if (hidden < 1 || hidden > EWG_MAX_HIDDEN) return fail(EWG_ERR_UNSUPPORTED, "hidden outside [1, EWG_MAX_HIDDEN]");
  return EWG_OK;
}

// A [rows][hidden] array of rows: its checks and its bytes.
int check_rows(const char* name, const void* p, int dtype, int64_t rows, int64_t hidden, int64_t stride,
               DeviceMemory& mem, Array* out) {
  // byte offsets stay within 62 bits
  if ((rows > 1 && stride < hidden) || stride < 0 || stride > (int64_t(1) << 62) / (rows * 4))
    return fail(EWG_ERR_UNSUPPORTED, std::string(name) + " row stride must be >= hidden");
  const size_t es = elem_size(dtype);
  *out = {name, p, span(p, rows, hidden, stride, es)};
  return check_array(*out, es, mem);
}

// An array that may be left out.
int check_optional(const Array& a, size_t align, DeviceMemory& mem) { return a.p ? check_array(a, align, mem) : EWG_OK; }

bool same_rows(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int64_t rows) {
  return a == b && (rows == 1 || a_stride == b_stride);
}

// Whether a step of the entry's tensor writes memory of `r`.
bool writes(const ewg::AdamwEntry& e, int state_bits, const Range& r) {
  const int64_t n = e.count, blocks = (n + ewg::kAdamwBlock - 1) / ewg::kAdamwBlock, state = state_bits / 8;
  auto in = [&](const void* p, int64_t count, size_t size) { return p && overlap(span(p, 1, count, count, size), r); };
  return in(e.param, n, e.flags & ewg::kAdamwParamBf16 ? 2 : 4) || in(e.exp_avg, n, state) || in(e.exp_avg_sq, n, state) ||
         in(e.scales, blocks, 8) || in(e.copy, n, 2);
}

int plan_adamw(const ewg_adamw_tensor* tensors, int64_t num, int state_bits, void* plan, size_t plan_bytes) {
  int dev = 0, sms = 0;
  int rc = current_device(&dev, &sms);
  if (rc) return rc;
  if (state_bits != 8 && state_bits != 32) return fail(EWG_ERR_UNSUPPORTED, "state_bits must be 8 or 32");
  const size_t need = ewg_adamw_plan_bytes(num);
  if (need == 0) return fail(EWG_ERR_UNSUPPORTED, "num_tensors outside [0, 2^20]");
  if (!plan || !aligned(plan, 8) || plan_bytes < need || (num > 0 && !tensors))
    return fail(EWG_ERR_INVALID, "plan or tensors null, or plan misaligned or smaller than ewg_adamw_plan_bytes(num_tensors)");
  DeviceMemory mem(dev);
  struct Used {
    Range r;
    bool written;
    int64_t tensor;
  };
  std::vector<Used> used;
  std::vector<ewg::AdamwEntry> entries;
  used.reserve(6 * num);
  entries.reserve(num);
  int64_t tile = 0;
  for (int64_t i = 0; i < num; ++i) {
    const ewg_adamw_tensor& t = tensors[i];
    const std::string at = "tensor " + std::to_string(i) + ": ";
    auto refuse = [&](const char* why) { return fail(EWG_ERR_UNSUPPORTED, at + why); };
    if (!is_float(t.param_dtype) || !is_float(t.grad_dtype)) return refuse("param and grad must be bf16 or fp32");
    if (t.count < 0 || t.count > (int64_t(1) << 40)) return refuse("count outside [0, 2^40]");
    if (!(t.weight_decay >= 0) || !std::isfinite(static_cast<float>(t.weight_decay)))
      return refuse("weight_decay must be finite and >= 0");
    if (t.copy && t.param_dtype != EWG_FP32) return refuse("a copy needs an fp32 param");
    if ((state_bits == 8) != (t.scales != nullptr) && t.count > 0)
      return refuse("scales belong to states in 8 bits, and only to them");
    if (t.count == 0) continue;
    const int64_t n = t.count, blocks = (n + ewg::kAdamwBlock - 1) / ewg::kAdamwBlock;
    const size_t ps = elem_size(t.param_dtype), gs = elem_size(t.grad_dtype), ss = state_bits / 8;
    const struct {
      Array a;
      size_t align;
      bool written, optional;
    } arrays[6] = {{flat("param", t.param, n, ps), ps, true, false},
                   {flat("grad", t.grad, n, gs), gs, false, false},
                   {flat("exp_avg", t.exp_avg, n, ss), ss, true, false},
                   {flat("exp_avg_sq", t.exp_avg_sq, n, ss), ss, true, false},
                   {flat("scales", t.scales, blocks, 8), 8, true, true},
                   {flat("copy", t.copy, n, 2), 2, true, true}};
    for (const auto& x : arrays) {
      if (x.optional && !x.a.p) continue;
      if ((rc = check_array(x.a, x.align, mem))) return fail(rc, at + ewg_last_error());
      used.push_back({x.a.r, x.written, i});
    }
    ewg::AdamwEntry e{};
    e.param = t.param;
    e.grad = t.grad;
    e.exp_avg = t.exp_avg;
    e.exp_avg_sq = t.exp_avg_sq;
    e.scales = reinterpret_cast<float2*>(t.scales);
    e.copy = t.copy;
    e.count = n;
    e.weight_decay = static_cast<float>(t.weight_decay);
    if (entries.size() % ewg::kAdamwEntries == 0) tile = 0;
    const int64_t tiles = (n + ewg::kAdamwTile - 1) / ewg::kAdamwTile;
    if (tile + tiles > INT32_MAX) return refuse("too many elements in one plan");
    e.first_tile = static_cast<int>(tile);
    tile += tiles;
    e.flags = (t.param_dtype == EWG_BF16 ? ewg::kAdamwParamBf16 : 0) | (t.grad_dtype == EWG_BF16 ? ewg::kAdamwGradBf16 : 0);
    if (aligned(t.param, 8 * ps) && aligned(t.grad, 8 * gs) && aligned(t.exp_avg, 8 * ss) &&
        aligned(t.exp_avg_sq, 8 * ss) && aligned(t.copy, 16))
      e.flags |= ewg::kAdamwAligned;
    entries.push_back(e);
  }
  // by address: what is written may not begin before the end of anything, nor what is read
  // before the end of something written
  std::sort(used.begin(), used.end(), [](const Used& a, const Used& b) { return a.r.lo < b.r.lo; });
  const Used *last = nullptr, *last_written = nullptr;         // those that end last so far
  for (const Used& u : used) {
    const Used* before = u.written ? last : last_written;
    if (before && u.r.lo < before->r.hi)
      return fail(EWG_ERR_UNSUPPORTED, "memory of tensor " + std::to_string(u.tensor) + " overlaps memory of tensor " +
                                           std::to_string(before->tensor));
    if (!last || u.r.hi > last->r.hi) last = &u;
    if (u.written && (!last_written || u.r.hi > last_written->r.hi)) last_written = &u;
  }
  ewg::AdamwPlan head{};
  head.magic = ewg::kAdamwMagic;
  head.device = dev;
  head.state_bits = state_bits;
  head.entries = static_cast<long long>(entries.size());
  head.bytes = static_cast<long long>(need);
  std::memcpy(plan, &head, sizeof head);
  if (!entries.empty())
    std::memcpy(static_cast<char*>(plan) + sizeof head, entries.data(), entries.size() * sizeof entries[0]);
  return EWG_OK;
}

}  // namespace

extern "C" {

int ewg_layer_norm(const void* x, int x_dtype, int64_t rows, int64_t hidden, int64_t row_stride, const void* weight,
                   const void* bias, int weight_dtype, double eps, void* out, int64_t out_row_stride, float* mean,
                   float* rstd, void* stream) {
  ewg::set_last_error("");
  int dev = 0, sms = 0;
  int rc = current_device(&dev, &sms);
  if (rc) return rc;
  DeviceMemory mem(dev);
  if (!is_float(x_dtype)) return fail(EWG_ERR_UNSUPPORTED, "x must be bf16 or fp32");
  if ((weight || bias) && !is_float(weight_dtype)) return fail(EWG_ERR_UNSUPPORTED, "weight and bias must be bf16 or fp32");
  if ((rc = check_eps(eps))) return rc;
  if ((rc = check_norm_sizes(rows, hidden))) return rc;
  if (rows == 0) return EWG_OK;
  if (!mean != !rstd) return fail(EWG_ERR_UNSUPPORTED, "mean and rstd belong together");
  const size_t ws = weight || bias ? elem_size(weight_dtype) : 0;
  Array in[3] = {{}, flat("weight", weight, hidden, ws), flat("bias", bias, hidden, ws)};
  Array res[3] = {{}, flat("mean", mean, rows, 4), flat("rstd", rstd, rows, 4)};
  if ((rc = check_rows("x", x, x_dtype, rows, hidden, row_stride, mem, &in[0])) ||
      (rc = check_optional(in[1], ws, mem)) || (rc = check_optional(in[2], ws, mem)) ||
      (rc = check_rows("out", out, x_dtype, rows, hidden, out_row_stride, mem, &res[0])) ||
      (rc = check_optional(res[1], 4, mem)) || (rc = check_optional(res[2], 4, mem)))
    return rc;
  const bool in_place = same_rows(x, row_stride, out, out_row_stride, rows);
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j)
      if (!(i == 0 && j == 0 && in_place) && (rc = check_apart(res[i], in[j]))) return rc;
    for (int j = 0; j < i; ++j)
      if ((rc = check_apart(res[i], res[j]))) return rc;
  }
  ewg::NormArgs a{};
  a.x = x;
  a.x_stride = rows > 1 ? row_stride : hidden;
  a.weight = weight;
  a.bias = bias;
  a.weight_bf16 = weight_dtype == EWG_BF16;
  a.n = static_cast<int>(rows);
  a.H = static_cast<int>(hidden);
  a.eps = static_cast<float>(eps);
  a.inv_h = static_cast<float>(1.0 / static_cast<double>(hidden));
  a.out = out;
  a.out_stride = rows > 1 ? out_row_stride : hidden;
  a.mean = mean;
  a.rstd = rstd;
  a.dev = dev;
  a.num_sms = sms;
  const cudaError_t e = ewg::launch_norm(a, x_dtype == EWG_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EWG_OK : cuda_fail(e, "layer norm launch");
}

size_t ewg_layer_norm_workspace_bytes(int64_t rows, int64_t hidden) {
  if (rows < 0 || rows > INT32_MAX || hidden < 1 || hidden > EWG_MAX_HIDDEN) return 0;
  return ewg::make_norm_grad_layout(rows > 0 ? rows : 1, hidden).total;
}

int ewg_layer_norm_backward(const void* grad, int64_t grad_row_stride, const void* x, int64_t x_row_stride, int dtype,
                            int64_t rows, int64_t hidden, const float* mean, const float* rstd, const void* weight,
                            int weight_dtype, void* grad_x, int64_t grad_x_row_stride, void* weight_main_grad,
                            void* bias_main_grad, int main_grad_dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  ewg::set_last_error("");
  int dev = 0, sms = 0;
  int rc = current_device(&dev, &sms);
  if (rc) return rc;
  DeviceMemory mem(dev);
  if (!is_float(dtype)) return fail(EWG_ERR_UNSUPPORTED, "grad and x must be bf16 or fp32");
  if (weight && !is_float(weight_dtype)) return fail(EWG_ERR_UNSUPPORTED, "weight must be bf16 or fp32");
  const bool sums = weight_main_grad || bias_main_grad;
  if (sums && !is_float(main_grad_dtype)) return fail(EWG_ERR_UNSUPPORTED, "main_grads must be bf16 or fp32");
  if ((rc = check_norm_sizes(rows, hidden))) return rc;
  if (rows == 0) return EWG_OK;
  const size_t ws = weight ? elem_size(weight_dtype) : 0, ms = sums ? elem_size(main_grad_dtype) : 0;
  const ewg::NormGradLayout L = ewg::make_norm_grad_layout(rows, hidden);
  Array in[5] = {{}, {}, flat("mean", mean, rows, 4), flat("rstd", rstd, rows, 4), flat("weight", weight, hidden, ws)};
  Array res[4] = {{}, flat("weight_main_grad", weight_main_grad, hidden, ms),
                  flat("bias_main_grad", bias_main_grad, hidden, ms),
                  flat("workspace", workspace, static_cast<int64_t>(L.total), 1)};
  if ((rc = check_rows("grad", grad, dtype, rows, hidden, grad_row_stride, mem, &in[0])) ||
      (rc = check_rows("x", x, dtype, rows, hidden, x_row_stride, mem, &in[1])) || (rc = check_array(in[2], 4, mem)) ||
      (rc = check_array(in[3], 4, mem)) || (rc = check_optional(in[4], ws, mem)) ||
      (rc = check_rows("grad_x", grad_x, dtype, rows, hidden, grad_x_row_stride, mem, &res[0])) ||
      (rc = check_optional(res[1], ms, mem)) || (rc = check_optional(res[2], ms, mem)))
    return rc;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < L.total || !mem.has(workspace))
    return fail(EWG_ERR_INVALID, "workspace null, misaligned, not on the device or smaller than "
                                 "ewg_layer_norm_workspace_bytes(rows, hidden)");
  const bool over[2] = {same_rows(grad, grad_row_stride, grad_x, grad_x_row_stride, rows),
                        same_rows(x, x_row_stride, grad_x, grad_x_row_stride, rows)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 5; ++j)
      if (!(i == 0 && j < 2 && over[j]) && (rc = check_apart(res[i], in[j]))) return rc;
    for (int j = 0; j < i; ++j)
      if ((rc = check_apart(res[i], res[j]))) return rc;
  }
  ewg::NormGradArgs a{};
  a.grad = grad;
  a.grad_stride = rows > 1 ? grad_row_stride : hidden;
  a.x = x;
  a.x_stride = rows > 1 ? x_row_stride : hidden;
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.weight_bf16 = weight_dtype == EWG_BF16;
  a.n = static_cast<int>(rows);
  a.H = static_cast<int>(hidden);
  a.inv_h = static_cast<float>(1.0 / static_cast<double>(hidden));
  a.grad_x = grad_x;
  a.grad_x_stride = rows > 1 ? grad_x_row_stride : hidden;
  a.weight_main_grad = weight_main_grad;
  a.bias_main_grad = bias_main_grad;
  a.main_grad_bf16 = main_grad_dtype == EWG_BF16;
  a.row_sums = reinterpret_cast<float2*>(static_cast<char*>(workspace) + L.row_sums);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.partial);
  a.parts = L.parts;
  a.dev = dev;
  a.num_sms = sms;
  const cudaError_t e = ewg::launch_norm_grad(a, dtype == EWG_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EWG_OK : cuda_fail(e, "layer norm gradient launch");
}

size_t ewg_adamw_plan_bytes(int64_t num_tensors) {
  if (num_tensors < 0 || num_tensors > (int64_t(1) << 20)) return 0;
  return sizeof(ewg::AdamwPlan) + static_cast<size_t>(num_tensors) * sizeof(ewg::AdamwEntry);
}

int ewg_adamw_plan(const ewg_adamw_tensor* tensors, int64_t num_tensors, int state_bits, void* plan, size_t plan_bytes) {
  try {
    ewg::set_last_error("");
    return plan_adamw(tensors, num_tensors, state_bits, plan, plan_bytes);
  } catch (const std::bad_alloc&) {
    return EWG_ERR_INVALID;        // no host memory for the check, nor for a message
  }
}

int ewg_adamw_step(const void* plan, size_t plan_bytes, int64_t step, const int64_t* step_on_device, double lr,
                   const float* lr_on_device, double beta1, double beta2, double eps, double grad_scale,
                   const float* grad_scale_on_device, void* stream) {
  ewg::set_last_error("");
  int dev = 0, sms = 0;
  int rc = current_device(&dev, &sms);
  if (rc) return rc;
  ewg::AdamwPlan head{};
  if (!plan || !aligned(plan, 8) || plan_bytes < sizeof head) return fail(EWG_ERR_INVALID, "plan null, misaligned or too small");
  std::memcpy(&head, plan, sizeof head);
  if (head.magic != ewg::kAdamwMagic || plan_bytes < sizeof head + head.entries * sizeof(ewg::AdamwEntry))
    return fail(EWG_ERR_INVALID, "plan was not made by ewg_adamw_plan, or is cut off");
  if (head.device != dev) return fail(EWG_ERR_INVALID, "plan was made on another device than the current one");
  auto fine = [](double v) { return std::isfinite(static_cast<float>(v)); };
  if (!step_on_device && step < 1) return fail(EWG_ERR_UNSUPPORTED, "step must be >= 1");
  if (!lr_on_device && !(fine(lr) && lr >= 0)) return fail(EWG_ERR_UNSUPPORTED, "lr must be finite and >= 0");
  if (!grad_scale_on_device && !fine(grad_scale)) return fail(EWG_ERR_UNSUPPORTED, "grad_scale must be finite");
  for (double b : {beta1, beta2})
    if (!(b >= 0 && static_cast<float>(b) < 1.0f)) return fail(EWG_ERR_UNSUPPORTED, "betas must be in [0, 1)");
  if ((rc = check_eps(eps))) return rc;
  DeviceMemory mem(dev);
  const auto* entries = reinterpret_cast<const ewg::AdamwEntry*>(static_cast<const char*>(plan) + sizeof head);
  // blocks read these when they start, others have written by then
  for (const Array& scalar : {flat("step", step_on_device, 1, 8), flat("lr", lr_on_device, 1, 4),
                              flat("grad_scale", grad_scale_on_device, 1, 4)}) {
    if (!scalar.p) continue;
    if ((rc = check_array(scalar, scalar.r.hi - scalar.r.lo, mem))) return rc;
    for (int64_t i = 0; i < head.entries; ++i)
      if (writes(entries[i], head.state_bits, scalar.r))
        return fail(EWG_ERR_UNSUPPORTED, std::string(scalar.name) + " lies in memory that is written by the step");
  }
  ewg::AdamwHyper h{};
  h.step = step;
  h.step_ptr = reinterpret_cast<const long long*>(step_on_device);
  h.lr = static_cast<float>(lr);
  h.lr_ptr = lr_on_device;
  h.grad_scale = static_cast<float>(grad_scale);
  h.grad_scale_ptr = grad_scale_on_device;
  h.beta1 = static_cast<float>(beta1);
  h.rest1 = static_cast<float>(1.0 - beta1);
  h.log_beta1 = static_cast<float>(std::log(beta1));
  h.beta2 = static_cast<float>(beta2);
  h.rest2 = static_cast<float>(1.0 - beta2);
  h.log_beta2 = static_cast<float>(std::log(beta2));
  h.eps = static_cast<float>(eps);
  for (int64_t i = 0; i < head.entries; i += ewg::kAdamwEntries) {
    const int num = static_cast<int>(std::min<int64_t>(ewg::kAdamwEntries, head.entries - i));
    const cudaError_t e = ewg::launch_adamw(entries + i, num, head.state_bits, h, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "AdamW launch");
  }
  return EWG_OK;
}

}  // extern "C"
