// One AdamW step of many tensors, the moments held in 32 bits or in 8.
//
// Per element, t the step's number:
//
//     g = s grad     m = b1 m + (1 - b1) g     v = b2 v + (1 - b2) g^2
//     p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// In 8 bits a block of 256 elements, counted from its tensor's first, holds e4m3 codes of m and of
// sqrt(v), each relative to a scale (largest magnitude / 448).  A second average changes by
// a thousandth of itself a step, and e4m3 has steps of a tenth: rounded to nearest, it would stay
// where it is.  So the rounding's threshold runs evenly through [0, 1) over steps and elements
// (an additive sequence), and the changes add up.  Rounding is an integer addition: times 2^-120,
// e4m3's exponents are fp32's lowest, its steps below 2^-6 fp32's subnormals, and a code the
// upper 7 bits of a number's 27.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ewg_train.cuh"

namespace ewg {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kTop = 448.0f;                                        // e4m3's largest number
constexpr float kTopInverse = static_cast<float>(1.0 / 448.0);
constexpr float kLowestScale = 0x1p-120f;
// the first two powers of the plastic number's inverse, of 2^32
constexpr uint32_t kWeylA = 0xC13FA9A9u, kWeylB = 0x91E10DA5u;

template <int kTable>
struct Launch {
  AdamwHyper hyper;
  int num, tiles;
  AdamwEntry entry[kTable];
};

// What a step's elements have in common.
struct Step {
  float grad_scale, lr, rate, root_factor;      // rate: lr / (1 - b1^t), factor: 1 / sqrt(1 - b2^t)
  uint32_t t;
};

__device__ __forceinline__ Step make_step(const AdamwHyper& h) {
  Step s;
  long long t = h.step_ptr ? *h.step_ptr : h.step;
  t = t < 1 ? 1 : t;
  s.lr = h.lr_ptr ? *h.lr_ptr : h.lr;
  s.grad_scale = h.grad_scale_ptr ? *h.grad_scale_ptr : h.grad_scale;
  // 1 - b^t without the digits that b^t near 1 would lose
  s.rate = s.lr / -expm1f(static_cast<float>(t) * h.log_beta1);
  s.root_factor = 1.0f / sqrtf(-expm1f(static_cast<float>(t) * h.log_beta2));
  s.t = static_cast<uint32_t>(t);
  return s;
}

__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }

// 8 neighbouring elements, in one access.
template <typename T>
struct Eight;

template <>
struct Eight<float> {
  static __device__ __forceinline__ void read(const float* p, float (&f)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p) : "memory");
  }
  static __device__ __forceinline__ void write(float* p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]) : "memory");
  }
};

template <>
struct Eight<__nv_bfloat16> {
  static __device__ __forceinline__ void read(const __nv_bfloat16* p, float (&f)[8]) {
    uint32_t u[4];
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "l"(p) : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void write(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// e4m3 codes: the values that they stand for.
__device__ __forceinline__ void eight_codes(const uint8_t* p, float (&f)[8]) {
  uint32_t u[2];
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(u[0]), "=r"(u[1]) : "l"(p) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[i / 2] >> (i % 2 * 16)), __NV_E4M3));
    const float2 v = __half22float2(h);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ float from_code(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// The moments after a gradient.  In 8 bits their rounding goes by every bit, so each
// operation is rounded by itself, whatever the compiler would join.
__device__ __forceinline__ void moments(const AdamwHyper& h, float g, float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, h.beta1), __fmul_rn(g, h.rest1));
  v = __fadd_rn(__fmul_rn(v, h.beta2), __fmul_rn(__fmul_rn(g, g), h.rest2));
}

__device__ __forceinline__ float updated(const AdamwHyper& h, const Step& s, float decay, float p, float m, float root) {
  // (the quotient of two units in the last place: it is scaled by lr before it meets the param)
  return p * (1.0f - s.lr * decay) - __fdividef(s.rate * m, root * s.root_factor + h.eps);
}

// A block's scale from its largest magnitude's bits (NaN is above every other), and what values are
// multiplied by for it.
__device__ __forceinline__ float block_scale(uint32_t bits, float& inverse) {
  const float scale = __fmul_rn(__uint_as_float(bits), kTopInverse);
  const bool none = scale < kLowestScale;
  inverse = none ? 0.0f : __frcp_rn(scale);
  return none ? 0.0f : scale;
}

// e4m3 code of x relative to its block's scale, `threshold` of 20 bits.
__device__ __forceinline__ uint32_t to_code(float x, float inverse, uint32_t threshold) {
  const uint32_t bits = __float_as_uint(__fmul_rn(__fmul_rn(x, inverse), 0x1p-120f));
  const uint32_t code = ((bits & 0x7fffffffu) + threshold) >> 20;
  return (code < 126u ? code : 126u) | (bits >> 31 << 7);
}

// A warp's 256 elements from `base` on.
template <typename P, typename G, int kBits>
__device__ __forceinline__ void update_block(const AdamwEntry& e, const AdamwHyper& h, const Step& s, long long base, int lane) {
  P* param = static_cast<P*>(e.param) + base;
  const G* grad = static_cast<const G*>(e.grad) + base;
  __nv_bfloat16* copy = e.copy ? static_cast<__nv_bfloat16*>(e.copy) + base : nullptr;
  const int count = e.count - base < kAdamwBlock ? static_cast<int>(e.count - base) : kAdamwBlock;
  if constexpr (kBits == 32) {
    float* mp = static_cast<float*>(e.exp_avg) + base;
    float* vp = static_cast<float*>(e.exp_avg_sq) + base;
    for (int i = lane; i < count; i += 32) {
      float m = mp[i], v = vp[i];
      moments(h, load(grad + i) * s.grad_scale, m, v);
      const float p = updated(h, s, e.weight_decay, load(param + i), m, sqrtf(v));
      mp[i] = m;
      vp[i] = v;
      store(param + i, p);
      if (copy) store(copy + i, p);
    }
  } else {
    uint8_t* mp = static_cast<uint8_t*>(e.exp_avg) + base;
    uint8_t* rp = static_cast<uint8_t*>(e.exp_avg_sq) + base;
    float2* at = e.scales + base / kAdamwBlock;
    const float2 scale = *at;
    float m[8], root[8];
    uint32_t top_m = 0, top_root = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = k * 32 + lane;
      m[k] = root[k] = 0.0f;
      if (i < count) {
        m[k] = __fmul_rn(from_code(mp[i]), scale.x);
        const float r = __fmul_rn(from_code(rp[i]), scale.y);
        float v = __fmul_rn(r, r);
        moments(h, __fmul_rn(load(grad + i), s.grad_scale), m[k], v);
        root[k] = sqrtf(v);
        const float p = updated(h, s, e.weight_decay, load(param + i), m[k], root[k]);
        store(param + i, p);
        if (copy) store(copy + i, p);
      }
      const uint32_t am = __float_as_uint(m[k]) & 0x7fffffffu, ar = __float_as_uint(root[k]) & 0x7fffffffu;
      top_m = am > top_m ? am : top_m;
      top_root = ar > top_root ? ar : top_root;
    }
    top_m = __reduce_max_sync(kAll, top_m);
    top_root = __reduce_max_sync(kAll, top_root);
    float inverse_m, inverse_root;
    float2 now;
    now.x = block_scale(top_m, inverse_m);
    now.y = block_scale(top_root, inverse_root);
    if (lane == 0) *at = now;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = k * 32 + lane;
      if (i < count) {
        const uint32_t n = static_cast<uint32_t>(base) + i;
        mp[i] = static_cast<uint8_t>(to_code(m[k], inverse_m, (n * kWeylA + s.t * kWeylB) >> 12));
        uint32_t c = to_code(root[k], inverse_root, (n * kWeylB + s.t * kWeylA) >> 12);
        // an element that has had gradients keeps a root to divide by
        if (c == 0 && root[k] > 0.0f && inverse_root > 0.0f) c = 1;
        rp[i] = static_cast<uint8_t>(c);
      }
    }
  }
}

// The same of a whole block where every array can be moved eight elements at a time; lanes take eight
// neighbouring ones each.
template <typename P, typename G, int kBits>
__device__ __forceinline__ void update_whole_block(const AdamwEntry& e, const AdamwHyper& h, const Step& s, long long base,
                                                   int lane) {
  const long long first = base + lane * 8;
  P* param = static_cast<P*>(e.param) + first;
  float p[8], g[8], m[8], v[8];
  Eight<P>::read(param, p);
  Eight<G>::read(static_cast<const G*>(e.grad) + first, g);
  if constexpr (kBits == 32) {
    float* mp = static_cast<float*>(e.exp_avg) + first;
    float* vp = static_cast<float*>(e.exp_avg_sq) + first;
    Eight<float>::read(mp, m);
    Eight<float>::read(vp, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      moments(h, g[k] * s.grad_scale, m[k], v[k]);
      p[k] = updated(h, s, e.weight_decay, p[k], m[k], sqrtf(v[k]));
    }
    Eight<float>::write(mp, m);
    Eight<float>::write(vp, v);
  } else {
    uint8_t* mp = static_cast<uint8_t*>(e.exp_avg) + first;
    uint8_t* rp = static_cast<uint8_t*>(e.exp_avg_sq) + first;
    eight_codes(mp, m);
    eight_codes(rp, v);
    float2* at = e.scales + base / kAdamwBlock;
    const float2 scale = *at;
    uint32_t top_m = 0, top_root = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m[k] = __fmul_rn(m[k], scale.x);
      const float r = __fmul_rn(v[k], scale.y);
      v[k] = __fmul_rn(r, r);
      moments(h, __fmul_rn(g[k], s.grad_scale), m[k], v[k]);
      v[k] = sqrtf(v[k]);
      p[k] = updated(h, s, e.weight_decay, p[k], m[k], v[k]);
      top_m = max(top_m, __float_as_uint(m[k]) & 0x7fffffffu);
      top_root = max(top_root, __float_as_uint(v[k]) & 0x7fffffffu);
    }
    top_m = __reduce_max_sync(kAll, top_m);
    top_root = __reduce_max_sync(kAll, top_root);
    float inverse_m, inverse_root;
    float2 now;
    now.x = block_scale(top_m, inverse_m);
    now.y = block_scale(top_root, inverse_root);
    if (lane == 0) *at = now;
    const uint32_t n = static_cast<uint32_t>(first);
    const uint32_t from_m = n * kWeylA + s.t * kWeylB, from_root = n * kWeylB + s.t * kWeylA;
    uint32_t cm[2] = {}, cr[2] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      cm[k / 4] |= to_code(m[k], inverse_m, (from_m + k * kWeylA) >> 12) << (k % 4 * 8);
      uint32_t c = to_code(v[k], inverse_root, (from_root + k * kWeylB) >> 12);
      if (c == 0 && v[k] > 0.0f && inverse_root > 0.0f) c = 1;
      cr[k / 4] |= c << (k % 4 * 8);
    }
    *reinterpret_cast<uint2*>(mp) = make_uint2(cm[0], cm[1]);
    *reinterpret_cast<uint2*>(rp) = make_uint2(cr[0], cr[1]);
  }
  Eight<P>::write(param, p);
  if constexpr (sizeof(P) == 4)
    if (e.copy) Eight<__nv_bfloat16>::write(static_cast<__nv_bfloat16*>(e.copy) + first, p);
}

template <typename P, typename G, int kBits>
__device__ __forceinline__ void update(const AdamwEntry& e, const AdamwHyper& h, const Step& s, long long base, int lane) {
  if ((e.flags & kAdamwWhole) && base + kAdamwBlock <= e.count) update_whole_block<P, G, kBits>(e, h, s, base, lane);
  else update_block<P, G, kBits>(e, h, s, base, lane);
}

template <int kBits, int kTable>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Launch<kTable> a) {
  const Step s = make_step(a.hyper);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int at = 0;
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    for (int end = a.num; end - at > 1;) {               // the last entry that begins at or before the tile
      const int mid = (at + end) / 2;
      if (a.entry[mid].first_tile <= tile) at = mid;
      else end = mid;
    }
    const AdamwEntry& e = a.entry[at];
    const long long base = static_cast<long long>(tile - e.first_tile) * kAdamwTile + warp * kAdamwBlock;
    if (base >= e.count) continue;
    switch (e.flags & (kAdamwParamBf16 | kAdamwGradBf16)) {
      case 0: update<float, float, kBits>(e, a.hyper, s, base, lane); break;
      case kAdamwParamBf16: update<__nv_bfloat16, float, kBits>(e, a.hyper, s, base, lane); break;
      case kAdamwGradBf16: update<float, __nv_bfloat16, kBits>(e, a.hyper, s, base, lane); break;
      default: update<__nv_bfloat16, __nv_bfloat16, kBits>(e, a.hyper, s, base, lane);
    }
  }
}

template <int kBits, int kTable>
cudaError_t launch(const AdamwEntry* entries, int num, const AdamwHyper& h, int num_sms, cudaStream_t stream) {
  Launch<kTable> a;
  a.hyper = h;
  a.num = num;
  for (int i = 0; i < num; ++i) a.entry[i] = entries[i];
  const AdamwEntry& last = entries[num - 1];
  a.tiles = last.first_tile + static_cast<int>((last.count + kAdamwTile - 1) / kAdamwTile);
  const int most = num_sms * 8;
  adamw_kernel<kBits, kTable><<<a.tiles < most ? a.tiles : most, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamwEntry* entries, int num, int state_bits, const AdamwHyper& h, int num_sms,
                         cudaStream_t stream) {
  return state_bits == 32 ? launch<32, kAdamwEntries>(entries, num, h, num_sms, stream)
                          : launch<8, kAdamwEntries>(entries, num, h, num_sms, stream);
}

}  // namespace ewg
