// One AdamW step of many tensors, the moments held in 32 bits or in 8.
//
// Per element, t the step's number:
//
//     g = s grad     m = b1 m + (1 - b1) g     v = b2 v + (1 - b2) g^2
//     p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// In 8 bits a block of 256 elements, counted from its tensor's first, holds e4m3 codes of m and of
// sqrt(v), each relative to a scale (largest magnitude / 448).  A second average changes by
// a thousandth of itself a step, and e4m3 has steps of a tenth: rounded to nearest, an element keeps
// its code for good unless the whole block's scale moves (with b2 = 0.999, where half of a block's
// gradients fall to 0.3 of what they were, their roots are still 2.2 times too large after 2000 steps).  So the
// rounding's threshold runs evenly through [0, 1) over steps and elements (an additive sequence: M. Roberts's
// R2, by the plastic number), and the changes add up (the roots are then 0.95 of what they should be; where the gradients
// triple 1.04, rounded to nearest 0.35).  Rounding is an integer addition: times 2^-120,
// e4m3's exponents are fp32's lowest, its steps below 2^-6 fp32's subnormals, and a code the upper 7
// bits of a number's 27.
//
// A warp takes 256 elements, eight neighbours a lane in one access of each array; where an array is not
// aligned to that, one of every 32.  In 32 bits the step is bound by memory (50257 x 1024 fp32 with a bf16 copy, 30 bytes
// an element: 224 us, 7.0 TB/s), in 8 with fp32 params too (129280 x 7168: 2540 us, 6.6 TB/s); with bf16 params and
// gradients, 10 bytes an element, by its 63 instructions and its loads (50257 x 1024: 114 us, 4.5 TB/s; three
// elements off alignment 130), of which the root takes ten and the two codes twelve.  The tensors' addresses are the
// launch's argument, so that nothing has to be uploaded and a captured call keeps them.
//
// Tried and slower: a warp's next block loaded ahead (bf16 in 8 bits the same, fp32 in 32 bits 3 % slower:
// neighbouring blocks are then further apart in time), four neighbouring blocks a warp (6 %), bf16 arrays off
// alignment by aligned accesses and shuffles (30 %), the first block's loads begun before the wait for the step's own
// numbers (8 bits 4 to 11 %, 32 bits the same).
#include <cfloat>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ewg_ptx.cuh"
#include "ewg_train.cuh"

namespace ewg {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kTopInverse = static_cast<float>(1.0 / 448.0);      // of e4m3's largest number
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

// How a warp's 256 elements lie with its lanes, eight each.  kAligned: neighbours, moved by one access, of a whole
// block of arrays that are aligned to eight of their elements; kWhole: one of every 32, of a whole block;
// kPart: the same of a tensor's last block, of which those that are there are moved.
enum Mode { kAligned, kWhole, kPart };

template <int kMode>
struct Place {
  static constexpr int kStep = kMode == kAligned ? 1 : 32;
  long long first;           // of the tensor, the lane's first element
  int left;                  // elements of the block from that one on

  __device__ __forceinline__ bool there(int k) const { return kMode != kPart || k * 32 < left; }
  __device__ __forceinline__ void read(const float* p, float2 (&f)[4]) const {
    p += first;
    if constexpr (kMode == kAligned) {
      asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y), "=f"(f[2].x), "=f"(f[2].y), "=f"(f[3].x),
                     "=f"(f[3].y) : "l"(p) : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) at(f, k) = there(k) ? p[k * 32] : 0.0f;
    }
  }
  __device__ __forceinline__ void read(const __nv_bfloat16* p, float2 (&f)[4]) const {
    p += first;
    if constexpr (kMode == kAligned) {
      uint32_t u[4];
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "l"(p) : "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) at(f, k) = there(k) ? __bfloat162float(p[k * 32]) : 0.0f;
    }
  }
  // e4m3 codes: the values that they stand for
  __device__ __forceinline__ void read(const uint8_t* p, float2 (&f)[4]) const {
    p += first;
    uint32_t u[4];                                          // two codes each
    if constexpr (kMode == kAligned) {
      uint32_t v[2];
      asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p) : "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = v[i / 2] >> (i % 2 * 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = (there(2 * i) ? p[2 * i * 32] : 0) | (there(2 * i + 1) ? p[2 * i * 32 + 32] << 8 : 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[i]), __NV_E4M3)));
  }
  __device__ __forceinline__ void write(float* p, const float2 (&f)[4]) const {
    p += first;
    if constexpr (kMode == kAligned) {
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0].x), "f"(f[0].y), "f"(f[1].x),
                   "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x), "f"(f[3].y) : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (there(k)) p[k * 32] = k % 2 ? f[k / 2].y : f[k / 2].x;
    }
  }
  __device__ __forceinline__ void write(__nv_bfloat16* p, const float2 (&f)[4]) const {
    p += first;
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(f[i].y), "f"(f[i].x));
    if constexpr (kMode == kAligned) {
      *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (there(k)) reinterpret_cast<unsigned short*>(p)[k * 32] = static_cast<unsigned short>(u[k / 2] >> (k % 2 * 16));
    }
  }
  // codes, each in the upper byte of a word
  __device__ __forceinline__ void write(uint8_t* p, const uint32_t (&c)[8]) const {
    p += first;
    if constexpr (kMode == kAligned) {
      uint32_t v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0073), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0073), 0x5410);
      *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (there(k)) p[k * 32] = static_cast<uint8_t>(c[k] >> 24);
    }
  }
  static __device__ __forceinline__ float& at(float2 (&f)[4], int k) { return k % 2 ? f[k / 2].y : f[k / 2].x; }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// (Not the packed addition: the compiler joins it with the products before it, which then are not
// rounded.)
__device__ __forceinline__ float2 rounded_sum(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// 1 / x to a unit in the last place; x is no subnormal (a root is 0 or above 2^-75).
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x, or the largest number of its sign where it is infinite: an infinite param stays what it is.
__device__ __forceinline__ float finite(float x) {
  float y;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(FLT_MAX));
  return y;
}

// The larger magnitude (of either sign), NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
  float y;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ float largest(const float2 (&f)[4]) {
  return larger(larger(larger(f[0].x, f[0].y), larger(f[1].x, f[1].y)), larger(larger(f[2].x, f[2].y), larger(f[3].x, f[3].y)));
}

// A block's scale from its largest magnitude's bits (NaN is above every other), and what values are
// multiplied by for it.
__device__ __forceinline__ float block_scale(uint32_t bits, float& inverse) {
  const float scale = __fmul_rn(__uint_as_float(bits), kTopInverse);
  const bool none = scale < kLowestScale;
  inverse = none ? 0.0f : __frcp_rn(scale);
  return none ? 0.0f : scale;
}

// e4m3 codes of x relative to its block's scale, in the upper bytes; their thresholds are the upper
// 20 bits of `from` and what follows it by steps of `by`.  `lowest`: the least that a number above
// 0 becomes (for numbers that are not negative), in the same place as a code before it is moved up.
template <bool kSigned>
__device__ __forceinline__ void to_codes(const float2 (&x)[4], float inverse, uint32_t from, uint32_t by, uint32_t lowest,
                                         uint32_t (&c)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = ptx::mul2(ptx::mul2(x[i], both(inverse)), both(0x1p-120f));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 2 * i + h;
      const uint32_t bits = __float_as_uint(h ? y.y : y.x);
      const uint32_t sum = bits + ((from + k * by) >> 12);
      constexpr uint32_t kMost = (126u << 20) | 0xfffffu;
      if constexpr (kSigned) {
        c[k] = min(sum & 0x7fffffffu, kMost) << 4 | (sum & 0x80000000u);
      } else {
        const uint32_t least = min(__float_as_uint(h ? x[i].y : x[i].x), lowest);
        c[k] = max(min(sum, kMost), least) << 4;
      }
    }
  }
}

// A warp's block of 256 elements.
template <typename P, typename G, int kBits, int kMode>
__device__ __forceinline__ void update_block(const AdamwEntry& e, const AdamwHyper& h, const Step& s, long long base, int lane) {
  using ptx::add2;
  using ptx::fma2;
  using ptx::mul2;
  const int count = e.count - base < kAdamwBlock ? static_cast<int>(e.count - base) : kAdamwBlock;
  const Place<kMode> place{base + (kMode == kAligned ? lane * 8 : lane), count - lane};
  using State = typename std::conditional<kBits == 32, float, uint8_t>::type;
  P* param = static_cast<P*>(e.param);
  State* exp_avg = static_cast<State*>(e.exp_avg);
  State* exp_avg_sq = static_cast<State*>(e.exp_avg_sq);
  float2 p[4], g[4], m[4], v[4], root[4];
  place.read(param, p);
  place.read(static_cast<const G*>(e.grad), g);
  place.read(exp_avg, m);
  place.read(exp_avg_sq, v);
  if constexpr (kBits == 8) {
    const float2 scale = e.scales[base / kAdamwBlock];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = mul2(m[i], both(scale.x));
      v[i] = mul2(v[i], both(scale.y));
      v[i] = mul2(v[i], v[i]);
    }
  }
  const float2 decay = both(-s.lr * e.weight_decay);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (each operation rounded by itself: the codes go by every bit of the moments)
    g[i] = mul2(g[i], both(s.grad_scale));
    m[i] = rounded_sum(mul2(m[i], both(h.beta1)), mul2(g[i], both(h.rest1)));
    v[i] = rounded_sum(mul2(v[i], both(h.beta2)), mul2(mul2(g[i], g[i]), both(h.rest2)));
    root[i] = make_float2(sqrtf(v[i].x), sqrtf(v[i].y));
    const float2 under = fma2(root[i], both(s.root_factor), both(h.eps));
    const float2 over = mul2(m[i], both(-s.rate));
    // The decay is added to the step and both to the param: 1 - lr wd by itself would be rounded by up to 2^-25, which
    // is as much as a small decay.
    const float2 lost = mul2(make_float2(finite(p[i].x), finite(p[i].y)), decay);
    p[i] = add2(p[i], fma2(over, make_float2(reciprocal(under.x), reciprocal(under.y)), lost));
  }
  place.write(param, p);
  if constexpr (sizeof(P) == 4)
    if (e.copy) place.write(static_cast<__nv_bfloat16*>(e.copy), p);
  if constexpr (kBits == 32) {
    place.write(exp_avg, m);
    place.write(exp_avg_sq, v);
  } else {
    const uint32_t top_m = __reduce_max_sync(kAll, __float_as_uint(largest(m)) & 0x7fffffffu);
    const uint32_t top_root = __reduce_max_sync(kAll, __float_as_uint(largest(root)) & 0x7fffffffu);
    float inverse_m, inverse_root;
    float2 now;
    now.x = block_scale(top_m, inverse_m);
    now.y = block_scale(top_root, inverse_root);
    if (lane == 0) e.scales[base / kAdamwBlock] = now;
    const uint32_t n = static_cast<uint32_t>(place.first);
    uint32_t c[8];
    to_codes<true>(m, inverse_m, n * kWeylA + s.t * kWeylB, place.kStep * kWeylA, 0, c);
    place.write(exp_avg, c);
    // a root above 0 keeps a code above 0: its element goes on to be divided by it
    to_codes<false>(root, inverse_root, n * kWeylB + s.t * kWeylA, place.kStep * kWeylB, inverse_root > 0.0f ? 1u << 20 : 0u, c);
    place.write(exp_avg_sq, c);
  }
}

template <typename P, typename G, int kBits>
__device__ __forceinline__ void update(const AdamwEntry& e, const AdamwHyper& h, const Step& s, long long base, int lane) {
  if (base + kAdamwBlock > e.count) update_block<P, G, kBits, kPart>(e, h, s, base, lane);
  else if (e.flags & kAdamwAligned) update_block<P, G, kBits, kAligned>(e, h, s, base, lane);
  else update_block<P, G, kBits, kWhole>(e, h, s, base, lane);
}

template <int kBits, int kTable>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Launch<kTable> a) {
  __shared__ Step shared_step;
  if (threadIdx.x == 0) shared_step = make_step(a.hyper);
  __syncthreads();
  const Step s = shared_step;
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
  // In 32 bits a block of threads takes one tile, so that the tiles on the way are neighbours in memory (50257 x
  // 1024 fp32 with a bf16 copy: 224 us; 8 blocks an SM that go on in steps of the grid: 242).  In 8 bits the step's
  // own numbers cost more than that brings: 32 blocks an SM (the same 140 us, bf16 without a copy 114; one tile
  // each 150 and 135, 8 blocks an SM 149 and 115).
  const int most = kBits == 32 ? a.tiles : num_sms * 32;
  adamw_kernel<kBits, kTable><<<a.tiles < most ? a.tiles : most, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamwEntry* entries, int num, int state_bits, const AdamwHyper& h, int num_sms,
                         cudaStream_t stream) {
  // (a launch's argument is copied whole, whatever it holds)
  if (num <= kAdamwFew)
    return state_bits == 32 ? launch<32, kAdamwFew>(entries, num, h, num_sms, stream)
                            : launch<8, kAdamwFew>(entries, num, h, num_sms, stream);
  return state_bits == 32 ? launch<32, kAdamwEntries>(entries, num, h, num_sms, stream)
                          : launch<8, kAdamwEntries>(entries, num, h, num_sms, stream);
}

}  // namespace ewg
