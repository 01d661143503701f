// 4-bit weights with group scales (w4.cuh): quantisation and the values that
// codes stand for.  Load-time steps, of simple form: bound by their small loads and stores (and the quantiser's divisions),
// not by bytes.  Measured (GB300, 262144 x 768, bf16 scales): from bf16 in groups of 128 262 us (1.9 TB/s), of 32 with zero points
// 451 (1.2); from fp32 262 and 442; back to bf16 436 and 481 us (1.2 and 1.1 TB/s), to fp32 617 and 665.
#include "common.cuh"
#include "internal.h"
#include "w4.cuh"

namespace semmoe {
namespace {

using namespace w4;

constexpr int kThreads = 256;

// One group per thread of a warp's 32 consecutive groups would read memory in strides;
// instead eight lanes share a group: each takes every eighth pair of values.
//   with zero points: lo = min(0, min x), hi = max(0, max x), s = (hi - lo) / 15, z = round(-lo / s)
//   without:          s = max |x| / 7, z = 8
//   code = clamp(round(x / s) + z, 0, 15), s rounded to its type first; s = 0 gives code z
// A group that holds NaN or an infinity gets the scale NaN.
template <typename T, typename S>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* __restrict__ x, long long groups, int group, uint8_t* __restrict__ codes, S* __restrict__ scales,
                uint8_t* __restrict__ zeros) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32, part = lane % 8;
  const long long stride = (long long)gridDim.x * (kThreads / 8);
  // groups of one warp differ in number only past the end: its lanes stay together
  for (long long base = ((long long)blockIdx.x * kThreads + threadIdx.x - lane) / 8; base < groups; base += stride) {
    const long long g = base + lane / 8;
    const bool live = g < groups;
    const T* row = x + (live ? g : 0) * group;
    float lo = 0.f, hi = 0.f;
    bool bad = false;
    for (int i = 2 * part; i < group; i += 16) {
      const float a = to_f32(row[i]), b = to_f32(row[i + 1]);
      lo = fminf(lo, fminf(a, b));
      hi = fmaxf(hi, fmaxf(a, b));
      bad |= !(a - a == 0.f) || !(b - b == 0.f);
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
      bad |= __shfl_xor_sync(0xffffffffu, (int)bad, d) != 0;
    }
    const float range = zeros != nullptr ? hi * (1.0f / 16) - lo * (1.0f / 16) : fmaxf(hi, -lo);
    float s = to_f32(from_f32<S>(zeros != nullptr ? __fdiv_rn(range, 15.0f / 16) : __fdiv_rn(range, 7.0f)));
    const bool none = bad || s == 0.f;
    if (bad) s = __int_as_float(0x7fc00000);
    const int z = zeros != nullptr ? (none ? 0 : (int)fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f)) : 8;
    if (!live) continue;
    for (int i = 2 * part; i < group; i += 16) {
      uint32_t c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        c[j] = none ? (uint32_t)z : (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(to_f32(row[i + j]), s)) + (float)z, 0.f), 15.f);
      codes[(g * group + i) / 2] = (uint8_t)(c[0] | (c[1] << 4));
    }
    if (part == 0) {
      scales[g] = from_f32<S>(s);
      if (zeros != nullptr) zeros[g] = (uint8_t)z;
    }
  }
}

// d * s rounded once: to bf16 through fp32, a product that fp32 rounds onto the middle between two
// bf16 numbers is first moved off it, to the side of what that rounding dropped.
template <typename T>
__device__ __forceinline__ T scaled(float d, float s) {
  float p = __fmul_rn(d, s);
  if constexpr (sizeof(T) == 2) {
    const float rest = fmaf(d, s, -p);
    if ((__float_as_uint(p) & 0xffffu) == 0x8000u && rest != 0.f)
      p = __uint_as_float(__float_as_uint(p) + ((rest > 0.f) == (p > 0.f) ? 1u : -1u));
  }
  return from_f32<T>(p);
}

// Eight codes (a word) per thread and step; a word lies in one group.
template <typename S, typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint32_t* __restrict__ codes, const S* __restrict__ scales, const uint8_t* __restrict__ zeros,
                  long long words, int group, T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < words; i += (long long)gridDim.x * kThreads) {
    const uint32_t w = codes[i];
    const long long g = i * 8 / group;
    const float s = load_scale(scales + g);
    const int z = zeros != nullptr ? zeros[g] & 15 : 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) out[i * 8 + j] = scaled<T>((float)((int)((w >> (4 * j)) & 15u) - z), s);
  }
}

template <typename K, typename... A>
cudaError_t launch_flat(K kern, long long items, cudaStream_t s, A... args) {
  long long blocks = (items + kThreads - 1) / kThreads;
  const long long cap = 16LL * sm_count();
  if (blocks > cap) blocks = cap;
  cudaError_t e = launch_kernel(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, 1, true, args...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_w4_quantize(const void* x, int dtype, long long rows, int K, int group, uint8_t* codes, void* scales,
                               int scale_dtype, uint8_t* zeros, cudaStream_t s) {
  const long long n = rows * (K / group);
  auto go = [&](auto* xp, auto* sp) {
    using T = std::remove_cv_t<std::remove_pointer_t<decltype(xp)>>;
    using S = std::remove_pointer_t<decltype(sp)>;
    return launch_flat(quantize_kernel<T, S>, n * 8, s, static_cast<const T*>(x), n, group, codes, static_cast<S*>(scales),
                       zeros);
  };
  const __nv_bfloat16* b = nullptr;
  const float* f = nullptr;
  __nv_bfloat16* sb = nullptr;
  float* sf = nullptr;
  if (dtype == SEMMOE_BF16) return scale_dtype == SEMMOE_BF16 ? go(b, sb) : go(b, sf);
  return scale_dtype == SEMMOE_BF16 ? go(f, sb) : go(f, sf);
}

cudaError_t launch_w4_dequantize(const Weights& w, long long rows, int K, int group, void* out, int dtype, cudaStream_t s) {
  const long long words = rows * (K / 8);
  auto go = [&](auto* sp, auto* op) {
    using S = std::remove_cv_t<std::remove_pointer_t<decltype(sp)>>;
    using T = std::remove_pointer_t<decltype(op)>;
    return launch_flat(dequantize_kernel<S, T>, words, s, reinterpret_cast<const uint32_t*>(w.codes), sp, w.zeros, words,
                       group, op);
  };
  if (w.scales_bf16) {
    const auto* sp = static_cast<const __nv_bfloat16*>(w.scales);
    return dtype == SEMMOE_BF16 ? go(sp, static_cast<__nv_bfloat16*>(out)) : go(sp, static_cast<float*>(out));
  }
  const auto* sp = static_cast<const float*>(w.scales);
  return dtype == SEMMOE_BF16 ? go(sp, static_cast<__nv_bfloat16*>(out)) : go(sp, static_cast<float*>(out));
}

}  // namespace semmoe
