// Quantisation to 4-bit microscaled values and back (format and layouts:
// mx4.cuh).  Pure data movement: per value 2 or 4 bytes in and 17/32 of a byte
// out, so the bound is HBM bandwidth; a lane takes 16 values of a row (two
// 16-byte loads of bf16), two lanes share a block, eight one 128-column tile.
// Measured (GB300): 180224 x 2048 bf16 to 4 bits 131 us and back 143 us (934 MB each: 7.1 and
// 6.5 TB/s, at the rate of a plain copy; with 8 values a lane and a grid that fills the
// GPU once 178 and 228 us); 16384 rows of 2048 into 131072 sorted rows 38 us (210 MB, 5.5 TB/s).
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"

namespace semmoe {
namespace {

using namespace mx4;

__device__ int g_err;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSpan = 512;  // columns a warp takes at once, 16 per lane

// Sixteen consecutive values of a row, as loaded and as fp32.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 a, b;
};
template <> struct Raw<float> {
  float4 a, b, c, d;
};
__device__ __forceinline__ void load16(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
  r.a = __ldg(reinterpret_cast<const uint4*>(p));
  r.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
}
__device__ __forceinline__ void load16(const float* p, Raw<float>& r) {
  const float4* q = reinterpret_cast<const float4*>(p);
  r.a = __ldg(q), r.b = __ldg(q + 1), r.c = __ldg(q + 2), r.d = __ldg(q + 3);
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&v)[16]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&v)[16]) {
  const float w[16] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w,
                       r.c.x, r.c.y, r.c.z, r.c.w, r.d.x, r.d.y, r.d.z, r.d.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = w[i];
}

// The lane's sixteen codes, and in every lane of an 8-lane group the group's four
// scales as one word (block j at byte j).  Whole warp.
template <typename T>
__device__ __forceinline__ uint2 quantise16(const Raw<T>& raw, uint32_t& scales) {
  float v[16];
  widen(raw, v);
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  const uint32_t b = scale_code(a);
  const float f = inverse_scale(b);
  uint32_t w = b << (8 * ((threadIdx.x >> 1) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 2);
  scales = w | __shfl_xor_sync(0xffffffffu, w, 4);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= f;
  return make_uint2(encode8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]),
                    encode8(v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]));
}

// Groups of group_rows rows.  A warp takes rows r, r + 32, r + 64, r + 96 of a
// row tile -- whose scales of one tile are 16 consecutive bytes -- and walks K.
template <typename T>
__global__ void __launch_bounds__(kThreads)
mx4_quantize_kernel(const T* __restrict__ x, int groups, int group_rows, int K, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const int tiles = row_tiles(group_rows), kc = col_tiles(K);
  const long long units = (long long)groups * tiles * 32;
  for (long long u = (long long)blockIdx.x * kWarps + threadIdx.x / 32; u < units; u += (long long)gridDim.x * kWarps) {
    const long long tile = u / 32;
    const int r0 = (int)(u % 32);
    const long long g = tile / tiles;
    const int in_group = (int)(tile % tiles) * kTileRows + r0;
    const size_t row = (size_t)g * group_rows + in_group;
    for (int c0 = 0; c0 < K; c0 += kSpan) {
      const int c = c0 + lane * 16;
      Raw<T> v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = Raw<T>{};
        if (c < K && in_group + 32 * i < group_rows) load16(x + (row + 32 * i) * K + c, v[i]);
      }
      uint32_t s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 w = quantise16(v[i], s[i]);
        if (c < K && in_group + 32 * i < group_rows)
          *reinterpret_cast<uint2*>(codes + ((row + 32 * i) * K + c) / 2) = w;
      }
      const int ct = c / kTileCols;
      if ((lane & 7) == 0 && ct < kc)
        *reinterpret_cast<uint4*>(scales + ((size_t)tile * kc + ct) * kTileBytes + 16 * r0) =
            make_uint4(s[0], s[1], s[2], s[3]);
    }
  }
}

// Token rows into expert order: one warp per token quantises its row once and
// writes the codes and scales to each of its pairs' sorted rows.
constexpr int kMaxE = 256;
constexpr int kBatch = 4;  // column spans held in registers: 2048 columns

template <typename T>
__global__ void __launch_bounds__(kThreads)
mx4_quantize_rows_kernel(const T* __restrict__ x, int n_tok, int K, const int32_t* __restrict__ pair_to_sorted,
                         int k_max, int P, const int32_t* __restrict__ expert_offsets, int E,
                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ int off[kMaxE + 1], first[kMaxE];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  Raw<T> v[kBatch];
  auto load = [&](int t, int c0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int c = c0 + i * kSpan + lane * 16;
      v[i] = Raw<T>{};
      if (c < K) load16(x + (size_t)t * K + c, v[i]);
    }
  };
  const int t_first = blockIdx.x * kWarps + threadIdx.x / 32;
  if (t_first < n_tok) load(t_first, 0);  // in flight beside the offsets
  if (threadIdx.x < 32) {  // row tile at which each expert's rows start, 8 experts per lane
    int o[9], cnt[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) o[i] = lane * 8 + i <= E ? expert_offsets[lane * 8 + i] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      cnt[i] = 0;
      if (e < E) {
        off[e] = o[i];
        if (e == E - 1) off[E] = o[i + 1];
        if (o[i] < 0 || o[i + 1] < o[i] || o[i + 1] > P) atomicOr(&g_err, SEMMOE_DEVERR_PAIRS);
        else cnt[i] = row_tiles(o[i + 1] - o[i]);
      }
      sum += cnt[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += u;
    }
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (lane * 8 + i < E) first[lane * 8 + i] = run;
      run += cnt[i];
    }
  }
  __syncthreads();
  const int kc = col_tiles(K);
  const int max_tiles = P / kTileRows + E;  // what the caller's scales hold
  for (int t = blockIdx.x * kWarps + threadIdx.x / 32; t < n_tok; t += gridDim.x * kWarps) {
    for (int c0 = 0; c0 < K; c0 += kBatch * kSpan) {
      if (t != t_first || c0 > 0) load(t, c0);
      uint2 w[kBatch];
      uint32_t s[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) w[i] = quantise16(v[i], s[i]);
      for (int j0 = 0; j0 < k_max; j0 += 32) {
        int q = j0 + lane < k_max ? pair_to_sorted[(size_t)t * k_max + j0 + lane] : -1;
        int at = 0;  // byte of the row's scales in its tile, and its row tile
        int rt = 0;
        if (q >= 0) {
          int lo = 0, hi = E - 1;  // largest e with off[e] <= q
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (off[mid] <= q) lo = mid;
            else hi = mid - 1;
          }
          const int r = q - off[lo];
          rt = first[lo] + r / kTileRows;
          at = row_byte(r % kTileRows);
          if (q >= P || r < 0 || q >= off[lo + 1] || rt >= max_tiles) {
            atomicOr(&g_err, SEMMOE_DEVERR_PAIRS);
            q = -1;
          }
        }
        const int n = k_max - j0 < 32 ? k_max - j0 : 32;
        for (int j = 0; j < n; ++j) {
          const int qj = __shfl_sync(0xffffffffu, q, j), rj = __shfl_sync(0xffffffffu, rt, j),
                    aj = __shfl_sync(0xffffffffu, at, j);
          if (qj < 0) continue;
          uint8_t* row = codes + (size_t)qj * (K / 2);
          uint8_t* sc = scales + (size_t)rj * kc * kTileBytes + aj;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int c = c0 + i * kSpan + lane * 16;
            if (c < K) *reinterpret_cast<uint2*>(row + c / 2) = w[i];
            if ((lane & 7) == 0 && c < K) *reinterpret_cast<uint32_t*>(sc + (size_t)(c / kTileCols) * kTileBytes) = s[i];
          }
        }
      }
    }
  }
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// Value of one e2m1 code: the two exponent bits and the mantissa bit are fp32's
// top ones at exponent bias 1, so the bits shifted into place, times 2^126, are
// the magnitude (0.5 is the format's one subnormal, and fp32's too).
__device__ __forceinline__ float decode(uint32_t code) {
  const float m = __uint_as_float((code & 7u) << 22) * 0x1p126f;
  return (code & 8u) ? -m : m;
}

// Every value is exact in fp32 and, with its two significant bits, in bf16.
template <typename T>
__global__ void __launch_bounds__(kThreads)
mx4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int groups,
                      int group_rows, int K, T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const int tiles = row_tiles(group_rows), kc = col_tiles(K);
  const long long units = (long long)groups * tiles * 32;
  for (long long u = (long long)blockIdx.x * kWarps + threadIdx.x / 32; u < units; u += (long long)gridDim.x * kWarps) {
    const long long tile = u / 32;
    const int r0 = (int)(u % 32);
    const long long g = tile / tiles;
    const int in_group = (int)(tile % tiles) * kTileRows + r0;
    const size_t row = (size_t)g * group_rows + in_group;
    for (int c = lane * 16; c < K; c += kSpan) {
      const uint4 sw = __ldg(reinterpret_cast<const uint4*>(
          scales + ((size_t)tile * kc + c / kTileCols) * kTileBytes + 16 * r0));
      const uint32_t s[4] = {sw.x, sw.y, sw.z, sw.w};
      uint2 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (in_group + 32 * i < group_rows)
          w[i] = __ldg(reinterpret_cast<const uint2*>(codes + ((row + 32 * i) * K + c) / 2));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (in_group + 32 * i >= group_rows) break;
        const float f = scale_value((s[i] >> (8 * ((c / kBlock) & 3))) & 255u);
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = decode((j < 8 ? w[i].x : w[i].y) >> (4 * (j & 7))) * f;
        store16(out + (row + 32 * i) * K + c, v);
      }
    }
  }
}

// CTAs for `units` warps' work, each warp a few units at most (a grid that fills the GPU
// once left the last units to a few warps: 8% on 45056 units of 2048 columns).
int grid_for(long long units) {
  const long long blocks = (units + kWarps - 1) / kWarps, cap = 1 << 20;
  return (int)(blocks < cap ? blocks : cap);
}

}  // namespace

int mx4_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

size_t mx4_scale_bytes(long long rows, int K, int groups) { return scale_bytes(rows, K, groups); }

cudaError_t launch_mx4_quantize(const void* x, int dtype, int groups, int group_rows, int K, uint8_t* codes,
                                uint8_t* scales, cudaStream_t s) {
  const int grid = grid_for((long long)groups * row_tiles(group_rows) * 32);
  cudaError_t e;
  if (dtype == SEMMOE_BF16)
    e = launch_kernel(mx4_quantize_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, s, 1, true,
                      static_cast<const __nv_bfloat16*>(x), groups, group_rows, K, codes, scales);
  else
    e = launch_kernel(mx4_quantize_kernel<float>, dim3(grid), dim3(kThreads), 0, s, 1, true,
                      static_cast<const float*>(x), groups, group_rows, K, codes, scales);
  count_launches(1);
  return e;
}

cudaError_t launch_mx4_quantize_rows(const void* x, int dtype, int T, int K, const int32_t* pair_to_sorted, int k_max,
                                     int P, const int32_t* expert_offsets, int E, uint8_t* codes, uint8_t* scales,
                                     cudaStream_t s) {
  const long long cap = 8LL * sm_count();  // each CTA first scans the offsets
  const int grid = (int)(ceil_div(T, kWarps) < cap ? ceil_div(T, kWarps) : cap);
  cudaError_t e;
  if (dtype == SEMMOE_BF16)
    e = launch_kernel(mx4_quantize_rows_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, s, 1, true,
                      static_cast<const __nv_bfloat16*>(x), T, K, pair_to_sorted, k_max, P, expert_offsets, E, codes,
                      scales);
  else
    e = launch_kernel(mx4_quantize_rows_kernel<float>, dim3(grid), dim3(kThreads), 0, s, 1, true,
                      static_cast<const float*>(x), T, K, pair_to_sorted, k_max, P, expert_offsets, E, codes, scales);
  count_launches(1);
  return e;
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int groups, int group_rows, int K,
                                  void* out, int dtype, cudaStream_t s) {
  const int grid = grid_for((long long)groups * row_tiles(group_rows) * 32);
  cudaError_t e;
  if (dtype == SEMMOE_BF16)
    e = launch_kernel(mx4_dequantize_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, s, 1, true, codes, scales,
                      groups, group_rows, K, static_cast<__nv_bfloat16*>(out));
  else
    e = launch_kernel(mx4_dequantize_kernel<float>, dim3(grid), dim3(kThreads), 0, s, 1, true, codes, scales, groups,
                      group_rows, K, static_cast<float*>(out));
  count_launches(1);
  return e;
}

}  // namespace semmoe
