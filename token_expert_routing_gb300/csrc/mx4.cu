// Quantisation to 4-bit microscaled values and back (format and layouts:
// mx4.cuh).  Pure data movement: per value 2 or 4 bytes in and 17/32 of a byte
// out, so the bound is HBM bandwidth; a lane takes 8 values of a row (one
// 16-byte load of bf16), four lanes share a block, sixteen one 128-column tile.
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"

namespace semmoe {
namespace {

using namespace mx4;

__device__ int g_err;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSpan = 256;  // columns a warp takes at once, 8 per lane

// Eight consecutive values of a row as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// The lane's eight codes, and in every lane of a 16-lane half the half's four
// scales as one word (block j at byte j).  Whole warp.
__device__ __forceinline__ uint32_t quantise8(const float (&v)[8], uint32_t& scales) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  const uint32_t b = scale_code(a);
  const float f = inverse_scale(b);
  uint32_t w = b << (8 * ((threadIdx.x >> 2) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  scales = w | __shfl_xor_sync(0xffffffffu, w, 8);
  return encode8(v[0] * f, v[1] * f, v[2] * f, v[3] * f, v[4] * f, v[5] * f, v[6] * f, v[7] * f);
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
      const int c = c0 + lane * 8;
      float v[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c < K && in_group + 32 * i < group_rows) {
          load8(x + (row + 32 * i) * K + c, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
      }
      uint32_t s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = quantise8(v[i], s[i]);
        if (c < K && in_group + 32 * i < group_rows)
          *reinterpret_cast<uint32_t*>(codes + ((row + 32 * i) * K + c) / 2) = w;
      }
      const int ct = c / kTileCols;
      if ((lane & 15) == 0 && ct < kc)
        *reinterpret_cast<uint4*>(scales + ((size_t)tile * kc + ct) * kTileBytes + 16 * r0) =
            make_uint4(s[0], s[1], s[2], s[3]);
    }
  }
}

// Token rows into expert order: one warp per token quantises its row once and
// writes the codes and scales to each of its pairs' sorted rows.
constexpr int kMaxE = 256;
constexpr int kBatch = 8;  // column spans held in registers: 2048 columns

template <typename T>
__global__ void __launch_bounds__(kThreads)
mx4_quantize_rows_kernel(const T* __restrict__ x, int n_tok, int K, const int32_t* __restrict__ pair_to_sorted,
                         int k_max, int P, const int32_t* __restrict__ expert_offsets, int E,
                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ int off[kMaxE + 1], first[kMaxE], scan[kThreads];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  // row tile at which each expert's rows start
  for (int e = threadIdx.x; e <= E; e += kThreads) off[e] = expert_offsets[e];
  __syncthreads();
  int mine = 0;
  if ((int)threadIdx.x < E) {
    const int lo = off[threadIdx.x], hi = off[threadIdx.x + 1];
    if (lo < 0 || hi < lo || hi > P) atomicOr(&g_err, SEMMOE_DEVERR_PAIRS);
    else mine = row_tiles(hi - lo);
  }
  scan[threadIdx.x] = mine;
  __syncthreads();
  for (int d = 1; d < kThreads; d <<= 1) {
    const int v = (int)threadIdx.x >= d ? scan[threadIdx.x - d] : 0;
    __syncthreads();
    scan[threadIdx.x] += v;
    __syncthreads();
  }
  if ((int)threadIdx.x < E) first[threadIdx.x] = scan[threadIdx.x] - mine;
  __syncthreads();
  const int kc = col_tiles(K);
  const int max_tiles = P / kTileRows + E;  // what the caller's scales hold
  for (int t = blockIdx.x * kWarps + threadIdx.x / 32; t < n_tok; t += gridDim.x * kWarps) {
    for (int c0 = 0; c0 < K; c0 += kBatch * kSpan) {
      float v[kBatch][8];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * kSpan + lane * 8;
        if (c < K) {
          load8(x + (size_t)t * K + c, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
      }
      uint32_t w[kBatch], s[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) w[i] = quantise8(v[i], s[i]);
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
            const int c = c0 + i * kSpan + lane * 8;
            if (c < K) *reinterpret_cast<uint32_t*>(row + c / 2) = w[i];
            if ((lane & 15) == 0 && c < K) *reinterpret_cast<uint32_t*>(sc + (size_t)(c / kTileCols) * kTileBytes) = s[i];
          }
        }
      }
    }
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 w;
  uint32_t* a = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    a[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
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
    for (int c = lane * 8; c < K; c += kSpan) {
      const uint4 sw = __ldg(reinterpret_cast<const uint4*>(
          scales + ((size_t)tile * kc + c / kTileCols) * kTileBytes + 16 * r0));
      const uint32_t s[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (in_group + 32 * i >= group_rows) break;
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + ((row + 32 * i) * K + c) / 2));
        const float f = scale_value((s[i] >> (8 * ((c / kBlock) & 3))) & 255u);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = decode(w >> (4 * j)) * f;
        store8(out + (row + 32 * i) * K + c, v);
      }
    }
  }
}

// One warp per unit until every SM holds eight CTAs, then a grid-stride loop.
int grid_for(long long units) {
  const long long blocks = (units + kWarps - 1) / kWarps, cap = 8LL * sm_count();
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
  const int grid = grid_for(T);
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
