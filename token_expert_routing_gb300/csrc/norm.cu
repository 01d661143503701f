// Norms around the layer, and the layer's end in one pass:
//   norm:          out[t] = N(x[t])
//   combine_norm:  y = y_shared[t] + sum_{j<k_t} w[t,j] y_perm[pair_to_sorted[t*k_max+j]]  (or a dense row y[t])
//                  o = residual_scale * residual[t] + block_scale * gate * N_post(y),  z = N_next(o)
// with N(v) = (v - m) / sqrt(mean((v - m)^2) + eps) * (offset + weight) + bias, m = 0
// (root mean square) or the row's mean.
//
// What bounds them: bytes.  A row stays in registers from its loads to its
// stores, so every input is read once and y never reaches memory; the squares are taken
// about the mean in a second sweep over the registers, not as a difference of sums.
// A row belongs to one warp while it fits 32 lanes x 4 pieces of 16 bytes, else to one
// CTA with 1, 2 or 4 pieces a thread.
#include "common.cuh"
#include "internal.h"
#include "vec16.cuh"

namespace semmoe {
namespace {

__device__ int g_err;
__device__ __forceinline__ void flag(int bit) { atomicOr(&g_err, bit); }

constexpr int kWarpRows = 4;     // rows of a CTA whose rows belong to warps
constexpr int kMaxWarps = 32;
constexpr unsigned kAll = 0xffffffffu;

// Threads of a CTA (plan below): rows of up to 512 pieces take 256, longer ones up to 512.
template <bool WARP, int CH>
constexpr int max_threads() { return WARP ? 32 * kWarpRows : CH == 4 ? 512 : 256; }

// VEC weights from `col` on, fp32 or bf16 (16-byte aligned base; col a multiple of VEC).
template <int VEC>
__device__ __forceinline__ void load_weights(const void* p, bool bf16, int col, float (&v)[VEC]) {
  if (bf16) {
    const uint2* q = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + col);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint2 a = q[i];
      v[4 * i] = __uint_as_float(a.x << 16), v[4 * i + 1] = __uint_as_float(a.x & 0xffff0000u);
      v[4 * i + 2] = __uint_as_float(a.y << 16), v[4 * i + 3] = __uint_as_float(a.y & 0xffff0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + col);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 a = q[i];
      v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
    }
  }
}

// Sum (or maximum) over the threads that share a row: a warp, or the whole CTA
// through shared memory.  Two buffers in turn: a thread writes one again only after
// the barrier of the reduction between, which every reader of it has reached.
struct RowReduce {
  float (*part)[kMaxWarps];
  int buf;
  template <bool WARP, bool MAX>
  __device__ __forceinline__ float run(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(kAll, v, d);
      v = MAX ? fmaxf(v, o) : v + o;
    }
    if (WARP) return v;
    const int n = blockDim.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) part[buf][threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < n ? part[buf][lane] : 0.f;
    buf ^= 1;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(kAll, v, d);
      v = MAX ? fmaxf(v, o) : v + o;
    }
    return v;
  }
};

// What turns a row's values into normalised ones: (v * scale - mean) * rstd.
struct RowStats {
  float scale, mean, rstd;
};

// Columns past the row's end hold 0 and are left out of the squares about the mean.
// A row whose squares (or sum) leave fp32's range -- values past 1e18, or rows all
// below 1e-15 beside a tiny eps -- is taken again with its values scaled so that its
// largest magnitude comes to [1, 2); the branch is the same for all its threads.
template <bool WARP, int CH, int VEC>
__device__ __forceinline__ RowStats row_stats(const float (&v)[CH][VEC], int kind, int H, float eps, int col0, int step,
                                              RowReduce& red) {
  const float inv = 1.0f / (float)H;
  RowStats st{1.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    if (kind == SEMMOE_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += v[c][i] * st.scale;
      st.mean = red.run<WARP, false>(s) * inv;
    }
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (col0 + c * step < H) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float d = fmaf(v[c][i], st.scale, -st.mean);
          ss = fmaf(d, d, ss);
        }
      }
    }
    ss = red.run<WARP, false>(ss);
    st.rstd = rsqrtf(fmaf(ss, inv, eps * st.scale * st.scale));
    if (pass || ((ss >= 1e-30f || eps >= 1e-20f) && ss <= 1e36f)) return st;
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(v[c][i]));
    m = red.run<WARP, true>(m);
    const unsigned e = __float_as_uint(m) >> 23;
    if (e == 0 || e == 255) return st;  // zeros or denormals, or an infinity (the maximum is never NaN)
    // at most 1 / sqrt(eps): eps keeps its place beside the squares
    st.scale = fminf(__uint_as_float((e < 254 ? 254u - e : 1u) << 23), rsqrtf(eps));
  }
}

// v, normalised by st, times (offset + weight) plus bias.
template <int VEC>
__device__ __forceinline__ void apply_norm(float (&v)[VEC], const RowStats& st, const void* weight, const void* bias,
                                           bool w_bf16, float offset, int col) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = fmaf(v[i], st.scale, -st.mean) * st.rstd;
  if (weight != nullptr) {
    float w[VEC];
    load_weights(weight, w_bf16, col, w);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] *= offset + w[i];
  }
  if (bias != nullptr) {
    float b[VEC];
    load_weights(bias, w_bf16, col, b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] += b[i];
  }
}

// One row at a time per warp or CTA; the next row's loads are issued before this
// row's reductions.
template <typename T, bool WARP, int CH>
__global__ void __launch_bounds__(max_threads<WARP, CH>())
norm_kernel(const T* x, int T_, int H, NormArgs n, T* out) {
  using V = Vec16<T>;
  constexpr int VEC = V::N;
  __shared__ float part[2][kMaxWarps];
  RowReduce red{part, 0};
  pdl_trigger();
  pdl_wait();
  const int tid = WARP ? threadIdx.x % 32 : threadIdx.x, per = WARP ? 32 : blockDim.x;
  const int rows = WARP ? kWarpRows : 1, row_of = WARP ? threadIdx.x / 32 : 0;
  const int col0 = tid * VEC, step = per * VEC;
  uint4 raw[CH];
  auto fetch = [&](long long t) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      raw[c] = t < T_ && col < H ? *reinterpret_cast<const uint4*>(x + (size_t)t * H + col) : make_uint4(0, 0, 0, 0);
    }
  };
  long long t = (long long)blockIdx.x * rows + row_of;
  const long long stride = (long long)gridDim.x * rows;
  fetch(t);
  for (; t < T_; t += stride) {
    float v[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) V::unpack(raw[c], v[c]);
    fetch(t + stride);
    const RowStats st = row_stats<WARP, CH, VEC>(v, n.kind, H, n.eps, col0, step, red);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      if (col < H) {
        apply_norm<VEC>(v[c], st, n.weight, n.bias, n.w_bf16, n.offset, col);
        V::store(out + (size_t)t * H + col, v[c]);
      }
    }
  }
}

// As norm_kernel, with the row summed from the token's expert rows (JB slots' loads in
// flight at a time; lane j of each warp holds slot j's sorted row and gate).
template <typename T, bool WARP, int CH>
__global__ void __launch_bounds__(max_threads<WARP, CH>(), WARP ? (CH == 1 ? 8 : 4) : CH == 1 ? 4 : CH == 2 ? 2 : 1)
combine_norm_kernel(const T* y_perm, const int32_t* __restrict__ pair_to_sorted, const float* __restrict__ topk_w,
                    const T* y_shared, int T_, int H, int k_max, int P, NormArgs post, NormArgs next, const void* gate,
                    bool gate_bf16, bool gate_per_row, float block_scale, const T* residual, float residual_scale, T* out,
                    T* next_out) {
  using V = Vec16<T>;
  constexpr int VEC = V::N, JB = CH == 1 ? 4 : CH == 2 ? 3 : 2;
  __shared__ float part[2][kMaxWarps];
  RowReduce red{part, 0};
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const int tid = WARP ? lane : threadIdx.x, per = WARP ? 32 : blockDim.x;
  const int rows = WARP ? kWarpRows : 1, row_of = WARP ? threadIdx.x / 32 : 0;
  const int col0 = tid * VEC, step = per * VEC;
  const bool dense = pair_to_sorted == nullptr;
  const int kk = dense ? 1 : k_max < 32 ? k_max : 32;
  int q_l = -1;
  float w_l = 0.f;
  auto fetch_slots = [&](long long t) {
    q_l = -1, w_l = 0.f;
    if (t >= T_ || lane >= kk) return;
    if (dense) {
      q_l = (int)t, w_l = 1.f;
    } else {
      q_l = pair_to_sorted[(size_t)t * k_max + lane];
      w_l = topk_w[(size_t)t * k_max + lane];
    }
  };
  long long t = (long long)blockIdx.x * rows + row_of;
  const long long stride = (long long)gridDim.x * rows;
  fetch_slots(t);
  for (; t < T_; t += stride) {
    if (!dense && q_l >= P) {
      flag(SEMMOE_DEVERR_PAIRS);
      q_l = -1;
    }
    uint4 res[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      res[c] = residual != nullptr && col < H ? *reinterpret_cast<const uint4*>(residual + (size_t)t * H + col)
                                              : make_uint4(0, 0, 0, 0);
    }
    float v[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      if (y_shared != nullptr && col < H) {
        V::load(y_shared + (size_t)t * H + col, v[c]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] = 0.f;
      }
    }
    for (int j0 = 0; j0 < kk; j0 += JB) {
      uint4 raw[JB][CH];
      float wj[JB];
      bool ok[JB];
#pragma unroll
      for (int b = 0; b < JB; ++b) {
        const int q = __shfl_sync(kAll, q_l, (j0 + b) & 31);
        wj[b] = __shfl_sync(kAll, w_l, (j0 + b) & 31);
        ok[b] = j0 + b < kk && q >= 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int col = col0 + c * step;
          raw[b][c] = ok[b] && col < H ? *reinterpret_cast<const uint4*>(y_perm + (size_t)q * H + col) : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int b = 0; b < JB; ++b) {
        if (!ok[b]) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float r[VEC];
          V::unpack(raw[b][c], r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[c][i] = fmaf(wj[b], r[i], v[c][i]);
        }
      }
    }
    for (int j = 32; !dense && j < k_max; ++j) {  // budgets above 32 experts: read the slot directly
      const int q = pair_to_sorted[(size_t)t * k_max + j];
      if (q < 0) continue;
      if (q >= P) {
        flag(SEMMOE_DEVERR_PAIRS);
        continue;
      }
      const float w = topk_w[(size_t)t * k_max + j];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = col0 + c * step;
        if (col < H) {
          float r[VEC];
          V::load(y_perm + (size_t)q * H + col, r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[c][i] = fmaf(w, r[i], v[c][i]);
        }
      }
    }
    fetch_slots(t + stride);
    RowStats st{1.f, 0.f, 1.f};
    if (post.kind != SEMMOE_NORM_NONE) st = row_stats<WARP, CH, VEC>(v, post.kind, H, post.eps, col0, step, red);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      if (col < H) {
        if (post.kind != SEMMOE_NORM_NONE) apply_norm<VEC>(v[c], st, post.weight, post.bias, post.w_bf16, post.offset, col);
        if (gate != nullptr) {
          float g[VEC];
          const size_t at = gate_per_row ? (size_t)t * H : 0;
          load_weights(gate_bf16 ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(gate) + at)
                                 : static_cast<const void*>(static_cast<const float*>(gate) + at),
                       gate_bf16, col, g);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[c][i] *= g[i];
        }
        float r[VEC];
        V::unpack(res[c], r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] = residual != nullptr ? fmaf(residual_scale, r[i], block_scale * v[c][i]) : block_scale * v[c][i];
        V::store(out + (size_t)t * H + col, v[c]);
      }
    }
    if (next.kind == SEMMOE_NORM_NONE) continue;
    st = row_stats<WARP, CH, VEC>(v, next.kind, H, next.eps, col0, step, red);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      if (col < H) {
        apply_norm<VEC>(v[c], st, next.weight, next.bias, next.w_bf16, next.offset, col);
        V::store(next_out + (size_t)t * H + col, v[c]);
      }
    }
  }
}

// How the rows are spread: a warp or a CTA of `threads` for each, `pieces` of 16 bytes a thread.
struct RowPlan {
  bool warp;
  int pieces, threads;
};
RowPlan plan(int H, int vec) {
  const int n = ceil_div(H, vec);
  if (n <= 128) return RowPlan{true, n <= 32 ? 1 : n <= 64 ? 2 : 4, 32 * kWarpRows};
  const int pieces = n <= 256 ? 1 : n <= 512 ? 2 : 4;
  return RowPlan{false, pieces, ceil_div(ceil_div(n, pieces), 32) * 32};
}

// CTAs that are resident at once, for a grid whose CTAs take rows in turn.
template <typename K>
cudaError_t resident_grid(K kern, int threads, long long want, unsigned* grid) {
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0);
  if (e != cudaSuccess) return e;
  const long long cap = (long long)(per_sm > 0 ? per_sm : 1) * sm_count();
  *grid = (unsigned)(want < cap ? want : cap);
  return cudaSuccess;
}

template <typename T, bool WARP, int CH>
cudaError_t launch_norm_t(const RowPlan& p, const void* x, int T_, int H, const NormArgs& n, void* out, cudaStream_t s) {
  auto kern = norm_kernel<T, WARP, CH>;
  unsigned grid;
  cudaError_t e = resident_grid(kern, p.threads, WARP ? ceil_div(T_, kWarpRows) : T_, &grid);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid), dim3(p.threads), 0, s, 1, true, static_cast<const T*>(x), T_, H, n,
                       static_cast<T*>(out));
}

template <typename T, bool WARP, int CH>
cudaError_t launch_combine_norm_t(const RowPlan& p, const CombineNorm& a, cudaStream_t s) {
  auto kern = combine_norm_kernel<T, WARP, CH>;
  unsigned grid;
  cudaError_t e = resident_grid(kern, p.threads, WARP ? ceil_div(a.T, kWarpRows) : a.T, &grid);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid), dim3(p.threads), 0, s, 1, true, static_cast<const T*>(a.y_perm),
                       a.pair_to_sorted, a.topk_w, static_cast<const T*>(a.y_shared), a.T, a.H, a.k_max, a.P, a.post,
                       a.next, a.gate, a.gate_bf16, a.gate_rows > 1, a.block_scale, static_cast<const T*>(a.residual),
                       a.residual_scale, static_cast<T*>(a.out), static_cast<T*>(a.next_out));
}

template <typename F>
cudaError_t by_plan(const RowPlan& p, F&& f) {
  using std::integral_constant;
  using yes = std::true_type;
  using no = std::false_type;
  if (p.warp) {
    if (p.pieces == 1) return f(yes{}, integral_constant<int, 1>{});
    if (p.pieces == 2) return f(yes{}, integral_constant<int, 2>{});
    return f(yes{}, integral_constant<int, 4>{});
  }
  if (p.pieces == 1) return f(no{}, integral_constant<int, 1>{});
  if (p.pieces == 2) return f(no{}, integral_constant<int, 2>{});
  return f(no{}, integral_constant<int, 4>{});
}

}  // namespace

int norm_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_norm(const void* x, int dtype, int T, int H, const NormArgs& n, void* out, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const RowPlan p = plan(H, dtype == SEMMOE_BF16 ? 8 : 4);
  cudaError_t e = by_plan(p, [&](auto warp, auto ch) {
    constexpr bool W = decltype(warp)::value;
    constexpr int C = decltype(ch)::value;
    return dtype == SEMMOE_BF16 ? launch_norm_t<__nv_bfloat16, W, C>(p, x, T, H, n, out, s)
                                : launch_norm_t<float, W, C>(p, x, T, H, n, out, s);
  });
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_combine_norm(const CombineNorm& a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const RowPlan p = plan(a.H, dtype == SEMMOE_BF16 ? 8 : 4);
  cudaError_t e = by_plan(p, [&](auto warp, auto ch) {
    constexpr bool W = decltype(warp)::value;
    constexpr int C = decltype(ch)::value;
    return dtype == SEMMOE_BF16 ? launch_combine_norm_t<__nv_bfloat16, W, C>(p, a, s)
                                : launch_combine_norm_t<float, W, C>(p, a, s);
  });
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace semmoe
