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
// Norms about the mean have kernels of their own (MEAN, MEANS): one for both would slow the others down (the norm of
// 16384 x 2048 23.7 us where it takes 22.9, the combine below 137 where it takes 129).
// A row belongs to one warp while it fits 32 lanes x 4 pieces of 16 bytes, else to one CTA.
// Measured (GB300, calls of a captured graph): the norm of 16384 x 2048 bf16, 22.9 us (5.9 TB/s); the combine of 8 rows a token
// with both norms, a gate per channel and the residual, 16384 x 2048 bf16, 129 us (5.7 TB/s); a dense block's row with a gate a
// token, the residual and one norm about the mean, 4096 x 2048 bf16, 17.1 us (4.9 TB/s).
#include "common.cuh"
#include "internal.h"
#include "vec16.cuh"

namespace semmoe {
namespace {

__device__ int g_err;
__device__ __forceinline__ void flag(int bit) { atomicOr(&g_err, bit); }

constexpr int kWarpRows = 4;     // rows of a CTA whose rows belong to warps
constexpr int PIECES = 2;        // of 16 bytes a thread, of many rows (more only where a CTA's threads would not do)
constexpr int RING = 4;          // rows on their way to a row's threads, and the one in use
constexpr int kMaxWarps = 16;    // of a CTA
constexpr unsigned kAll = 0xffffffffu;
static_assert(kMaxWarps == 16, "half of a warp's lanes add up one sum of the warps'");

// Threads of a CTA (plan below), and CTAs that an SM's registers have to hold: as many as come without spills that matter
// (4 CTAs of the combine's two-piece form 129 us at 16384 x 2048, 3 of them 139, 5 142; 4 of the dense one's 27 us at
// 4096 x 2048, 3 of them 17.1).
template <bool WARP, int CH>
constexpr int max_threads() { return WARP ? 32 * kWarpRows : CH == 4 ? 512 : 256; }
template <bool WARP, int CH>
constexpr int norm_ctas() { return WARP ? (CH == 4 ? 6 : 8) : CH == 1 ? 5 : CH == 2 ? 4 : 1; }
template <bool WARP, int CH>
constexpr int min_ctas() { return WARP ? (CH == 4 ? 6 : 8) : CH == 1 ? 4 : CH == 2 ? 4 : 1; }

template <bool WARP, int CH>
constexpr int dense_ctas() { return WARP ? (CH == 4 ? 3 : CH == 2 ? 6 : 8) : CH == 1 ? 4 : CH == 2 ? 3 : 1; }

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
  float (*part)[2 * kMaxWarps];
  int buf;
  template <bool MAX>
  static __device__ __forceinline__ float add(float v, float o) { return MAX ? fmaxf(v, o) : v + o; }
  // over the warps' values, from `from` on in the buffer; each half of a warp
  template <bool MAX>
  __device__ __forceinline__ float warps(int from) {
    const int n = blockDim.x / 32, j = threadIdx.x % kMaxWarps;
    float v = j < n ? part[buf][from + j] : 0.f;
    buf ^= 1;
#pragma unroll
    for (int d = kMaxWarps / 2; d > 0; d >>= 1) v = add<MAX>(v, __shfl_xor_sync(kAll, v, d));
    return v;
  }
  template <bool WARP, bool MAX>
  __device__ __forceinline__ float run(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = add<MAX>(v, __shfl_xor_sync(kAll, v, d));
    if (WARP) return v;
    if (threadIdx.x % 32 == 0) part[buf][threadIdx.x / 32] = v;
    __syncthreads();
    return warps<MAX>(0);
  }
  // two sums at once: half of the lanes add up one, half the other
  template <bool WARP>
  __device__ __forceinline__ float2 pair(float x, float y) {
    const bool up = threadIdx.x & 16;
    float v = (up ? y : x) + __shfl_xor_sync(kAll, up ? x : y, 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    if (!WARP) {
      if (threadIdx.x % 16 == 0) part[buf][(up ? kMaxWarps : 0) + threadIdx.x / 32] = v;
      __syncthreads();
      v = warps<false>(up ? kMaxWarps : 0);
    }
    const float o = __shfl_xor_sync(kAll, v, 16);
    return up ? make_float2(o, v) : make_float2(v, o);
  }
};

// What turns a row's values into normalised ones: v * a, or (v * scale - mean) * a + b about the mean.
struct RowStats {
  float scale, mean, a, b;
};

// Columns past the row's end hold 0 and are left out of the squares about the mean.
// about_mean: SEMMOE_NORM_LAYER, else SEMMOE_NORM_RMS.
// A row whose squares (or sum) leave fp32's range -- values past 1e18, or rows all
// below 1e-15 beside a tiny eps -- is taken again with its values scaled so that its
// largest magnitude comes to [1, 2); the branch is the same for all its threads.
// The mean, as a sum in fp32 has it, is off by some steps of the largest value, which may be more than the values
// differ by.  So the differences from it are summed beside their squares: what they come to on average is taken off each of
// them, and its square off theirs, and no error of the mean is left but that of numbers as small as the differences.  In rows
// that differ by a few steps of fp32 those are small multiples of one step, whose sums are exact, and the mean comes out
// as a sum of two numbers: a constant row gives 0 whatever its value, with a variance that is kept above 0.
template <bool WARP, int CH, int VEC>
__device__ __forceinline__ RowStats row_stats(const float (&v)[CH][VEC], bool about_mean, int H, float eps, int col0, int step,
                                              RowReduce& red) {
  const float inv = 1.0f / (float)H;
  float scale = 1.0f, mean = 0.0f;
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    if (about_mean) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += pass ? v[c][i] * scale : v[c][i];
      mean = red.run<WARP, false>(s) * inv;
    }
    float ss = 0.f, off = 0.f;  // off: the differences' own mean
    if (pass || about_mean) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (col0 + c * step < H) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float d = fmaf(v[c][i], scale, -mean);
            s += d;
            ss = fmaf(d, d, ss);
          }
        }
      }
      if (about_mean) {
        const float2 both = red.pair<WARP>(ss, s);
        ss = both.x, off = both.y * inv;
        off = fmaf(fmaf(-off, (float)H, both.y), inv, off);  // exact where a quotient is
      } else {
        ss = red.run<WARP, false>(ss);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss = fmaf(v[c][i], v[c][i], ss);
      ss = red.run<WARP, false>(ss);
    }
    const float least = eps * scale * scale;
    float var = fmaf(ss, inv, least);
    if (about_mean) var = fmaxf(fmaf(-off, off, var), fmaxf(least, 1.17549435e-38f));  // (a NaN comes through b)
    const float rstd = rsqrtf(var);
    RowStats st{scale, mean, scale * rstd, 0.f};
    if (about_mean) {  // mean + off = st.mean + rest, exactly
      st.mean = mean + off;
      const float o = st.mean - mean, rest = (mean - (st.mean - o)) + (off - o);
      st.a = rstd, st.b = -rest * rstd;
    }
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
    scale = fminf(__uint_as_float((e < 254 ? 254u - e : 1u) << 23), rsqrtf(eps));
  }
}

// v, normalised by st, times (offset + weight) plus bias.
template <int VEC>
__device__ __forceinline__ void apply_norm(float (&v)[VEC], const RowStats& st, bool about_mean, const NormArgs& n,
                                           int col) {
  if (about_mean) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = fmaf(fmaf(v[i], st.scale, -st.mean), st.a, st.b);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] *= st.a;
  }
  if (n.weight != nullptr) {
    float w[VEC];
    load_weights(n.weight, n.w_bf16, col, w);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] *= n.offset + w[i];
  }
  if (n.bias != nullptr) {
    float b[VEC];
    load_weights(n.bias, n.w_bf16, col, b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] += b[i];
  }
}

// One row at a time per warp or CTA: the loads of the AHEAD next rows are in flight, in registers, through this row's reductions.
template <typename T, bool WARP, int CH, bool MEAN>
__global__ void __launch_bounds__(max_threads<WARP, CH>(), norm_ctas<WARP, CH>())
norm_kernel(const T* x, int T_, int H, const __grid_constant__ NormArgs n, T* out) {
  using V = Vec16<T>;
  constexpr int VEC = V::N, AHEAD = CH == 1 ? 2 : 1;
  __shared__ float part[2][2 * kMaxWarps];
  RowReduce red{part, 0};
  pdl_trigger();
  pdl_wait();
  const int tid = WARP ? threadIdx.x % 32 : threadIdx.x, per = WARP ? 32 : blockDim.x;
  const int rows = WARP ? kWarpRows : 1, row_of = WARP ? threadIdx.x / 32 : 0;
  const int col0 = tid * VEC, step = per * VEC;
  uint4 raw[AHEAD][CH];
  auto fetch = [&](long long t, uint4 (&r)[CH]) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      r[c] = t < T_ && col < H ? *reinterpret_cast<const uint4*>(x + (size_t)t * H + col) : make_uint4(0, 0, 0, 0);
    }
  };
  long long t = (long long)blockIdx.x * rows + row_of;
  const long long stride = (long long)gridDim.x * rows;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(t + i * stride, raw[i]);
  while (t < T_) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (t >= T_) break;
      float v[CH][VEC];
#pragma unroll
      for (int c = 0; c < CH; ++c) V::unpack(raw[i][c], v[c]);
      fetch(t + AHEAD * stride, raw[i]);
      const RowStats st = row_stats<WARP, CH, VEC>(v, MEAN, H, n.eps, col0, step, red);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = col0 + c * step;
        if (col < H) {
          apply_norm<VEC>(v[c], st, MEAN, n, col);
          V::store(out + (size_t)t * H + col, v[c]);
        }
      }
      t += stride;
    }
  }
}

// From the block's row on: norm, gate, residual, the sum's row stored, the next block's norm, its row stored.  `next` comes to
// the gate's own row (of type T), then the residual's; `piece` reads 16 bytes a thread of it.
template <typename T, bool WARP, int CH, bool MEANS, typename Next, typename Piece>
__device__ __forceinline__ void finish_row(const CombineNorm& a, long long t, float (&v)[CH][Vec16<T>::N], int col0, int step,
                                           RowReduce& red, bool own_gate, Next&& next, Piece&& piece) {
  using V = Vec16<T>;
  constexpr int VEC = V::N;
  const int H = a.H;
  const bool mean_post = MEANS && a.post.kind == SEMMOE_NORM_LAYER, mean_next = MEANS && a.next.kind == SEMMOE_NORM_LAYER;
  if (a.post.kind != SEMMOE_NORM_NONE) {
    const RowStats st = row_stats<WARP, CH, VEC>(v, mean_post, H, a.post.eps, col0, step, red);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      if (col < H) apply_norm<VEC>(v[c], st, mean_post, a.post, col);
    }
  }
  if (a.gate != nullptr) {
    const int at = own_gate ? next(true) : 0;
    const size_t row = a.gate_rows > 1 ? (size_t)t * H : 0;
    const void* p = a.gate_bf16 ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(a.gate) + row)
                                : static_cast<const void*>(static_cast<const float*>(a.gate) + row);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col0 + c * step;
      if (col < H) {
        float g[VEC];
        if (own_gate) piece(true, at, c, g);
        else load_weights(p, a.gate_bf16, col, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] *= g[i];
      }
    }
  }
  const int at = a.residual != nullptr ? next(false) : 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = col0 + c * step;
    if (col < H) {
      if (a.residual != nullptr) {
        float r[VEC];
        piece(false, at, c, r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] = fmaf(a.residual_scale, r[i], a.block_scale * v[c][i]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] *= a.block_scale;
      }
      V::store(static_cast<T*>(a.out) + (size_t)t * H + col, v[c]);
    }
  }
  if (a.next.kind == SEMMOE_NORM_NONE) return;
  const RowStats st = row_stats<WARP, CH, VEC>(v, mean_next, H, a.next.eps, col0, step, red);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = col0 + c * step;
    if (col < H) {
      apply_norm<VEC>(v[c], st, mean_next, a.next, col);
      V::store(static_cast<T*>(a.next_out) + (size_t)t * H + col, v[c]);
    }
  }
}

// A dense block's row (no slots).  A token needs the same two or three rows each time, so they need no list and no ring: their
// next pieces are fetched into registers as soon as this token's have been used (17.1 us at 4096 x 2048 bf16, 23.9 through
// the ring below).  A shared row, which a dense block seldom has, is read where it is added.
template <typename T, bool WARP, int CH, bool MEANS>
__global__ void __launch_bounds__(max_threads<WARP, CH>(), dense_ctas<WARP, CH>())
dense_norm_kernel(const __grid_constant__ CombineNorm a) {
  using V = Vec16<T>;
  constexpr int VEC = V::N;
  __shared__ float part[2][2 * kMaxWarps];
  RowReduce red{part, 0};
  pdl_trigger();
  pdl_wait();
  const int tid = WARP ? threadIdx.x % 32 : threadIdx.x, per = WARP ? 32 : blockDim.x;
  const int rows = WARP ? kWarpRows : 1, row_of = WARP ? threadIdx.x / 32 : 0;
  const int col0 = tid * VEC, step = per * VEC, T_ = a.T, H = a.H;
  const T *y = static_cast<const T*>(a.y_perm), *y_shared = static_cast<const T*>(a.y_shared),
          *residual = static_cast<const T*>(a.residual),
          *gate_rows = a.gate_rows > 1 && a.gate_bf16 == (sizeof(T) == 2) ? static_cast<const T*>(a.gate) : nullptr;
  uint4 raw[3][CH];  // pieces of the block's row, the gate's, the residual's
  auto fetch = [&](long long t, int c, const T* p, uint4& r) {
    const int col = col0 + c * step;
    r = p != nullptr && t < T_ && col < H ? *reinterpret_cast<const uint4*>(p + (size_t)t * H + col) : make_uint4(0, 0, 0, 0);
  };
  long long t = (long long)blockIdx.x * rows + row_of;
  const long long stride = (long long)gridDim.x * rows;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    fetch(t, c, y, raw[0][c]);
    fetch(t, c, gate_rows, raw[1][c]);
    fetch(t, c, residual, raw[2][c]);
  }
  for (; t < T_; t += stride) {
    float v[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      V::unpack(raw[0][c], v[c]);
      fetch(t + stride, c, y, raw[0][c]);
    }
    if (y_shared != nullptr) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = col0 + c * step;
        if (col < H) {
          float r[VEC];
          V::load(y_shared + (size_t)t * H + col, r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[c][i] += r[i];
        }
      }
    }
    finish_row<T, WARP, CH, MEANS>(
        a, t, v, col0, step, red, gate_rows != nullptr, [&](bool) { return 0; },
        [&](bool gate, int, int c, float (&r)[VEC]) {
          uint4& mine = gate ? raw[1][c] : raw[2][c];
          V::unpack(mine, r);
          fetch(t + stride, c, gate ? gate_rows : residual, mine);
        });
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The rows that a token needs, in the order in which they are used, as a warp's lanes write them down when the copies come
// to it: the shared experts', its slots', a gate's own, the residual's.  At most 32 slots; an empty list has one item, NULL.
struct Token {
  const void* row[36];
  float weight[32];  // of the slots
  int items, slots;
};

// One row at a time per warp or CTA.  The rows that a token needs -- the shared experts', its slots', a gate's, the residual's
// -- pass one after the other through a ring of RING of them in shared memory: a thread copies its own pieces of the next
// RING - 1 rows asynchronously, into the next tokens' too, so that bytes stay in flight through the reductions and nothing is
// waited for but its own copies.
// Lane j of each warp reads slot j's sorted row and gate, one token ahead of the copies (up to 32 slots; the ones behind
// are read where they are used).
template <typename T, bool WARP, int CH, bool MEANS>
__global__ void __launch_bounds__(max_threads<WARP, CH>(), min_ctas<WARP, CH>())
combine_norm_kernel(const __grid_constant__ CombineNorm a) {
  using V = Vec16<T>;
  constexpr int VEC = V::N;
  extern __shared__ uint4 ring[];  // [RING][CH][threads], then the lists of RING tokens a warp
  __shared__ float part[2][2 * kMaxWarps];
  RowReduce red{part, 0};
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, T_ = a.T, H = a.H;
  const int tid = WARP ? lane : threadIdx.x, per = WARP ? 32 : blockDim.x;
  const int rows = WARP ? kWarpRows : 1, row_of = WARP ? warp : 0;
  const int col0 = tid * VEC, step = per * VEC;
  const int kk = a.k_max < 32 ? a.k_max : 32;
  const T *y_perm = static_cast<const T*>(a.y_perm), *y_shared = static_cast<const T*>(a.y_shared),
          *residual = static_cast<const T*>(a.residual), *gate_rows = static_cast<const T*>(a.gate);
  const bool own_gate = a.gate != nullptr && a.gate_rows > 1 && a.gate_bf16 == (sizeof(T) == 2);  // a row of its own, of type T
  const int first_slot = y_shared != nullptr ? 1 : 0;
  const uint32_t piece = blockDim.x * 16, base = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
  Token* tokens = reinterpret_cast<Token*>(ring + RING * CH * blockDim.x) + warp * RING;

  int q_l = -1;  // slot `lane` of the token after the copies' one
  float w_l = 0.f;
  auto read_slots = [&](long long t) {
    q_l = -1, w_l = 0.f;
    if (t >= T_ || lane >= kk) return;
    q_l = a.pair_to_sorted[(size_t)t * a.k_max + lane];
    w_l = a.topk_w[(size_t)t * a.k_max + lane];
  };
  const long long stride = (long long)gridDim.x * rows;
  // the copies' place: a token, its list (kept for the sums, RING of them in turn), the next item of it
  long long t_c = (long long)blockIdx.x * rows + row_of;
  int turn_c = 0, next = 0, items = 0, to = 0;
  auto enter = [&]() {
    if (q_l >= a.P) {
      flag(SEMMOE_DEVERR_PAIRS);
      q_l = -1;
    }
    Token& tk = tokens[turn_c];
    const unsigned live = __ballot_sync(kAll, q_l >= 0);
    const int n = __popc(live);
    items = first_slot + n;
    if (q_l >= 0) {
      const int j = __popc(live & lanemask_lt());
      tk.row[first_slot + j] = y_perm + (size_t)q_l * H;
      tk.weight[j] = w_l;
    }
    if (first_slot && lane == 0) tk.row[0] = y_shared + (size_t)t_c * H;
    if (own_gate) {
      if (lane == 0) tk.row[items] = gate_rows + (size_t)t_c * H;
      ++items;
    }
    if (residual != nullptr) {
      if (lane == 0) tk.row[items] = residual + (size_t)t_c * H;
      ++items;
    }
    if (items == 0) {
      if (lane == 0) tk.row[0] = nullptr;
      items = 1;
    }
    if (lane == 0) tk.items = items, tk.slots = n;
    next = 0;
    __syncwarp();
    read_slots(t_c + stride);
  };
  auto copy_next = [&]() {
    if (next == items && t_c < T_) {
      t_c += stride;
      turn_c = (turn_c + 1) % RING;
      if (t_c < T_) enter();
    }
    if (t_c < T_) {
      const T* src = static_cast<const T*>(tokens[turn_c].row[next++]);
      if (src != nullptr) {
        src += col0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (col0 + c * step < H) cp_async16(base + (to * CH + c) * piece, src + c * step);
      }
      to = (to + 1) % RING;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int from = 0;
  auto next_item = [&]() {  // the ring's place of the next item, once its pieces are there
    copy_next();
    asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
    const int at = from;
    from = (from + 1) % RING;
    return at;
  };
  auto values = [&](int at, int c, float (&v)[VEC]) { V::unpack(ring[(at * CH + c) * blockDim.x + threadIdx.x], v); };

  long long t = t_c;
  if (t < T_) {
    read_slots(t);
    enter();
  }
#pragma unroll
  for (int i = 0; i < RING - 1; ++i) copy_next();
  for (int turn = 0; t < T_; t += stride, turn = (turn + 1) % RING) {
    __syncwarp();
    float v[CH][VEC];
    if (y_shared != nullptr) {
      const int at = next_item();
#pragma unroll
      for (int c = 0; c < CH; ++c) values(at, c, v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] = 0.f;
    }
    const Token& tk = tokens[turn];
    const int n = tk.slots;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const float w = tk.weight[j];
      const int at = next_item();
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float r[VEC];
        values(at, c, r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] = fmaf(w, r[i], v[c][i]);
      }
    }
    if (tk.row[0] == nullptr) next_item();  // the list's only item, which holds nothing
    for (int j = 32; j < a.k_max; ++j) {  // budgets above 32 experts: read the slot directly
      const int q = a.pair_to_sorted[(size_t)t * a.k_max + j];
      if (q < 0) continue;
      if (q >= a.P) {
        flag(SEMMOE_DEVERR_PAIRS);
        continue;
      }
      const float w = a.topk_w[(size_t)t * a.k_max + j];
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
#pragma unroll
    for (int c = 0; c < CH; ++c) {  // columns past the row's end hold 0
      if (col0 + c * step >= H) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] = 0.f;
      }
    }
    finish_row<T, WARP, CH, MEANS>(
        a, t, v, col0, step, red, own_gate, [&](bool) { return next_item(); },
        [&](bool, int at, int c, float (&r)[VEC]) { values(at, c, r); });
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// How the rows are spread: a warp or a CTA of `threads` for each, `pieces` of 16 bytes a thread.
struct RowPlan {
  bool warp;
  int pieces, threads;
};
// Many rows: two pieces a thread, so that reductions and loop are shared by more bytes (the combine of 16384 x 2048 takes 166 us
// with one piece and 129 with two; four mean fewer warps at a time).  Few rows, whose time is one row's: as many threads as
// there are pieces.
RowPlan plan(int H, int vec, int T) {
  const int n = ceil_div(H, vec);
  if (T >= 4 * sm_count() && n <= 128) return RowPlan{true, n <= 32 ? 1 : n <= 64 ? 2 : 4, 32 * kWarpRows};
  const int few = n <= 256 ? 1 : n <= 512 ? 2 : 4, pieces = T < 4 * sm_count() || few > PIECES ? few : PIECES;
  return RowPlan{false, pieces, ceil_div(ceil_div(n, pieces), 32) * 32};
}

// CTAs that are resident at once, for a grid whose CTAs take rows in turn.
unsigned resident_grid(const RowPlan& p, int T, int per_sm) {
  const long long want = p.warp ? ceil_div(T, kWarpRows) : T, cap = (long long)per_sm * sm_count();
  return (unsigned)(want < cap ? want : cap);
}
// What registers (as the launch bounds have it) and shared memory let an SM hold.
int ctas_per_sm(const RowPlan& p, int by_bounds, int bound_threads, int smem) {
  int n = by_bounds * bound_threads / p.threads;
  const int by_smem = 233472 / (smem + 1024 + 256), by_threads = 2048 / p.threads;
  if (n > by_smem) n = by_smem;
  if (n > by_threads) n = by_threads;
  return n > 0 ? n : 1;
}

template <typename T, bool WARP, int CH>
cudaError_t launch_norm_t(const RowPlan& p, const void* x, int T_, int H, const NormArgs& n, void* out, cudaStream_t s) {
  const int per_sm = ctas_per_sm(p, norm_ctas<WARP, CH>(), max_threads<WARP, CH>(), 0);
  auto kern = n.kind == SEMMOE_NORM_LAYER ? norm_kernel<T, WARP, CH, true> : norm_kernel<T, WARP, CH, false>;
  return launch_kernel(kern, dim3(resident_grid(p, T_, per_sm)), dim3(p.threads), 0, s, 1, true, static_cast<const T*>(x), T_, H,
                       n, static_cast<T*>(out));
}

template <typename T, bool WARP, int CH, bool MEANS>
cudaError_t launch_t(const RowPlan& p, const CombineNorm& a, cudaStream_t s) {
  if (a.pair_to_sorted == nullptr) {
    const int n = ctas_per_sm(p, dense_ctas<WARP, CH>(), max_threads<WARP, CH>(), 0);
    return launch_kernel(dense_norm_kernel<T, WARP, CH, MEANS>, dim3(resident_grid(p, a.T, n)), dim3(p.threads), 0, s, 1, true, a);
  }
  auto kern = combine_norm_kernel<T, WARP, CH, MEANS>;
  const int smem = RING * (CH * p.threads * 16 + p.threads / 32 * (int)sizeof(Token));
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, RING * (CH * max_threads<WARP, CH>() * 16 + max_threads<WARP, CH>() / 32 * (int)sizeof(Token)), smem_set);
  if (e != cudaSuccess) return e;
  const int per_sm = ctas_per_sm(p, min_ctas<WARP, CH>(), max_threads<WARP, CH>(), smem);
  return launch_kernel(kern, dim3(resident_grid(p, a.T, per_sm)), dim3(p.threads), (size_t)smem, s, 1, true, a);
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

cudaError_t launch_combine_norm(const CombineNorm& a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const RowPlan p = plan(a.H, dtype == SEMMOE_BF16 ? 8 : 4, a.T);
  cudaError_t e = by_plan(p, [&](auto warp, auto ch) {
    constexpr bool W = decltype(warp)::value;
    constexpr int C = decltype(ch)::value;
    if (a.post.kind == SEMMOE_NORM_LAYER || a.next.kind == SEMMOE_NORM_LAYER)
      return dtype == SEMMOE_BF16 ? launch_t<__nv_bfloat16, W, C, true>(p, a, s) : launch_t<float, W, C, true>(p, a, s);
    return dtype == SEMMOE_BF16 ? launch_t<__nv_bfloat16, W, C, false>(p, a, s) : launch_t<float, W, C, false>(p, a, s);
  });
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_norm(const void* x, int dtype, int T, int H, const NormArgs& n, void* out, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const RowPlan p = plan(H, dtype == SEMMOE_BF16 ? 8 : 4, T);
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

}  // namespace semmoe
