// Grouped products of bf16 rows with 4-bit weights (w4.cuh), fp32 accumulation.
// Rows [off[b], off[b+1]) belong to expert pe[b]:
//   plain:  out = x W_e^T
//   SwiGLU: h = silu(x W1_e^T) * (x W3_e^T)      (both stored in bf16)
//
// Few rows per expert (w4_rows_kernel): the weights' bytes bound it, and a
// tensor-core tile of 128 rows would be all but empty, so the weights are the left operand
// of the warp-level m16n8k16 product and the rows its narrow side.
// A unit is NB = 8 NT rows of one group times 32 WM weight rows (SwiGLU: 16 WM gate rows
// and the same up rows); a CTA of four warps takes units in turn, WM warps
// along the weight rows, WK along the columns (summed through shared memory at
// the unit's end).  Codes and rows come in stages of 128 WK columns by asynchronous
// copies, STAGES - 1 of them in flight, across the ends of units.
// A lane's word of eight codes gives the A operands of two products as they lie: bits 0-3
// and 16-19 (columns 0, 4), 4-7 and 20-23 (1, 5), and so on; the row's eight values are
// put into that order instead.  The codes are exact in bf16 (128 + code, less 128 + z), a
// group's products are summed alone and multiplied by its scale in fp32, so no weight is
// rounded.
#include "common.cuh"
#include "internal.h"
#include "w4_groups.cuh"

namespace semmoe {
namespace {

using namespace w4;

__device__ int g_err;

constexpr int THREADS = 128;
constexpr int STAGES = 4;
constexpr int CHUNK = 128;            // columns of a warp's stage
constexpr int W_STAGE = 8192;         // bytes of codes a stage: 32 rows x 64 bytes x 4 warps
constexpr int X_STAGE = 8192;         // bytes of rows a stage: 8 NT x 256 bytes x WK
constexpr int STAGE_BYTES = W_STAGE + X_STAGE;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // nothing read, zeros written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// d = a b + c, a [16 x 16] bf16, b [16 x 8] bf16.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// GS: groups of scales in a chunk of 128 columns (4, 2, or 1 for groups of 128 and more).
template <int NT, int WM, bool GLU, typename S, int GS>
__global__ void __launch_bounds__(THREADS, 3)
w4_rows_kernel(Product pr) {
  constexpr int WK = 4 / WM, NB = 8 * NT, BK = CHUNK * WK;
  constexpr int MT = 2;                              // 16-row tiles of a warp
  constexpr int COLS = (GLU ? 16 : 32) * WM;         // output columns of a unit
  constexpr int RED = 32 * WM + 4;                   // floats per row of the sums (conflict-free over t)
  static_assert(NB * 256 * WK == X_STAGE, "a stage of rows");
  extern __shared__ __align__(128) unsigned char smem[];
  float* red = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);  // [WK][NB][RED]
  __shared__ Groups sh;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int wm = warp % WM, wk = warp / WM;
  pdl_trigger();
  pdl_wait();
  if (warp == 0) load_groups(sh, pr, NB, lane, &g_err);
  __syncthreads();
  const int G = pr.E, K = pr.K, KG = K / pr.group, ki = (K + BK - 1) / BK;
  const int rows_w = GLU ? 2 * pr.N : pr.N;          // weight rows of an expert
  const int total = sh.total * pr.n_tiles;
  // row r of the unit's weight rows (of warp block r / 32) among the expert's
  auto weight_row = [&](int nt, int r) {
    if (GLU) {
      const int c = nt * COLS + (r / 32) * 16 + r % 16;
      return (c < pr.N ? c : pr.N - 1) + (r % 32 >= 16 ? pr.N : 0);
    }
    const int c = nt * COLS + r;
    return c < pr.N ? c : pr.N - 1;
  };

  // ---- copies: this thread's 16-byte pieces of a stage, the same columns in four rows ----
  constexpr int WP = 4 * WK, XP = 16 * WK;           // pieces of a row
  constexpr int XN = X_STAGE / 16 / THREADS;
  const int w_seg = tid % WP, x_seg = tid % XP;
  const uint32_t base = smem_addr(smem);
  int lu = blockIdx.x, lg = 0, ug = 0;               // the unit being copied, its group ...
  int lkb = 0;                                       // ... and its k-block
  const uint8_t* wsrc[4];
  const __nv_bfloat16* xsrc[XN];
  auto copy_rows = [&]() {
    const Unit un = decode_unit(sh, G, lg, pr.n_tiles, NB, lu);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      wsrc[i] = pr.w.codes + ((size_t)un.e * rows_w + weight_row(un.nt, tid / WP + i * (THREADS / WP))) * (K / 2) + w_seg * 16;
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int n = tid / XP + i * (THREADS / XP);
      xsrc[i] = pr.x + (size_t)(un.row0 + (n < un.rows ? n : un.rows - 1)) * K + x_seg * 8;
    }
  };
  auto copy_stage = [&](int s) {
    if (lu < total) {
      const uint32_t ws = base + s * STAGE_BYTES, xs = ws + W_STAGE;
      const int k0 = lkb * BK;
      const bool w_live = k0 + w_seg * 32 < K, x_live = k0 + x_seg * 8 < K;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = tid / WP + i * (THREADS / WP), b = r / 32, q = r % 32;
        cp_async16(ws + (b * WK + w_seg / 4) * 2048 + q * 64 + (((w_seg & 3) ^ ((q >> 1) & 3)) << 4),
                   w_live ? wsrc[i] + k0 / 2 : pr.w.codes, w_live);
      }
#pragma unroll
      for (int i = 0; i < XN; ++i) {
        const int n = tid / XP + i * (THREADS / XP);
        cp_async16(xs + (x_seg / 16) * (NB * 256) + n * 256 + (((x_seg & 15) ^ ((n & 1) << 2)) << 4),
                   x_live ? (const void*)(xsrc[i] + k0) : (const void*)pr.x, x_live);
      }
      if (++lkb == ki) {
        lkb = 0;
        lu += gridDim.x;
        if (lu < total) copy_rows();
      }
    }
    cp_async_commit();
  };

  // ---- scales and zero points of this lane's rows in a chunk ----
  float sc[MT][2][GS];
  uint32_t zp[MT][2][GS];
  size_t srow[MT][2];
  auto scale_rows = [&](const Unit& un) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        srow[m][h] = ((size_t)un.e * rows_w + weight_row(un.nt, wm * 32 + m * 16 + h * 8 + g)) * KG;
  };
  auto load_scales = [&](int kb, float (&s)[MT][2][GS], uint32_t (&z)[MT][2][GS]) {
    const int k = kb * BK + wk * CHUNK;
#pragma unroll
    for (int j = 0; j < GS; ++j) {
      int i = (k + j * (CHUNK / GS)) / pr.group;
      if (i >= KG) i = KG - 1;  // past K: codes and rows are 0
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[m][h][j] = load_scale(static_cast<const S*>(pr.w.scales) + srow[m][h] + i);
          z[m][h][j] = pr.w.zeros != nullptr ? __ldg(pr.w.zeros + srow[m][h] + i) : 8u;
        }
    }
  };

  int u = blockIdx.x;
  if (u >= total) return;
  copy_rows();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) copy_stage(s);
  Unit un = decode_unit(sh, G, ug, pr.n_tiles, NB, u);
  scale_rows(un);
  load_scales(0, sc, zp);
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

  int stage = 0, kb = 0;
  while (true) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();
    copy_stage((stage + STAGES - 1) % STAGES);  // the stage that every warp has left
    // the next stage's scales, one stage ahead
    const bool last = kb == ki - 1;
    Unit nx = un;
    float nsc[MT][2][GS];
    uint32_t nzp[MT][2][GS];
    const bool more = !last || u + (int)gridDim.x < total;
    if (last && more) {
      nx = decode_unit(sh, G, ug, pr.n_tiles, NB, u + gridDim.x);
      scale_rows(nx);
    }
    load_scales(last ? 0 : kb + 1, nsc, nzp);  // (of this unit again where there is none: not used)

    const uint32_t ws = base + stage * STAGE_BYTES + (wm * WK + wk) * 2048;
    const uint32_t xs = base + stage * STAGE_BYTES + W_STAGE + wk * (NB * 256);
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    float part[MT][NT][4];
#pragma unroll
    for (int jp = 0; jp < 2; ++jp) {
      uint32_t w[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = m * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, seg = 2 * jp + (lane >> 4);
        ldmatrix_x4(w[m], ws + r * 64 + ((seg ^ ((r >> 1) & 3)) << 4));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 2 * jp + h, gi = j * GS / 4;            // 32 columns, their group
        const bool first = j % (4 / GS) == 0, end = (j + 1) % (4 / GS) == 0;
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = lds128(xs + (n * 8 + g) * 256 + (((4 * j + t) ^ ((g & 1) << 2)) << 4));
          b[n][0] = __byte_perm(v.x, v.z, 0x5410);
          b[n][1] = __byte_perm(v.x, v.z, 0x7632);
          b[n][2] = __byte_perm(v.y, v.w, 0x5410);
          b[n][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t lo = w[m][2 * h], hi = w[m][2 * h + 1], z0 = zero_pair(zp[m][0][gi]), z1 = zero_pair(zp[m][1][gi]);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t a0 = sub_bf16x2(code_pair(lo, 8 * p), z0), a1 = sub_bf16x2(code_pair(hi, 8 * p), z1),
                           a2 = sub_bf16x2(code_pair(lo, 8 * p + 4), z0), a3 = sub_bf16x2(code_pair(hi, 8 * p + 4), z1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (first && p == 0) mma(part[m][n], a0, a1, a2, a3, b[n][0], b[n][1], zero);
              else mma(part[m][n], a0, a1, a2, a3, b[n][2 * p], b[n][2 * p + 1], part[m][n]);
            }
          }
          if (end) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[m][n][i] = fmaf(sc[m][i / 2][gi], part[m][n][i], acc[m][n][i]);
          }
        }
      }
    }
    if (last) {  // the unit's sums: over the warps along the columns, then stored
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            red[(wk * NB + n * 8 + 2 * t + (i & 1)) * RED + wm * 32 + m * 16 + (i / 2) * 8 + g] = acc[m][n][i];
            acc[m][n][i] = 0.f;
          }
      __syncthreads();
      const int n0 = un.nt * COLS;
      for (int i = tid; i < NB * COLS / 2; i += THREADS) {
        const int n = i / (COLS / 2), c = 2 * (i % (COLS / 2));
        if (n >= un.rows || n0 + c >= pr.N) continue;
        const int r = GLU ? (c / 16) * 32 + c % 16 : c;
        float v[2] = {0.f, 0.f}, up[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < WK; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            v[j] += red[(k * NB + n) * RED + r + j];
            if (GLU) up[j] += red[(k * NB + n) * RED + r + 16 + j];
          }
        if (GLU) v[0] = swiglu(v[0], up[0]), v[1] = swiglu(v[1], up[1]);
        *reinterpret_cast<__nv_bfloat162*>(pr.out + (size_t)(un.row0 + n) * pr.N + n0 + c) = __floats2bfloat162_rn(v[0], v[1]);
      }
      if (!more) break;
      u += gridDim.x;
      un = nx;
      kb = 0;
    } else {
      ++kb;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < GS; ++j) sc[m][h][j] = nsc[m][h][j], zp[m][h][j] = nzp[m][h][j];
    stage = (stage + 1) % STAGES;
  }
  cp_async_wait<0>();
}

template <int NT, int WM, bool GLU, typename S, int GS>
cudaError_t launch_rows_t(Product pr, cudaStream_t s) {
  constexpr int cols = (GLU ? 16 : 32) * WM, smem = STAGES * STAGE_BYTES + (4 / WM) * 8 * NT * (32 * WM + 4) * 4;
  auto kern = w4_rows_kernel<NT, WM, GLU, S, GS>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, smem, smem_set);
  if (e != cudaSuccess) return e;
  pr.n_tiles = (pr.N + cols - 1) / cols;
  const long long units = ((long long)pr.P / (8 * NT) + (pr.E < pr.P ? pr.E : pr.P)) * pr.n_tiles;
  constexpr int per_sm = 232448 / (smem + (int)sizeof(Groups) + 1024);  // CTAs that an SM's shared memory holds
  const long long cap = (per_sm < 3 ? per_sm : 3) * (long long)sm_count();
  e = launch_kernel(kern, dim3((unsigned)(units < cap ? units : cap)), dim3(THREADS), smem, s, 1, true, pr);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <bool GLU>
cudaError_t launch_product(const Product& pr, cudaStream_t s) {
  // a few rows whose 128-row weight tiles would not fill the SMs
  const int used = pr.E < pr.P ? pr.E : pr.P;
  if (pr.P > 8LL * used || (long long)used * ((pr.N + 127) / 128) >= sm_count())
    return GLU ? launch_w4_tc_glu(pr, s) : launch_w4_tc_plain(pr, s);
  if (pr.w.scales_bf16) {
    if (pr.group == 32) return launch_rows_t<1, 1, GLU, __nv_bfloat16, 4>(pr, s);
    if (pr.group == 64) return launch_rows_t<1, 1, GLU, __nv_bfloat16, 2>(pr, s);
    return launch_rows_t<1, 1, GLU, __nv_bfloat16, 1>(pr, s);
  }
  if (pr.group == 32) return launch_rows_t<1, 1, GLU, float, 4>(pr, s);
  if (pr.group == 64) return launch_rows_t<1, 1, GLU, float, 2>(pr, s);
  return launch_rows_t<1, 1, GLU, float, 1>(pr, s);
}

}  // namespace

int w4_gemm_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

size_t w4_ffn_ws_bytes(int P, int I) { return align_up((size_t)(P > 0 ? P : 1) * I * 2, 256); }

cudaError_t launch_w4_grouped_gemm(const void* x, const int32_t* offsets, const int32_t* experts, const Weights& w, int P,
                                   int E, int N, int K, int group, void* out, cudaStream_t s) {
  return launch_product<false>(Product{static_cast<const __nv_bfloat16*>(x), offsets, experts, w, P, E, N, K, group, 0,
                                       static_cast<__nv_bfloat16*>(out)},
                               s);
}

cudaError_t launch_w4_grouped_ffn(const void* x, const int32_t* offsets, const int32_t* experts, const Weights& w13,
                                  const Weights& w2, int P, int E, int H, int I, int group, void* y, void* ws,
                                  cudaStream_t s) {
  __nv_bfloat16* h = static_cast<__nv_bfloat16*>(ws);
  cudaError_t e = launch_product<true>(Product{static_cast<const __nv_bfloat16*>(x), offsets, experts, w13, P, E, I, H,
                                               group, 0, h},
                                       s);
  if (e != cudaSuccess) return e;
  return launch_product<false>(Product{h, offsets, experts, w2, P, E, H, I, group, 0, static_cast<__nv_bfloat16*>(y)}, s);
}

}  // namespace semmoe
