// Grouped products of bf16 rows with 4-bit weights (w4.cuh), fp32 accumulation.
// Rows [off[b], off[b+1]) belong to expert pe[b]:
//   plain:  out = x W_e^T
//   SwiGLU: h = silu(x W1_e^T) * (x W3_e^T)      (both stored in bf16)
//
// Few rows per expert (w4_rows_kernel): the weights' bytes bound it, and so few 128-row weight tiles
// would not fill the SMs, so the weights are the left operand of the warp-level m16n8k16 product
// and the rows its narrow side.
// A unit is 8 rows of one group times 32 weight rows (SwiGLU: 16 gate rows and the same up
// rows); a CTA of four warps takes units in turn, the warps side by side along the columns
// (summed through shared memory at the unit's end).  Codes and rows come in stages of 512
// columns by asynchronous copies, STAGES - 1 of them in flight, across the ends of units.
// A lane's word of eight codes gives the A operands of two products as they lie: bits 0-3
// and 16-19 (columns 0, 4), 4-7 and 20-23 (1, 5), and so on; the row's eight values are
// put into that order instead.  A code is made bf16 as 128 + code, one masked OR, and 128 + z is subtracted from a pair of
// them at once, exactly; the scale is applied to the sums of its group of columns.
// No weight is rounded: code - z and the rows' values are exact in bf16, the sums fp32.  (Sums of (128 + code) x, put right by
// the sum of x at a group's end, took as long, and lost what large values on weights of 0 left of the others.)
// What bounds it: a few microseconds of latency, the tables, the first codes and the unit's end one after the other; the weights
// of one token take 0.3 to 3 us.  Measured (GB300, calls of a captured graph): one row by 2048 x 2048 4.3 us, by 8192 x 2048 5.7 us;
// one token through 8 of 128 experts of 2048 x 768 14.3 us, through 6 of 64 of 2048 x 1408 16.6 us (20 us for the first before the
// second product read its tables and codes while the first one ends).
#include "common.cuh"
#include "internal.h"
#include "w4_groups.cuh"

namespace semmoe {
namespace {

using namespace w4;

__device__ int g_err;

constexpr int THREADS = 128;
constexpr int WK = 4;                 // warps, side by side along the columns
constexpr int STAGES = 3;
constexpr int CHUNK = 128;            // columns of a warp's stage
constexpr int BK = CHUNK * WK;
constexpr int NB = 8;                 // rows of a unit
constexpr int MT = 2;                 // 16-row tiles of weight rows
constexpr int W_STAGE = 32 * BK / 2;  // bytes of codes a stage
constexpr int X_STAGE = NB * BK * 2;  // bytes of rows a stage
constexpr int STAGE_BYTES = W_STAGE + X_STAGE;
constexpr int RED = 36;               // floats of a row of the sums (conflict-free over a warp)
constexpr int SMEM = STAGES * STAGE_BYTES + WK * NB * RED * 4;
constexpr int PER_SM = 4;             // CTAs that an SM holds

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
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// BYTES (2, 4, 8 or 16) that lie together, aligned to their size.
template <int BYTES>
__device__ __forceinline__ void load_raw(const void* p, uint32_t* r) {
  if (BYTES == 2) r[0] = __ldg(static_cast<const unsigned short*>(p));
  if (BYTES == 4) r[0] = __ldg(static_cast<const uint32_t*>(p));
  if (BYTES == 8) {
    const uint2 v = __ldg(static_cast<const uint2*>(p));
    r[0] = v.x, r[BYTES / 4 - 1] = v.y;
  }
  if (BYTES == 16) {
    const uint4 v = __ldg(static_cast<const uint4*>(p));
    r[0] = v.x, r[BYTES / 4 - 3 > 0 ? 1 : 0] = v.y, r[BYTES / 4 - 2 > 0 ? 2 : 0] = v.z, r[BYTES / 4 - 1] = v.w;
  }
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// GS: groups of scales in a chunk of 128 columns (4, 2, or 1 for groups of 128 and more).
template <bool GLU, typename S, int GS>
__global__ void __launch_bounds__(THREADS, PER_SM)
w4_rows_kernel(const __grid_constant__ Product pr) {
  constexpr int COLS = GLU ? 16 : 32;                // output columns of a unit
  extern __shared__ __align__(128) unsigned char smem[];
  float* red = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);  // [WK][NB][RED]
  __shared__ Groups sh;
  const int tid = threadIdx.x, wk = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  if (!pr.early) pdl_wait();
  pdl_trigger();
  if (wk == 0) load_groups(sh, pr, NB, lane, &g_err);
  __syncthreads();
  const int G = pr.E, K = pr.K, KG = K / pr.group, ki = (K + BK - 1) / BK;
  const int rows_w = GLU ? 2 * pr.N : pr.N;          // weight rows of an expert
  const int total = sh.total * pr.n_tiles;
  // row r of the unit's weight rows among the expert's
  auto weight_row = [&](int nt, int r) {
    const int c = nt * COLS + (GLU ? r % 16 : r);
    return (c < pr.N ? c : pr.N - 1) + (GLU && r >= 16 ? pr.N : 0);
  };

  // ---- copies: this thread's 16-byte pieces of a stage, the same columns in four rows ----
  constexpr int WP = 4 * WK, XP = 16 * WK;           // pieces of a row of codes, of a row
  constexpr int WN = W_STAGE / 16 / THREADS, XN = X_STAGE / 16 / THREADS;
  const int w_seg = tid % WP, x_seg = tid % XP;
  const uint32_t base = smem_addr(smem);
  uint32_t w_to[WN], x_to[XN];                       // places in a stage
#pragma unroll
  for (int i = 0; i < WN; ++i) {
    const int r = tid / WP + i * (THREADS / WP);
    w_to[i] = base + (w_seg / 4) * 2048 + r * 64 + (((w_seg & 3) ^ ((r >> 1) & 3)) << 4);
  }
#pragma unroll
  for (int i = 0; i < XN; ++i) {
    const int n = tid / XP + i * (THREADS / XP);
    x_to[i] = base + W_STAGE + (x_seg / 16) * (NB * 256) + n * 256 + (((x_seg & 15) ^ ((n & 1) << 2)) << 4);
  }
  int lu = blockIdx.x;                               // the unit being copied ...
  int lkb = 0;                                       // ... and its k-block
  int lrows = 0;                                     // its rows: places of rows past them keep what they hold, no sum of
  const uint8_t* wsrc[WN];                           // which is stored (and a row read for all eight is one L2 line for
  const __nv_bfloat16* xsrc[XN];                     // every CTA)
  auto copy_rows = [&](const Unit& un) {
#pragma unroll
    for (int i = 0; i < WN; ++i)
      wsrc[i] = pr.w.codes + ((size_t)un.e * rows_w + weight_row(un.nt, tid / WP + i * (THREADS / WP))) * (K / 2) + w_seg * 16;
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int n = tid / XP + i * (THREADS / XP);
      xsrc[i] = pr.x + (size_t)(un.row0 + (n < un.rows ? n : 0)) * K + x_seg * 8;
    }
    lrows = un.rows;
  };
  auto copy_codes = [&](int s, int kb) {
    const bool live = kb * BK + w_seg * 32 < K;
#pragma unroll
    for (int i = 0; i < WN; ++i)
      cp_async16(w_to[i] + s * STAGE_BYTES, live ? wsrc[i] + kb * (BK / 2) : pr.w.codes, live);
  };
  auto copy_stage = [&](int s, bool codes = true) {
    if (lu < total) {
      if (codes) copy_codes(s, lkb);
      const bool x_live = lkb * BK + x_seg * 8 < K;
#pragma unroll
      for (int i = 0; i < XN; ++i) {
        if (tid / XP + i * (THREADS / XP) < lrows)
          cp_async16(x_to[i] + s * STAGE_BYTES, x_live ? (const void*)(xsrc[i] + lkb * BK) : (const void*)pr.x, x_live);
      }
      if (++lkb == ki) {
        lkb = 0;
        lu += gridDim.x;
        if (lu < total) copy_rows(decode_unit(sh, G, pr.n_tiles, NB, lu));
      }
    }
    cp_async_commit();
  };

  // ---- scales and zero points of this lane's rows in a chunk ----
  const bool whole = GS == 1 || K % CHUNK == 0;      // a chunk's scales are aligned to their size
  const int per = pr.group > CHUNK ? pr.group / CHUNK : 1;  // chunks of a scale
  size_t srow[MT][2];
  auto scale_rows = [&](const Unit& un) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        srow[m][h] = ((size_t)un.e * rows_w + weight_row(un.nt, m * 16 + h * 8 + g)) * KG;
  };
  // as they lie in memory; unpacked where they are used, so that nothing waits for them before
  constexpr int NR = GS * (int)sizeof(S) <= 4 ? 1 : GS * (int)sizeof(S) / 4;
  struct Scales {
    uint32_t s[MT][2][NR], z[MT][2];
  };
  auto load_scales = [&](int kb, Scales& r) {
    const int ch = kb * WK + wk;
    int i0 = GS > 1 ? ch * GS : per > 1 ? ch / per : ch;
    if (whole && i0 + GS > KG) i0 = KG - GS;  // a chunk past K: codes and rows are 0
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const S* p = static_cast<const S*>(pr.w.scales) + srow[m][h];
        const uint8_t* q = pr.w.zeros + srow[m][h];
        r.z[m][h] = 0x08080808u;
        if (whole) {
          load_raw<GS * (int)sizeof(S)>(p + i0, r.s[m][h]);
          if (pr.w.zeros != nullptr) {
            if (GS == 1) r.z[m][h] = __ldg(q + i0);
            if (GS == 2) r.z[m][h] = __ldg(reinterpret_cast<const unsigned short*>(q + i0));
            if (GS == 4) r.z[m][h] = __ldg(reinterpret_cast<const uint32_t*>(q + i0));
          }
        } else {  // one by one; past K, which a whole chunk may be, the row's last one again
          uint32_t v[GS], z = 0;
#pragma unroll
          for (int j = 0; j < GS; ++j) {
            const int o = i0 + j < KG ? i0 + j : KG - 1;
            v[j] = sizeof(S) == 4 ? __ldg(reinterpret_cast<const uint32_t*>(p) + o)
                                  : __ldg(reinterpret_cast<const unsigned short*>(p) + o);
            z |= (pr.w.zeros != nullptr ? (uint32_t)__ldg(q + o) : 8u) << (8 * j);
          }
          r.z[m][h] = z;
#pragma unroll
          for (int j = 0; j < NR; ++j)
            r.s[m][h][j] = sizeof(S) == 4 ? v[j] : v[2 * j % GS] | (GS > 1 ? v[(2 * j + 1) % GS] << 16 : 0u);
        }
      }
  };
  auto scale_of = [&](const Scales& r, int m, int h, int j) {
    if (sizeof(S) == 4) return __uint_as_float(r.s[m][h][j % NR]);
    return __uint_as_float(j & 1 ? r.s[m][h][j / 2 % NR] & 0xffff0000u : r.s[m][h][j / 2 % NR] << 16);
  };
  auto zero_of = [&](const Scales& r, int m, int h, int j) { return ((r.z[m][h] >> (8 * j)) & 15u) * 0x00010001u | 0x43004300u; };

  int u = blockIdx.x;
  if (u >= total) {
    if (pr.early) pdl_wait();  // a kernel ends after the one before it
    return;
  }
  Unit un = decode_unit(sh, G, pr.n_tiles, NB, u);
  copy_rows(un);
  if (pr.early) {
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
      if (s < ki) copy_codes(s, s);
  }
  Scales sc;
  scale_rows(un);
  load_scales(0, sc);
  if (pr.early) pdl_wait();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) copy_stage(s, !pr.early || s >= ki);
  float acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;

  // this lane's places in a stage: ldmatrix rows, its row's values
  const int mr = (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t w_at = base + wk * 2048 + mr * 64, w_turn = ((mr >> 1) & 3) << 4, seg0 = (lane >> 4) << 4;
  const uint32_t x_at = base + W_STAGE + wk * (NB * 256) + g * 256 + (t << 4), x_turn = (g & 1) << 6;
  int stage = 0, kb = 0;
  while (true) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();
    copy_stage((stage + STAGES - 1) % STAGES);  // the stage that every warp has left
    // the next stage's scales, one stage ahead
    const bool last = kb == ki - 1;
    Unit nx = un;
    Scales nsc;
    const bool more = !last || u + (int)gridDim.x < total;
    if (last && more) {
      nx = decode_unit(sh, G, pr.n_tiles, NB, u + gridDim.x);
      scale_rows(nx);
    }
    if (more) load_scales(last ? 0 : kb + 1, nsc);

    const uint32_t off = stage * STAGE_BYTES;
    const int left = K - (kb * BK + wk * CHUNK);  // columns from this chunk's first one on
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    float part[MT][4];
#pragma unroll
    for (int jp = 0; jp < 2; ++jp) {
      uint32_t w[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) ldmatrix_x4(w[m], w_at + off + m * 1024 + ((32 * jp + seg0) ^ w_turn));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 2 * jp + h, gi = j * GS / 4;            // 32 columns, their group
        const bool first = j % (4 / GS) == 0, end = (j + 1) % (4 / GS) == 0;
        const uint4 v = lds128(x_at + off + ((64 * j) ^ x_turn));
        const uint32_t b[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                               __byte_perm(v.y, v.w, 0x7632)};
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t lo = w[m][2 * h], hi = w[m][2 * h + 1], zl = zero_of(sc, m, 0, gi), zh = zero_of(sc, m, 1, gi);
          auto weight = [](uint32_t c, int sh, uint32_t z) { return sub_bf16x2(code_pair(c, sh), z); };
          if (first) mma(part[m], weight(lo, 0, zl), weight(hi, 0, zh), weight(lo, 4, zl), weight(hi, 4, zh), b[0], b[1], zero);
          else mma(part[m], weight(lo, 0, zl), weight(hi, 0, zh), weight(lo, 4, zl), weight(hi, 4, zh), b[0], b[1], part[m]);
          mma(part[m], weight(lo, 8, zl), weight(hi, 8, zh), weight(lo, 12, zl), weight(hi, 12, zh), b[2], b[3], part[m]);
          if (end) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a group past K has scale 0: its sums are 0, which an infinite scale would make NaN.  (Put in here rather than at
              // the loads, which it would delay: one token through 8 of 128 experts 14.3 us here, 14.9 there.)
              const float s = gi * (CHUNK / GS) < left ? scale_of(sc, m, i / 2, gi) : 0.f;
              acc[m][i] = fmaf(s, part[m][i], acc[m][i]);
            }
          }
        }
      }
    }
    if (last) {  // the unit's sums: over the warps along the columns, then stored
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          red[(wk * NB + 2 * t + (i & 1)) * RED + m * 16 + (i / 2) * 8 + g] = acc[m][i];
          acc[m][i] = 0.f;
        }
      __syncthreads();
      const int n0 = un.nt * COLS, n = tid / (COLS / 2), c = 2 * (tid % (COLS / 2));  // a pair of columns a thread
      if (n < un.rows && n0 + c < pr.N) {
        float v[2] = {0.f, 0.f}, up[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < WK; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            v[j] += red[(k * NB + n) * RED + c + j];
            if (GLU) up[j] += red[(k * NB + n) * RED + 16 + c + j];
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
    sc = nsc;
    stage = (stage + 1) % STAGES;
  }
  cp_async_wait<0>();
}

template <bool GLU, typename S, int GS>
cudaError_t launch_rows(Product pr, cudaStream_t s) {
  constexpr int COLS = GLU ? 16 : 32;
  static_assert(PER_SM * (SMEM + (int)sizeof(Groups) + 1024) <= 233472, "shared memory of an SM");
  auto kern = w4_rows_kernel<GLU, S, GS>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, SMEM, smem_set);
  if (e != cudaSuccess) return e;
  pr.n_tiles = (pr.N + COLS - 1) / COLS;
  const long long units = ((long long)pr.P / NB + (pr.E < pr.P ? pr.E : pr.P)) * pr.n_tiles, cap = PER_SM * (long long)sm_count();
  e = launch_kernel(kern, dim3((unsigned)(units < cap ? units : cap)), dim3(THREADS), SMEM, s, 1, true, pr);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <bool GLU>
cudaError_t launch_product(const Product& pr, cudaStream_t s) {
  // A few rows, whose 128-row weight tiles would not fill the SMs, by this file's kernel (the other one takes 8.1 us for one row by
  // 2048 x 2048, this one 4.3; 18.4 and 14.3 for one token through 8 of 128 experts of 768), all else on the tensor cores' own
  // path (384 rows through 64 matrices of 1408 x 2048: 34.6 us, 51.6 here).
  const int used = pr.E < pr.P ? pr.E : pr.P;
  if (pr.P > (long long)NB * used || (long long)used * ((pr.N + 127) / 128) >= sm_count())
    return GLU ? launch_w4_tc_glu(pr, s) : launch_w4_tc_plain(pr, s);
  if (pr.w.scales_bf16) {
    if (pr.group == 32) return launch_rows<GLU, __nv_bfloat16, 4>(pr, s);
    if (pr.group == 64) return launch_rows<GLU, __nv_bfloat16, 2>(pr, s);
    return launch_rows<GLU, __nv_bfloat16, 1>(pr, s);
  }
  if (pr.group == 32) return launch_rows<GLU, float, 4>(pr, s);
  if (pr.group == 64) return launch_rows<GLU, float, 2>(pr, s);
  return launch_rows<GLU, float, 1>(pr, s);
}

}  // namespace

int w4_gemm_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

size_t w4_ffn_ws_bytes(int P, int I) { return align_up((size_t)(P > 0 ? P : 1) * I * 2, 256); }

cudaError_t launch_w4_grouped_gemm(const void* x, const int32_t* offsets, const int32_t* experts, const Weights& w, int P,
                                   int E, int N, int K, int group, void* out, cudaStream_t s) {
  return launch_product<false>(Product{static_cast<const __nv_bfloat16*>(x), offsets, experts, w, P, E, N, K, group, 0,
                                       false, static_cast<__nv_bfloat16*>(out)},
                               s);
}

cudaError_t launch_selftest_w4_wait(const void* x, const int32_t* offsets, const int32_t* experts, const Weights& w, int P,
                                    int E, int N, int K, int group, void* out, cudaStream_t s) {
  return launch_w4_tc_plain(Product{static_cast<const __nv_bfloat16*>(x), offsets, experts, w, P, E, N, K, group, 0, false,
                                    static_cast<__nv_bfloat16*>(out), true},
                            s);
}

cudaError_t launch_w4_grouped_ffn(const void* x, const int32_t* offsets, const int32_t* experts, const Weights& w13,
                                  const Weights& w2, int P, int E, int H, int I, int group, void* y, void* ws,
                                  cudaStream_t s) {
  __nv_bfloat16* h = static_cast<__nv_bfloat16*>(ws);
  cudaError_t e = launch_product<true>(Product{static_cast<const __nv_bfloat16*>(x), offsets, experts, w13, P, E, I, H,
                                               group, 0, false, h},
                                       s);
  if (e != cudaSuccess) return e;
  return launch_product<false>(Product{h, offsets, experts, w2, P, E, H, I, group, 0, true, static_cast<__nv_bfloat16*>(y)}, s);
}

}  // namespace semmoe
