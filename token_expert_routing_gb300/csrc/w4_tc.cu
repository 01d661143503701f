// Grouped products of bf16 rows with 4-bit weights (w4.cuh) on the 5th-generation
// tensor cores, for experts with more than a few rows.
//
// The weights are the left operand (M = 128 weight rows), held in tensor memory: a
// thread turns the 64 codes of its row's k-block into bf16 in registers and
// writes them to its TMEM lane, so the expanded weights never pass through shared memory, whose
// bandwidth bounds the bf16 products (ffn_tc.cu).  The token rows are the right
// operand (N = up to 128 rows of a group, a multiple of 16), by TMA.
//
// A unit has two accumulators of up to 128 columns (tokens):
//   plain:  128 weight rows x 256 token rows; both halves read one A block
//   SwiGLU: 128 gate rows and the 128 up rows x 128 token rows; two A blocks
// TMEM holds three accumulators and a ring of four A blocks (32 columns each): a
// unit's first accumulator is free while the epilogue still reads the unit before.
//
// One persistent CTA per SM takes units in turn.  Warp roles:
//   warps 0..7    expand the weights, two groups of four (plain: k-blocks in turn; SwiGLU: gate, up)
//   warps 8..15   epilogue, two groups of four (token columns 0-63 and 64-127 of a half)
//   warp 16       TMA producer of codes, [128 rows x 256 columns] a slot
//   warp 17       TMA producer of token rows, boxes of [32 rows x 64 columns]
//   warp 18       allocates TMEM, issues the MMAs (M128 N16..128 K16)
//
// A weight is (code - zero) exactly, times its scale rounded once to bf16 (an fp32
// scale enters as the sum of two bf16 numbers, the smaller product first): at most half a step, as in
// any bf16 copy of the weights.
//
// Every wait is bounded; a wait that runs out sets the timeout bit of the device error
// word and an abort flag, after which every role stops, loads and MMAs in flight are
// drained (again with a bound), and TMEM is freed before the CTA exits.
#include "common.cuh"
#include "internal.h"
#include "tc_common.cuh"
#include "w4_groups.cuh"

namespace semmoe {
namespace {

using namespace tc;
using namespace w4;

__device__ int g_err;

constexpr int BM = 128;               // weight rows of an A block
constexpr int HN = 128;               // columns of an accumulator
constexpr int BK = 64;                // columns of an A block
constexpr int UK = 16;                // K per MMA
constexpr int CK = 256;               // columns of a slot of codes: 128 bytes a row
constexpr int C_BYTES = BM * CK / 2;  // 16 KB
constexpr int XR = 32;                // rows of a box of token rows
constexpr int X_BOX = XR * BK * 2;
constexpr int C_SLOTS = 6;
constexpr int A_SLOTS = 4;
constexpr int ACCS = 3;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t A_COL = ACCS * HN, A_COLS = BK / 2;
static_assert(A_COL + A_SLOTS * A_COLS == TMEM_COLS, "TMEM columns");
constexpr int EXPAND_WARPS = 8, THREADS = 19 * 32;
constexpr int ROUND = 16;             // token rows of a unit: a multiple of this

template <bool GLU>
struct Shape {
  static constexpr int ROWS = GLU ? HN : 2 * HN;       // token rows of a unit, at most
  static constexpr int X_BYTES = ROWS * BK * 2;        // a stage of them
  static constexpr int X_STAGES = 98304 / X_BYTES;     // 96 KB
  static constexpr int AB = GLU ? 2 : 1;               // A blocks of a k-block
  static constexpr size_t smem = 1024 + (size_t)C_SLOTS * C_BYTES + 98304;
};

template <bool GLU>
struct Shared {
  uint64_t cfull[C_SLOTS], cempty[C_SLOTS], xfull[Shape<GLU>::X_STAGES], xempty[Shape<GLU>::X_STAGES];
  uint64_t afull[A_SLOTS], aempty[A_SLOTS], tfull[ACCS], tempty[ACCS], done;
  uint32_t tmem_base;
  int abort_flag;
  int c_armed, x_armed;  // slots and stages that the producers have armed
  Groups groups;
};

// D[tmem] (+)= A[tmem] * B[smem]^T.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// A scale as bf16 pairs: the scale, and what is left of an fp32 one.
struct ScalePair {
  uint32_t hi, lo;
};
__device__ __forceinline__ uint32_t both(__nv_bfloat16 v) {
  const uint32_t b = *reinterpret_cast<const unsigned short*>(&v);
  return b | (b << 16);
}
template <typename S>
__device__ __forceinline__ ScalePair scale_pair(float s) {
  const __nv_bfloat16 h = __float2bfloat16_rn(s);
  if (sizeof(S) == 2) return ScalePair{both(h), 0u};
  const float rest = s - __bfloat162float(h);
  return ScalePair{both(h), both(__float2bfloat16_rn(rest == rest ? rest : 0.f))};  // (an infinite scale has no rest)
}

// The eight codes of a word as bf16 weights, in column order.
template <typename S>
__device__ __forceinline__ void expand(uint32_t w, uint32_t z, const ScalePair& s, uint32_t* r) {
  const uint32_t t = w >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = (__byte_perm(w, t, (uint32_t)(i | ((4 + i) << 8))) & 0x000f000fu) | 0x43004300u;
    const uint32_t d = sub_bf16x2(p, z);
    r[i] = sizeof(S) == 2 ? mul_bf16x2(d, s.hi) : fma_bf16x2(d, s.hi, mul_bf16x2(d, s.lo));
  }
}

// mbar_wait by a whole converged warp, polling a few times before it looks at the clock.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return mbar_wait_warp(bar, parity, abort_flag, &g_err);
}

// Two tokens' columns of a warp's 32 weight rows (v0, v1: this lane's row): even lanes
// store the first token's pair of rows, odd lanes the second's.
__device__ __forceinline__ void store_pair(float v0, float v1, __nv_bfloat16* first, size_t stride, int left, bool live, int lane) {
  const __nv_bfloat162 own2 = __floats2bfloat162_rn(v0, v1);
  const uint32_t own = *reinterpret_cast<const uint32_t*>(&own2);
  const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
  const int odd = lane & 1;
  const uint32_t v = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
  if (live && odd < left) *reinterpret_cast<uint32_t*>(first + (odd ? stride : 0)) = v;
}

template <bool GLU, typename S, bool G32>
__global__ void __launch_bounds__(THREADS, 1)
w4_tc_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_x, Product pr) {
  using SH = Shape<GLU>;
  constexpr int AB = SH::AB, X_STAGES = SH::X_STAGES;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ Shared<GLU> sh;
  unsigned char* codes = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* xs = codes + C_SLOTS * C_BYTES;
  volatile int* abort_flag = &sh.abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C_SLOTS; ++i) {
      mbar_init(&sh.cfull[i], 1);
      mbar_init(&sh.cempty[i], GLU ? 4 : 8);  // the warps that read it
    }
    for (int i = 0; i < X_STAGES; ++i) {
      mbar_init(&sh.xfull[i], 1);
      mbar_init(&sh.xempty[i], 1);
    }
    for (int i = 0; i < A_SLOTS; ++i) {
      mbar_init(&sh.afull[i], 4);
      mbar_init(&sh.aempty[i], 1);
    }
    for (int i = 0; i < ACCS; ++i) {
      mbar_init(&sh.tfull[i], 1);
      mbar_init(&sh.tempty[i], 8);
    }
    mbar_init(&sh.done, 1);
    sh.abort_flag = 0;
    sh.c_armed = sh.x_armed = 0;
    mbar_init_fence();
    prefetch_map(&map_c);
    prefetch_map(&map_x);
  }
  if (warp == 18) tmem_alloc(&sh.tmem_base, TMEM_COLS);
  pdl_wait();
  pdl_trigger();
  if (warp == 0) load_groups(sh.groups, pr, SH::ROWS, lane, &g_err);
  fence_before();
  __syncthreads();
  fence_after();

  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);
  const int G = pr.E, n_tiles = pr.n_tiles, K = pr.K;
  const long long total = (long long)__shfl_sync(0xffffffffu, sh.groups.total, 0) * n_tiles;
  const int kb_n = (K + BK - 1) / BK, ks_n = (K + CK - 1) / CK;
  auto unit_at = [&](long long u) { return decode_unit(sh.groups, G, n_tiles, SH::ROWS, u, ROUND); };

  if (warp < EXPAND_WARPS) {
    // ---------------- codes to bf16 weights in TMEM ----------------
    const int wg = warp / 4, r = (warp % 4) * 32 + lane;
    const int KG = K / pr.group, rows_w = GLU ? 2 * pr.N : pr.N;
    constexpr int STEP = GLU ? 1 : 2, NS = G32 ? 2 : 1;  // k-blocks between this group's, scales of one
    const S* scales = static_cast<const S*>(pr.w.scales);
    const uint32_t a_lane = tmem + ((uint32_t)((warp % 4) * 32) << 16) + A_COL;
    auto row_at = [&](const Unit& un) {
      int n = un.nt * BM + r;
      if (n >= pr.N) n = pr.N - 1;  // a row past the matrix: its codes are 0, nothing of it is stored
      return ((size_t)un.e * rows_w + n + (GLU && wg ? pr.N : 0)) * KG;
    };
    // this row's scales and zero points of k-block kb: loaded one block ahead
    size_t srow = 0;
    int kg = 0, rem = 0;  // the block's group, and its first column within that
    float sc[NS];
    uint32_t zc[NS];
    auto load = [&](float (&s)[NS], uint32_t (&z)[NS]) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int g = kg + i < KG ? kg + i : KG - 1;  // past K: token rows are 0
        s[i] = load_scale(scales + srow + g);
        z[i] = pr.w.zeros != nullptr ? __ldg(pr.w.zeros + srow + g) : 8u;
      }
    };
    auto begin = [&](int kb) {  // of a unit
      kg = 0;
      rem = kb * BK;
      while (rem >= pr.group) rem -= pr.group, ++kg;
    };
    auto advance = [&]() {
      rem += STEP * BK;
      while (rem >= pr.group) rem -= pr.group, ++kg;
    };
    const int kb0 = GLU ? 0 : wg;
    uint32_t kbase = 0, cbase = 0;  // k-blocks and slots of the units before
    long long u = blockIdx.x;
    bool ok = true;
    if (u < total && kb0 < kb_n) {
      srow = row_at(unit_at(u));
      begin(kb0);
      load(sc, zc);
    }
    for (; ok && u < total; u += gridDim.x, kbase += kb_n, cbase += ks_n) {
      for (int ks = 0; ok && ks < ks_n; ++ks) {
        const uint32_t j = GLU ? 2 * (cbase + ks) + wg : cbase + ks, slot = j % C_SLOTS;
        if (!(ok = wait_warp(&sh.cfull[slot], (j / C_SLOTS) & 1, abort_flag))) break;
        const unsigned char* src = codes + slot * C_BYTES + r * 128;
        for (int q = GLU ? 0 : wg; q < CK / BK; q += STEP) {
          const int kb = ks * (CK / BK) + q;
          if (kb >= kb_n) break;
          uint4 c[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) c[i] = *reinterpret_cast<const uint4*>(src + (((2 * q + i) ^ (r & 7)) << 4));
          uint32_t z[NS];
          ScalePair s[NS];
#pragma unroll
          for (int i = 0; i < NS; ++i) z[i] = zero_pair(zc[i]), s[i] = scale_pair<S>(sc[i]);
          // the next block's scales
          if (kb + STEP < kb_n) {
            advance();
            load(sc, zc);
          } else if (u + gridDim.x < total) {
            srow = row_at(unit_at(u + gridDim.x));
            begin(kb0);
            load(sc, zc);
          }
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int g = G32 ? i : 0;
            expand<S>(c[i].x, z[g], s[g], w + 16 * i);
            expand<S>(c[i].y, z[g], s[g], w + 16 * i + 4);
            expand<S>(c[i].z, z[g], s[g], w + 16 * i + 8);
            expand<S>(c[i].w, z[g], s[g], w + 16 * i + 12);
          }
          const uint32_t a = GLU ? 2 * (kbase + kb) + wg : kbase + kb, as = a % A_SLOTS;
          if (!(ok = wait_warp(&sh.aempty[as], ((a / A_SLOTS) & 1) ^ 1, abort_flag))) break;
          fence_after();
          tmem_st32(a_lane + as * A_COLS, w);
          tmem_st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.afull[as]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.cempty[slot]);
      }
    }
  } else if (warp < 16) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, w = (warp - 8) >> 2;
    const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + 64 * w;
    uint32_t half = 0;
    auto wait_acc = [&](uint32_t h) { return wait_warp(&sh.tfull[h % ACCS], (h / ACCS) & 1, abort_flag); };
    auto leave_acc = [&](uint32_t h) {
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tempty[h % ACCS]);
    };
    for (long long u = blockIdx.x; u < total; u += gridDim.x) {
      const Unit un = unit_at(u);
      const int n = un.nt * BM + q * 32 + lane;  // this lane's output column
      const bool live = n < pr.N;
      __nv_bfloat16* col = pr.out + (size_t)un.row0 * pr.N + (live ? n & ~1 : 0);
      if (GLU) {
        if (!wait_acc(half) || !wait_acc(half + 1)) break;
        fence_after();
        const int left = un.rows - 64 * w;
        const uint32_t tg = t_row + (half % ACCS) * HN, tu = t_row + ((half + 1) % ACCS) * HN;
        uint32_t g[2][32];
        if (left > 0) {
          tmem_ld32(tg, g[0]);
          if (left > 32) tmem_ld32(tg + 32, g[1]);
          tmem_ld_wait();
        }
        leave_acc(half);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (left > 16 * c) {
            uint32_t up[16];
            tmem_ld16(tu + 16 * c, up);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const uint32_t* gc = g[c / 2] + 16 * (c & 1);
              const int t = 16 * c + i;
              const float v0 = swiglu(__uint_as_float(gc[i]), __uint_as_float(up[i]));
              const float v1 = swiglu(__uint_as_float(gc[i + 1]), __uint_as_float(up[i + 1]));
              store_pair(v0, v1, col + (size_t)(64 * w + t) * pr.N, pr.N, left - t, live, lane);
            }
          }
        }
        leave_acc(half + 1);
        half += 2;
      } else {
        const int nh = un.rows > HN ? 2 : 1;
        bool ok = true;
        for (int h = 0; h < nh; ++h, ++half) {
          if (!(ok = wait_acc(half))) break;
          fence_after();
          const int t0 = h * HN + 64 * w, left = un.rows - t0;
          const uint32_t ty = t_row + (half % ACCS) * HN;
          uint32_t y[2][32];
          if (left > 0) {
            tmem_ld32(ty, y[0]);
            if (left > 32) tmem_ld32(ty + 32, y[1]);
            tmem_ld_wait();
          }
          leave_acc(half);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (left > 32 * c) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const int t = 32 * c + i;
                store_pair(__uint_as_float(y[c][i]), __uint_as_float(y[c][i + 1]), col + (size_t)(t0 + t) * pr.N, pr.N,
                           left - t, live, lane);
              }
            }
          }
        }
        if (!ok) break;
      }
    }
  } else if (warp == 16) {
    // ---------------- producer of codes ----------------
    uint32_t j = 0;
    bool ok = true;
    for (long long u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const Unit un = unit_at(u);
      for (int i = 0; i < ks_n * AB; ++i, ++j) {
        const uint32_t slot = j % C_SLOTS;
        if (!(ok = wait_warp(&sh.cempty[slot], ((j / C_SLOTS) & 1) ^ 1, abort_flag))) break;
        if (elect_one()) {
          mbar_expect_tx(&sh.cfull[slot], C_BYTES);
          if (GLU) tma_load_4d(codes + slot * C_BYTES, &map_c, &sh.cfull[slot], (i / 2) * (CK / 2), un.nt * BM, i & 1, un.e);
          else tma_load_3d(codes + slot * C_BYTES, &map_c, &sh.cfull[slot], i * (CK / 2), un.nt * BM, un.e);
        }
        __syncwarp();
      }
    }
    if (lane == 0) *reinterpret_cast<volatile int*>(&sh.c_armed) = (int)j;
  } else if (warp == 17) {
    // ---------------- producer of token rows ----------------
    uint32_t it = 0;
    bool ok = true;
    for (long long u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const Unit un = unit_at(u);
      const int boxes = (un.rows + XR - 1) / XR;
      for (int kb = 0; kb < kb_n; ++kb, ++it) {
        const uint32_t s = it % X_STAGES;
        if (!(ok = wait_warp(&sh.xempty[s], ((it / X_STAGES) & 1) ^ 1, abort_flag))) break;
        if (elect_one()) {
          mbar_expect_tx(&sh.xfull[s], boxes * X_BOX);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(xs + s * SH::X_BYTES + b * X_BOX, &map_x, &sh.xfull[s], kb * BK, un.row0 + b * XR);
        }
        __syncwarp();
      }
    }
    if (lane == 0) *reinterpret_cast<volatile int*>(&sh.x_armed) = (int)it;
  } else {
    // ---------------- MMA issuer ----------------
    uint32_t it = 0, a = 0, half = 0;
    bool ok = true;
    const uint64_t desc_x = sw128_desc(smem_u32(xs));  // its address field counts 16 bytes
    for (long long u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const Unit un = unit_at(u);
      const int n = (un.rows + ROUND - 1) / ROUND * ROUND;
      const int nh = GLU || n > HN ? 2 : 1;
      for (int h = 0; ok && h < nh; ++h)  // the epilogue has left the accumulators (three halves ago)
        if (half + h >= ACCS) ok = wait_warp(&sh.tempty[(half + h) % ACCS], ((half + h) / ACCS - 1) & 1, abort_flag);
      if (!ok) break;
      fence_after();
      const uint32_t d0 = tmem + (half % ACCS) * HN, d1 = tmem + ((half + 1) % ACCS) * HN;
      const uint32_t id0 = idesc_bf16_f32(BM, n < HN ? n : HN), id1 = idesc_bf16_f32(BM, GLU ? n : n - HN);
      for (int kb = 0; kb < kb_n; ++kb, ++it) {
        const uint32_t s = it % X_STAGES;
        if (!(ok = wait_warp(&sh.xfull[s], (it / X_STAGES) & 1, abort_flag))) break;
#pragma unroll
        for (int b = 0; b < AB; ++b, ++a) {
          const uint32_t as = a % A_SLOTS;
          if (!(ok = wait_warp(&sh.afull[as], (a / A_SLOTS) & 1, abort_flag))) break;
          fence_after();
          if (elect_one()) {
            const uint64_t dx = desc_x + s * (SH::X_BYTES / 16);
            const uint32_t ta = tmem + A_COL + as * A_COLS;
#pragma unroll
            for (int k = 0; k < BK / UK; ++k) {
              const uint32_t acc = (kb | k) != 0;
              mma_ts(GLU && b ? d1 : d0, ta + k * (UK / 2), dx + k * (UK * 2 / 16), GLU && b ? id1 : id0, acc);
              if (!GLU && nh == 2) mma_ts(d1, ta + k * (UK / 2), dx + HN * BK * 2 / 16 + k * (UK * 2 / 16), id1, acc);
            }
            commit(&sh.aempty[as]);
            if (b == AB - 1) {
              commit(&sh.xempty[s]);
              if (kb == kb_n - 1) {
                commit(&sh.tfull[half % ACCS]);
                if (nh == 2) commit(&sh.tfull[(half + 1) % ACCS]);
              }
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      half += nh;
    }
    if (elect_one()) commit(&sh.done);
    __syncwarp();
    if (lane == 0) mbar_drain(&sh.done, 0, &g_err);
  }

  fence_before();
  __syncthreads();
  if (lane == 0 && *abort_flag) {  // no TMA write may still be landing when the CTA exits
    if (warp == 16)
      for (int j = sh.c_armed > C_SLOTS ? sh.c_armed - C_SLOTS : 0; j < sh.c_armed; ++j)
        mbar_drain(&sh.cfull[j % C_SLOTS], (j / C_SLOTS) & 1, &g_err);
    if (warp == 17)
      for (int j = sh.x_armed > X_STAGES ? sh.x_armed - X_STAGES : 0; j < sh.x_armed; ++j)
        mbar_drain(&sh.xfull[j % X_STAGES], (j / X_STAGES) & 1, &g_err);
  }
  if (warp == 18) {
    __syncwarp();
    fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

bool map_codes(CUtensorMap* m, const Product& pr, bool glu) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t row = (cuuint64_t)pr.K / 2, n = (cuuint64_t)pr.N, e = (cuuint64_t)pr.E;
  const cuuint64_t dims4[4] = {row, n, 2, e}, strides4[3] = {row, row * n, row * n * 2};
  const cuuint64_t dims3[3] = {row, n, e}, strides3[2] = {row, row * n};
  const cuuint32_t box[4] = {CK / 2, BM, 1, 1}, step[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, glu ? 4 : 3, const_cast<uint8_t*>(pr.w.codes), glu ? dims4 : dims3,
             glu ? strides4 : strides3, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool GLU, typename S, bool G32>
cudaError_t launch_t(Product pr, cudaStream_t s) {
  CUtensorMap mc, mx;
  const cuuint64_t dims[2] = {(cuuint64_t)pr.K, (cuuint64_t)pr.P}, strides[1] = {(cuuint64_t)pr.K * 2};
  const cuuint32_t box[2] = {BK, XR};
  if (!map_codes(&mc, pr, GLU) || !make_map_bf16(&mx, pr.x, 2, dims, strides, box)) return cudaErrorInvalidValue;
  auto kern = w4_tc_kernel<GLU, S, G32>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, (int)Shape<GLU>::smem, smem_set);
  if (e != cudaSuccess) return e;
  pr.n_tiles = (pr.N + BM - 1) / BM;
  const long long units = ((long long)pr.P / Shape<GLU>::ROWS + (pr.E < pr.P ? pr.E : pr.P)) * pr.n_tiles;
  const int sms = sm_count();
  e = launch_kernel(kern, dim3((unsigned)(units < sms ? units : sms)), dim3(THREADS), Shape<GLU>::smem, s, 1, true, mc, mx, pr);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <bool GLU>
cudaError_t launch_s(const Product& pr, cudaStream_t s) {
  if (pr.w.scales_bf16)
    return pr.group == 32 ? launch_t<GLU, __nv_bfloat16, true>(pr, s) : launch_t<GLU, __nv_bfloat16, false>(pr, s);
  return pr.group == 32 ? launch_t<GLU, float, true>(pr, s) : launch_t<GLU, float, false>(pr, s);
}

}  // namespace

int w4_tc_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_w4_tc(const Product& pr, bool glu, cudaStream_t s) {
  return glu ? launch_s<true>(pr, s) : launch_s<false>(pr, s);
}

}  // namespace semmoe
