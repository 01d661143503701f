// Grouped products of bf16 rows with 4-bit weights (w4.cuh) on the 5th-generation
// tensor cores, for all but a few rows.
//
// The weights are the left operand (M = 128 weight rows), held in tensor memory: a
// thread turns the codes of its row into bf16 in registers and writes them to its
// TMEM lane, so the expanded weights never pass through shared memory, whose
// bandwidth bounds the bf16 products (ffn_tc.cu).  The token rows are the right
// operand (N = up to 128 rows of a group, a multiple of 16), by TMA.
//
// A unit has two accumulators of up to 128 columns (tokens):
//   plain:  128 weight rows x up to 256 token rows; both halves read one A block
//   SwiGLU: 128 gate rows and the 128 up rows x up to 128 token rows; two A blocks
// TMEM holds three accumulators and a ring of A blocks: a unit's first accumulator
// is free while the epilogue still reads the unit before.
//
// One persistent CTA per SM takes units in turn.  Warp roles:
//   expansion   EXP / 4 groups of four warps, a chunk of 128 columns at a time in turn
//               (SwiGLU: half of the groups for gate rows, half for up rows)
//   epilogue    EPI / 4 groups of four, the columns of an accumulator divided between them
//   producers   one warp for codes ([128 rows x 128 columns] a slot), one for token rows
//   issuer      allocates TMEM, issues the MMAs (M128 N16..128 K16)
// 16 warps expand; four (few token rows a unit) or eight read the accumulators.  With few rows a k-block has 128
// columns, which halves the barriers a weight, else 64, so that more A blocks are on their way.
//
// What bounds it.  Many rows: the MMAs (a SwiGLU k-block of 128 rows takes 630 to 650 clocks of MMAs and 850 to 900 in
// all; the rest is waited for accumulators, token rows and A blocks in turn).  A decode batch: half of the time the
// expansion's instructions (their count times two clocks, whichever pipe they use), half the chain codes, registers, tensor
// memory, MMA, place free again; a second issuing warp changes nothing.
// Measured (GB300, 128 experts of 2048 x 768 or 64 of 2048 x 1408, groups of 128, bf16 scales): 131072 rows through the FFN
// 923 to 939 us in a captured graph (1.3 PFLOP/s; 860 between flushes of L2, before the power cap), 384 rows 72 us (4.4 TB/s of weights; 88 with groups of 64 and zero points, 102 with
// fp32 scales), 384 rows through one 1408 x 2048 product with zero points 34 us.
// Tried and slower: 24 expansion warps; accumulators split by k-step; a single lane for the issuer's whole loop; decode
// batches on the warp-level product with codes straight into registers (48.6 us where this took 34.5, its loads alone 33).
//
// Expansion of a word of eight codes: two masked halves (codes of even columns, and of odd ones, shifted or as they lie, 16
// times as large), then one byte permutation a pair of columns, whose result reads as bf16 numbers: integers below 256 times
// 2^-133, since the exponents 0 and 1 have the same steps.  Then, where odd columns' are 16 times as large with a sixteenth
// of the factor,
//   without zero points, bf16 scales:  w = code * (s 2^93) - 8 s 2^-40      one fused operation, one rounding
//   with zero points, bf16 scales:  16 - z is added to the codes, four bytes an addition; then the same with 16 s
//   fp32 scales: d = code * 2^127 - z 2^-6 (exact),  w = d * (s 2^-34) with the scale as the sum of two bf16 numbers, the
//   smaller product first
// So a weight is held as w 2^-40 (the sums are multiplied by 2^40), rounded once to bf16: at most half a
// step off, as in any bf16 copy of the weights (with fp32 scales 2^-17 of it more, as two bf16 numbers hold the scale to 2^-18).
// That is 10 (shifted 11), 13 and 18 instructions a word, and each of them adds some 3 us to the FFN of 384 rows above.
//
// Every wait is bounded; a wait that runs out sets the timeout bit of the device error
// word and an abort flag, after which every role stops, loads and MMAs in flight are
// drained (again with a bound), and TMEM is freed before the CTA exits.
#pragma once

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
constexpr int UK = 16;                // K per MMA
constexpr int CHUNK = 128;            // columns of a slot of codes: 64 bytes a row
constexpr int C_BYTES = BM * CHUNK / 2;
constexpr int XR = 32;                // rows of a box of token rows
constexpr int XC = 64;                // its columns: a 128-byte swizzle row
constexpr int X_BOX = XR * XC * 2;
constexpr int ACCS = 3;
constexpr uint32_t TMEM_COLS = 512;
constexpr int ROUND = 16;             // token rows of a unit: a multiple of this
constexpr uint32_t DONES = 16;        // barriers of finished k-blocks

enum Mode { SYM, ZEROS, F32 };        // bf16 scales without and with zero points; fp32 scales

// ROWS: token rows of a unit, at most.
template <bool GLU, int ROWS>
struct Shape {
  static constexpr bool few = ROWS <= 64;
  static constexpr int HN = ROWS < 128 ? ROWS : 128;   // columns of an accumulator
  static constexpr int BK = few ? 128 : 64;            // columns of a k-block
  static constexpr int EXP = 16, EPI = few ? 4 : 8;
  static constexpr int THREADS = (EXP + EPI + 3) * 32;
  static constexpr int AB = GLU ? 2 : 1;               // A blocks of a k-block
  static constexpr int A_COLS = AB * BK / 2;           // TMEM columns of a k-block's
  static constexpr int AD = (TMEM_COLS - ACCS * HN) / A_COLS;
  static constexpr int X_BYTES = ROWS * BK * 2;        // a stage of token rows
  static constexpr int XD = ROWS == 32 ? 8 : ROWS == 256 ? 5 : 6;
  static constexpr int C_FIT = (208 * 1024 - XD * X_BYTES) / C_BYTES, C_SLOTS = C_FIT < 16 ? C_FIT : 16;
  static constexpr size_t smem = 1024 + (size_t)C_SLOTS * C_BYTES + (size_t)XD * X_BYTES;
  static constexpr int STEP = EXP / 4 / AB, BLOCKS = CHUNK / BK;  // chunks between an expansion group's, k-blocks of one
  static_assert(AD >= 2 && AD <= (int)DONES && XD <= (int)DONES, "rings");
  // A wait tells a barrier's phase from the one before it only: whoever waits for a phase must know that the one before it
  // is over.  Roles that take every turn know; an expansion group, which skips the others' turns, knows that the k-blocks
  // AD before its last one are done.
  static_assert((STEP - 1) * BLOCKS + 1 <= (int)DONES, "the turns of done[] that a group skips");
  static_assert(C_SLOTS >= AB * (STEP + (AD + BLOCKS - 1) / BLOCKS), "the turns of cfull[] that a group skips");
};

template <int C_SLOTS, int XD, int AD>
struct Shared {
  uint64_t cfull[C_SLOTS], cempty[C_SLOTS], xfull[XD], afull[AD];
  uint64_t done[DONES];  // a k-block's MMAs: its token rows and A blocks may be overwritten
  uint64_t tfull[ACCS], tempty[ACCS], last;
  uint32_t tmem_base;
  int abort_flag;
  int c_armed, x_armed;  // slots and stages that the producers have armed
  Groups groups;
};

// A k-block's places in the rings of token rows and A blocks, and the phases of their barriers.
struct Turn {
  uint32_t s, s_phase, a, a_phase;
  __device__ __forceinline__ void step(uint32_t stages, uint32_t blocks) {
    if (++s == stages) s = 0, s_phase ^= 1;
    if (++a == blocks) a = 0, a_phase ^= 1;
  }
};

// D[tmem] (+)= A[tmem] * B[smem]^T.  b: the low word of B's descriptor, which holds its address; the high word is that of
// every K-major tile with 128-byte swizzle (sw128_desc).  Few instructions an MMA: with few columns they take longer than it.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool ACCUMULATE>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate = 1) {
  if (ACCUMULATE)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 d;\n\t"
        "setp.eq.u32 p, 0, 0;\n\tmov.b64 d, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], d, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(idesc), "n"(kDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 d;\n\t"
        "setp.ne.u32 p, %5, 0;\n\tmov.b64 d, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], d, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(idesc), "n"(kDescHigh), "r"(accumulate)
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
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t both(float v) { return pack_bf16x2(v, v); }

// Whether odd columns' codes are shifted into place, or taken where they lie, 16 times as large.  Shifted: with zero points,
// which need the byte's upper bits, and in units of many rows without them (131072 rows through the FFN 862 to 868 us, 872 with the
// codes where they lie; 384 rows 74.6 and 71.6; fp32 scales 1069 and 1047, 107 and 102).
template <int MODE, bool FEW>
constexpr bool shifted() { return MODE == ZEROS || (MODE == SYM && !FEW); }

// What a group's codes are expanded with.
struct Factors {
  uint32_t f[3];
};
template <int MODE, bool FEW>
__device__ __forceinline__ Factors factors(float s, uint32_t z) {
  constexpr float k93 = 9903520314283042199192993792.0f, k89 = k93 / 16, k40 = 9.094947017729282379150390625e-13f,
                  k34 = 5.82076609134674072265625e-11f;  // 2^93, 2^-40, 2^-34
  if (MODE == SYM) return Factors{{pack_bf16x2(s * k93, shifted<MODE, FEW>() ? s * k93 : s * k89), both(-8.0f * k40 * s), 0u}};
  if (MODE == ZEROS) return Factors{{both(s * k93), both(-16.0f * k40 * s), (16u - (z & 15u)) * 0x01010101u}};
  const uint32_t zero = both(-0.015625f * (float)(z & 15u));
  const float hi = __bfloat162float(__float2bfloat16_rn(s)), rest = s - hi;
  return Factors{{zero, both(hi * k34), both(rest == rest ? rest * k34 : 0.0f)}};  // (an infinite scale has no rest)
}

// The eight codes of a word as bf16 weights, in column order.
template <int MODE, bool FEW>
__device__ __forceinline__ void expand(uint32_t w, const Factors& f, uint32_t* r) {
  uint32_t even = w & 0x0f0f0f0fu, odd = shifted<MODE, FEW>() ? (w >> 4) & 0x0f0f0f0fu : w & 0xf0f0f0f0u;
  if (MODE == ZEROS) even += f.f[2], odd += f.f[2];  // code - z + 16, 1 to 31 in each byte
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    uint32_t q;  // byte i of each, with copies of the even one's sign bit, 0, above
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(q) : "r"(even), "r"(odd), "r"(i | ((8 + i) << 4) | ((4 + i) << 8) | ((8 + i) << 12)));
    if (MODE != F32) {
      r[i] = fma_bf16x2(q, f.f[0], f.f[1]);
    } else {
      const uint32_t d = fma_bf16x2(q, 0x7d007f00u, f.f[0]);
      r[i] = fma_bf16x2(d, f.f[1], mul_bf16x2(d, f.f[2]));
    }
  }
}

// silu(g) * u of sums held as g 2^-40 and u 2^-40.
__device__ __forceinline__ float unscaled_swiglu(float g, float u) {
  constexpr float k40 = 1099511627776.0f;
  const float z = g * k40;
  return __fdividef(z, 1.0f + __expf(-z)) * (u * k40);
}

// mbar_wait by a whole converged warp, polling a few times before it looks at the clock.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return mbar_wait_warp(bar, parity, abort_flag, &g_err);
}

// Whether a phase has completed, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// 2 N tokens' columns of a warp's 32 weight rows, v[i]: this lane's row of tokens 2 i and 2 i + 1 in bf16.  Even lanes store
// the first token's pair of rows, odd lanes the second's.  left: tokens from the first one on that are the unit's.
// All exchanges come before the first store, and the stores are predicated: a branch around each one made the epilogue nearly
// twice as long (4465 clocks a SwiGLU unit's half, 2381 without).
template <int N>
__device__ __forceinline__ void store_pairs(const uint32_t (&v)[N], __nv_bfloat16* first, size_t stride, int left, bool live, int lane) {
  const int odd = lane & 1;
  uint32_t out[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, v[i], 1);
    out[i] = odd ? __byte_perm(other, v[i], 0x7632) : __byte_perm(v[i], other, 0x5410);
  }
  if (odd) first += stride;
  const int mine = live ? left - odd : 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %0, %3;\n\t@p st.global.b32 [%1], %2;\n\t}" ::"r"(mine),
                 "l"(first + 2 * i * stride), "r"(out[i]), "r"(2 * i)
                 : "memory");
}

template <bool GLU, int ROWS, int MODE>
__global__ void __launch_bounds__(Shape<GLU, ROWS>::THREADS, 1)
w4_tc_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_x, Product pr) {
  using SH = Shape<GLU, ROWS>;
  constexpr int AB = SH::AB, XD = SH::XD, AD = SH::AD, C_SLOTS = SH::C_SLOTS, BK = SH::BK, HN = SH::HN;
  constexpr uint32_t A_COL = ACCS * HN;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ Shared<C_SLOTS, XD, AD> sh;
  unsigned char* xs = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* codes = xs + XD * SH::X_BYTES;
  volatile int* abort_flag = &sh.abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  constexpr int EPI0 = SH::EXP, C_WARP = EPI0 + SH::EPI, X_WARP = C_WARP + 1, MMA_WARP = C_WARP + 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C_SLOTS; ++i) {
      mbar_init(&sh.cfull[i], 1);
      mbar_init(&sh.cempty[i], 4);  // the warps that read it
    }
    for (int i = 0; i < XD; ++i) mbar_init(&sh.xfull[i], 1);
    for (uint32_t i = 0; i < DONES; ++i) mbar_init(&sh.done[i], 1);
    for (int i = 0; i < AD; ++i) mbar_init(&sh.afull[i], 4 * AB);
    for (int i = 0; i < ACCS; ++i) {
      mbar_init(&sh.tfull[i], 1);
      mbar_init(&sh.tempty[i], SH::EPI);
    }
    mbar_init(&sh.last, 1);
    sh.abort_flag = 0;
    sh.c_armed = sh.x_armed = 0;
    mbar_init_fence();
    prefetch_map(&map_c);
    prefetch_map(&map_x);
  }
  if (warp == MMA_WARP) tmem_alloc(&sh.tmem_base, TMEM_COLS);
  if (!pr.early) pdl_wait();
  pdl_trigger();
  if (warp == 0) load_groups(sh.groups, pr, ROWS, lane, &g_err);
  fence_before();
  __syncthreads();
  fence_after();

  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);
  const int G = pr.E, n_tiles = pr.n_tiles, K = pr.K, units = gridDim.x;
  const int total = __shfl_sync(0xffffffffu, sh.groups.total, 0) * n_tiles;
  const int kb_n = (K + BK - 1) / BK, ch_n = (K + CHUNK - 1) / CHUNK;
  auto unit_at = [&](int u) { return decode_unit(sh.groups, G, n_tiles, ROWS, u, ROUND); };

  if (warp < SH::EXP) {
    // ---------------- codes to bf16 weights in TMEM ----------------
    constexpr int STEP = SH::STEP;
    constexpr int SB = MODE == F32 ? 4 : 2;             // bytes of a scale
    constexpr int NR = MODE == F32 ? 4 : 2;             // registers of a chunk's scales
    const int wg = warp / 4, ab = GLU ? wg & 1 : 0, r = (warp % 4) * 32 + lane;
    const int KG = K / pr.group, rows_w = GLU ? 2 * pr.N : pr.N;
    const int gs = pr.group >= CHUNK ? 1 : CHUNK / pr.group;    // scales of a chunk
    const bool whole = gs == 1 || K % CHUNK == 0;               // a chunk's scales are aligned to their size
    const int per = pr.group > CHUNK ? pr.group / CHUNK : 1;    // chunks of a scale
    const uint32_t a_lane = tmem + ((uint32_t)((warp % 4) * 32) << 16) + A_COL + ab * (BK / 2);
    const unsigned char* srow = nullptr;  // the row's scales and zero points
    const uint8_t* zrow = nullptr;
    auto at_row = [&](const Unit& un) {
      int n = un.nt * BM + r;
      if (n >= pr.N) n = pr.N - 1;  // a row past the matrix: its codes are 0, nothing of it is stored
      const size_t at = ((size_t)un.e * rows_w + n + (GLU && ab ? pr.N : 0)) * KG;
      srow = static_cast<const unsigned char*>(pr.w.scales) + at * SB;
      if (MODE != SYM) zrow = pr.w.zeros != nullptr ? pr.w.zeros + at : nullptr;
    };
    // a chunk's scales and zero points as they lie in memory, loaded one chunk of this group ahead
    uint32_t raw[NR], rawz = 0x08080808u;
    auto load = [&](int ch) {
      const int i0 = per > 1 ? ch / per : ch * gs;
      if (whole) {
        const unsigned char* p = srow + i0 * SB;
        if (gs * SB == 2) raw[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
        if (gs * SB == 4) raw[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        if (gs * SB == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
          raw[0] = v.x, raw[1] = v.y;
        }
        if (MODE == F32 && gs == 4) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
          raw[0] = v.x, raw[1] = v.y, raw[NR - 2] = v.z, raw[NR - 1] = v.w;
        }
        if (MODE != SYM && zrow != nullptr) {
          if (gs == 1) rawz = __ldg(zrow + i0);
          if (gs == 2) rawz = __ldg(reinterpret_cast<const unsigned short*>(zrow + i0));
          if (gs == 4) rawz = __ldg(reinterpret_cast<const uint32_t*>(zrow + i0));
        }
        return;
      }
      uint32_t v[4], z = 0;  // scale by scale; past K, where token rows are 0, a scale of 0 (an infinite one would give NaN)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = i0 + i < KG ? i0 + i : KG - 1;
        v[i] = MODE == F32 ? __ldg(reinterpret_cast<const uint32_t*>(srow) + j)
                           : __ldg(reinterpret_cast<const unsigned short*>(srow) + j);
        if (i0 + i >= KG) v[i] = 0;
        if (MODE != SYM) z |= (zrow != nullptr ? (uint32_t)__ldg(zrow + j) : 8u) << (8 * i);
      }
      if (MODE != SYM) rawz = z;
      if (MODE == F32) {
        raw[0] = v[0], raw[1] = v[1], raw[NR - 2] = v[2], raw[NR - 1] = v[3];
      } else {
        raw[0] = v[0] | (v[1] << 16), raw[1] = v[2] | (v[3] << 16);
      }
    };
    // the factors of scale j of a chunk
    auto factors_of = [&](const uint32_t (&v)[NR], uint32_t z, int j) {
      uint32_t s;
      if (MODE == F32) s = j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[NR - 2] : v[NR - 1];
      else s = j & 1 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16;
      return factors<MODE, SH::few>(__uint_as_float(s), z >> (8 * j));
    };
    // this group's place: unit u, chunk ch of it; its slot of codes and first k-block, counted from the start
    int u = blockIdx.x, ch = GLU ? wg >> 1 : wg;
    uint32_t slot = ch * AB + ab, slot_phase = 0, first = 0;  // first: k-blocks of the units before
    auto settle = [&]() {
      while (ch >= ch_n) ch -= ch_n, u += units, first += kb_n;
    };
    settle();
    int loaded = -1;  // the unit of srow
    if (u < total) {
      at_row(unit_at(u));
      loaded = u;
      load(ch);
    }
    bool ok = true;
    while (u < total) {
      uint32_t now[NR];
      const uint32_t nowz = rawz;
#pragma unroll
      for (int i = 0; i < NR; ++i) now[i] = raw[i];
      const uint32_t it0 = first + ch * (CHUNK / BK);
      const int blocks = kb_n - ch * (CHUNK / BK);  // k-blocks from here on
      ch += STEP;
      settle();
      if (u < total) {
        if (u != loaded) {
          at_row(unit_at(u));
          loaded = u;
        }
        load(ch);
      }
      if (!(ok = wait_warp(&sh.cfull[slot], slot_phase, abort_flag))) break;
      const unsigned char* src = codes + slot * C_BYTES + r * 64;
      Factors fa, fb;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 64 columns
        if (BK == 64 && h >= blocks) break;
        uint4 c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = *reinterpret_cast<const uint4*>(src + (((2 * h + i) ^ ((r >> 1) & 3)) << 4));
        if (gs == 4) {
          fa = factors_of(now, nowz, 2 * h);
          fb = factors_of(now, nowz, 2 * h + 1);
        } else if (h == 0 || gs == 2) {
          fb = fa = factors_of(now, nowz, h);
        }
        uint32_t w[32];
        expand<MODE, SH::few>(c[0].x, fa, w);
        expand<MODE, SH::few>(c[0].y, fa, w + 4);
        expand<MODE, SH::few>(c[0].z, fa, w + 8);
        expand<MODE, SH::few>(c[0].w, fa, w + 12);
        expand<MODE, SH::few>(c[1].x, fb, w + 16);
        expand<MODE, SH::few>(c[1].y, fb, w + 20);
        expand<MODE, SH::few>(c[1].z, fb, w + 24);
        expand<MODE, SH::few>(c[1].w, fb, w + 28);
        const uint32_t it = it0 + (BK == 64 ? h : 0), place = it % AD;
        if ((BK == 64 || h == 0) && it >= AD) {  // the MMAs that read this place
          if (!(ok = wait_warp(&sh.done[(it - AD) % DONES], ((it - AD) / DONES) & 1, abort_flag))) break;
          fence_after();
        }
        tmem_st32(a_lane + place * SH::A_COLS + (BK == 128 ? h * 32 : 0), w);
        if (BK == 64 || h == 1) {
          tmem_st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.afull[place]);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.cempty[slot]);
      slot += STEP * AB;
      if (slot >= C_SLOTS) slot -= C_SLOTS, slot_phase ^= 1;
    }
  } else if (warp < C_WARP) {
    // ---------------- epilogue ----------------
    constexpr int PART = HN / (SH::EPI / 4);              // columns of a group of four warps
    constexpr float kUnscale = 1099511627776.0f;          // 2^40
    const int q = warp & 3, w = (warp - EPI0) >> 2;
    const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + PART * w;
    uint32_t half = 0;
    auto wait_acc = [&](uint32_t h) { return wait_warp(&sh.tfull[h % ACCS], (h / ACCS) & 1, abort_flag); };
    auto leave_acc = [&](uint32_t h) {
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tempty[h % ACCS]);
    };
    for (int u = blockIdx.x; u < total; u += units) {
      const Unit un = unit_at(u);
      const int n = un.nt * BM + q * 32 + lane;  // this lane's output column
      const bool live = n < pr.N;
      __nv_bfloat16* col = pr.out + (size_t)un.row0 * pr.N + (live ? n & ~1 : 0);
      if (GLU) {
        if (!wait_acc(half) || !wait_acc(half + 1)) break;
        fence_after();
        const int left = un.rows - PART * w;
        const uint32_t tg = t_row + (half % ACCS) * HN, tu = t_row + ((half + 1) % ACCS) * HN;
        // pieces of 16 columns: the registers of 27 warps hold no more (the accumulators are held for the whole of it)
#pragma unroll 1
        for (int c = 0; c < PART; c += 16) {
          if (left <= c) break;
          uint32_t g[16], up[16];
          tmem_ld16(tg + c, g);
          tmem_ld16(tu + c, up);
          tmem_ld_wait();
          if (c + 16 >= PART || left <= c + 16) leave_acc(half), leave_acc(half + 1);
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = pack_bf16x2(unscaled_swiglu(__uint_as_float(g[2 * i]), __uint_as_float(up[2 * i])),
                               unscaled_swiglu(__uint_as_float(g[2 * i + 1]), __uint_as_float(up[2 * i + 1])));
          store_pairs(v, col + (size_t)(PART * w + c) * pr.N, pr.N, left - c, live, lane);
        }
        if (left <= 0) leave_acc(half), leave_acc(half + 1);
        half += 2;
      } else {
        const int nh = un.rows > HN ? 2 : 1;
        bool ok = true;
        for (int h = 0; h < nh; ++h, ++half) {
          if (!(ok = wait_acc(half))) break;
          fence_after();
          const int t0 = h * HN + PART * w, left = un.rows - t0;
          const uint32_t ty = t_row + (half % ACCS) * HN;
#pragma unroll 1
          for (int c = 0; c < PART; c += 32) {
            if (left <= c) break;
            uint32_t y[32];
            tmem_ld32(ty + c, y);
            tmem_ld_wait();
            if (c + 32 >= PART || left <= c + 32) leave_acc(half);
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[i] = pack_bf16x2(__uint_as_float(y[2 * i]) * kUnscale, __uint_as_float(y[2 * i + 1]) * kUnscale);
            store_pairs(v, col + (size_t)(t0 + c) * pr.N, pr.N, left - c, live, lane);
          }
          if (left <= 0) leave_acc(half);
        }
        if (!ok) break;
      }
    }
  } else if (warp == C_WARP) {
    // ---------------- producer of codes ----------------
    uint32_t j = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < total; u += units) {
      const Unit un = unit_at(u);
      for (int i = 0; i < ch_n * AB; ++i, ++j) {
        const uint32_t slot = j % C_SLOTS;
        if (!(ok = wait_warp(&sh.cempty[slot], ((j / C_SLOTS) & 1) ^ 1, abort_flag))) break;
        if (elect_one()) {
          mbar_expect_tx(&sh.cfull[slot], C_BYTES);
          if (GLU)
            tma_load_4d(codes + slot * C_BYTES, &map_c, &sh.cfull[slot], (i / 2) * (CHUNK / 2), un.nt * BM, i & 1, un.e);
          else tma_load_3d(codes + slot * C_BYTES, &map_c, &sh.cfull[slot], i * (CHUNK / 2), un.nt * BM, un.e);
        }
        __syncwarp();
      }
    }
    if (lane == 0) *reinterpret_cast<volatile int*>(&sh.c_armed) = (int)j;
  } else if (warp == X_WARP) {
    // ---------------- producer of token rows ----------------
    if (pr.early) pdl_wait();  // (also by a CTA without units: a kernel ends after the one before it)
    uint32_t it = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < total; u += units) {
      const Unit un = unit_at(u);
      const int boxes = (un.rows + XR - 1) / XR;
      for (int kb = 0; kb < kb_n; ++kb, ++it) {
        const uint32_t s = it % XD;
        if (it >= XD && !(ok = wait_warp(&sh.done[(it - XD) % DONES], ((it - XD) / DONES) & 1, abort_flag))) break;
        if (elect_one()) {
          mbar_expect_tx(&sh.xfull[s], boxes * (BK / XC) * X_BOX);
          for (int b = 0; b < boxes; ++b)
#pragma unroll
            for (int k = 0; k < BK / XC; ++k)
              tma_load_2d(xs + s * SH::X_BYTES + k * (ROWS * XC * 2) + b * X_BOX, &map_x, &sh.xfull[s], kb * BK + k * XC,
                          un.row0 + b * XR);
        }
        __syncwarp();
      }
    }
    if (lane == 0) *reinterpret_cast<volatile int*>(&sh.x_armed) = (int)it;
  } else {
    // ---------------- MMA issuer ----------------
    uint32_t it = 0, half = 0;      // k-block, half tile
    Turn next{0, 0, 0, 0};
    bool ready = false;             // the next operands have been seen
    bool ok = !pr.stall || wait_warp(&sh.last, 0, abort_flag);
    const uint32_t desc_x = (uint32_t)sw128_desc(smem_u32(xs));  // its address field counts 16 bytes
    for (int u = blockIdx.x; ok && u < total; u += units) {
      const Unit un = unit_at(u);
      const int n = (un.rows + ROUND - 1) / ROUND * ROUND;
      const int nh = GLU || n > HN ? 2 : 1;
      for (int h = 0; ok && h < nh; ++h)  // the epilogue has left the accumulators (three halves ago)
        if (half + h >= ACCS) ok = wait_warp(&sh.tempty[(half + h) % ACCS], ((half + h) / ACCS - 1) & 1, abort_flag);
      if (!ok) break;
      fence_after();
      const uint32_t d0 = tmem + (half % ACCS) * HN, d1 = tmem + ((half + 1) % ACCS) * HN;
      const uint32_t id0 = idesc_bf16_f32(BM, n < HN ? n : HN), id1 = idesc_bf16_f32(BM, GLU ? n : n - HN);
      // `turn`: a k-block's places in the rings
      auto issue = [&](int kb, const Turn& turn, int k0, int k1) {
        const uint32_t dx = desc_x + turn.s * (SH::X_BYTES / 16), ta = tmem + A_COL + turn.a * SH::A_COLS;
#pragma unroll
        for (int k = k0; k < k1; ++k) {
          const uint32_t b = dx + (k / 4) * (ROWS * XC * 2 / 16) + (k % 4) * (UK * 2 / 16);
          auto mma = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
            if (k > 0) mma_ts<true>(d, a, b, id);
            else mma_ts<false>(d, a, b, id, kb);
          };
          mma(d0, ta + k * (UK / 2), b, id0);
          if (GLU) mma(d1, ta + BK / 2 + k * (UK / 2), b, id1);
          else if (nh == 2) mma(d1, ta + k * (UK / 2), b + HN * XC * 2 / 16, id1);
        }
      };
      auto finish = [&](int kb) {
        commit(&sh.done[it % DONES]);
        if (kb == kb_n - 1) {
          commit(&sh.tfull[half % ACCS]);
          if (nh == 2) commit(&sh.tfull[(half + 1) % ACCS]);
        }
      };
      auto wait_for = [&](const Turn& turn) {
        return wait_warp(&sh.xfull[turn.s], turn.s_phase, abort_flag) && wait_warp(&sh.afull[turn.a], turn.a_phase, abort_flag);
      };
      auto seen = [&](const Turn& turn) { return mbar_test(&sh.xfull[turn.s], turn.s_phase) & mbar_test(&sh.afull[turn.a], turn.a_phase); };
      // The issue of a long MMA waits for the ones before it, and a look at a barrier takes as long as one or two of them,
      // so the next k-block's barriers are looked at before this one's last MMAs; short ones are issued at once.
      constexpr int FIRST = SH::few ? BK / UK : BK / UK - 1;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!ready && !(ok = wait_for(next))) break;
        fence_after();
        if (elect_one()) {
          issue(kb, next, 0, FIRST);
          if (FIRST == BK / UK) finish(kb);
        }
        __syncwarp();
        Turn after = next;
        after.step(XD, AD);
        const bool look = seen(after);
        if (FIRST < BK / UK) {
          if (elect_one()) {
            issue(kb, next, FIRST, BK / UK);
            finish(kb);
          }
          __syncwarp();
        }
        ++it;
        next = after;
        ready = __all_sync(0xffffffffu, look);
      }
      half += nh;
    }
    if (elect_one()) commit(&sh.last);
    __syncwarp();
    if (lane == 0) mbar_drain(&sh.last, 0, &g_err);
  }

  fence_before();
  __syncthreads();
  if (lane == 0 && *abort_flag) {  // no TMA write may still be landing when the CTA exits
    if (warp == C_WARP)
      for (int j = sh.c_armed > C_SLOTS ? sh.c_armed - C_SLOTS : 0; j < sh.c_armed; ++j)
        mbar_drain(&sh.cfull[j % C_SLOTS], (j / C_SLOTS) & 1, &g_err);
    if (warp == X_WARP)
      for (int j = sh.x_armed > XD ? sh.x_armed - XD : 0; j < sh.x_armed; ++j)
        mbar_drain(&sh.xfull[j % XD], (j / XD) & 1, &g_err);
  }
  if (warp == MMA_WARP) {
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
  const cuuint32_t box[4] = {CHUNK / 2, BM, 1, 1}, step[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, glu ? 4 : 3, const_cast<uint8_t*>(pr.w.codes), glu ? dims4 : dims3,
             glu ? strides4 : strides3, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool GLU, int ROWS, int MODE>
cudaError_t launch_t(Product pr, cudaStream_t s) {
  using SH = Shape<GLU, ROWS>;
  CUtensorMap mc, mx;
  const cuuint64_t dims[2] = {(cuuint64_t)pr.K, (cuuint64_t)pr.P}, strides[1] = {(cuuint64_t)pr.K * 2};
  const cuuint32_t box[2] = {XC, XR};
  if (!map_codes(&mc, pr, GLU) || !make_map_bf16(&mx, pr.x, 2, dims, strides, box)) return cudaErrorInvalidValue;
  auto kern = w4_tc_kernel<GLU, ROWS, MODE>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, (int)SH::smem, smem_set);
  if (e != cudaSuccess) return e;
  pr.n_tiles = (pr.N + BM - 1) / BM;
  const long long units = ((long long)pr.P / ROWS + (pr.E < pr.P ? pr.E : pr.P)) * pr.n_tiles;
  const int sms = sm_count();
  e = launch_kernel(kern, dim3((unsigned)(units < sms ? units : sms)), dim3(SH::THREADS), SH::smem, s, 1, true, mc, mx, pr);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <bool GLU, int ROWS>
cudaError_t launch_mode(const Product& pr, cudaStream_t s) {
  if (!pr.w.scales_bf16) return launch_t<GLU, ROWS, F32>(pr, s);
  return pr.w.zeros != nullptr ? launch_t<GLU, ROWS, ZEROS>(pr, s) : launch_t<GLU, ROWS, SYM>(pr, s);
}

}  // namespace
}  // namespace semmoe
