// Grouped products of 4-bit microscaled operands on the 5th-generation tensor
// cores (tcgen05.mma kind::mxf4, fp32 accumulation in TMEM; format: mx4.cuh).
// Rows [off[b], off[b+1]) belong to expert pe[b]:
//   plain:  out = a B_e^T                                      (bf16 or fp32)
//   SwiGLU: h = silu(a W1_e^T) * (a W3_e^T), quantised per 32 columns (4 bits)
//
// One persistent CTA per SM walks the (m-tile, n-tile) list of all groups, in
// M128 x N256 tiles.  Warp roles:
//   warp 0      TMA producer: A [128 x 256] and B [256 x 256] values per stage
//               (128-byte rows, 128-byte swizzle) and their scales (512-byte tiles)
//   warp 1      allocates TMEM; one thread copies the stage's scales to TMEM
//               (tcgen05.cp) and issues the MMAs (K 64 each)
//   warps 2..9  epilogue: two groups of four, each one half of the tile's columns
// TMEM: two accumulators of 256 columns that share 48 of them, [0, 256) and
// [208, 464), and two sets of scales in the 48 columns left, so that the epilogue
// of a tile runs beside the next tile's MMAs: it loads the shared columns first
// and then lets the MMAs go on.  A set of scales is overwritten only after the
// commit of the MMAs that read it, two stages before.
//
// Every wait is bounded; a wait that runs out sets the timeout bit of the device
// error word and an abort flag, after which every role stops, loads and MMAs in
// flight are drained (again with a bound), and TMEM is freed before the CTA exits.
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "tc_common.cuh"

namespace semmoe {
namespace {

using namespace tc;
using namespace mx4;

__device__ int g_err;

constexpr int BM = 128, BN = 256;      // tile = one MMA's M and N
constexpr int BK = 256;                // K per stage: one 128-byte swizzle row of packed values
constexpr int UK = 64;                 // K per tcgen05.mma, kind::mxf4
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK / 2;   // 16 KB
constexpr int B_BYTES = BN * BK / 2;   // 32 KB
constexpr int SC_BYTES = 6 * kTileBytes;  // two column tiles of A's and of B's two row tiles
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 320;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SC_COLS = 24;       // columns of one set of scales: 2 x (4 for A + 8 for B)
constexpr uint32_t SC_COL = TMEM_COLS - 2 * SC_COLS;  // the scales' first column
constexpr uint32_t ACC1_COL = SC_COL - BN;            // the second accumulator's first column (the first one's is 0)
static_assert(BN - ACC1_COL <= 64, "the epilogue's first pieces hold the shared columns");
constexpr int MAX_GROUPS = 256;

struct Shared {
  uint64_t full[STAGES], empty[STAGES], tfull[2], tempty, done;
  uint32_t tmem_base;
  int abort_flag;
  int armed;  // stage positions the producer has armed
  int total_mtiles;
  int off[MAX_GROUPS + 1];
  int pe[MAX_GROUPS];
  int tp[MAX_GROUPS + 1];
};

constexpr int OUT_STAGE_BYTES = 8 * 2048;  // 2 KB per epilogue warp
constexpr size_t kSmemBytes =
    1024 + (size_t)STAGES * (STAGE_BYTES + SC_BYTES) + OUT_STAGE_BYTES + sizeof(Shared);

// Instruction descriptor, kind::mxf4: A and B e2m1 (bits 7-9 and 10-11 = 1), both
// K-major, N >> 3 at bits 17-22, scales with 8 exponent bits (bit 23), M >> 7 at
// bits 27-28, K = 64 (bit 31 = 0); the scales' first byte within their 32-bit
// word (0 or 2) at bits 4-5 (B) and 29-30 (A).
__device__ __forceinline__ constexpr uint32_t idesc_mx4(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) |
         (sf << 29);
}

// Shared-memory descriptor of one 512-byte scale tile: 32 rows of 16 bytes, no
// swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// One thread: a scale tile to 4 TMEM columns, replicated in the four 32-lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void mma_mx4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float swiglu(uint32_t gw, uint32_t uw) {
  const float g = __uint_as_float(gw), u = __uint_as_float(uw);
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// m-tile mu -> (first row, valid rows, expert)
__device__ __forceinline__ void decode_mtile(const Shared& sh, int G, int mu, int& row0, int& rows, int& e) {
  int lo = 0, hi = G - 1;  // largest g with tp[g] <= mu
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh.tp[mid] <= mu) lo = mid;
    else hi = mid - 1;
  }
  row0 = sh.off[lo] + (mu - sh.tp[lo]) * BM;
  const int left = sh.off[lo + 1] - row0;
  rows = left < BM ? left : BM;
  e = sh.pe[lo];
}

// Output of a 64-byte piece of an epilogue warp's 32 tile rows (w: the thread's
// row, 16 words): transposed through the warp's 2 KB of shared memory (16-byte
// piece v of row r at piece v ^ (r / 2 & 3)) so that four lanes write one row's
// 64 bytes.  orow0: the warp's first row at the piece's first column; bytes: row
// bytes left from there (a multiple of 16); rows: valid rows.
__device__ __forceinline__ void emit(unsigned char* stage, const uint32_t* w, unsigned char* orow0, size_t stride,
                                     int bytes, int rows, int lane) {
  __syncwarp();
#pragma unroll
  for (int v = 0; v < 4; ++v)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
  __syncwarp();
  const int v = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    const uint4 d = *reinterpret_cast<const uint4*>(stage + r * 64 + ((v ^ ((r >> 1) & 3)) << 4));
    if (r < rows && v * 16 < bytes) *reinterpret_cast<uint4*>(orow0 + (size_t)r * stride + v * 16) = d;
  }
}

// What a launch multiplies.
struct Product {
  const int32_t* offsets;
  const int32_t* experts;
  const uint8_t* a_scales;
  const uint8_t* b_scales;
  int G, P, E, N, K, n_tiles;
  void* out;             // plain: [P, N]; SwiGLU: the packed h [P, N / 2]
  uint8_t* out_scales;   // SwiGLU: h's scales
};

// GLU: N = I, B rows 0..127 of a tile are gate rows, 128..255 the matching up rows.
template <bool GLU, typename OUT>
__global__ void __launch_bounds__(THREADS, 1)
mx4_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, Product pr) {
  pdl_trigger();
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  unsigned char* stage_a = smem_raw + pad;
  unsigned char* stage_b = stage_a + STAGES * A_BYTES;
  unsigned char* stage_s = stage_a + STAGES * STAGE_BYTES;  // scales: A's two tiles, then B's (row tile, column tile)
  unsigned char* out_stage = stage_s + STAGES * SC_BYTES;
  Shared& sh = *reinterpret_cast<Shared*>(out_stage + OUT_STAGE_BYTES);
  volatile int* abort_flag = &sh.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = pr.G;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) mbar_init(&sh.tfull[a], 1);
    mbar_init(&sh.tempty, 256);
    mbar_init(&sh.done, 1);
    sh.abort_flag = 0;
    sh.armed = 0;
    mbar_init_fence();
    prefetch_map(&map_a);
    prefetch_map(&map_b);
  }
  if (warp == 1) tmem_alloc(&sh.tmem_base, TMEM_COLS);
  pdl_wait();
  for (int g = threadIdx.x; g <= G; g += blockDim.x) sh.off[g] = pr.offsets[g];
  for (int g = threadIdx.x; g < G; g += blockDim.x) sh.pe[g] = pr.experts[g];
  __syncthreads();
  if (warp == 0) {  // exclusive prefix of m-tiles per group, 8 groups per lane
    int cnt[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      int c = 0;
      if (g < G) {
        const int lo = sh.off[g], hi = sh.off[g + 1], e = sh.pe[g];
        if (lo < 0 || hi < lo || hi > pr.P) atomicOr(&g_err, SEMMOE_DEVERR_PAIRS);
        else if (e < 0 || e >= pr.E) atomicOr(&g_err, SEMMOE_DEVERR_EXPERT);
        else c = row_tiles(hi - lo);
      }
      cnt[i] = c;
      sum += c;
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      if (g < G) sh.tp[g] = run;
      run += cnt[i];
    }
    if (lane == 31) {
      // more tiles than any split of P rows has: offsets that step back, and scales that end before them
      const bool bad = incl > pr.P / BM + G;
      if (bad) atomicOr(&g_err, SEMMOE_DEVERR_PAIRS);
      sh.tp[G] = incl;
      sh.total_mtiles = bad ? 0 : incl;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();

  const uint32_t tmem = sh.tmem_base;
  const int n_tiles = pr.n_tiles, total = sh.total_mtiles * n_tiles;
  const int kb_n = (pr.K + BK - 1) / BK, kc = col_tiles(pr.K);
  const int unit0 = blockIdx.x, units = gridDim.x;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      const int b_tiles = row_tiles(pr.N);  // scale row tiles of one matrix (or of its gate half)
      for (int tile = unit0; ok && tile < total; tile += units) {
        const int mt = tile / n_tiles, nt = tile % n_tiles;
        int row0, rows, e;
        decode_mtile(sh, G, mt, row0, rows, e);
        const uint8_t* as = pr.a_scales + (size_t)mt * kc * kTileBytes;
        const int b0 = GLU ? 2 * e * b_tiles + nt : e * b_tiles + 2 * nt;
        const int b1 = GLU ? b0 + b_tiles : b0 + 1;
        const bool two = GLU || 2 * nt + 1 < b_tiles;  // the tile's second 128 columns exist
        const uint8_t* bs0 = pr.b_scales + (size_t)b0 * kc * kTileBytes;
        const uint8_t* bs1 = pr.b_scales + (size_t)b1 * kc * kTileBytes;
        for (int kb = 0; kb < kb_n; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&sh.empty[s], ((it / STAGES) & 1) ^ 1, abort_flag, &g_err)) {
            ok = false;
            break;
          }
          const int ct = kc - 2 * kb < 2 ? kc - 2 * kb : 2;
          const uint32_t sb = (uint32_t)ct * kTileBytes;
          mbar_expect_tx(&sh.full[s], STAGE_BYTES + (two ? 3 : 2) * sb);
          unsigned char* b = stage_b + s * B_BYTES;
          unsigned char* sc = stage_s + s * SC_BYTES;
          tma_load_2d(stage_a + s * A_BYTES, &map_a, &sh.full[s], kb * (BK / 2), row0);
          if (GLU) {
            tma_load_4d(b, &map_b, &sh.full[s], kb * (BK / 2), nt * 128, 0, e);
            tma_load_4d(b + B_BYTES / 2, &map_b, &sh.full[s], kb * (BK / 2), nt * 128, 1, e);
          } else {
            tma_load_3d(b, &map_b, &sh.full[s], kb * (BK / 2), nt * BN, e);
          }
          const size_t o = (size_t)(2 * kb) * kTileBytes;
          bulk_load_1d(sc, as + o, sb, &sh.full[s]);
          bulk_load_1d(sc + 2 * kTileBytes, bs0 + o, sb, &sh.full[s]);
          if (two) bulk_load_1d(sc + 4 * kTileBytes, bs1 + o, sb, &sh.full[s]);
        }
      }
      *reinterpret_cast<volatile int*>(&sh.armed) = (int)it;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0, acc_it = 0;
      bool ok = true;
      for (int tile = unit0; ok && tile < total; tile += units, ++acc_it) {
        // the epilogue of the tile before has left the shared columns (and that of two tiles before has ended)
        if (acc_it > 0 && !mbar_wait(&sh.tempty, (acc_it - 1) & 1, abort_flag, &g_err)) break;
        fence_after();
        const uint32_t d = tmem + (acc_it & 1) * ACC1_COL;
        for (int kb = 0; kb < kb_n; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&sh.full[s], (it / STAGES) & 1, abort_flag, &g_err)) {
            ok = false;
            break;
          }
          // the MMAs of two stages before have read this set of scales
          if (it >= 2 && !mbar_wait(&sh.empty[(it - 2) % STAGES], ((it - 2) / STAGES) & 1, abort_flag, &g_err)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t sa = smem_u32(stage_a + s * A_BYTES), sb = smem_u32(stage_b + s * B_BYTES);
          const uint32_t ss = smem_u32(stage_s + s * SC_BYTES);
          const uint32_t ta = tmem + SC_COL + (it & 1) * SC_COLS, tb = ta + 8;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            copy_scales(ta + 4 * c, scale_desc(ss + c * kTileBytes));
            copy_scales(tb + 8 * c, scale_desc(ss + (2 + c) * kTileBytes));
            copy_scales(tb + 8 * c + 4, scale_desc(ss + (4 + c) * kTileBytes));
          }
          const int left = pr.K - kb * BK;  // columns past K are zeros, their scales undefined
#pragma unroll
          for (int k = 0; k < BK / UK; ++k)
            if (k * UK < left)
              mma_mx4(d, sw128_desc(sa + k * UK / 2), sw128_desc(sb + k * UK / 2),
                      idesc_mx4(BM, BN, (uint32_t)(k & 1) * 2), ta + 4 * (k / 2), tb + 8 * (k / 2), (kb | k) != 0);
          commit(&sh.empty[s]);
        }
        if (!ok) break;
        commit(&sh.tfull[acc_it & 1]);
      }
      commit(&sh.done);
      mbar_drain(&sh.done, 0, &g_err);
    }
  } else {
    // Epilogue group w takes pieces (64 output columns; SwiGLU: 32) 3 - w and 1 - w
    // of the first accumulator, w and 2 + w of the second: the shared columns are
    // in the first pieces taken.
    const int q = warp & 3, w = (warp - 2) >> 2;
    const int r = q * 32 + lane;
    uint32_t acc_it = 0;
    unsigned char* stage = out_stage + (warp - 2) * 2048;
    for (int tile = unit0; tile < total; tile += units, ++acc_it) {
      const int mt = tile / n_tiles, nt = tile % n_tiles;
      int row0, rows, e;
      decode_mtile(sh, G, mt, row0, rows, e);
      const uint32_t a = acc_it & 1;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&sh.tfull[a], (acc_it >> 1) & 1, abort_flag, &g_err);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      fence_after();
      const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + a * ACC1_COL;
      const int wrows = rows - q * 32;  // valid rows of this warp
      uint8_t* hrow = static_cast<uint8_t*>(pr.out) + (size_t)(row0 + (r < rows ? r : 0)) * (pr.N / 2) + nt * 64;
      uint8_t* hs = GLU ? pr.out_scales + ((size_t)mt * n_tiles + nt) * kTileBytes + row_byte(r) : nullptr;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int j = a == 0 ? 3 - w - 2 * i : w + 2 * i;
        uint32_t x0[32], x1[32];  // SwiGLU: gate and up values; else 64 columns
        tmem_ld32(t_row + (GLU ? 32 * j : 64 * j), x0);
        tmem_ld32(t_row + (GLU ? 128 + 32 * j : 64 * j + 32), x1);
        tmem_ld_wait();
        if (i == 0) {
          fence_before();
          mbar_arrive(&sh.tempty);
        }
        if (GLU) {
          // a block past N is outside h: only its scale, 0, is kept
          uint32_t b = 0;
          if (nt * 128 + 32 * j < pr.N) {
            uint32_t m = 0;
#pragma unroll
            for (int i2 = 0; i2 < 32; ++i2) {
              const float h = swiglu(x0[i2], x1[i2]);
              x0[i2] = __float_as_uint(h);
              m = max(m, x0[i2] & 0x7fffffffu);
            }
            b = scale_code(m);
            const float f = inverse_scale(b);
            uint32_t c[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float h[8];
#pragma unroll
              for (int i2 = 0; i2 < 8; ++i2) h[i2] = __uint_as_float(x0[8 * v + i2]) * f;
              c[v] = encode8(h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7]);
            }
            if (r < rows) *reinterpret_cast<uint4*>(hrow + j * 16) = make_uint4(c[0], c[1], c[2], c[3]);
          }
          if (r < rows) hs[j] = (uint8_t)b;
        } else if (wrows > 0) {
          constexpr int PIECE = 64 / (int)sizeof(OUT);  // columns of an emitted piece
          uint32_t y[sizeof(OUT) == 4 ? 1 : 32];
          if (sizeof(OUT) == 2) {
#pragma unroll
            for (int i2 = 0; i2 < 16; ++i2) {
              __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(x0[2 * i2]), __uint_as_float(x0[2 * i2 + 1]));
              y[i2] = *reinterpret_cast<uint32_t*>(&p);
              p = __floats2bfloat162_rn(__uint_as_float(x1[2 * i2]), __uint_as_float(x1[2 * i2 + 1]));
              y[16 + i2] = *reinterpret_cast<uint32_t*>(&p);
            }
          }
#pragma unroll
          for (int c = 0; c < 64; c += PIECE) {
            const int col = nt * BN + 64 * j + c;
            if (col >= pr.N) break;
            const uint32_t* src = sizeof(OUT) == 2 ? y + c / 2 : (c < 32 ? x0 + c : x1 + c - 32);
            emit(stage, src, static_cast<unsigned char*>(pr.out) + ((size_t)(row0 + q * 32) * pr.N + col) * sizeof(OUT),
                 (size_t)pr.N * sizeof(OUT), (pr.N - col) * (int)sizeof(OUT), wrows, lane);
          }
        }
      }
    }
  }

  fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {  // no TMA write may still be landing when the CTA exits
    const int armed = sh.armed;
    for (int j = armed > STAGES ? armed - STAGES : 0; j < armed; ++j)
      mbar_drain(&sh.full[j % STAGES], (j / STAGES) & 1, &g_err);
  }
  if (warp == 1) {
    __syncwarp();
    fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

bool make_map_u8(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed rows [P, K / 2], boxes of 128 rows x 128 bytes.
bool map_rows(CUtensorMap* m, const void* base, int P, int K) {
  const cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)P}, strides[1] = {(cuuint64_t)K / 2};
  const cuuint32_t box[2] = {BK / 2, BM};
  return make_map_u8(m, base, 2, dims, strides, box);
}

template <bool GLU, typename OUT>
cudaError_t launch_one(const void* a, const void* b, const Product& pr, cudaStream_t s) {
  CUtensorMap ma, mb;
  bool ok = map_rows(&ma, a, pr.P, pr.K);
  const cuuint64_t kb = (cuuint64_t)pr.K / 2;
  if (GLU) {
    const cuuint64_t dims[4] = {kb, (cuuint64_t)pr.N, 2, (cuuint64_t)pr.E};
    const cuuint64_t strides[3] = {kb, kb * pr.N, kb * pr.N * 2};
    const cuuint32_t box[4] = {BK / 2, 128, 1, 1};
    ok = ok && make_map_u8(&mb, b, 4, dims, strides, box);
  } else {
    const cuuint64_t dims[3] = {kb, (cuuint64_t)pr.N, (cuuint64_t)pr.E};
    const cuuint64_t strides[2] = {kb, kb * pr.N};
    const cuuint32_t box[3] = {BK / 2, BN, 1};
    ok = ok && make_map_u8(&mb, b, 3, dims, strides, box);
  }
  if (!ok) return cudaErrorInvalidValue;
  auto kern = mx4_gemm_kernel<GLU, OUT>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, (int)kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  const long long tiles = ((long long)pr.P / BM + pr.G) * pr.n_tiles;  // at most
  const int grid = (int)(tiles < sm_count() ? tiles : sm_count());
  e = launch_kernel(kern, dim3(grid), dim3(THREADS), kSmemBytes, s, 1, true, ma, mb, pr);
  count_launches(1);
  return e;
}

}  // namespace

int mx4_gemm_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_mx4_grouped_gemm(const uint8_t* a, const uint8_t* a_scales, const int32_t* offsets,
                                    const int32_t* experts, const uint8_t* b, const uint8_t* b_scales, int P, int E,
                                    int N, int K, void* out, int out_dtype, cudaStream_t s) {
  const Product pr{offsets, experts, a_scales, b_scales, E, P, E, N, K, (N + BN - 1) / BN, out, nullptr};
  return out_dtype == SEMMOE_BF16 ? launch_one<false, __nv_bfloat16>(a, b, pr, s) : launch_one<false, float>(a, b, pr, s);
}

// Workspace: h's codes [P, I / 2], then its scales.
size_t mx4_ffn_ws_bytes(int P, int E, int I) {
  return align_up((size_t)(P > 0 ? P : 1) * (I / 2), 256) + scale_bytes(P, I, E);
}

cudaError_t launch_mx4_grouped_ffn(const uint8_t* x, const uint8_t* x_scales, const int32_t* offsets,
                                   const int32_t* experts, const uint8_t* w13, const uint8_t* w13_scales,
                                   const uint8_t* w2, const uint8_t* w2_scales, int P, int E, int H, int I, void* y,
                                   void* ws, cudaStream_t s) {
  uint8_t* h = static_cast<uint8_t*>(ws);
  uint8_t* hs = h + align_up((size_t)P * (I / 2), 256);
  const Product p1{offsets, experts, x_scales, w13_scales, E, P, E, I, H, (I + 127) / 128, h, hs};
  cudaError_t e = launch_one<true, __nv_bfloat16>(x, w13, p1, s);
  if (e != cudaSuccess) return e;
  return launch_mx4_grouped_gemm(h, hs, offsets, experts, w2, w2_scales, P, E, H, I, y, SEMMOE_BF16, s);
}

}  // namespace semmoe
