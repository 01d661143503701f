// Grouped products of 4-bit microscaled operands on the 5th-generation tensor
// cores (tcgen05.mma kind::mxf4, fp32 accumulation in TMEM; format: mx4.cuh).
// Rows [off[b], off[b+1]) belong to expert pe[b]:
//   plain:  out = a B_e^T                                      (bf16 or fp32)
//   SwiGLU: h = silu(a W1_e^T) * (a W3_e^T), quantised per 32 columns (4 bits)
//
// One persistent CTA per SM walks the (m-tile, n-tile) list of all groups, in M128 x
// N256 tiles.  Warp roles:
//   warp 0      TMA producer: A [128 x 256] and B [256 x 256] values per stage
//               (128-byte rows, 128-byte swizzle) and their scales (512-byte tiles)
//   warp 1      allocates TMEM; copies the stage's scales to TMEM (tcgen05.cp) and
//               issues the MMAs (M128 N128 K64)
//   warps 2..9  epilogue, two groups of four
// A tile has two halves of 128 columns (SwiGLU: gate and up) with an accumulator
// each, and TMEM holds three: the first half of a tile always finds one free, and the
// second half the one that the epilogue of the tile before leaves first; until it
// has, the first halves of up to three stages go ahead.  (Two accumulators of 256 columns
// would leave no TMEM for the scales; sharing some columns left the tensor cores idle
// for a round trip per tile.)
// A stage's scales have TMEM columns of their own, so they are overwritten only after
// the commit of the MMAs that read them.
//
// What bounds it (GB300).  Long groups: each stage's own time.  A stage is 51 KB for
// 16.8 MFLOP, four of them in flight; its MMAs take 0.2 us at the tensor cores' rate, the
// stage 0.45-0.5 us with no output.  32768 rows x 2048 x 1536: 53 us, 3.9 PFLOP/s; 45 us
// with no output stored, 42 with nothing loaded either, so the loads are 3 us of it, the stores 8, and
// more than half of what is left is neither, nor the MMAs' own rate: the scale copies in front of
// a stage's MMAs, those MMAs' reads of shared memory (64 KB a stage) and the commit and wait between
// stages have not been told apart.
// 131072 rows x 768 x 2048 (537 MB of bf16 out): 130 us, 5.4 TB/s.  Pairs of CTAs
// (cta_group::2, M256, 35 KB a stage and CTA, five in flight) took 61 us on the first and
// 178 us on the second when stages were still released in twos and descriptors built for each
// MMA; they were not measured again after this form had both mended.  Three stages of this
// form: 68 and 146 us.
// Few rows per group: the weights' bytes, 64 experts of 2048 x 1408 and 384 rows in 23 us
// (98 MB, 4.3 TB/s, of which some 7 us are the launch, the first loads and the last tiles).
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

constexpr int BM = 128, BN = 256;      // tile
constexpr int HN = BN / 2;             // columns of a half: one MMA's N
constexpr int BK = 256;                // K per stage: one 128-byte swizzle row of packed values
constexpr int UK = 64;                 // K per tcgen05.mma, kind::mxf4
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK / 2;   // 16 KB
constexpr int B_BYTES = BN * BK / 2;   // 32 KB
constexpr int SC_BYTES = 6 * kTileBytes;  // two column tiles of A's rows and of B's two row tiles
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SC_BYTES;  // a multiple of 1024
constexpr int THREADS = 320;
constexpr int ACCS = 3;                // accumulators of HN columns
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SC_COL = ACCS * HN; // the scales' first column
constexpr uint32_t SC_COLS = 24;       // columns of one stage's scales: 2 x (4 for A + 4 for each half of B)
static_assert(SC_COL + STAGES * SC_COLS <= TMEM_COLS, "TMEM columns");
constexpr int MAX_GROUPS = 256;

struct Shared {
  uint64_t full[STAGES], empty[STAGES], tfull[ACCS], tempty[ACCS], done;
  uint32_t tmem_base;
  int abort_flag;
  int armed;        // stage positions that the producer has armed
  int total_mtiles;
  int off[MAX_GROUPS + 1];
  int pe[MAX_GROUPS];
  int tp[MAX_GROUPS + 1];  // row tiles of work before each group
  int skipped[MAX_GROUPS]; // row tiles before each group that are no work (an expert out of range): they have scales
};

constexpr int OUT_STAGE_BYTES = 8 * 2048;  // 2 KB per epilogue warp
constexpr size_t kSmemBytes = 1024 + (size_t)STAGES * STAGE_BYTES + OUT_STAGE_BYTES + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

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

// A row tile: its first row, valid rows, expert, and its place among the scales' row tiles.
struct RowTile {
  int row0, rows, expert, scales;
};
// Tiles come in increasing order, so a role keeps the group `g` it is at: the next tile
// is a few groups on where groups are long, and anywhere after it where they are empty.
__device__ __forceinline__ RowTile decode_mtile(const Shared& sh, int G, int& g, int mt) {
  // the group: the first one with tp[g + 1] > mt
  int steps = 4;
  while (sh.tp[g + 1] <= mt && --steps) ++g;
  if (steps == 0) {
    int hi = G - 1;
    while (g < hi) {
      const int mid = (g + hi) >> 1;
      if (sh.tp[mid + 1] > mt) hi = mid;
      else g = mid + 1;
    }
  }
  const int row0 = sh.off[g] + (mt - sh.tp[g]) * BM, left = sh.off[g + 1] - row0;
  return RowTile{row0, left < BM ? left : BM, sh.pe[g], mt + sh.skipped[g]};
}

// mbar_wait (same bounds), polling a few times before it looks at the clock, whose
// reading takes longer than most of the waits here.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, &g_err);
}
// The same by a whole converged warp, with one answer for all lanes (mbar_wait_warp).
__device__ __forceinline__ bool wait_for_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return mbar_wait_warp(bar, parity, abort_flag, &g_err);
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
  int G, P, E, N, K, n_tiles;
  // early: launched as the dependent of a kernel of this file that triggers after its own wait (so that everything
  // before that kernel is complete): tables and B are read before this kernel's wait, only A is its output
  int early;
  int stall;             // failure-path self-test only: the issuer first waits for what never comes
  void* out;             // plain: [P, N]; SwiGLU: the packed h [P, N / 2]
  uint8_t* out_scales;   // SwiGLU: h's scales
};

// GLU: N = I, a tile's first half are gate rows, its second half the matching up rows.
template <bool GLU, typename OUT>
__global__ void __launch_bounds__(THREADS, 1)
mx4_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_as,
                const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_bs,
                const __grid_constant__ CUtensorMap map_out, Product pr) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  unsigned char* ring = smem_raw + pad;  // stage s: A, B, the scales (A's two tiles, then B's by row tile, column tile)
  unsigned char* out_stage = ring + STAGES * STAGE_BYTES;
  Shared& sh = *reinterpret_cast<Shared*>(out_stage + OUT_STAGE_BYTES);
  volatile int* abort_flag = &sh.abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int G = pr.G;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int a = 0; a < ACCS; ++a) {
      mbar_init(&sh.tfull[a], 1);
      mbar_init(&sh.tempty[a], GLU ? 8 : 4);  // the epilogue warps that read it
    }
    mbar_init(&sh.done, 1);
    sh.abort_flag = 0;
    sh.armed = 0;
    mbar_init_fence();
    prefetch_map(&map_a);
    prefetch_map(&map_as);
    prefetch_map(&map_b);
    prefetch_map(&map_bs);
  }
  if (warp == 1) tmem_alloc(&sh.tmem_base, TMEM_COLS);
  if (!pr.early) pdl_wait();
  pdl_trigger();
  // The tables, and the exclusive prefixes per group of row tiles and of those to skip: 8 groups per lane.  The
  // offsets alone say where a group's scales are, so a group whose expert is out of range keeps its row tiles
  // there while it has none in the list of work.
  if (warp == 0) {
    int off[9], cnt[8], skip[8], sum = 0, sum_skip = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) off[i] = lane * 8 + i <= G ? pr.offsets[lane * 8 + i] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      int c = 0, c_skip = 0;
      if (g < G) {
        const int lo = off[i], hi = off[i + 1], e = pr.experts[g];
        sh.off[g] = lo;
        sh.pe[g] = e;
        if (g == G - 1) sh.off[G] = hi;
        if (lo < 0 || hi < lo || hi > pr.P) atomicOr(&g_err, SEMMOE_DEVERR_PAIRS);
        else if (e < 0 || e >= pr.E) {
          atomicOr(&g_err, SEMMOE_DEVERR_EXPERT);
          c_skip = row_tiles(hi - lo);
        } else c = row_tiles(hi - lo);
      }
      cnt[i] = c, skip[i] = c_skip;
      sum += c, sum_skip += c_skip;
    }
    int incl = sum, incl_skip = sum_skip;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d), v_skip = __shfl_up_sync(0xffffffffu, incl_skip, d);
      if (lane >= d) incl += v, incl_skip += v_skip;
    }
    int run = incl - sum, run_skip = incl_skip - sum_skip;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      if (g < G) sh.tp[g] = run, sh.skipped[g] = run_skip;
      run += cnt[i], run_skip += skip[i];
    }
    if (lane == 31) {
      // more tiles than any split of P rows has: offsets that step back, and scales that end before them
      const bool bad = (long long)incl + incl_skip > pr.P / BM + G;
      if (bad) atomicOr(&g_err, SEMMOE_DEVERR_PAIRS);
      sh.tp[G] = incl;
      sh.total_mtiles = bad ? 0 : incl;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();

  // from shared memory through a shuffle, so that they are known to be the same in a warp
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);
  const int n_tiles = pr.n_tiles, total = __shfl_sync(0xffffffffu, sh.total_mtiles, 0) * n_tiles;
  const int kb_n = (pr.K + BK - 1) / BK, kc = col_tiles(pr.K);
  const int unit0 = blockIdx.x, units = gridDim.x;

  // Producer and issuer: the whole warp runs the loop, so that addresses and descriptors
  // stay in uniform registers, and one elected lane issues.  With loops of one lane alone
  // K = 2048 products took 83 us instead of 54 (32768 rows x 1536).
  if (warp == 0) {
    const int b_tiles = row_tiles(pr.N);  // scale row tiles of one matrix (or of its gate half)
    // Positions: the producer's place in the (tile, k-block) list.
    struct Place {
      int tile, kb, g;
      RowTile rt;
    };
    auto begin = [&](Place& p) {
      if (p.tile < total) p.rt = decode_mtile(sh, G, p.g, p.tile / n_tiles);
    };
    auto next = [&](Place& p) {
      if (++p.kb == kb_n) {
        p.kb = 0;
        p.tile += units;
        begin(p);
      }
    };
    auto load_a = [&](const Place& p, int s) {
      unsigned char* a = ring + (size_t)s * STAGE_BYTES;
      tma_load_2d(a, &map_a, &sh.full[s], p.kb * (BK / 2), p.rt.row0);
      // two column tiles (of the next row tile, or past the end, where K has only one more: not used)
      tma_load_2d(a + A_BYTES + B_BYTES, &map_as, &sh.full[s], 0, p.rt.scales * kc + 2 * p.kb);
    };
    auto load_b = [&](const Place& p, int s) {
      const int nt = p.tile % n_tiles, e = p.rt.expert, x = p.kb * (BK / 2);
      const int b0 = GLU ? 2 * e * b_tiles + nt : e * b_tiles + 2 * nt;  // row tiles of B's two halves
      const int b1 = GLU ? b0 + b_tiles : b0 + 1;
      uint64_t* bar = &sh.full[s];
      unsigned char* b = ring + (size_t)s * STAGE_BYTES + A_BYTES;
      unsigned char* sc = b + B_BYTES;
      mbar_expect_tx(bar, STAGE_BYTES);
      if (GLU) {
        tma_load_4d(b, &map_b, bar, x, nt * HN, 0, e);
        tma_load_4d(b + B_BYTES / 2, &map_b, bar, x, nt * HN, 1, e);
      } else {
        tma_load_3d(b, &map_b, bar, x, nt * BN, e);
      }
      tma_load_2d(sc + 2 * kTileBytes, &map_bs, bar, 0, b0 * kc + 2 * p.kb);
      tma_load_2d(sc + 4 * kTileBytes, &map_bs, bar, 0, b1 * kc + 2 * p.kb);
    };
    Place p{unit0, 0, 0, {}};
    begin(p);
    uint32_t it = 0;
    if (pr.early) {  // the ring's first turn: B while the kernel before ends, then A
      Place q = p;
      for (uint32_t s = 0; s < STAGES && q.tile < total; ++s, next(q)) {
        if (elect_one()) load_b(q, s);
        __syncwarp();
      }
      pdl_wait();
      for (; it < STAGES && p.tile < total; ++it, next(p)) {
        if (elect_one()) load_a(p, it);
        __syncwarp();
      }
    }
    for (; p.tile < total; ++it, next(p)) {
      const int s = it % STAGES;
      if (!wait_for_warp(&sh.empty[s], ((it / STAGES) & 1) ^ 1, abort_flag)) break;
      if (elect_one()) {
        load_b(p, s);
        load_a(p, s);
      }
      __syncwarp();
    }
    if (lane == 0) *reinterpret_cast<volatile int*>(&sh.armed) = (int)it;
  } else if (warp == 1) {
    uint32_t it = 0, half = 0;  // stage position; half tiles begun
    bool ok = !pr.stall || wait_for_warp(&sh.done, 0, abort_flag);
    // descriptors of stage 0; their address field counts 16 bytes
    const uint64_t desc_a = sw128_desc(smem_u32(ring)), desc_b = sw128_desc(smem_u32(ring) + A_BYTES),
                   desc_s = scale_desc(smem_u32(ring) + A_BYTES + B_BYTES);
    auto stage_mma = [&](uint32_t pos, int kb, int h, uint32_t acc) {  // one half's MMAs of a stage
      const uint32_t s = pos % STAGES;
      const uint64_t da = desc_a + s * (STAGE_BYTES / 16), db = desc_b + s * (STAGE_BYTES / 16) + h * (B_BYTES / 32);
      const uint32_t ta = tmem + SC_COL + s * SC_COLS, tb = ta + 8 + 8 * h, d = tmem + acc * HN;
      const int left = pr.K - kb * BK;  // columns past K are zeros, their scales undefined
#pragma unroll
      for (int k = 0; k < BK / UK; ++k)
        if (k * UK < left)
          mma_mx4(d, da + k * (UK / 32), db + k * (UK / 32), idesc_mx4(BM, HN, (uint32_t)(k & 1) * 2), ta + 4 * (k / 2),
                  tb + 4 * (k / 2), (kb | k) != 0);
    };
    for (int tile = unit0; ok && tile < total; tile += units, half += 2) {
      const uint32_t a0 = half % ACCS, a1 = (half + 1) % ACCS;
      // the epilogue has left the accumulator (three halves ago)
      if (half >= ACCS && !wait_for_warp(&sh.tempty[a0], (half / ACCS - 1) & 1, abort_flag)) break;
      int done1 = 0;                // stages whose second half is issued
      bool free1 = half + 1 < ACCS; // the second half's accumulator is free
      for (int kb = 0; kb < kb_n; ++kb) {
        const uint32_t pos = it + kb, s = pos % STAGES;
        if (!wait_for_warp(&sh.full[s], (pos / STAGES) & 1, abort_flag)) {
          ok = false;
          break;
        }
        fence_after();
        if (elect_one()) {
          const uint64_t ds = desc_s + s * (STAGE_BYTES / 16);
          const uint32_t ta = tmem + SC_COL + s * SC_COLS;
#pragma unroll
          for (int c = 0; c < 6; ++c) copy_scales(ta + 4 * c, ds + c * (kTileBytes / 16));
          stage_mma(pos, kb, 0, a0);
          if (kb == kb_n - 1) commit(&sh.tfull[a0]);
        }
        __syncwarp();
        if (!free1) {  // first halves go on while the epilogue still reads it, as far as the ring reaches
          const uint32_t ph = ((half + 1) / ACCS - 1) & 1;
          if (kb + 1 < kb_n && kb + 1 < STAGES - 1) free1 = __all_sync(0xffffffffu, mbar_try_wait(&sh.tempty[a1], ph));
          else free1 = ok = wait_for_warp(&sh.tempty[a1], ph, abort_flag);
          if (!free1) {
            if (!ok) break;
            continue;
          }
          fence_after();
        }
        if (elect_one()) {
          for (int i = done1; i <= kb; ++i) {
            stage_mma(it + i, i, 1, a1);
            commit(&sh.empty[(it + i) % STAGES]);
          }
          if (kb == kb_n - 1) commit(&sh.tfull[a1]);
        }
        done1 = kb + 1;
        __syncwarp();
      }
      it += kb_n;
    }
    if (elect_one()) commit(&sh.done);
    __syncwarp();
    if (lane == 0) mbar_drain(&sh.done, 0, &g_err);
  } else {
    const int q = warp & 3, w = (warp - 2) >> 2;  // TMEM lane quarter, group
    const int r = q * 32 + lane;
    uint32_t half = 0;
    int g = 0;
    unsigned char* stage = out_stage + (warp - 2) * 2048;
    auto wait_acc = [&](uint32_t h) {  // half tile h has been summed
      int ok = 1;
      if (lane == 0) ok = wait_for(&sh.tfull[h % ACCS], (h / ACCS) & 1, abort_flag);
      return __shfl_sync(0xffffffffu, ok, 0);
    };
    auto leave_acc = [&](uint32_t h) {  // this warp has loaded its part
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tempty[h % ACCS]);
    };
    const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16);
    for (int tile = unit0; tile < total; tile += units, half += 2) {
      const int nt = tile % n_tiles;
      const RowTile rt = decode_mtile(sh, G, g, tile / n_tiles);
      const int row0 = rt.row0, rows = rt.rows;
      if (GLU) {  // group w takes blocks w and w + 2 of 32 columns
        if (!wait_acc(half) || !wait_acc(half + 1)) break;
        fence_after();
        const uint32_t tg = t_row + (half % ACCS) * HN, tu = t_row + ((half + 1) % ACCS) * HN;
        uint32_t x[2][32];
        tmem_ld32(tg + 32 * w, x[0]);
        tmem_ld32(tg + 32 * w + 64, x[1]);
        tmem_ld_wait();
        leave_acc(half);
        uint8_t* hrow = static_cast<uint8_t*>(pr.out) + (size_t)(row0 + (r < rows ? r : 0)) * (pr.N / 2) + nt * 64;
        uint8_t* hs = pr.out_scales + ((size_t)rt.scales * n_tiles + nt) * kTileBytes + row_byte(r);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = w + 2 * i;
          uint32_t u[32];
          tmem_ld32(tu + 32 * j, u);
          tmem_ld_wait();
          if (i == 1) leave_acc(half + 1);
          // a block past N is outside h: only its scale, 0, is kept
          uint32_t b = 0;
          if (nt * HN + 32 * j < pr.N) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              x[i][k] = __float_as_uint(swiglu(x[i][k], u[k]));
              m = max(m, x[i][k] & 0x7fffffffu);
            }
            b = scale_code(m);
            const float f = inverse_scale(b);
            uint32_t c[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float h[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) h[k] = __uint_as_float(x[i][8 * v + k]) * f;
              c[v] = encode8(h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7]);
            }
            if (r < rows) *reinterpret_cast<uint4*>(hrow + j * 16) = make_uint4(c[0], c[1], c[2], c[3]);
          }
          if (r < rows) hs[j] = (uint8_t)b;
        }
      } else {  // group w takes half w
        if (!wait_acc(half + w)) break;
        fence_after();
        const uint32_t ty = t_row + ((half + w) % ACCS) * HN;
        const int wrows = rows - q * 32;  // valid rows of this warp
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          uint32_t x0[32], x1[32];
          tmem_ld32(ty + 64 * i, x0);
          tmem_ld32(ty + 64 * i + 32, x1);
          tmem_ld_wait();
          if (i == 1) leave_acc(half + w);
          if (wrows <= 0) continue;
          constexpr int PIECE = 64 / (int)sizeof(OUT);  // columns of an emitted piece
          uint32_t y[sizeof(OUT) == 4 ? 1 : 32];
          if (sizeof(OUT) == 2) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(x0[2 * k]), __uint_as_float(x0[2 * k + 1]));
              y[k] = *reinterpret_cast<uint32_t*>(&p);
              p = __floats2bfloat162_rn(__uint_as_float(x1[2 * k]), __uint_as_float(x1[2 * k + 1]));
              y[16 + k] = *reinterpret_cast<uint32_t*>(&p);
            }
          }
#pragma unroll
          for (int c = 0; c < 64; c += PIECE) {
            const int col = nt * BN + HN * w + 64 * i + c;
            if (col >= pr.N) break;
            const uint32_t* src = sizeof(OUT) == 2 ? y + c / 2 : (c < 32 ? x0 + c : x1 + c - 32);
            if (sizeof(OUT) == 2 && wrows >= 32) {  // whole rows: by TMA
              if (lane == 0) bulk_wait_read<0>();  // the store before has read the buffer
              __syncwarp();
#pragma unroll
              for (int v = 0; v < 4; ++v)
                *reinterpret_cast<uint4*>(stage + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) =
                    make_uint4(src[4 * v], src[4 * v + 1], src[4 * v + 2], src[4 * v + 3]);
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&map_out, stage, col, row0 + q * 32);
                bulk_commit();
              }
              continue;
            }
            if (sizeof(OUT) == 2 && lane == 0) bulk_wait_read<0>();
            emit(stage, src, static_cast<unsigned char*>(pr.out) + ((size_t)(row0 + q * 32) * pr.N + col) * sizeof(OUT),
                 (size_t)pr.N * sizeof(OUT), (pr.N - col) * (int)sizeof(OUT), wrows, lane);
          }
        }
      }
    }
  }

  if (!GLU && warp >= 2 && lane == 0) bulk_wait_all();  // this warp's stores are complete
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

bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, type, rank, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed values, 128-byte rows of a box with 128-byte swizzle.
bool map_codes(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
               const cuuint32_t* box) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rank, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles, 512 bytes each, in boxes of two.
bool map_scales(CUtensorMap* m, const void* base, long long row_tiles, int K) {
  const cuuint64_t dims[2] = {kTileBytes / 4, (cuuint64_t)(row_tiles * col_tiles(K))}, strides[1] = {kTileBytes};
  const cuuint32_t box[2] = {kTileBytes / 4, 2};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, base, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <bool GLU, typename OUT>
cudaError_t launch_one(const void* a, const void* a_scales, const void* b, const void* b_scales, const Product& pr,
                       cudaStream_t s) {
  CUtensorMap ma, mas, mb, mbs;
  const cuuint64_t kb = (cuuint64_t)pr.K / 2;
  bool ok;
  {
    const cuuint64_t dims[2] = {kb, (cuuint64_t)pr.P}, strides[1] = {kb};
    const cuuint32_t box[2] = {BK / 2, BM};
    ok = map_codes(&ma, a, 2, dims, strides, box);
  }
  if (GLU) {
    const cuuint64_t dims[4] = {kb, (cuuint64_t)pr.N, 2, (cuuint64_t)pr.E};
    const cuuint64_t strides[3] = {kb, kb * pr.N, kb * pr.N * 2};
    const cuuint32_t box[4] = {BK / 2, HN, 1, 1};
    ok = ok && map_codes(&mb, b, 4, dims, strides, box);
  } else {
    const cuuint64_t dims[3] = {kb, (cuuint64_t)pr.N, (cuuint64_t)pr.E};
    const cuuint64_t strides[2] = {kb, kb * pr.N};
    const cuuint32_t box[3] = {BK / 2, BN, 1};
    ok = ok && map_codes(&mb, b, 3, dims, strides, box);
  }
  ok = ok && map_scales(&mas, a_scales, (long long)pr.P / BM + pr.G, pr.K) &&
       map_scales(&mbs, b_scales, (long long)(GLU ? 2 : 1) * pr.E * row_tiles(pr.N), pr.K);
  CUtensorMap mo = {};
  if (!GLU && sizeof(OUT) == 2) {  // boxes of 32 rows x 32 columns, 64-byte swizzle
    const cuuint64_t dims[2] = {(cuuint64_t)pr.N, (cuuint64_t)pr.P}, strides[1] = {(cuuint64_t)pr.N * 2};
    const cuuint32_t box[2] = {32, 32};
    ok = ok && make_map(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pr.out, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  if (!ok) return cudaErrorInvalidValue;
  auto kern = mx4_gemm_kernel<GLU, OUT>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = ensure_smem_limit(kern, (int)kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  const long long tiles = ((long long)pr.P / BM + pr.G) * pr.n_tiles;  // of any grouping, at most
  const int grid = (int)(tiles < sm_count() ? tiles : sm_count());
  e = launch_kernel(kern, dim3(grid), dim3(THREADS), kSmemBytes, s, 1, true, ma, mas, mb, mbs, mo, pr);
  count_launches(1);
  return e;
}

}  // namespace

int mx4_gemm_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_mx4_grouped_gemm(const uint8_t* a, const uint8_t* a_scales, const int32_t* offsets,
                                    const int32_t* experts, const uint8_t* b, const uint8_t* b_scales, int P, int E,
                                    int N, int K, void* out, int out_dtype, cudaStream_t s, bool early, bool stall) {
  const Product pr{offsets, experts, E, P, E, N, K, (N + BN - 1) / BN, early, stall, out, nullptr};
  return out_dtype == SEMMOE_BF16 ? launch_one<false, __nv_bfloat16>(a, a_scales, b, b_scales, pr, s)
                                  : launch_one<false, float>(a, a_scales, b, b_scales, pr, s);
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
  const Product p1{offsets, experts, E, P, E, I, H, (I + 127) / 128, 0, 0, h, hs};
  cudaError_t e = launch_one<true, __nv_bfloat16>(x, x_scales, w13, w13_scales, p1, s);
  if (e != cudaSuccess) return e;
  return launch_mx4_grouped_gemm(h, hs, offsets, experts, w2, w2_scales, P, E, H, I, y, SEMMOE_BF16, s, true);
}

}  // namespace semmoe
