// What the grouped products of 4-bit weights multiply, and how their rows are split (w4_gemm.cu, w4_tc.cuh).
#pragma once

#include "common.cuh"
#include "w4.cuh"

namespace semmoe {
namespace w4 {

constexpr int MAX_GROUPS = 256;

// One product.  N: columns of the output (SwiGLU: I, with 2 I weight rows an expert).
struct Product {
  const __nv_bfloat16* x;
  const int32_t* offsets;
  const int32_t* experts;
  Weights w;
  int P, E, N, K, group, n_tiles;
  // launched as the dependent of a kernel of these files, which triggers after its own wait (so that everything before it is
  // complete): tables and weights are read before this kernel's wait, only x is its output
  bool early;
  __nv_bfloat16* out;
  bool stall = false;  // failure-path self-test only: the issuer first waits for what never comes (w4_tc.cuh)
};

struct Groups {
  int total;                 // blocks of rows, of all groups
  int off[MAX_GROUPS + 1];
  int pe[MAX_GROUPS];
  int tp[MAX_GROUPS + 1];    // blocks of rows before each group
};

// One warp: the tables and the exclusive prefix of the groups' blocks of at most `block` rows, 8 groups per lane.
__device__ inline void load_groups(Groups& sh, const Product& pr, int block, int lane, int* err) {
  const int G = pr.E;
  int off[9], ex[8], cnt[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 9; ++i) off[i] = lane * 8 + i <= G ? pr.offsets[lane * 8 + i] : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) ex[i] = lane * 8 + i < G ? pr.experts[lane * 8 + i] : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int g = lane * 8 + i;
    int c = 0;
    if (g < G) {
      const int lo = off[i], hi = off[i + 1], e = ex[i];
      sh.off[g] = lo;
      sh.pe[g] = e;
      if (g == G - 1) sh.off[G] = hi;
      if (lo < 0 || hi < lo || hi > pr.P) atomicOr(err, SEMMOE_DEVERR_PAIRS);
      else if (e < 0 || e >= pr.E) atomicOr(err, SEMMOE_DEVERR_EXPERT);
      else c = (hi - lo + block - 1) / block;
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
    // more blocks than any split of P rows has: offsets that step back
    const bool bad = incl > pr.P / block + G;
    if (bad) atomicOr(err, SEMMOE_DEVERR_PAIRS);
    sh.tp[G] = incl;
    sh.total = bad ? 0 : incl;
  }
}

// A whole warp: unit u of the (group, weight tile, block of rows) list, blocks innermost:
// rows [row0, row0 + rows) with expert e, weight tile nt.  round > 0: a group's blocks are
// of one size, rounded up to that many rows (at most `block`).
struct Unit {
  int row0, rows, e, nt;
};
__device__ __forceinline__ Unit decode_unit(const Groups& sh, int G, int n_tiles, int block, int u, int round = 0) {
  const int at = u / n_tiles, lane = threadIdx.x % 32;
  // the group: the last g with tp[g] <= at, looked for in steps of eight, then among eight
  const int eights = 31 - __clz(__ballot_sync(0xffffffffu, lane * 8 < G && sh.tp[lane * 8 < G ? lane * 8 : 0] <= at));
  const int mine = eights * 8 + (lane & 7);
  const int g = eights * 8 + 31 - __clz(__ballot_sync(0xffffffffu, lane < 8 && mine < G && sh.tp[mine < G ? mine : 0] <= at));
  const int v = u - sh.tp[g] * n_tiles, blocks = sh.tp[g + 1] - sh.tp[g];
  int nt = v, b = 0, rows = sh.off[g + 1] - sh.off[g];
  if (blocks > 1) {
    nt = v / blocks;
    b = v - nt * blocks;
    if (round > 0) block = ((rows + blocks - 1) / blocks + round - 1) / round * round;
  }
  const int left = rows - b * block;
  return Unit{sh.off[g] + b * block, left < block ? left : block, sh.pe[g], nt};
}

__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

}  // namespace w4

// Many rows per expert (w4_tc.cuh): the plain product, and the SwiGLU form.
cudaError_t launch_w4_tc_plain(const w4::Product& pr, cudaStream_t s);
cudaError_t launch_w4_tc_glu(const w4::Product& pr, cudaStream_t s);

}  // namespace semmoe
