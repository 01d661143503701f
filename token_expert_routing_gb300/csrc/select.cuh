// Expert choice by score (semmoe_route_select) of one token by one warp, lane l
// holding the experts l + 32 i.
//   s_e = sigmoid(l_e), or the softmax of l;  c_e = s_e + bias_e  (fp32)
// and experts are taken by c -- by l without a bias, which s never reorders and
// which has no ties that rounding s would make.  Experts whose c is -inf are off.
// Groups: `per_group` consecutive experts; L lanes share a group (L = 32 over
// the next power of two of G, one lane per group and several groups per lane
// past 32), each finds the two largest of its share of c and they are merged.
// A group's rank is the number of groups with a larger score, or an equal one
// and a lower index; ranks below topk_group stay.
// Picks: each lane sorts the keys of its experts (order-preserving, 0: not to be
// taken; equal keys by index), then k_t rounds take the largest head of any lane; only
// when several lanes hold it does a second reduction find the lowest index.
// Weights: s_j, or s_j over the sum of the picks'; where that sum is close to
// underflow, exp(log s_j - max log s) over its sum (log sigmoid(l) = min(l, 0) -
// log1p(exp(-|l|))), so that picks whose scores all underflow still share one.
// Bound by instructions where the GPU is full of tokens (16384 tokens, 128 experts, 8
// picks: 69% of the issue slots, 690 instructions a token, 16 us beside 20 us of the
// product) and by the latency of its steps where it is not (one token, 256 experts in 8
// groups: about 5 us of the call's 13 on the device).
#pragma once

#include <float.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace semmoe {

// Words of scratch per warp: logits, choice scores, group scores, picks.
__host__ __device__ constexpr int select_scratch(int E, int G, int k_max) { return 2 * E + G + k_max; }

// Within 3 ulp: the quotient of numbers at most 1 apart in magnitude needs no slow path (0 for l < -88).
__device__ __forceinline__ float sigmoid_f32(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }
__device__ __forceinline__ float log_sigmoid_f32(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }

// (a, b) = the two largest of (a, b) and (c, d), each pair in descending order.
__device__ __forceinline__ void merge_top2(float& a, float& b, float c, float d) {
  const float lo = fminf(a, c);
  a = fmaxf(a, c);
  b = fmaxf(lo, fmaxf(b, d));
}

// The lane's biases, loaded once per warp (0 without a bias); bits: what is not finite.
template <int NPER>
__device__ __forceinline__ int load_bias(const Select& sel, int E, float (&bias)[NPER]) {
  int bits = 0;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = (threadIdx.x & 31) + 32 * i;
    bias[i] = sel.bias != nullptr && e < E ? __ldg(sel.bias + e) : 0.0f;
    if (!(bias[i] < INFINITY)) {  // NaN or +inf: the expert is off
      bits = SEMMOE_DEVERR_NONFINITE;
      bias[i] = -INFINITY;
    }
  }
  return bits;
}

// v: the token's logits, -inf where not finite and past E.  idx / w: its k_max output
// slots; picked(e) is called once for each expert taken.  Every lane of the warp calls.
template <int NPER, typename F>
__device__ __forceinline__ void warp_choose(const float (&v)[NPER], const float (&bias)[NPER], int E, int kt, int k_max, const Select& sel,
                                           float* scratch, int32_t* __restrict__ idx, float* __restrict__ w,
                                           F&& picked) {
  const int lane = threadIdx.x & 31;
  const int G = sel.n_group;
  const bool soft = sel.score == SEMMOE_SCORE_SOFTMAX, grouped = sel.topk_group < G;
  float* lg = scratch;
  float* ch = lg + E;
  float* gs = ch + E;
  int* pick = reinterpret_cast<int*>(gs + G);
  float m = -INFINITY, z = 1.0f;  // the softmax's maximum and sum over all experts
  if (soft) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.0f;  // no finite logit (flagged): nothing is taken
    z = 0.0f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) z += expf(v[i] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  float c[NPER];  // what experts are taken by
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    if (lane + 32 * i < E) lg[lane + 32 * i] = v[i];
    c[i] = v[i];
  }
  if (sel.bias != nullptr || grouped) {
    float s[NPER];
    if (soft) {
      const float r = 1.0f / z;
#pragma unroll
      for (int i = 0; i < NPER; ++i) s[i] = expf(v[i] - m) * r;
    } else {
#pragma unroll
      for (int i = 0; i < NPER; ++i) s[i] = sigmoid_f32(v[i]);
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const float b = v[i] == -INFINITY ? -INFINITY : s[i] + bias[i];
      if (lane + 32 * i < E && grouped) ch[lane + 32 * i] = b;
      if (sel.bias != nullptr) c[i] = b;
    }
  }
  if (grouped) {
    const int per_group = E / G;
    // an expert's group without an integer division: (e + 1/2) / per_group is at least 1/512 from a whole number
    const float per_group_inv = 1.0f / (float)per_group;
    auto group_of = [&](int e) { return __float2int_rz(((float)e + 0.5f) * per_group_inv); };
    const int lsh = G <= 32 ? __clz(G - 1) - 27 : 0, L = 1 << lsh;  // lanes per group, a power of two
    __syncwarp();
    for (int g0 = 0; g0 < G; g0 += 32 >> lsh) {
      const int g = g0 + (lane >> lsh);
      float a = -INFINITY, b = -INFINITY;
      if (g < G)
        for (int i = lane & (L - 1); i < per_group; i += L) merge_top2(a, b, ch[g * per_group + i], -INFINITY);
      for (int o = L / 2; o > 0; o >>= 1) {
        const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
        merge_top2(a, b, a2, b2);
      }
      // a sum past the lowest float (biases of the type's lowest value) still beats a group that is off
      if (g < G && (lane & (L - 1)) == 0) gs[g] = sel.group_top == 2 && b > -INFINITY ? fmaxf(a + b, -FLT_MAX) : a;
    }
    __syncwarp();
    if (G <= 32) {  // lane g ranks group g
      const float mine = lane < G ? gs[lane] : 0.0f;
      int rank = 0;
      for (int o = 0; o < G; ++o) {
        const float other = __shfl_sync(0xffffffffu, mine, o);
        rank += other > mine || (other == mine && o < lane);
      }
      const unsigned keep = __ballot_sync(0xffffffffu, lane < G && rank < sel.topk_group);
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((keep >> group_of(e)) & 1u)) c[i] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        if (e < E) {
          const int g = group_of(e);
          const float mine = gs[g];
          int rank = 0;
          for (int o = 0; o < G; ++o) rank += gs[o] > mine || (gs[o] == mine && o < g);
          if (rank >= sel.topk_group) c[i] = -INFINITY;
        }
      }
    }
  }
  uint32_t key[NPER];  // descending once sorted
  int at[NPER];        // the experts' indices
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const uint32_t b = __float_as_uint(__fadd_rn(c[i], 0.0f));  // -0.0 -> +0.0
    key[i] = c[i] == -INFINITY ? 0u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    at[i] = lane + 32 * i;
  }
#pragma unroll
  for (int i = 1; i < NPER; ++i)
#pragma unroll
    for (int j = i; j > 0; --j) {  // strictly larger keys move ahead: equal ones stay in index order
      const bool up = key[j] > key[j - 1];
      const uint32_t hi = up ? key[j] : key[j - 1], lo = up ? key[j - 1] : key[j];
      const int ih = up ? at[j] : at[j - 1], il = up ? at[j - 1] : at[j];
      key[j - 1] = hi, key[j] = lo;
      at[j - 1] = ih, at[j] = il;
    }
  int taken = 0;
  for (; taken < kt; ++taken) {
    const uint32_t mk = __reduce_max_sync(0xffffffffu, key[0]);
    if (mk == 0u) break;  // none left to take
    bool won = key[0] == mk;
    const unsigned holders = __ballot_sync(0xffffffffu, won);
    if (holders & (holders - 1)) won = at[0] == (int)__reduce_min_sync(0xffffffffu, won ? (unsigned)at[0] : 0xffffffffu);
    if (won) pick[taken] = at[0];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {  // the next head
      key[i] = won ? (i + 1 < NPER ? key[i + 1] : 0u) : key[i];
      at[i] = won && i + 1 < NPER ? at[i + 1] : at[i];
    }
  }
  __syncwarp();
  // the pick of this lane, and the sum of the first 32 (the rest are added below)
  float mine = 0.0f, den = soft ? z : 1.0f, top = 0.0f;
  bool logs = false;
  if (lane < taken) {
    const float l = lg[pick[lane]];
    mine = soft ? expf(l - m) : sigmoid_f32(l);
  }
  if (sel.renorm) {
    den = mine;
    for (int j = lane + 32; j < taken; j += 32) {
      const float l = lg[pick[j]];
      den += soft ? expf(l - m) : sigmoid_f32(l);
    }
    if (taken <= 8) {
      den += __shfl_xor_sync(0xffffffffu, den, 4);
      den += __shfl_xor_sync(0xffffffffu, den, 2);
      den += __shfl_xor_sync(0xffffffffu, den, 1);
      den = __shfl_sync(0xffffffffu, den, 0);
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    logs = !(den > 1e-30f);
    if (logs) {
      top = -INFINITY;
      for (int j = lane; j < taken; j += 32) {
        const float l = lg[pick[j]];
        top = fmaxf(top, soft ? l : log_sigmoid_f32(l));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      den = 0.0f;
      for (int j = lane; j < taken; j += 32) {
        const float l = lg[pick[j]];
        den += expf((soft ? l : log_sigmoid_f32(l)) - top);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
  }
  for (int j = lane; j < k_max; j += 32) {
    int e = -1;
    float g = 0.0f;
    if (j < taken) {
      e = pick[j];
      g = mine;
      if (logs || j >= 32) {
        const float l = lg[e];
        g = logs ? expf((soft ? l : log_sigmoid_f32(l)) - top) : soft ? expf(l - m) : sigmoid_f32(l);
      }
      g = g / den * sel.scale;  // a single pick's renormalised weight is exactly the scale
      picked(e);
    }
    idx[j] = e;
    w[j] = g;
  }
  __syncwarp();  // the scratch may be written again
}

}  // namespace semmoe
