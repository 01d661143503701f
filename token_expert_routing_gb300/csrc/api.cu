// C ABI of the semmoe library: host-side argument validation, error
// reporting, and the launch of each step's kernels.  See include/semmoe.h.
#include <stdarg.h>
#include <stdio.h>

#include <atomic>
#include <string>

#include "common.cuh"
#include "internal.h"
#include "w4.cuh"

namespace {

thread_local std::string g_msg;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_msg = buf;
  return code;
}

int cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return SEMMOE_OK;
  return fail(SEMMOE_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Whether na bytes from a on and nb from b on share any.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && na > 0 && nb > 0 && (x < y ? y - x < na : x - y < nb);
}
bool valid_dtype(int d) { return d == SEMMOE_F32 || d == SEMMOE_BF16; }
// Router weights may also come as the split of an fp32 weight, for bf16
// activations with 16-byte rows (the tensor-core router).
bool valid_router_dtype(int w, int x, int H) {
  return valid_dtype(w) || (w == SEMMOE_F32_SPLIT && x == SEMMOE_BF16 && H % 8 == 0);
}
size_t elem_size(int d) { return d == SEMMOE_BF16 ? 2 : 4; }

// The kernels are built for sm_103a only.
int require_sm103(const char* fn) {
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return cuda_status(e, fn);
  if (major != 10 || minor != 3)
    return fail(SEMMOE_ERR_UNSUPPORTED, "%s: built for sm_103a, device is sm_%d%d", fn, major, minor);
  return SEMMOE_OK;
}

#define REQUIRE(cond, ...)                                              \
  do {                                                                  \
    if (!(cond)) return fail(SEMMOE_ERR_INVALID_ARG, __VA_ARGS__);      \
  } while (0)

#define CHECK_DEVICE(fn)                   \
  do {                                     \
    int _rc = require_sm103(fn);           \
    if (_rc != SEMMOE_OK) return _rc;      \
  } while (0)

std::atomic<unsigned long long> g_launches{0};

}  // namespace

void semmoe::count_launches(int n) { g_launches.fetch_add((unsigned long long)n, std::memory_order_relaxed); }

using namespace semmoe;

extern "C" {

const char* semmoe_last_error(void) { return g_msg.c_str(); }

int semmoe_version(void) { return 100; }

unsigned long long semmoe_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

int semmoe_check_errors(void* stream, int* bits) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e, "semmoe_check_errors");
  int b = 0;
  if (route_take_errors(s, &b) || permute_take_errors(s, &b) || ffn_take_errors(s, &b) ||
      combine_take_errors(s, &b) || schedule_take_errors(s, &b) || selftest_take_errors(s, &b) ||
      mx4_take_errors(s, &b) || mx4_gemm_take_errors(s, &b) || norm_take_errors(s, &b) ||
      w4_gemm_take_errors(s, &b) || w4_tc_plain_take_errors(s, &b) ||
      w4_tc_glu_take_errors(s, &b))
    return cuda_status(cudaGetLastError(), "semmoe_check_errors: reading the device error word");
  if (bits != nullptr) *bits = b;
  if (b & SEMMOE_DEVERR_TIMEOUT) return fail(SEMMOE_ERR_DEVICE_TIMEOUT, "a bounded in-kernel wait ran out (bits 0x%x)", b);
  if (b) return fail(SEMMOE_ERR_DEVICE_CHECK, "kernels saw invalid data (device error bits 0x%x)", b);
  return SEMMOE_OK;
}

size_t semmoe_route_workspace_size(int T, int H, int E, int x_dtype, int w_dtype) {
  if (T < 0 || H < 1 || E < 1 || !valid_dtype(x_dtype) || !valid_router_dtype(w_dtype, x_dtype, H)) return 0;
  const size_t b = route_ws_bytes(T, H, E, x_dtype, w_dtype);
  return b > 0 ? b : 256;
}

size_t semmoe_pair_counts_size(int T, int E) {
  if (T < 0 || E < 1) return 0;
  return pair_counts_bytes(T, E);
}

int semmoe_pair_counts_stride(int T) { return T < 0 ? 0 : pair_counts_stride(T); }

int semmoe_route(const void* x, int x_dtype, const void* w_router, int w_dtype, const float* logits_in,
                 float* logits_out, const int32_t* k_per_token, int k_uniform, int T, int H, int E, int k_max,
                 int32_t* topk_idx, float* topk_w, int32_t* pair_counts, void* ws, size_t ws_bytes, void* stream) {
  REQUIRE(T >= 0, "semmoe_route: T = %d < 0", T);
  REQUIRE(E >= 1 && E <= 256, "semmoe_route: E = %d outside [1, 256]", E);
  REQUIRE(k_max >= 1 && k_max <= E, "semmoe_route: k_max = %d outside [1, E = %d]", k_max, E);
  REQUIRE((long long)T * (k_max > E ? k_max : E) < (1LL << 31), "semmoe_route: T * E too large");
  REQUIRE(k_per_token != nullptr || (k_uniform >= 1 && k_uniform <= k_max),
          "semmoe_route: k_uniform = %d outside [1, k_max = %d]", k_uniform, k_max);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(topk_idx != nullptr && topk_w != nullptr, "semmoe_route: null output pointer");
  if (logits_in == nullptr) {
    REQUIRE(x != nullptr && w_router != nullptr, "semmoe_route: null x or w_router without logits_in");
    REQUIRE(valid_dtype(x_dtype) && valid_router_dtype(w_dtype, x_dtype, H), "semmoe_route: bad dtype (%d, %d)",
            x_dtype, w_dtype);
    REQUIRE(H >= 1, "semmoe_route: H = %d < 1", H);
    REQUIRE(aligned(x, 16) && aligned(w_router, 16), "semmoe_route: x and w_router must be 16-byte aligned");
    const size_t need = route_ws_bytes(T, H, E, x_dtype, w_dtype);
    REQUIRE(need == 0 || (ws != nullptr && aligned(ws, 256) && ws_bytes >= need),
            "semmoe_route: workspace null, not 256-byte aligned or below %zu bytes", need);
  } else {
    REQUIRE(aligned(logits_in, 4), "semmoe_route: misaligned logits_in");
  }
  REQUIRE(aligned(topk_idx, 4) && aligned(topk_w, 4) && aligned(logits_out, 4) && aligned(k_per_token, 4) &&
              aligned(pair_counts, 16),
          "semmoe_route: misaligned output or k_per_token");
  CHECK_DEVICE("semmoe_route");
  return cuda_status(launch_route(x, x_dtype, w_router, w_dtype, logits_in, logits_out, k_per_token, k_uniform, T,
                                  H, E, k_max, topk_idx, topk_w, pair_counts, ws, static_cast<cudaStream_t>(stream)),
                     "semmoe_route");
}

size_t semmoe_route_split_size(int H, int E) {
  if (H < 8 || H % 8 != 0 || E < 1 || E > 256) return 0;
  return route_split_size(H, E);
}

int semmoe_route_split_weight(const float* w, int H, int E, void* split, void* stream) {
  REQUIRE(H >= 8 && H % 8 == 0, "semmoe_route_split_weight: H = %d must be a positive multiple of 8", H);
  REQUIRE(E >= 1 && E <= 256, "semmoe_route_split_weight: E = %d outside [1, 256]", E);
  REQUIRE(w != nullptr && split != nullptr, "semmoe_route_split_weight: null pointer");
  REQUIRE(aligned(w, 4) && aligned(split, 256), "semmoe_route_split_weight: misaligned pointer");
  CHECK_DEVICE("semmoe_route_split_weight");
  return cuda_status(launch_route_split(w, H, E, split, static_cast<cudaStream_t>(stream)),
                     "semmoe_route_split_weight");
}

size_t semmoe_route_hier_workspace_size(int T, int H, int Ep, int x_dtype, int w_dtype) {
  if (T < 0 || H < 1 || Ep < 1 || !valid_dtype(x_dtype) || !valid_router_dtype(w_dtype, x_dtype, H)) return 0;
  const size_t b = route_hier_ws_bytes(T, H, Ep, x_dtype, w_dtype);
  return b > 0 ? b : 256;
}

int semmoe_route_hier(const void* x, int x_dtype, const void* w_parent, int w_dtype, const float* logits_in,
                      float* logits_out, const float* sub_logw, int N, const int32_t* k_per_token, int k_uniform,
                      int T, int H, int Ep, int k_max, int32_t* topk_idx, float* topk_w, int32_t* pair_counts,
                      void* ws, size_t ws_bytes, void* stream) {
  REQUIRE(T >= 0, "semmoe_route_hier: T = %d < 0", T);
  REQUIRE(N >= 1 && Ep >= 1 && (long long)Ep * N <= 256, "semmoe_route_hier: Ep * N = %lld outside [1, 256]",
          (long long)Ep * N);
  const int E = Ep * N;
  REQUIRE(k_max >= 1 && k_max <= E, "semmoe_route_hier: k_max = %d outside [1, Ep*N = %d]", k_max, E);
  REQUIRE((long long)T * E < (1LL << 31), "semmoe_route_hier: T * Ep * N too large");
  REQUIRE(k_per_token != nullptr || (k_uniform >= 1 && k_uniform <= k_max),
          "semmoe_route_hier: k_uniform = %d outside [1, k_max = %d]", k_uniform, k_max);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(topk_idx != nullptr && topk_w != nullptr && sub_logw != nullptr, "semmoe_route_hier: null pointer");
  if (logits_in == nullptr) {
    REQUIRE(x != nullptr && w_parent != nullptr, "semmoe_route_hier: null x or w_parent without logits_in");
    REQUIRE(valid_dtype(x_dtype) && valid_router_dtype(w_dtype, x_dtype, H), "semmoe_route_hier: bad dtype (%d, %d)",
            x_dtype, w_dtype);
    REQUIRE(H >= 1, "semmoe_route_hier: H = %d < 1", H);
    REQUIRE(aligned(x, 16) && aligned(w_parent, 16), "semmoe_route_hier: x and w_parent must be 16-byte aligned");
    const size_t need = route_hier_ws_bytes(T, H, Ep, x_dtype, w_dtype);
    REQUIRE(need == 0 || (ws != nullptr && aligned(ws, 256) && ws_bytes >= need),
            "semmoe_route_hier: workspace null, not 256-byte aligned or below %zu bytes", need);
  } else {
    REQUIRE(aligned(logits_in, 4), "semmoe_route_hier: misaligned logits_in");
  }
  REQUIRE(aligned(topk_idx, 4) && aligned(topk_w, 4) && aligned(logits_out, 4) && aligned(k_per_token, 4) &&
              aligned(sub_logw, 4) && aligned(pair_counts, 16),
          "semmoe_route_hier: misaligned pointer");
  CHECK_DEVICE("semmoe_route_hier");
  return cuda_status(launch_route_hier(x, x_dtype, w_parent, w_dtype, logits_in, logits_out, sub_logw, N,
                                       k_per_token, k_uniform, T, H, Ep, k_max, topk_idx, topk_w, pair_counts, ws,
                                       static_cast<cudaStream_t>(stream)),
                     "semmoe_route_hier");
}

// Rows of one call: a kernel's next row after the last, and the rows rounded up to a tile, still fit 32 bits.
static constexpr long long kMaxRows = (1LL << 31) - (1 << 16);

size_t semmoe_route_select_workspace_size(int T, int H, int E, int x_dtype, int w_dtype) {
  if (T < 0 || H < 1 || E < 1 || E > 256 || !valid_dtype(x_dtype) || !valid_router_dtype(w_dtype, x_dtype, H)) return 0;
  const size_t b = route_select_ws_bytes(T, H, E, x_dtype, w_dtype);
  return b > 0 ? b : 256;
}

int semmoe_route_select(const void* x, int x_dtype, const void* w_router, int w_dtype, const float* logits_in,
                        float* logits_out, int score, const float* bias, int n_group, int topk_group, int group_top,
                        int renorm, float scale, const int32_t* k_per_token, int k_uniform, int T, int H, int E,
                        int k_max, int32_t* topk_idx, float* topk_w, int32_t* pair_counts, void* ws, size_t ws_bytes,
                        void* stream) {
  const char* fn = "semmoe_route_select";
  REQUIRE(T >= 0, "%s: T = %d < 0", fn, T);
  REQUIRE(E >= 1 && E <= 256, "%s: E = %d outside [1, 256]", fn, E);
  REQUIRE(k_max >= 1 && k_max <= E, "%s: k_max = %d outside [1, E = %d]", fn, k_max, E);
  REQUIRE((long long)T * E < (1LL << 31) && T <= kMaxRows, "%s: T * E too large", fn);
  REQUIRE(score == SEMMOE_SCORE_SIGMOID || score == SEMMOE_SCORE_SOFTMAX, "%s: bad score %d", fn, score);
  REQUIRE(n_group >= 1 && E % n_group == 0, "%s: n_group = %d does not divide E = %d", fn, n_group, E);
  REQUIRE(topk_group >= 1 && topk_group <= n_group, "%s: topk_group = %d outside [1, n_group = %d]", fn, topk_group,
          n_group);
  REQUIRE(group_top == 1 || group_top == 2, "%s: group_top = %d is neither 1 nor 2", fn, group_top);
  REQUIRE(k_max <= (long long)topk_group * (E / n_group), "%s: k_max = %d exceeds the %d experts of %d groups", fn,
          k_max, topk_group * (E / n_group), topk_group);
  REQUIRE(scale == scale && scale - scale == 0.0f, "%s: scale is not finite", fn);
  REQUIRE(k_per_token != nullptr || (k_uniform >= 1 && k_uniform <= k_max), "%s: k_uniform = %d outside [1, k_max = %d]",
          fn, k_uniform, k_max);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(topk_idx != nullptr && topk_w != nullptr, "%s: null output pointer", fn);
  if (logits_in == nullptr) {
    REQUIRE(x != nullptr && w_router != nullptr, "%s: null x or w_router without logits_in", fn);
    REQUIRE(valid_dtype(x_dtype) && valid_router_dtype(w_dtype, x_dtype, H), "%s: bad dtype (%d, %d)", fn, x_dtype,
            w_dtype);
    REQUIRE(H >= 1, "%s: H = %d < 1", fn, H);
    REQUIRE(aligned(x, 16) && aligned(w_router, 16), "%s: x and w_router must be 16-byte aligned", fn);
    const size_t need = route_select_ws_bytes(T, H, E, x_dtype, w_dtype);
    REQUIRE(need == 0 || (ws != nullptr && aligned(ws, 256) && ws_bytes >= need),
            "%s: workspace null, not 256-byte aligned or below %zu bytes", fn, need);
  } else {
    REQUIRE(aligned(logits_in, 4), "%s: misaligned logits_in", fn);
  }
  REQUIRE(aligned(topk_idx, 4) && aligned(topk_w, 4) && aligned(logits_out, 4) && aligned(k_per_token, 4) &&
              aligned(bias, 4) && aligned(pair_counts, 16),
          "%s: misaligned pointer", fn);
  CHECK_DEVICE(fn);
  return cuda_status(launch_route_select(x, x_dtype, w_router, w_dtype, logits_in, logits_out,
                                         Select{score, bias, n_group, topk_group, group_top, renorm != 0, scale},
                                         k_per_token, k_uniform, T, H, E, k_max, topk_idx, topk_w, pair_counts, ws,
                                         static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_affinity_lookup(const int32_t* token_ids, const int32_t* lut, int V, int R, int T, int32_t* pred_rank,
                           void* stream) {
  REQUIRE(T >= 0 && V >= 1 && R >= 1, "semmoe_affinity_lookup: bad sizes T=%d V=%d R=%d", T, V, R);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(token_ids && lut && pred_rank, "semmoe_affinity_lookup: null pointer");
  REQUIRE(aligned(token_ids, 4) && aligned(lut, 4) && aligned(pred_rank, 4), "semmoe_affinity_lookup: misaligned");
  CHECK_DEVICE("semmoe_affinity_lookup");
  return cuda_status(launch_affinity_lookup(token_ids, lut, V, R, T, pred_rank, static_cast<cudaStream_t>(stream)),
                     "semmoe_affinity_lookup");
}

int semmoe_remote_count(const int32_t* topk_idx, const int32_t* pred_rank, const int32_t* expert_rank, int T,
                        int k_max, int E, int R, int32_t* counts, int32_t* remote, void* stream) {
  REQUIRE(T >= 0 && k_max >= 1 && E >= 1 && E <= 256, "semmoe_remote_count: bad sizes T=%d k_max=%d E=%d", T, k_max,
          E);
  REQUIRE(R >= 1 && R <= 64, "semmoe_remote_count: R = %d outside [1, 64]", R);
  REQUIRE(counts && remote && expert_rank, "semmoe_remote_count: null pointer");
  REQUIRE(T == 0 || (topk_idx && pred_rank), "semmoe_remote_count: null topk_idx or pred_rank");
  REQUIRE((long long)T * k_max < (1LL << 31), "semmoe_remote_count: T * k_max too large");
  CHECK_DEVICE("semmoe_remote_count");
  return cuda_status(launch_remote_count(topk_idx, pred_rank, expert_rank, T, k_max, E, R, counts, remote,
                                         static_cast<cudaStream_t>(stream)),
                     "semmoe_remote_count");
}

size_t semmoe_permute_workspace_size(int T, int k_max, int E) {
  if (T < 0 || k_max < 1 || E < 1) return 0;
  return permute_ws_bytes(T, k_max, E);
}

int semmoe_permute(const int32_t* topk_idx, const int32_t* expert_rank, const void* x, int dtype, int T, int H,
                   int E, int R, int k_max, int P, int32_t* expert_offsets, int32_t* rank_offsets,
                   int32_t* phys_to_expert, int32_t* expert_counts, int32_t* sorted_to_pair,
                   int32_t* pair_to_sorted, void* x_perm, const int32_t* pair_counts, void* ws, size_t ws_bytes,
                   void* stream) {
  REQUIRE(T >= 0, "semmoe_permute: T = %d < 0", T);
  REQUIRE(E >= 1 && E <= 256, "semmoe_permute: E = %d outside [1, 256]", E);
  REQUIRE(R >= 1 && R <= E, "semmoe_permute: R = %d outside [1, E]", R);
  REQUIRE(k_max >= 1 && k_max <= E, "semmoe_permute: k_max = %d outside [1, E]", k_max);
  REQUIRE((long long)T * k_max < (1LL << 31), "semmoe_permute: T * k_max too large");
  REQUIRE(P >= 0 && (long long)P <= (long long)T * k_max, "semmoe_permute: P = %d outside [0, T*k_max]", P);
  REQUIRE(expert_rank && expert_offsets && rank_offsets && phys_to_expert && expert_counts,
          "semmoe_permute: null table pointer");
  REQUIRE(T == 0 || (topk_idx && pair_to_sorted), "semmoe_permute: null topk_idx or pair_to_sorted");
  REQUIRE(P == 0 || sorted_to_pair, "semmoe_permute: null sorted_to_pair");
  REQUIRE((x == nullptr) == (x_perm == nullptr), "semmoe_permute: x and x_perm must both be set or both NULL");
  if (x != nullptr) {
    REQUIRE(valid_dtype(dtype), "semmoe_permute: bad dtype %d", dtype);
    REQUIRE(H >= 1 && (H * elem_size(dtype)) % 16 == 0, "semmoe_permute: H * elem size must be a multiple of 16");
    REQUIRE(aligned(x, 16) && aligned(x_perm, 16), "semmoe_permute: x / x_perm not 16-byte aligned");
  }
  REQUIRE(ws != nullptr && aligned(ws, 256), "semmoe_permute: workspace null or not 256-byte aligned");
  REQUIRE(ws_bytes >= permute_ws_bytes(T, k_max, E), "semmoe_permute: workspace %zu < %zu bytes", ws_bytes,
          permute_ws_bytes(T, k_max, E));
  REQUIRE(aligned(pair_counts, 16), "semmoe_permute: pair_counts not 16-byte aligned");
  CHECK_DEVICE("semmoe_permute");
  return cuda_status(launch_permute(topk_idx, expert_rank, x, dtype, T, H, E, R, k_max, P, expert_offsets,
                                    rank_offsets, phys_to_expert, expert_counts, sorted_to_pair, pair_to_sorted,
                                    x_perm, pair_counts, ws, static_cast<cudaStream_t>(stream)),
                     "semmoe_permute");
}

int semmoe_permute_noalloc(const int32_t* topk_idx, const int32_t* expert_rank, const void* x, int dtype, int T,
                           int H, int E, int R, int k_max, int P, int32_t* expert_offsets, int32_t* rank_offsets,
                           int32_t* phys_to_expert, int32_t* expert_counts, int32_t* sorted_to_pair,
                           int32_t* pair_to_sorted, void* x_perm, void* stream) {
  REQUIRE(T >= 0, "semmoe_permute_noalloc: T = %d < 0", T);
  REQUIRE(E >= 1 && E <= 256, "semmoe_permute_noalloc: E = %d outside [1, 256]", E);
  REQUIRE(R >= 1 && R <= E, "semmoe_permute_noalloc: R = %d outside [1, E]", R);
  REQUIRE(k_max >= 1 && k_max <= E, "semmoe_permute_noalloc: k_max = %d outside [1, E]", k_max);
  REQUIRE((long long)T * k_max < (1LL << 31), "semmoe_permute_noalloc: T * k_max too large");
  REQUIRE(permute_ws_bytes(T, k_max, E) <= permute_noalloc_max_scratch(),
          "semmoe_permute_noalloc: T=%d, k_max=%d, E=%d need %zu bytes of scratch; the built-in scratch holds "
          "%zu bytes (use semmoe_permute with a caller workspace)",
          T, k_max, E, permute_ws_bytes(T, k_max, E), permute_noalloc_max_scratch());
  REQUIRE(P >= 0 && (long long)P <= (long long)T * k_max, "semmoe_permute_noalloc: P = %d outside [0, T*k_max]", P);
  REQUIRE(expert_rank && expert_offsets && rank_offsets && phys_to_expert && expert_counts,
          "semmoe_permute_noalloc: null table pointer");
  REQUIRE(T == 0 || (topk_idx && pair_to_sorted), "semmoe_permute_noalloc: null topk_idx or pair_to_sorted");
  REQUIRE(P == 0 || sorted_to_pair, "semmoe_permute_noalloc: null sorted_to_pair");
  REQUIRE((x == nullptr) == (x_perm == nullptr),
          "semmoe_permute_noalloc: x and x_perm must both be set or both NULL");
  if (x != nullptr) {
    REQUIRE(valid_dtype(dtype), "semmoe_permute_noalloc: bad dtype %d", dtype);
    REQUIRE(H >= 1 && (H * elem_size(dtype)) % 16 == 0,
            "semmoe_permute_noalloc: H * elem size must be a multiple of 16");
    REQUIRE(aligned(x, 16) && aligned(x_perm, 16), "semmoe_permute_noalloc: x / x_perm not 16-byte aligned");
  }
  CHECK_DEVICE("semmoe_permute_noalloc");
  return cuda_status(launch_permute_noalloc(topk_idx, expert_rank, x, dtype, T, H, E, R, k_max, P, expert_offsets,
                                            rank_offsets, phys_to_expert, expert_counts, sorted_to_pair,
                                            pair_to_sorted, x_perm, static_cast<cudaStream_t>(stream)),
                     "semmoe_permute_noalloc");
}

size_t semmoe_grouped_ffn_workspace_size(int P, int I, int dtype) {
  if (P < 0 || I < 1 || !valid_dtype(dtype)) return 0;
  return ffn_ws_bytes(P, I, dtype);
}

static int check_ffn_args(const char* fn, const void* x, const void* w13, const void* w2, int dtype, int P, int H,
                          int I, const void* y, const void* ws, size_t ws_bytes) {
  REQUIRE(valid_dtype(dtype), "%s: bad dtype %d", fn, dtype);
  REQUIRE(P >= 0 && H >= 8 && I >= 8 && H % 8 == 0 && I % 8 == 0, "%s: need P >= 0 and H, I multiples of 8 (P=%d H=%d I=%d)",
          fn, P, H, I);
  REQUIRE((long long)P * (H > I ? H : I) < (1LL << 40), "%s: P too large", fn);
  REQUIRE(w13 && w2 && (P == 0 || (x && y)), "%s: null pointer", fn);  // no rows: x and y may be empty
  REQUIRE(aligned(x, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(y, 16), "%s: pointers must be 16-byte aligned",
          fn);
  REQUIRE(ws != nullptr && aligned(ws, 256), "%s: workspace null or not 256-byte aligned", fn);
  REQUIRE(ws_bytes >= ffn_ws_bytes(P, I, dtype), "%s: workspace %zu < %zu bytes", fn, ws_bytes,
          ffn_ws_bytes(P, I, dtype));
  return SEMMOE_OK;
}

int semmoe_grouped_ffn(const void* x_perm, const int32_t* expert_offsets, const int32_t* phys_to_expert,
                       const void* w13, const void* w2, int dtype, int P, int E, int H, int I, void* y_perm,
                       void* ws, size_t ws_bytes, void* stream) {
  REQUIRE(E >= 1 && E <= 256, "semmoe_grouped_ffn: E = %d outside [1, 256]", E);
  REQUIRE(expert_offsets && phys_to_expert, "semmoe_grouped_ffn: null offsets");
  int rc = check_ffn_args("semmoe_grouped_ffn", x_perm, w13, w2, dtype, P, H, I, y_perm, ws, ws_bytes);
  if (rc != SEMMOE_OK) return rc;
  if (P == 0) return SEMMOE_OK;
  CHECK_DEVICE("semmoe_grouped_ffn");
  return cuda_status(launch_ffn(x_perm, expert_offsets, phys_to_expert, w13, w2, dtype, P, E, H, I, y_perm, ws,
                                nullptr, 1, 0, static_cast<cudaStream_t>(stream)),
                     "semmoe_grouped_ffn");
}

int semmoe_grouped_ffn_gather(const void* x, const int32_t* sorted_to_pair, int k_max, int T,
                              const int32_t* expert_offsets, const int32_t* phys_to_expert, const void* w13,
                              const void* w2, int dtype, int P, int E, int H, int I, void* y_perm, void* ws,
                              size_t ws_bytes, void* stream) {
  REQUIRE(E >= 1 && E <= 256, "semmoe_grouped_ffn_gather: E = %d outside [1, 256]", E);
  REQUIRE(T >= 0 && k_max >= 1 && (long long)T * k_max < (1LL << 31),
          "semmoe_grouped_ffn_gather: bad sizes T=%d k_max=%d", T, k_max);
  REQUIRE(P <= (long long)T * k_max, "semmoe_grouped_ffn_gather: P = %d > T * k_max", P);
  REQUIRE(expert_offsets && phys_to_expert, "semmoe_grouped_ffn_gather: null offsets");
  REQUIRE(P == 0 || sorted_to_pair, "semmoe_grouped_ffn_gather: null sorted_to_pair");
  int rc = check_ffn_args("semmoe_grouped_ffn_gather", x, w13, w2, dtype, P, H, I, y_perm, ws, ws_bytes);
  if (rc != SEMMOE_OK) return rc;
  if (P == 0) return SEMMOE_OK;
  CHECK_DEVICE("semmoe_grouped_ffn_gather");
  return cuda_status(launch_ffn(x, expert_offsets, phys_to_expert, w13, w2, dtype, P, E, H, I, y_perm, ws,
                                sorted_to_pair, k_max, T, static_cast<cudaStream_t>(stream)),
                     "semmoe_grouped_ffn_gather");
}

int semmoe_grouped_ffn_form(const void* x, const int32_t* sorted_to_pair, int k_max, int T,
                            const int32_t* expert_offsets, const int32_t* phys_to_expert, const void* w13,
                            const void* w2, int dtype, int P, int E, int H, int I, void* y_perm, void* ws,
                            size_t ws_bytes, int form1, int form2, void* stream) {
  const char* fn = "semmoe_grouped_ffn_form";
  REQUIRE(E >= 1 && E <= 256, "%s: E = %d outside [1, 256]", fn, E);
  REQUIRE(expert_offsets && phys_to_expert, "%s: null offsets", fn);
  const bool gathered = sorted_to_pair != nullptr;
  if (gathered) {
    REQUIRE(T >= 0 && k_max >= 1 && (long long)T * k_max < (1LL << 31), "%s: bad sizes T=%d k_max=%d", fn, T, k_max);
    REQUIRE(P <= (long long)T * k_max, "%s: P = %d > T * k_max", fn, P);
  }
  const bool cc1 = form1 == SEMMOE_FORM_CUDA_CORE, cc2 = form2 == SEMMOE_FORM_CUDA_CORE;
  const bool fu1 = form1 == SEMMOE_FORM_FUSED, fu2 = form2 == SEMMOE_FORM_FUSED;
  REQUIRE(form1 >= SEMMOE_FORM_DEFAULT && form1 <= SEMMOE_FORM_FUSED && form2 >= SEMMOE_FORM_DEFAULT &&
              form2 <= SEMMOE_FORM_FUSED && cc1 == cc2 && fu1 == fu2,
          "%s: bad form pair (%d, %d)", fn, form1, form2);
  REQUIRE(!fu1 || !gathered, "%s: SEMMOE_FORM_FUSED reads x_perm (no gathered rows)", fn);
  REQUIRE(form2 != SEMMOE_FORM_SINGLE_TMA_GATHER && (form1 != SEMMOE_FORM_SINGLE_TMA_GATHER || gathered),
          "%s: SEMMOE_FORM_SINGLE_TMA_GATHER applies to a GEMM1 with gathered rows only", fn);
  REQUIRE(dtype != SEMMOE_F32 || ((form1 == SEMMOE_FORM_DEFAULT || cc1) && (form2 == SEMMOE_FORM_DEFAULT || cc2)),
          "%s: fp32 runs on CUDA cores only (form SEMMOE_FORM_DEFAULT or SEMMOE_FORM_CUDA_CORE)", fn);
  int rc = check_ffn_args(fn, x, w13, w2, dtype, P, H, I, y_perm, ws, ws_bytes);
  if (rc != SEMMOE_OK) return rc;
  if (P == 0) return SEMMOE_OK;
  CHECK_DEVICE(fn);
  return cuda_status(launch_ffn(x, expert_offsets, phys_to_expert, w13, w2, dtype, P, E, H, I, y_perm, ws,
                                sorted_to_pair, gathered ? k_max : 1, gathered ? T : 0,
                                static_cast<cudaStream_t>(stream), form1, form2),
                     fn);
}

int semmoe_grouped_ffn_combine(const void* x, int x_rows_are_tokens, const int32_t* sorted_to_pair, int k_max, int T,
                               const int32_t* expert_offsets, const int32_t* phys_to_expert, const void* w13,
                               const void* w2, const float* topk_w, int dtype, int P, int E, int H, int I, float* acc,
                               void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "semmoe_grouped_ffn_combine";
  REQUIRE(E >= 1 && E <= 256, "%s: E = %d outside [1, 256]", fn, E);
  REQUIRE(T >= 0 && k_max >= 1 && (long long)T * k_max < (1LL << 31), "%s: bad sizes T=%d k_max=%d", fn, T, k_max);
  REQUIRE(P >= 0 && P <= (long long)T * k_max, "%s: P = %d outside [0, T * k_max]", fn, P);
  REQUIRE(H >= 8 && I >= 8 && H % 8 == 0 && I % 8 == 0, "%s: need H, I multiples of 8 (H=%d I=%d)", fn, H, I);
  if (dtype != SEMMOE_BF16) return fail(SEMMOE_ERR_UNSUPPORTED, "%s: bf16 activations and experts only", fn);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(expert_offsets && phys_to_expert && w13 && w2 && topk_w && acc, "%s: null pointer", fn);
  REQUIRE(P == 0 || (x && sorted_to_pair), "%s: null x or sorted_to_pair", fn);
  REQUIRE(aligned(x, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(acc, 16) && aligned(topk_w, 4),
          "%s: misaligned pointer", fn);
  REQUIRE(ws != nullptr && aligned(ws, 256) && ws_bytes >= ffn_ws_bytes(P, I, dtype),
          "%s: workspace null, not 256-byte aligned or below %zu bytes", fn, ffn_ws_bytes(P, I, dtype));
  CHECK_DEVICE(fn);
  return cuda_status(launch_ffn_combine(x, x_rows_are_tokens != 0, sorted_to_pair, k_max, T, expert_offsets,
                                        phys_to_expert, w13, w2, topk_w, P, E, H, I, acc, ws,
                                        static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_combine_finish(const float* acc, const void* y_shared, int dtype, int T, int H, void* out, void* stream) {
  const char* fn = "semmoe_combine_finish";
  REQUIRE(T >= 0 && H >= 8 && H % 8 == 0, "%s: bad sizes T=%d H=%d", fn, T, H);
  if (dtype != SEMMOE_BF16) return fail(SEMMOE_ERR_UNSUPPORTED, "%s: bf16 output only", fn);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(acc && out, "%s: null pointer", fn);
  REQUIRE(aligned(acc, 16) && aligned(y_shared, 16) && aligned(out, 16), "%s: misaligned pointer", fn);
  CHECK_DEVICE(fn);
  return cuda_status(launch_combine_finish(acc, y_shared, T, H, out, static_cast<cudaStream_t>(stream)), fn);
}

size_t semmoe_shared_ffn_workspace_size(int T, int I_s, int dtype) {
  if (T < 0 || I_s < 1 || !valid_dtype(dtype)) return 0;
  return ffn_ws_bytes(T, I_s, dtype);
}

int semmoe_shared_ffn(const void* x, const void* ws13, const void* ws2, int dtype, int T, int H, int I_s,
                      void* y_shared, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_ffn_args("semmoe_shared_ffn", x, ws13, ws2, dtype, T, H, I_s, y_shared, ws, ws_bytes);
  if (rc != SEMMOE_OK) return rc;
  if (T == 0) return SEMMOE_OK;
  CHECK_DEVICE("semmoe_shared_ffn");
  // not as programmatic dependents: it runs beside the layer's steps on another
  // stream, where CTAs waiting for their turn would hold SMs those steps could use
  return cuda_status(launch_ffn(x, nullptr, nullptr, ws13, ws2, dtype, T, 1, H, I_s, y_shared, ws, nullptr, 1, 0,
                                static_cast<cudaStream_t>(stream), SEMMOE_FORM_DEFAULT, SEMMOE_FORM_DEFAULT, false),
                     "semmoe_shared_ffn");
}

int semmoe_combine(const void* y_perm, const int32_t* pair_to_sorted, const float* topk_w, const void* y_shared,
                   int dtype, int T, int H, int k_max, int P, void* out, void* stream) {
  REQUIRE(valid_dtype(dtype), "semmoe_combine: bad dtype %d", dtype);
  REQUIRE(T >= 0 && k_max >= 1 && P >= 0, "semmoe_combine: bad sizes T=%d k_max=%d P=%d", T, k_max, P);
  REQUIRE(H >= 1 && (H * elem_size(dtype)) % 16 == 0, "semmoe_combine: H * elem size must be a multiple of 16");
  REQUIRE((long long)T * k_max < (1LL << 31), "semmoe_combine: T * k_max too large");
  if (T == 0) return SEMMOE_OK;
  REQUIRE(pair_to_sorted && topk_w && out, "semmoe_combine: null pointer");
  REQUIRE(P == 0 || y_perm, "semmoe_combine: null y_perm");
  REQUIRE(aligned(y_perm, 16) && aligned(y_shared, 16) && aligned(out, 16), "semmoe_combine: pointers must be 16-byte aligned");
  CHECK_DEVICE("semmoe_combine");
  return cuda_status(launch_combine(y_perm, pair_to_sorted, topk_w, y_shared, dtype, T, H, k_max, P, out,
                                    static_cast<cudaStream_t>(stream)),
                     "semmoe_combine");
}

static bool is_finite(float v) { return v - v == 0.0f; }

static int check_norm(const char* fn, const char* which, int kind, const void* weight, const void* bias, int w_dtype,
                      float offset, float eps) {
  REQUIRE(kind == SEMMOE_NORM_RMS || kind == SEMMOE_NORM_LAYER, "%s: bad %s %d", fn, which, kind);
  REQUIRE((weight == nullptr && bias == nullptr) || valid_dtype(w_dtype), "%s: bad w_dtype %d", fn, w_dtype);
  REQUIRE(is_finite(offset), "%s: weight_offset is not finite", fn);
  REQUIRE(is_finite(eps) && eps > 0.0f, "%s: eps must be finite and above 0", fn);
  REQUIRE(aligned(weight, 16) && aligned(bias, 16), "%s: weights and biases must be 16-byte aligned", fn);
  return SEMMOE_OK;
}

static int check_rows(const char* fn, int dtype, int T, int H) {
  REQUIRE(valid_dtype(dtype), "%s: bad dtype %d", fn, dtype);
  REQUIRE(T >= 0 && T <= kMaxRows, "%s: T = %d outside [0, 2^31 - 2^16]", fn, T);
  REQUIRE(H >= 1 && (H * elem_size(dtype)) % 16 == 0 && H * elem_size(dtype) <= (size_t)kNormMaxRowBytes,
          "%s: H = %d: rows are a multiple of 16 bytes, at most %d", fn, H, kNormMaxRowBytes);
  return SEMMOE_OK;
}

int semmoe_norm(const void* x, int dtype, int T, int H, int kind, const void* weight, const void* bias, int w_dtype,
                float weight_offset, float eps, void* out, void* stream) {
  const char* fn = "semmoe_norm";
  int rc = check_rows(fn, dtype, T, H);
  if (rc == SEMMOE_OK) rc = check_norm(fn, "kind", kind, weight, bias, w_dtype, weight_offset, eps);
  if (rc != SEMMOE_OK || T == 0) return rc;
  REQUIRE(x && out, "%s: null pointer", fn);
  REQUIRE(aligned(x, 16) && aligned(out, 16), "%s: pointers must be 16-byte aligned", fn);
  const size_t bytes = (size_t)T * H * elem_size(dtype), w_bytes = (size_t)H * elem_size(w_dtype);
  REQUIRE(out == x || !overlap(out, bytes, x, bytes), "%s: out overlaps x", fn);
  REQUIRE(!overlap(out, bytes, weight, w_bytes) && !overlap(out, bytes, bias, w_bytes), "%s: out overlaps the weight or bias", fn);
  CHECK_DEVICE(fn);
  return cuda_status(launch_norm(x, dtype, T, H, NormArgs{kind, weight, bias, w_dtype == SEMMOE_BF16, weight_offset, eps},
                                 out, static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_combine_norm(const void* y_perm, const int32_t* pair_to_sorted, const float* topk_w, const void* y_shared,
                        int dtype, int T, int H, int k_max, int P, int post_kind, const void* post_weight,
                        const void* post_bias, int next_kind, const void* next_weight, const void* next_bias,
                        int w_dtype, float weight_offset, float eps, const void* gate, int gate_dtype, int gate_rows,
                        float block_scale, const void* residual, float residual_scale, void* out, void* next_out,
                        void* stream) {
  const char* fn = "semmoe_combine_norm";
  int rc = check_rows(fn, dtype, T, H);
  if (rc == SEMMOE_OK && post_kind != SEMMOE_NORM_NONE)
    rc = check_norm(fn, "post_kind", post_kind, post_weight, post_bias, w_dtype, weight_offset, eps);
  if (rc == SEMMOE_OK && next_kind != SEMMOE_NORM_NONE)
    rc = check_norm(fn, "next_kind", next_kind, next_weight, next_bias, w_dtype, weight_offset, eps);
  if (rc != SEMMOE_OK) return rc;
  const bool dense = pair_to_sorted == nullptr;
  if (!dense) {
    REQUIRE(k_max >= 1 && P >= 0, "%s: bad sizes k_max=%d P=%d", fn, k_max, P);
    REQUIRE((long long)T * k_max < (1LL << 31), "%s: T * k_max too large", fn);
  }
  REQUIRE(gate == nullptr || valid_dtype(gate_dtype), "%s: bad gate_dtype %d", fn, gate_dtype);
  REQUIRE(gate == nullptr || gate_rows == 1 || gate_rows == T, "%s: gate_rows = %d is neither 1 nor T = %d", fn, gate_rows, T);
  REQUIRE(is_finite(block_scale) && is_finite(residual_scale), "%s: scales must be finite", fn);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(out && (dense || topk_w), "%s: null pointer", fn);
  REQUIRE(y_perm || (!dense && P == 0), "%s: null y_perm", fn);
  REQUIRE((next_kind != SEMMOE_NORM_NONE) == (next_out != nullptr), "%s: next_kind and next_out go together", fn);
  REQUIRE(next_out == nullptr || (next_out != out && next_out != residual && next_out != y_perm && next_out != y_shared),
          "%s: next_out is a buffer of its own", fn);
  REQUIRE(aligned(y_perm, 16) && aligned(y_shared, 16) && aligned(gate, 16) && aligned(residual, 16) && aligned(out, 16) &&
              aligned(next_out, 16),
          "%s: pointers must be 16-byte aligned", fn);
  REQUIRE(aligned(pair_to_sorted, 4) && aligned(topk_w, 4), "%s: misaligned table", fn);
  // rows of these are read for more than one token, and those of a gate of another type do not lie over out's
  const bool own_gate = gate_rows == T && gate_dtype == dtype;
  REQUIRE((dense || out != y_perm) && (gate == nullptr || (next_out != gate && (own_gate || out != gate))),
          "%s: out is neither y_perm (unless dense) nor a gate per channel or of another type, next_out no gate", fn);
  // beside those: a thread reads its pieces of a token's rows before it writes them, but those of no other token
  const size_t bytes = (size_t)T * H * elem_size(dtype), w_bytes = (size_t)H * elem_size(w_dtype);
  const size_t pairs = dense ? 0 : (size_t)T * k_max * 4;
  const struct {
    const char* name;
    const void* p;
    size_t n;
  } in[] = {{"y_perm", y_perm, dense ? bytes : (size_t)P * H * elem_size(dtype)},
            {"y_shared", y_shared, bytes},
            {"residual", residual, bytes},
            {"gate", gate, (size_t)gate_rows * H * elem_size(gate_dtype)},
            {"pair_to_sorted", pair_to_sorted, pairs},
            {"topk_w", dense ? nullptr : topk_w, pairs},
            {"post_weight", post_weight, w_bytes},
            {"post_bias", post_bias, w_bytes},
            {"next_weight", next_weight, w_bytes},
            {"next_bias", next_bias, w_bytes}};
  for (int i = 0; i < 10; ++i) {
    REQUIRE((i < 4 && out == in[i].p) || !overlap(out, bytes, in[i].p, in[i].n), "%s: out overlaps %s", fn, in[i].name);
    REQUIRE(!overlap(next_out, bytes, in[i].p, in[i].n), "%s: next_out overlaps %s", fn, in[i].name);
  }
  REQUIRE(!overlap(next_out, bytes, out, bytes), "%s: next_out overlaps out", fn);
  CHECK_DEVICE(fn);
  const bool wb = w_dtype == SEMMOE_BF16;
  const CombineNorm a{y_perm, pair_to_sorted, topk_w, y_shared, T, H, k_max, P,
                      NormArgs{post_kind, post_weight, post_bias, wb, weight_offset, eps},
                      NormArgs{next_kind, next_weight, next_bias, wb, weight_offset, eps},
                      gate, gate_dtype == SEMMOE_BF16, gate_rows, block_scale, residual, residual_scale, out, next_out};
  return cuda_status(launch_combine_norm(a, dtype, static_cast<cudaStream_t>(stream)), fn);
}

int semmoe_dp_schedule(const int32_t* pred_rank, const int32_t* req_offsets, int T, int n_req, int R, int32_t* hist,
                       int32_t* req_rank, int32_t* req_order, int32_t* rank_req_offsets, int32_t* req_tok_start,
                       int32_t* tok_order, int32_t* tok_rank, int32_t* rank_tok_offsets, void* stream) {
  REQUIRE(T >= 0 && n_req >= 0, "semmoe_dp_schedule: bad sizes T=%d n_req=%d", T, n_req);
  REQUIRE(R >= 1 && R <= 64, "semmoe_dp_schedule: R = %d outside [1, 64]", R);
  REQUIRE(n_req >= 1 || T == 0, "semmoe_dp_schedule: %d tokens but no request", T);
  REQUIRE((long long)n_req * R < (1LL << 31), "semmoe_dp_schedule: n_req * R too large");
  REQUIRE(req_offsets && rank_req_offsets && rank_tok_offsets, "semmoe_dp_schedule: null pointer");
  REQUIRE(n_req == 0 || (hist && req_rank && req_order && req_tok_start), "semmoe_dp_schedule: null request output");
  REQUIRE(T == 0 || (pred_rank && tok_order && tok_rank), "semmoe_dp_schedule: null token array");
  CHECK_DEVICE("semmoe_dp_schedule");
  return cuda_status(launch_dp_schedule(pred_rank, req_offsets, T, n_req, R, hist, req_rank, req_order,
                                        rank_req_offsets, req_tok_start, tok_order, tok_rank, rank_tok_offsets,
                                        static_cast<cudaStream_t>(stream)),
                     "semmoe_dp_schedule");
}

int semmoe_transition_lookup(const int32_t* topk_idx, const int32_t* k_per_token, int k_uniform, const float* trans,
                             int T, int k_max, int E, int R, int32_t* pred_next, void* stream) {
  REQUIRE(T >= 0 && k_max >= 1 && E >= 1, "semmoe_transition_lookup: bad sizes T=%d k_max=%d E=%d", T, k_max, E);
  REQUIRE(R >= 1 && R <= 64, "semmoe_transition_lookup: R = %d outside [1, 64]", R);
  REQUIRE((long long)T * k_max < (1LL << 31) && (long long)E * R < (1LL << 31),
          "semmoe_transition_lookup: T * k_max or E * R too large");
  REQUIRE(k_per_token != nullptr || (k_uniform >= 1 && k_uniform <= k_max),
          "semmoe_transition_lookup: k_uniform = %d outside [1, k_max = %d]", k_uniform, k_max);
  if (T == 0) return SEMMOE_OK;
  REQUIRE(topk_idx && trans && pred_next, "semmoe_transition_lookup: null pointer");
  REQUIRE(aligned(trans, 4) && aligned(topk_idx, 4) && aligned(pred_next, 4) && aligned(k_per_token, 4),
          "semmoe_transition_lookup: misaligned pointer");
  CHECK_DEVICE("semmoe_transition_lookup");
  return cuda_status(launch_transition_lookup(topk_idx, k_per_token, k_uniform, trans, T, k_max, E, R, pred_next,
                                              static_cast<cudaStream_t>(stream)),
                     "semmoe_transition_lookup");
}

size_t semmoe_mx4_scales_size(int rows, int K, int groups) {
  if (rows < 0 || K < 32 || K % 32 != 0 || groups < 1) return 0;
  return mx4_scale_bytes(rows, K, groups);
}

static int check_mx4_matrix(const char* fn, int groups, int group_rows, int K, const void* full, int dtype,
                            const void* codes, const void* scales) {
  REQUIRE(valid_dtype(dtype), "%s: bad dtype %d", fn, dtype);
  REQUIRE(groups >= 1 && group_rows >= 0, "%s: bad sizes groups=%d group_rows=%d", fn, groups, group_rows);
  REQUIRE(K >= 32 && K % 32 == 0, "%s: K = %d is not a positive multiple of 32", fn, K);
  REQUIRE((long long)groups * group_rows <= kMaxRows, "%s: groups * group_rows too large", fn);
  if (group_rows == 0) return SEMMOE_OK;
  REQUIRE(full && codes && scales, "%s: null pointer", fn);
  REQUIRE(aligned(full, 16) && aligned(codes, 16) && aligned(scales, 16), "%s: pointers must be 16-byte aligned", fn);
  return SEMMOE_OK;
}

int semmoe_mx4_quantize(const void* x, int dtype, int groups, int group_rows, int K, uint8_t* codes, uint8_t* scales,
                        void* stream) {
  const char* fn = "semmoe_mx4_quantize";
  int rc = check_mx4_matrix(fn, groups, group_rows, K, x, dtype, codes, scales);
  if (rc != SEMMOE_OK || group_rows == 0) return rc;
  CHECK_DEVICE(fn);
  return cuda_status(launch_mx4_quantize(x, dtype, groups, group_rows, K, codes, scales,
                                         static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int groups, int group_rows, int K, void* out,
                          int out_dtype, void* stream) {
  const char* fn = "semmoe_mx4_dequantize";
  int rc = check_mx4_matrix(fn, groups, group_rows, K, out, out_dtype, codes, scales);
  if (rc != SEMMOE_OK || group_rows == 0) return rc;
  CHECK_DEVICE(fn);
  return cuda_status(launch_mx4_dequantize(codes, scales, groups, group_rows, K, out, out_dtype,
                                           static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_mx4_quantize_rows(const void* x, int dtype, int T, int K, const int32_t* pair_to_sorted, int k_max, int P,
                             const int32_t* expert_offsets, int E, uint8_t* codes, uint8_t* scales, void* stream) {
  const char* fn = "semmoe_mx4_quantize_rows";
  REQUIRE(valid_dtype(dtype), "%s: bad dtype %d", fn, dtype);
  REQUIRE(K >= 32 && K % 32 == 0, "%s: K = %d is not a positive multiple of 32", fn, K);
  REQUIRE(E >= 1 && E <= 256, "%s: E = %d outside [1, 256]", fn, E);
  REQUIRE(T >= 0 && k_max >= 1 && (long long)T * k_max <= kMaxRows, "%s: bad sizes T=%d k_max=%d", fn, T, k_max);
  REQUIRE(P >= 0 && P <= (long long)T * k_max, "%s: P = %d outside [0, T * k_max]", fn, P);
  if (P == 0) return SEMMOE_OK;
  REQUIRE(x && pair_to_sorted && expert_offsets && codes && scales, "%s: null pointer", fn);
  REQUIRE(aligned(x, 16) && aligned(codes, 16) && aligned(scales, 16), "%s: pointers must be 16-byte aligned", fn);
  REQUIRE(aligned(pair_to_sorted, 4) && aligned(expert_offsets, 4), "%s: misaligned table", fn);
  CHECK_DEVICE(fn);
  return cuda_status(launch_mx4_quantize_rows(x, dtype, T, K, pair_to_sorted, k_max, P, expert_offsets, E, codes,
                                              scales, static_cast<cudaStream_t>(stream)),
                     fn);
}

static int check_mx4_product(const char* fn, int P, int E, int N, int K, const void* a, const void* a_scales,
                             const void* offsets, const void* experts, const void* b, const void* b_scales,
                             const void* out) {
  REQUIRE(E >= 1 && E <= 256, "%s: E = %d outside [1, 256]", fn, E);
  REQUIRE(P >= 0 && P <= kMaxRows, "%s: P = %d outside [0, 2^31 - 2^16]", fn, P);
  REQUIRE(K >= 32 && K % 32 == 0, "%s: K = %d is not a positive multiple of 32", fn, K);
  REQUIRE(N >= 8 && N % 8 == 0, "%s: N = %d is not a positive multiple of 8", fn, N);
  // tile counts and the tensor maps' coordinates are 32-bit
  REQUIRE((long long)P / 128 + E < (1LL << 31) / ((N + 127) / 128), "%s: P * N too large", fn);
  REQUIRE((long long)P / 128 + E < (1LL << 31) / ((K + 127) / 128), "%s: P * K too large", fn);
  REQUIRE(2LL * E * ((N + 127) / 128) < (1LL << 31) / ((K + 127) / 128), "%s: E * N * K too large", fn);
  if (P == 0) return SEMMOE_OK;
  REQUIRE(a && a_scales && offsets && experts && b && b_scales && out, "%s: null pointer", fn);
  REQUIRE(aligned(a, 16) && aligned(a_scales, 16) && aligned(b, 16) && aligned(b_scales, 16) && aligned(out, 16),
          "%s: pointers must be 16-byte aligned", fn);
  REQUIRE(aligned(offsets, 4) && aligned(experts, 4), "%s: misaligned table", fn);
  return SEMMOE_OK;
}

int semmoe_mx4_grouped_gemm(const uint8_t* a, const uint8_t* a_scales, const int32_t* expert_offsets,
                            const int32_t* phys_to_expert, const uint8_t* b, const uint8_t* b_scales, int P, int E,
                            int N, int K, void* out, int out_dtype, void* stream) {
  const char* fn = "semmoe_mx4_grouped_gemm";
  REQUIRE(valid_dtype(out_dtype), "%s: bad dtype %d", fn, out_dtype);
  int rc = check_mx4_product(fn, P, E, N, K, a, a_scales, expert_offsets, phys_to_expert, b, b_scales, out);
  if (rc != SEMMOE_OK || P == 0) return rc;
  CHECK_DEVICE(fn);
  return cuda_status(launch_mx4_grouped_gemm(a, a_scales, expert_offsets, phys_to_expert, b, b_scales, P, E, N, K, out,
                                             out_dtype, static_cast<cudaStream_t>(stream)),
                     fn);
}

size_t semmoe_mx4_grouped_ffn_workspace_size(int P, int E, int I) {
  if (P < 0 || E < 1 || I < 32 || I % 32 != 0) return 0;
  return mx4_ffn_ws_bytes(P, E, I);
}

int semmoe_mx4_grouped_ffn(const uint8_t* x, const uint8_t* x_scales, const int32_t* expert_offsets,
                           const int32_t* phys_to_expert, const uint8_t* w13, const uint8_t* w13_scales,
                           const uint8_t* w2, const uint8_t* w2_scales, int P, int E, int H, int I, void* y_perm,
                           void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "semmoe_mx4_grouped_ffn";
  REQUIRE(I >= 32 && I % 32 == 0, "%s: I = %d is not a positive multiple of 32", fn, I);
  int rc = check_mx4_product(fn, P, E, H > I ? H : I, H, x, x_scales, expert_offsets, phys_to_expert, w13, w13_scales,
                             y_perm);
  if (rc != SEMMOE_OK || P == 0) return rc;
  REQUIRE((long long)P / 128 + E < (1LL << 31) / ((I + 127) / 128), "%s: P * I too large", fn);
  REQUIRE(w2 && w2_scales, "%s: null pointer", fn);
  REQUIRE(aligned(w2, 16) && aligned(w2_scales, 16), "%s: pointers must be 16-byte aligned", fn);
  REQUIRE(ws != nullptr && aligned(ws, 256) && ws_bytes >= mx4_ffn_ws_bytes(P, E, I),
          "%s: workspace null, not 256-byte aligned or below %zu bytes", fn, mx4_ffn_ws_bytes(P, E, I));
  CHECK_DEVICE(fn);
  return cuda_status(launch_mx4_grouped_ffn(x, x_scales, expert_offsets, phys_to_expert, w13, w13_scales, w2,
                                            w2_scales, P, E, H, I, y_perm, ws, static_cast<cudaStream_t>(stream)),
                     fn);
}

static int check_w4_shape(const char* fn, int scale_dtype, int K, int group) {
  REQUIRE(valid_dtype(scale_dtype), "%s: bad scale_dtype %d", fn, scale_dtype);
  REQUIRE(group == 32 || group == 64 || (group >= 128 && group % 128 == 0),
          "%s: group = %d is neither 32, 64 nor a multiple of 128", fn, group);
  REQUIRE(K >= group && K % group == 0, "%s: %d columns are not a positive multiple of group = %d", fn, K, group);
  return SEMMOE_OK;
}

static int check_w4_matrix(const char* fn, int rows, int K, int group, const void* full, int dtype, const void* codes,
                           const void* scales, int scale_dtype, const void* zeros) {
  REQUIRE(valid_dtype(dtype), "%s: bad dtype %d", fn, dtype);
  REQUIRE(rows >= 0 && rows <= kMaxRows, "%s: rows = %d outside [0, 2^31 - 2^16]", fn, rows);
  int rc = check_w4_shape(fn, scale_dtype, K, group);
  if (rc != SEMMOE_OK || rows == 0) return rc;
  REQUIRE(full && codes && scales, "%s: null pointer", fn);
  REQUIRE(aligned(full, 16) && aligned(codes, 16) && aligned(scales, 16) && aligned(zeros, 16), "%s: misaligned pointer", fn);
  return SEMMOE_OK;
}

int semmoe_w4_quantize(const void* x, int dtype, int rows, int K, int group, uint8_t* codes, void* scales,
                       int scale_dtype, uint8_t* zeros, void* stream) {
  const char* fn = "semmoe_w4_quantize";
  int rc = check_w4_matrix(fn, rows, K, group, x, dtype, codes, scales, scale_dtype, zeros);
  if (rc != SEMMOE_OK || rows == 0) return rc;
  CHECK_DEVICE(fn);
  return cuda_status(launch_w4_quantize(x, dtype, rows, K, group, codes, scales, scale_dtype, zeros,
                                        static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_w4_dequantize(const uint8_t* codes, const void* scales, int scale_dtype, const uint8_t* zeros, int rows, int K,
                         int group, void* out, int out_dtype, void* stream) {
  const char* fn = "semmoe_w4_dequantize";
  int rc = check_w4_matrix(fn, rows, K, group, out, out_dtype, codes, scales, scale_dtype, zeros);
  if (rc != SEMMOE_OK || rows == 0) return rc;
  CHECK_DEVICE(fn);
  return cuda_status(launch_w4_dequantize(w4::Weights{codes, scales, zeros, scale_dtype == SEMMOE_BF16}, rows, K, group,
                                          out, out_dtype, static_cast<cudaStream_t>(stream)),
                     fn);
}

static int check_w4_product(const char* fn, const void* x, const void* offsets, const void* experts, const void* codes,
                            const void* scales, int scale_dtype, const void* zeros, int P, int E, int N, int K, int group,
                            const void* out) {
  REQUIRE(E >= 1 && E <= 256, "%s: E = %d outside [1, 256]", fn, E);
  REQUIRE(P >= 0 && P <= kMaxRows, "%s: P = %d outside [0, 2^31 - 2^16]", fn, P);
  int rc = check_w4_shape(fn, scale_dtype, K, group);
  if (rc != SEMMOE_OK) return rc;
  REQUIRE(N >= 8 && N % 8 == 0, "%s: N = %d is not a positive multiple of 8", fn, N);
  REQUIRE(N <= kMaxRows / 2 && K <= kMaxRows, "%s: N or K too large", fn);
  // units of work (at least 8 rows x 16 columns) are counted in 32 bits
  REQUIRE(((long long)P / 8 + E) * ((N + 15) / 16) <= kMaxRows, "%s: P * N too large", fn);
  if (P == 0) return SEMMOE_OK;
  REQUIRE(x && offsets && experts && codes && scales && out, "%s: null pointer", fn);
  REQUIRE(aligned(x, 16) && aligned(codes, 16) && aligned(out, 16) && aligned(scales, 16) && aligned(zeros, 16) &&
              aligned(offsets, 4) && aligned(experts, 4),
          "%s: misaligned pointer", fn);
  return SEMMOE_OK;
}

int semmoe_w4_grouped_gemm(const void* x, const int32_t* expert_offsets, const int32_t* phys_to_expert,
                           const uint8_t* codes, const void* scales, int scale_dtype, const uint8_t* zeros, int P, int E,
                           int N, int K, int group, void* out, void* stream) {
  const char* fn = "semmoe_w4_grouped_gemm";
  int rc = check_w4_product(fn, x, expert_offsets, phys_to_expert, codes, scales, scale_dtype, zeros, P, E, N, K, group, out);
  if (rc != SEMMOE_OK || P == 0) return rc;
  REQUIRE(!overlap(out, (size_t)P * N * 2, x, (size_t)P * K * 2), "%s: out overlaps x, of which all columns are read for each of out's", fn);
  CHECK_DEVICE(fn);
  return cuda_status(launch_w4_grouped_gemm(x, expert_offsets, phys_to_expert,
                                            w4::Weights{codes, scales, zeros, scale_dtype == SEMMOE_BF16}, P, E, N, K,
                                            group, out, static_cast<cudaStream_t>(stream)),
                     fn);
}

size_t semmoe_w4_grouped_ffn_workspace_size(int P, int I) {
  if (P < 0 || I < 32 || I % 32 != 0) return 0;
  return w4_ffn_ws_bytes(P, I);
}

int semmoe_w4_grouped_ffn(const void* x, const int32_t* expert_offsets, const int32_t* phys_to_expert,
                          const uint8_t* w13, const void* w13_scales, const uint8_t* w13_zeros, const uint8_t* w2,
                          const void* w2_scales, const uint8_t* w2_zeros, int scale_dtype, int P, int E, int H, int I,
                          int group, void* y_perm, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "semmoe_w4_grouped_ffn";
  int rc = check_w4_product(fn, x, expert_offsets, phys_to_expert, w13, w13_scales, scale_dtype, w13_zeros, P, E, H, H,
                            group, y_perm);
  if (rc != SEMMOE_OK) return rc;
  rc = check_w4_shape(fn, scale_dtype, I, group);
  if (rc != SEMMOE_OK || P == 0) return rc;
  REQUIRE(I <= kMaxRows / 2 && ((long long)P / 8 + E) * ((I + 15) / 16) <= kMaxRows, "%s: I or P * I too large", fn);
  REQUIRE(w2 && w2_scales, "%s: null pointer", fn);
  REQUIRE((w13_zeros == nullptr) == (w2_zeros == nullptr), "%s: zeros of w13 and w2 go together", fn);
  REQUIRE(aligned(w2, 16) && aligned(w2_scales, 16) && aligned(w2_zeros, 16), "%s: misaligned pointer", fn);
  REQUIRE(ws != nullptr && aligned(ws, 256) && ws_bytes >= w4_ffn_ws_bytes(P, I),
          "%s: workspace null, not 256-byte aligned or below %zu bytes", fn, w4_ffn_ws_bytes(P, I));
  const size_t rows = (size_t)P * H * 2, h = (size_t)P * I * 2;
  REQUIRE(!overlap(ws, h, x, rows) && !overlap(ws, h, y_perm, rows), "%s: the workspace overlaps x or y_perm", fn);
  CHECK_DEVICE(fn);
  const bool sb = scale_dtype == SEMMOE_BF16;
  return cuda_status(launch_w4_grouped_ffn(x, expert_offsets, phys_to_expert, w4::Weights{w13, w13_scales, w13_zeros, sb},
                                           w4::Weights{w2, w2_scales, w2_zeros, sb}, P, E, H, I, group, y_perm, ws,
                                           static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_selftest_bounded_wait(void* stream) {
  CHECK_DEVICE("semmoe_selftest_bounded_wait");
  return cuda_status(launch_selftest_bounded_wait(static_cast<cudaStream_t>(stream)), "semmoe_selftest_bounded_wait");
}

int semmoe_selftest_mx4_wait(const uint8_t* a, const uint8_t* a_scales, const int32_t* expert_offsets,
                             const int32_t* phys_to_expert, const uint8_t* b, const uint8_t* b_scales, int P, int E,
                             int N, int K, float* out, void* stream) {
  const char* fn = "semmoe_selftest_mx4_wait";
  int rc = check_mx4_product(fn, P, E, N, K, a, a_scales, expert_offsets, phys_to_expert, b, b_scales, out);
  if (rc != SEMMOE_OK) return rc;
  REQUIRE(P > 0 && P <= 4096, "%s: need 0 < P <= 4096 (P=%d)", fn, P);
  CHECK_DEVICE(fn);
  return cuda_status(launch_mx4_grouped_gemm(a, a_scales, expert_offsets, phys_to_expert, b, b_scales, P, E, N, K, out,
                                             SEMMOE_F32, static_cast<cudaStream_t>(stream), false, true),
                     fn);
}

int semmoe_selftest_w4_wait(const void* x, const int32_t* expert_offsets, const int32_t* phys_to_expert, const uint8_t* codes,
                            const void* scales, int scale_dtype, const uint8_t* zeros, int P, int E, int N, int K, int group,
                            void* out, void* stream) {
  const char* fn = "semmoe_selftest_w4_wait";
  int rc = check_w4_product(fn, x, expert_offsets, phys_to_expert, codes, scales, scale_dtype, zeros, P, E, N, K, group, out);
  if (rc != SEMMOE_OK) return rc;
  REQUIRE(P > 0 && P <= 4096, "%s: need 0 < P <= 4096 (P=%d)", fn, P);
  CHECK_DEVICE(fn);
  return cuda_status(launch_selftest_w4_wait(x, expert_offsets, phys_to_expert,
                                             w4::Weights{codes, scales, zeros, scale_dtype == SEMMOE_BF16}, P, E, N, K, group, out,
                                             static_cast<cudaStream_t>(stream)),
                     fn);
}

int semmoe_selftest_fused_ready_wait(const void* x_perm, const void* w13, const void* w2, int P, int H, int I,
                                     void* y_perm, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_ffn_args("semmoe_selftest_fused_ready_wait", x_perm, w13, w2, SEMMOE_BF16, P, H, I, y_perm, ws,
                          ws_bytes);
  if (rc != SEMMOE_OK) return rc;
  REQUIRE(P > 0 && P <= 4096, "semmoe_selftest_fused_ready_wait: need 0 < P <= 4096 (P=%d)", P);
  CHECK_DEVICE("semmoe_selftest_fused_ready_wait");
  return cuda_status(launch_selftest_fused_ready_wait(x_perm, w13, w2, P, H, I, y_perm, ws,
                                                      static_cast<cudaStream_t>(stream)),
                     "semmoe_selftest_fused_ready_wait");
}

}  // extern "C"
