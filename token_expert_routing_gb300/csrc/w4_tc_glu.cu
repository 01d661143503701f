// The SwiGLU form of w4_tc.cuh (two files, so that they compile side by side).
#include "w4_tc.cuh"

namespace semmoe {

int w4_tc_glu_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_w4_tc_glu(const w4::Product& pr, cudaStream_t s) {
  const int rows = pr.P / (pr.E < pr.P ? pr.E : pr.P);  // of a group, on average
  if (rows <= 24) return launch_mode<true, 32>(pr, s);
  return rows <= 48 ? launch_mode<true, 64>(pr, s) : launch_mode<true, 128>(pr, s);
}

}  // namespace semmoe
