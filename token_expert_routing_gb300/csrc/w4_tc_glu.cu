// The SwiGLU form of w4_tc.cuh (two files, so that they compile side by side).
#include "w4_tc.cuh"

namespace semmoe {

int w4_tc_glu_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_w4_tc_glu(const w4::Product& pr, cudaStream_t s) {
  const int rows = pr.P / (pr.E < pr.P ? pr.E : pr.P);  // of a group, on average
  // Units of 32, 64 or 128 rows, measured on 64 experts, 2048 -> 2 x 1408, us: 6 rows a group 41, 43, 54; 16 rows 44, 44, 55;
  // 24 rows 50, 46, 56; 48 rows 79, 55, 60; 64 rows 97, 64, 67; 80 rows 113, 75, 74; 96 rows 134, 87, 78.
  if (rows <= 16) return launch_mode<true, 32>(pr, s);
  return rows <= 64 ? launch_mode<true, 64>(pr, s) : launch_mode<true, 128>(pr, s);
}

}  // namespace semmoe
