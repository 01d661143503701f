// The plain product of w4_tc.cuh (two files, so that they compile side by side).
#include "w4_tc.cuh"

namespace semmoe {

int w4_tc_plain_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_w4_tc_plain(const w4::Product& pr, cudaStream_t s) {
  const int rows = pr.P / (pr.E < pr.P ? pr.E : pr.P);  // of a group, on average
  // Units of 32, 64 or 256 rows, measured on 64 experts, 1408 -> 2048, us: 6 rows a group 30.3, 30.5, 43.9; 12 rows 31.2, 30.9,
  // 44.0; 24 rows 37.8, 32.7, 44.7; 64 rows 69.8, 46.8, 47.9; 72 rows 75.2, 50.8, 48.6; 96 rows 95.1, 62.8, 51.3 (units of 128
  // rows: nowhere the best, 57.4 at 96).
  if (rows < 12) return launch_mode<false, 32>(pr, s);
  return rows <= 64 ? launch_mode<false, 64>(pr, s) : launch_mode<false, 256>(pr, s);
}

}  // namespace semmoe
