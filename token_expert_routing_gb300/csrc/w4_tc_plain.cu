// The plain product of w4_tc.cuh (two files, so that they compile side by side).
#include "w4_tc.cuh"

namespace semmoe {

int w4_tc_plain_take_errors(cudaStream_t s, int* bits) { return take_error_word(g_err, s, bits); }

cudaError_t launch_w4_tc_plain(const w4::Product& pr, cudaStream_t s) {
  const int rows = pr.P / (pr.E < pr.P ? pr.E : pr.P);  // of a group, on average
  if (rows <= 24) return launch_mode<false, 32>(pr, s);
  if (rows <= 48) return launch_mode<false, 64>(pr, s);
  return rows <= 96 ? launch_mode<false, 128>(pr, s) : launch_mode<false, 256>(pr, s);
}

}  // namespace semmoe
