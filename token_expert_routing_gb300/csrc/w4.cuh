// 4-bit weights with group scales: integer codes 0..15, and for each group of
// `group` columns of a row a scale s and a zero point z (8 where none is held):
//   w[r,k] = (code[r,k] - z[r,k/group]) * s[r,k/group]
// Codes row-major, two per byte, the lower column in the low four bits; scales and
// zero points row-major [rows, K / group].  Shared by the conversions (w4.cu) and
// the grouped products (w4_gemm.cu).
#pragma once

#include "common.cuh"

namespace semmoe {
namespace w4 {

// A weight tensor of `rows` rows of K columns.
struct Weights {
  const uint8_t* codes;
  const void* scales;    // fp32 or bf16
  const uint8_t* zeros;  // or NULL
  bool scales_bf16;
};

__device__ __forceinline__ float load_scale(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_scale(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

// Two codes of a word (bits sh.. and sh + 16..) as bf16 values 128 + code: the
// codes are the low bits of the mantissa.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int sh) { return ((w >> sh) & 0x000f000fu) | 0x43004300u; }

}  // namespace w4
}  // namespace semmoe
