// 4-bit microscaled values (blocks of 32 along K share one power-of-two scale):
// the conversion of a block and the layout of the scales, shared by the
// quantisation kernels (mx4.cu) and the grouped products (mx4_gemm.cu).
//
// A block x_0..x_31 with a = max |x_i| is held as a biased exponent
//   b = max(E(a) - 2, 0),  E(a) = the biased fp32 exponent of a   (scale 2^(b - 127))
// and 32 codes of e2m1 (sign, two exponent bits, one mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6), the round-to-nearest-even of x_i / 2^(b - 127), at most 6.
// a / scale lies in [4, 8), so the largest magnitudes use the grid's top; the
// division is by a power of two, hence exact, and each value is rounded once.
// E(a) = 255 (NaN or infinity in the block) gives b = 255, which stands for NaN.
//
// Codes: row-major, two per byte, the lower column in the low four bits.
// Scales: tiles of 128 rows x 128 columns, 512 bytes each: row r of a tile and
// its column block j (0..3) at byte 16 (r % 32) + 4 (r / 32) + j, which is the order
// in which the tensor cores read a tile's scales.  Tiles of one row tile are
// consecutive along K; each group of rows (an expert's rows or matrix) starts a
// row tile of its own.
#pragma once

#include "common.cuh"

namespace semmoe {
namespace mx4 {

constexpr int kBlock = 32;         // values per scale
constexpr int kTileRows = 128;
constexpr int kTileCols = 128;     // values per row and tile
constexpr int kTileBytes = 512;

__host__ __device__ inline int col_tiles(int K) { return (K + kTileCols - 1) / kTileCols; }
__host__ __device__ inline int row_tiles(int rows) { return (rows + kTileRows - 1) / kTileRows; }
// Bytes of the scales of `rows` rows in `groups` groups, however they are spread over the groups.
inline size_t scale_bytes(long long rows, int K, int groups) {
  return (size_t)(rows / kTileRows + groups) * col_tiles(K) * kTileBytes;
}
// Byte offset of row r of a row tile inside each of its 512-byte tiles.
__host__ __device__ inline int row_byte(int r) { return 16 * (r & 31) + 4 * (r >> 5); }

// Biased scale exponent of a block whose largest |x| has the fp32 bits `amax`
// (a maximum over magnitudes as integers, which orders NaN above infinity).
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - b): what the block's values are multiplied by (b = 255 never used for numbers).
__device__ __forceinline__ float inverse_scale(uint32_t b) { return __uint_as_float((b < 254u ? 254u - b : 1u) << 23); }
// 2^(b - 127), the scale itself; NaN for b = 255.
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}

// Eight values (already divided by their block's scale) -> eight codes, value i at bits 4i.
__device__ __forceinline__ uint32_t encode8(float v0, float v1, float v2, float v3, float v4, float v5, float v6,
                                            float v7) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3), "f"(v4), "f"(v5), "f"(v6), "f"(v7));
  return r;
}

}  // namespace mx4
}  // namespace semmoe
