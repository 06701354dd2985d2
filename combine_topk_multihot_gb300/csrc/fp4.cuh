// Microscaled 4-bit floating point: e2m1 codes with a power-of-two scale for
// each 32 of a row, after the OCP Microscaling Formats (MX) specification 1.0.
//
// A code is sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4,
// 6; two codes a byte, the lower four bits first.  A scale is its exponent's 8
// bits (e8m0): 2^(e - 127), 255 for NaN.  Scales lie in tiles of 128 rows and 4
// blocks, 512 bytes, as the tensor cores read them: row r's four bytes at
// 16 (r % 32) + 4 (r / 32); [row tiles, block tiles] of them a matrix.
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"
#include "fp8_quant.cuh"

namespace moe {

constexpr int FP4_BLOCK = 32;
constexpr int SCALE_TILE = 512;  // bytes

// Offset of the four scales of row `row` and codes [128 kt, 128 kt + 128) in a matrix of `kts` block tiles.
__host__ __device__ __forceinline__ long long scale_word(long long row, int kt, int kts) {
  return ((row >> 7) * kts + kt) * SCALE_TILE + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// A block's scale from its largest magnitude: the largest exponent that leaves
// amax / X below 7, since 7 and more lie nearer to the next code, 8, that X's
// double would have.  (X = 2^(floor(log2 amax) - 2) for every block would cut
// what lies between 7 X and 8 X to 6 X.)  X is at most 2^125, so that 6 X is an
// fp32 number.  NaN and infinity give 255, NaN.
__device__ __forceinline__ uint32_t e8m0_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7f800000u) return 255u;
  const uint32_t e = (u + (1u << 21)) >> 23;  // mantissas of 1.75 and more carry
  return e > 2u ? min(e - 2u, 252u) : 0u;
}

// 2^(127 - e), by which a block's values are multiplied: exact, barring values
// that lie 2^-100 below their block's largest.  (Not for 255: the codes of a NaN block are zeros.)
__device__ __forceinline__ float e8m0_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// 2^(e - 127)
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7fc00000u : e << 23);
}

// Eight codes (the first in the lowest bits) of values already divided by their scale.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_E2M1, cudaRoundNearest)) << (8 * i);
  return c;
}

// Eight e2m1 codes as e4m3 codes of 2^-6 times their values: the even ones
// (codes 0, 2, 4, 6 of the word, lowest byte first) and the odd ones.  Both
// formats have subnormals, so that moving sign, exponent and mantissa bits into
// place is exact for every code.
__device__ __forceinline__ uint32_t e4m3_of_even(uint32_t w) { return ((w << 4) & 0x80808080u) | ((w << 2) & 0x1c1c1c1cu); }
__device__ __forceinline__ uint32_t e4m3_of_odd(uint32_t w) { return (w & 0x80808080u) | ((w >> 2) & 0x1c1c1c1cu); }

__device__ __forceinline__ void mma_e4m3_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace moe
