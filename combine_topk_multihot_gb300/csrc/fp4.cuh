// Microscaled 4-bit floating point: e2m1 codes with a power-of-two scale for
// each 32 of a row, after the OCP Microscaling Formats (MX) specification 1.0.
//
// A code is sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4,
// 6; two codes a byte, the lower four bits first.  A scale is its exponent's 8
// bits (e8m0): 2^(e - 127), 255 for NaN.  Scales lie in tiles of 128 rows and 4
// blocks, 512 bytes, as the tensor cores read them: row r's four bytes at
// 16 (r % 32) + 4 (r / 32); [row tiles, block tiles] of them a matrix.
#pragma once

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

// The codes of eight values already divided by their scale, the first in the
// lowest bits: to nearest even, saturated.  (The conversions here are written
// as instructions: through the toolkit's header, 13.0, they took tens of others.)
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t c;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(c) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return c;
}
// The eight codes of a word as pairs of f16.
__device__ __forceinline__ void f16_of_e2m1x8(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(w));
}
// The four scales of a word as pairs of bf16.
__device__ __forceinline__ void bf16_of_e8m0x4(uint32_t w, uint32_t (&v)[2]) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\tcvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
      : "=r"(v[0]), "=r"(v[1]) : "r"(w));
}
// The four e4m3 codes of a word as pairs of f16.
__device__ __forceinline__ void f16_of_e4m3x4(uint32_t w, uint32_t (&v)[2]) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(v[0]), "=r"(v[1]) : "r"(w));
}
__device__ __forceinline__ void mma_f16_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace moe
