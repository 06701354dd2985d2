// Rowwise e4m3 quantization of bf16 rows, shared by the FP8 row kernels and
// the fused dispatch's FP8 rows.
//
// "Add the deepep expert-parallel implementation (huggingface/transformers
// #49638)", What this adds, scope note: FP8 dispatch is the named follow-up.
// Format: one fp32 scale per row, scale = amax(|row|) / 448 (1 for an
// all-zero row), code = e4m3(v / scale) rounded to nearest even and saturated
// at +-448, the division an IEEE fp32 division.  A warp owns a row: lane l
// holds the 8-value (16-byte) vectors l, l + 32, ...
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr float E4M3_MAX = 448.0f;

__device__ __forceinline__ float bf16_abs_max8(uint4 q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
  return m;
}

__device__ __forceinline__ uint32_t e4m3_of(float v) {
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}

// 8 bf16 values / scale -> 8 e4m3 codes, in element order (lowest byte first).
__device__ __forceinline__ uint2 quantize8(uint4 q, float scale) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3_of(bf16_lo(w[i]) / scale) | (e4m3_of(bf16_hi(w[i]) / scale) << 8);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The scale of a warp-owned row (V vectors per lane).
__device__ __forceinline__ float row_scale(const uint4* src, int V, int lane) {
  float amax = 0.f;
  for (int v = 0; v < V; ++v) amax = fmaxf(amax, bf16_abs_max8(__ldg(src + lane + 32 * v)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, o));
  return amax > 0.f ? amax / E4M3_MAX : 1.0f;
}

// ---------------------------------------------------------------- blocks of 128
// The same rule for blocks of 128 values, with two additions: the scale of a
// block that is not zero is at least 2^-126 (so that no quotient overflows for
// want of it), and a NaN or an infinity makes the block's scale non-finite
// (its products are then, too) instead of being passed over by the maximum.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The larger magnitudes of two pairs of bf16 values (NaN if there is one).
__device__ __forceinline__ uint32_t bf16x2_abs_max(uint32_t a, uint32_t b) {
  const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&a), y = *reinterpret_cast<const __nv_bfloat162*>(&b);
  const __nv_bfloat162 m = __hmax2_nan(__habs2(x), __habs2(y));
  return *reinterpret_cast<const uint32_t*>(&m);
}

__device__ __forceinline__ float block_scale(float amax) {
  if (amax >= 0x1p-90f && amax < 0x1p100f) {  // Markstein's residual again, see below
    constexpr float inv = 1.0f / E4M3_MAX;
    const float q = __fmul_rn(amax, inv);
    return __fmaf_rn(-__fmaf_rn(q, E4M3_MAX, -amax), inv, q);
  }
  return amax == 0.f ? 1.0f : max_nan(__fdiv_rn(amax, E4M3_MAX), 0x1p-126f);
}

// Four codes, lowest byte first.
__device__ __forceinline__ uint32_t e4m3x4(float v0, float v1, float v2, float v3) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v2, v3), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Quotients of bf16 values by one scale, rounded as an IEEE division rounds
// them, in three operations each: a product with y, the correctly rounded
// reciprocal of s, and Markstein's correction by the residual ("Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990).  His
// theorem wants q within an ulp of v / s, and here it may be 1.4 ulp off; but v
// and the maximum that s comes from have 8 significant bits, and for all 128 x
// 128 pairs of them the result is the correctly rounded quotient (checked in
// rational arithmetic, and on the GPU against a division).  The residual's last bit
// is above fp32's smallest for |v| >= 2^-103; with a scale of at
// least 2^-90 a smaller v has a code of zero either way.  The residual is taken as
// q s - v, which leaves the sign of a zero quotient v's.  Other scales (and
// non-finite ones) take the division.
// Bit-exactness matters here: a quotient of two bf16 values often lies midway
// between two codes, or an fp32 ulp from there.
struct BlockDivide {
  float s, y;
  bool fast;
  __device__ __forceinline__ explicit BlockDivide(float scale) {
    s = scale;
    y = __frcp_rn(scale);
    fast = scale >= 0x1p-90f && scale < 0x1p100f;
  }
  __device__ __forceinline__ float operator()(float v) const {
    const float q = __fmul_rn(v, y);
    return __fmaf_rn(-__fmaf_rn(q, s, -v), y, q);
  }
  // codes of eight bf16 values
  __device__ __forceinline__ uint2 codes(const uint32_t (&w)[4]) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
    if (fast) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (*this)(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], s);
    }
    return make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
  }
};

// silu(g) u with an exponential that is off by up to 2 + 1.2 |g| ulp and a
// quotient off by 2: h has no exact rounding to keep (g and u are fp32 sums), and
// its codes have 3 bits.  For the same reason its quotients by the block's
// scale are products with the scale's reciprocal.  (With expf and IEEE
// divisions for both, the experts of 4096 tokens, E = 128, H = 2048, I = 768,
// take 347 us for 269.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

}  // namespace moe
