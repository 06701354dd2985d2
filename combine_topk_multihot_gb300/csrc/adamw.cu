// One AdamW step over many tensors in one launch, the two averages held in
// fp32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit averages are codes with one fp32 scale per block of 256 elements:
//   m  e4m3, scale = max|m| / 448;
//   v  e5m2 (never negative, up to 0x7B), scale = max v / 57344.
// v is rounded at random: away from zero with the probability that keeps its
// mean.  It changes by about (1 - b2) of itself a step, far less than half the
// distance of two codes, so that rounding to nearest would hold it where it
// is.  A positive v never becomes zero: its root divides m.
// m is rounded at random in the same way wherever a step's decay is not
// clearly more than half the distance of two codes: all of it with b1 above
// 11/12 (half a distance is up to 1/16 of m), and the codes below the normal
// ones with any b1.  Held while v falls, it would make updates without end (gradients
// that stop, b1 = b2 = 0.95, 400 steps later: 9346 lr a step, at random 2e-5, fp64 3e-5; b1 =
// 0.9 with its four lowest codes held: 0.96 lr, now 0).  Elsewhere the
// nearer code is the better one (m of random gradients, rms error: 0.0124 of
// their deviation against 0.0176 at b1 = 0.9; halving takes 7 steps for 6.6).
// So it is for all of m in the first NEAREST_STEPS steps: m is then a sum of as many
// terms, of which the last is more than half a distance.
// Scales are at least 2^-120, so that their reciprocals are finite.  The
// parameter's own update uses m and v before they are rounded to 8 bits.
//
// The averages are computed with one rounding per operation (no fused
// multiply-add): what goes into the codes is then the same in any
// implementation that does the operations one by one.  The root and the quotient of the
// update may be off by a few units of 2^-23: they are multiplied by lr and added
// to p, whose own rounding is coarser by 1 / lr.  (Rounded ones take 293 us for 266
// with 8-bit averages, 389 for 375 with fp32 ones: 100 M bf16 parameters, fp32 gradients.)
//
// Bound by HBM: with bf16 parameters, fp32 masters and fp32 gradients 30 bytes
// an element with fp32 averages, 18 with 8-bit ones.  A warp takes a block of
// 256 elements at a time: lane l holds elements 4l .. 4l + 3 of each half of
// 128, so that each load and store of the warp is one contiguous piece and a
// block's maxima are warp maxima.  Warps stride over the blocks of all
// tensors, numbered through; the tensors' table is a kernel argument (no copy
// to the device), and a warp's tensor only ever moves forward in it.

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp8_quant.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int BLOCK = ADAMW_STATE_BLOCK;  // 256: 8 elements a lane
constexpr float SCALE_FLOOR = 0x1p-120f;
constexpr uint32_t E5M2_TOP = 0x7B;  // 57344
constexpr uint32_t E4M3_TOP = 0x7E;  // 448
constexpr long long NEAREST_STEPS = 8;

struct Table {
  AdamWTensor t[ADAMW_BATCH];
  int first[ADAMW_BATCH + 1];  // number of each tensor's first block
  int count;
};

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(FULL_MASK, v, o));
  return v;
}

// 32 mixed bits: shifts and odd multipliers, twice.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0xA3D95B4Fu;
  x ^= x >> 15;
  x *= 0xC2F1E6D3u;
  return x ^ (x >> 16);
}
__host__ __device__ __forceinline__ uint32_t chain(uint32_t key, uint32_t k) { return mix(key ^ k) + 0x9E3779B9u; }

// Four elements at p + i: WIDE when the tensor's address allows one access
// and all four exist, else one by one up to n.
template <bool WIDE>
__device__ __forceinline__ void load4_f32(const float* p, long long i, long long n, float (&v)[4]) {
  if constexpr (WIDE) {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(p + i));
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k < n ? p[i + k] : 0.f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void load4_bf16(const uint16_t* p, long long i, long long n, float (&v)[4]) {
  if constexpr (WIDE) {
    const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p + i));
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k < n ? __uint_as_float(static_cast<uint32_t>(p[i + k]) << 16) : 0.f;
  }
}
template <bool WIDE>
__device__ __forceinline__ uint32_t load4_u8(const uint8_t* p, long long i, long long n) {
  if constexpr (WIDE) {
    return __ldcs(reinterpret_cast<const uint32_t*>(p + i));
  } else {
    uint32_t q = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) q |= static_cast<uint32_t>(p[i + k]) << (8 * k);
    return q;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store4_f32(float* p, long long i, long long n, const float (&v)[4]) {
  if constexpr (WIDE) {
    __stcs(reinterpret_cast<float4*>(p + i), make_float4(v[0], v[1], v[2], v[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) p[i + k] = v[k];
  }
}
template <bool WIDE>
__device__ __forceinline__ void store4_bf16(uint16_t* p, long long i, long long n, const float (&v)[4]) {
  const uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
  if constexpr (WIDE) {
    __stcs(reinterpret_cast<uint2*>(p + i), make_uint2(a, b));
  } else {
    const uint16_t h[4] = {static_cast<uint16_t>(a), static_cast<uint16_t>(a >> 16), static_cast<uint16_t>(b),
                           static_cast<uint16_t>(b >> 16)};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) p[i + k] = h[k];
  }
}
template <bool WIDE>
__device__ __forceinline__ void store4_u8(uint8_t* p, long long i, long long n, uint32_t q) {
  if constexpr (WIDE) {
    __stcs(reinterpret_cast<uint32_t*>(p + i), q);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) p[i + k] = static_cast<uint8_t>(q >> (8 * k));
  }
}

__device__ __forceinline__ void decode_e4m3(uint32_t q, float scale, float (&v)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    v[2 * h] = f.x * scale;
    v[2 * h + 1] = f.y * scale;
  }
}
// An e5m2 code is the upper byte of the same number in fp16.
__device__ __forceinline__ void decode_e5m2(uint32_t q, float scale, float (&v)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t b = __byte_perm(q, 0, h ? 0x3424 : 0x1404);  // bytes 0, 2h, 0, 2h + 1
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b));
    v[2 * h] = f.x * scale;
    v[2 * h + 1] = f.y * scale;
  }
}

struct Step {  // what is the same for all tensors
  float b1, c1, b2, c2, eps;  // c = 1 - b
  float step_size;            // lr / (1 - b1^t)
  float root_bc2;             // 1 / sqrt(1 - b2^t)
  float grad_scale;
  uint32_t step_lo, step_hi;
  float m_random;             // m below this many units of its scale is rounded at random
};

// PARAM: 0 fp32, 1 bf16, 2 bf16 with an fp32 master.
template <int PARAM, bool GRAD_F32, bool EIGHT, bool WIDE>
__device__ __forceinline__ void update_block(const AdamWTensor& T, const Step& st, long long base, long long block,
                                             int lane, uint32_t key) {
  const long long n = T.n;
  float p[2][4], g[2][4], m[2][4], v[2][4];
  uint32_t mq[2], vq[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long i = base + 128 * h + 4 * lane;
    if constexpr (GRAD_F32) load4_f32<WIDE>(static_cast<const float*>(T.grad), i, n, g[h]);
    else load4_bf16<WIDE>(static_cast<const uint16_t*>(T.grad), i, n, g[h]);
    if constexpr (PARAM == 0) load4_f32<WIDE>(static_cast<const float*>(T.param), i, n, p[h]);
    if constexpr (PARAM == 1) load4_bf16<WIDE>(static_cast<const uint16_t*>(T.param), i, n, p[h]);
    if constexpr (PARAM == 2) load4_f32<WIDE>(T.master, i, n, p[h]);
    if constexpr (EIGHT) {
      mq[h] = load4_u8<WIDE>(static_cast<const uint8_t*>(T.exp_avg), i, n);
      vq[h] = load4_u8<WIDE>(static_cast<const uint8_t*>(T.exp_avg_sq), i, n);
    } else {
      load4_f32<WIDE>(static_cast<const float*>(T.exp_avg), i, n, m[h]);
      load4_f32<WIDE>(static_cast<const float*>(T.exp_avg_sq), i, n, v[h]);
    }
  }
  if constexpr (EIGHT) {
    const float ms = T.exp_avg_scale[block], vs = T.exp_avg_sq_scale[block];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      decode_e4m3(mq[h], ms, m[h]);
      decode_e5m2(vq[h], vs, v[h]);
    }
  }
  float m_top = 0.f, v_top = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float gk = g[h][k] * st.grad_scale;
      m[h][k] = __fadd_rn(__fmul_rn(m[h][k], st.b1), __fmul_rn(gk, st.c1));
      v[h][k] = __fadd_rn(__fmul_rn(v[h][k], st.b2), __fmul_rn(__fmul_rn(gk, gk), st.c2));
      // sqrt(v) < 2^64, root_bc2 < 2^27 (1 - b2^t >= 2^-53) and eps < 1e30 (else
      // refused): the divisor is below 2^101, and __fdividef's range, 2^126, is not left
      float root;
      asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v[h][k]));
      const float q = __fdividef(m[h][k], root * st.root_bc2 + st.eps);
      p[h][k] = p[h][k] * T.decay - st.step_size * q;
      if constexpr (EIGHT) {
        m_top = max_nan(m_top, fabsf(m[h][k]));
        v_top = max_nan(v_top, v[h][k]);
      }
    }
    const long long i = base + 128 * h + 4 * lane;
    if constexpr (PARAM == 0) store4_f32<WIDE>(static_cast<float*>(T.param), i, n, p[h]);
    else store4_bf16<WIDE>(static_cast<uint16_t*>(T.param), i, n, p[h]);
    if constexpr (PARAM == 2) store4_f32<WIDE>(T.master, i, n, p[h]);
    if constexpr (!EIGHT) {
      store4_f32<WIDE>(static_cast<float*>(T.exp_avg), i, n, m[h]);
      store4_f32<WIDE>(static_cast<float*>(T.exp_avg_sq), i, n, v[h]);
    }
  }
  if constexpr (EIGHT) {
    const float ms = max_nan(__fdiv_rn(warp_max_nan(m_top), 448.0f), SCALE_FLOOR);
    const float vs = max_nan(__fdiv_rn(warp_max_nan(v_top), 57344.0f), SCALE_FLOOR);
    const float mi = __frcp_rn(ms), vi = __frcp_rn(vs);
    // (a block's elements share the upper half of their number)
    const uint32_t inner = mix(static_cast<uint32_t>(static_cast<uint64_t>(base) >> 33) ^ key);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long i = base + 128 * h + 4 * lane;
      uint32_t qm = 0, qv = 0;
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        // one hash for two neighbours, 16 random bits each; m takes the bits
        // of the neighbour's v, so that an element's two roundings are independent
        const uint32_t r = mix(static_cast<uint32_t>(static_cast<uint64_t>(i + k) >> 1) ^ inner);
        uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(m[h][k] * mi, m[h][k + 1] * mi), __NV_SATFINITE, __NV_E4M3);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // as below, with the exponent moved by 120: the e4m3 code is what
          // lies above the 20th bit (a NaN is below nothing)
          const float t = m[h][k + e] * mi;
          if (fabsf(t) < st.m_random) {
            const uint32_t bits = __float_as_uint(__fmul_rn(fabsf(t), 0x1p-120f));
            const uint32_t code = min((bits + ((e ? r & 0xffffu : r >> 16) << 4)) >> 20, E4M3_TOP);
            two = (two & (e ? 0x80ffu : 0xff80u)) | code << (8 * e);  // (the sign is there)
          }
        }
        qm |= two << (8 * k);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // with its exponent moved by 112, an fp32's bits above the 21st are
          // the e5m2 code (subnormals too); random bits below them carry
          const float x = v[h][k + e];
          const uint32_t bits = __float_as_uint(__fmul_rn(__fmul_rn(x, vi), 0x1p-112f));
          uint32_t code = (bits + ((e ? r >> 16 : r & 0xffffu) << 5)) >> 21;
          if (x > 0.f) code = min(max(code, 1u), E5M2_TOP);
          qv |= (code & 0xffu) << (8 * (k + e));
        }
      }
      store4_u8<WIDE>(static_cast<uint8_t*>(T.exp_avg), i, n, qm);
      store4_u8<WIDE>(static_cast<uint8_t*>(T.exp_avg_sq), i, n, qv);
    }
    if (lane == 0) {
      T.exp_avg_scale[block] = ms;
      T.exp_avg_sq_scale[block] = vs;
    }
  }
}

template <bool EIGHT, bool WIDE>
__device__ __forceinline__ void update_any(const AdamWTensor& T, const Step& st, long long block, int lane, uint32_t key) {
  const long long base = block * BLOCK;
  switch (T.kind) {
    case 0: update_block<0, false, EIGHT, WIDE>(T, st, base, block, lane, key); break;
    case 1: update_block<1, false, EIGHT, WIDE>(T, st, base, block, lane, key); break;
    case 2: update_block<2, false, EIGHT, WIDE>(T, st, base, block, lane, key); break;
    case 3: update_block<0, true, EIGHT, WIDE>(T, st, base, block, lane, key); break;
    case 4: update_block<1, true, EIGHT, WIDE>(T, st, base, block, lane, key); break;
    case 5: update_block<2, true, EIGHT, WIDE>(T, st, base, block, lane, key); break;
  }
}

template <bool EIGHT>
// 8-bit states are bound by instructions as much as by HBM: 64 registers, for four
// CTAs an SM (2^28 elements with masters: 819 -> 782 us).
__global__ void __launch_bounds__(256, EIGHT ? 4 : 1) adamw_kernel(const __grid_constant__ Table table, const AdamWStep h) {
  __shared__ Step s_step;
  griddep_launch_dependents();
  griddep_wait();
  if (h.skip && *h.skip != 0) return;
  if (threadIdx.x == 0) {
    Step st;
    st.b1 = static_cast<float>(h.beta1), st.c1 = static_cast<float>(1.0 - h.beta1);
    st.b2 = static_cast<float>(h.beta2), st.c2 = static_cast<float>(1.0 - h.beta2);
    st.eps = static_cast<float>(h.eps);
    st.grad_scale = h.grad_scale ? *h.grad_scale : 1.0f;
    long long t = h.step;
    st.step_size = h.step_size, st.root_bc2 = h.root_bc2;
    if (h.step_dev) {  // the step's number is known on the device only
      t = *h.step_dev;
      st.step_size = static_cast<float>(h.lr / (1.0 - pow(h.beta1, static_cast<double>(t))));
      st.root_bc2 = static_cast<float>(1.0 / sqrt(1.0 - pow(h.beta2, static_cast<double>(t))));
    }
    st.step_lo = static_cast<uint32_t>(t);
    st.step_hi = static_cast<uint32_t>(static_cast<unsigned long long>(t) >> 32);
    st.m_random = t <= NEAREST_STEPS ? 0.f : h.beta1 > 11.0 / 12.0 ? INFINITY : 0x1p-6f;
    s_step = st;
  }
  __syncthreads();
  const Step st = s_step;
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (blockDim.x >> 5);
  int k = 0, keyed = -1;
  uint32_t key = 0;
  for (long long b = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); b < table.first[table.count]; b += warps) {
    while (b >= table.first[k + 1]) ++k;
    const AdamWTensor& T = table.t[k];
    const long long block = b - table.first[k];
    if (k != keyed) {
      key = chain(chain(T.key, st.step_lo), st.step_hi);
      keyed = k;
    }
    if (T.wide && (block + 1) * BLOCK <= T.n) update_any<EIGHT, true>(T, st, block, lane, key);
    else update_any<EIGHT, false>(T, st, block, lane, key);
  }
}

}  // namespace

uint32_t adamw_key(uint64_t seed, uint32_t tensor) {
  return chain(chain(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32)), tensor);
}

cudaError_t launch_adamw(const AdamWTensor* tensors, int count, const AdamWStep& h, bool eight, cudaStream_t s) {
  for (int at = 0; at < count; at += ADAMW_BATCH) {
    Table table;
    table.count = count - at < ADAMW_BATCH ? count - at : ADAMW_BATCH;
    long long blocks = 0;
    for (int k = 0; k < table.count; ++k) {
      table.t[k] = tensors[at + k];
      table.first[k] = static_cast<int>(blocks);
      blocks += (tensors[at + k].n + BLOCK - 1) / BLOCK;
      if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    }
    table.first[table.count] = static_cast<int>(blocks);
    if (blocks == 0) continue;
    const long long need = (blocks + 7) / 8, most = (eight ? 8LL : 6LL) * sm_count();
    const cudaError_t err = launch_dependent(eight ? adamw_kernel<true> : adamw_kernel<false>,
                                             static_cast<unsigned>(need < most ? need : most), 256, 0, s, table, h);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace moe
