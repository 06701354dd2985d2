// The RMS norms before and after a block, fused with the block's gate and
// residual scale.
//
//   r(v) = 1 / sqrt(mean(v^2) + eps),   w~ = offset + w
//   in:   n    = x r(x) w~
//   out:  out  = a x + s (y r(y) w~),   s = sigmoid(g), g, or 1
//         next = out r(out) w~2         (the next block's norm, same pass)
//
// One kernel computes all three forms: HAS_Y says whether there is a block
// output to add to the stream, HAS_NEXT whether the (updated) stream is
// normed.  `next` is the norm of the stream as it is held, i.e. after `out`'s
// rounding, so that it equals a separate call on `out`.
//
// Backward, with d the gradient of the stream (dout plus what comes through
// the next norm), all sums over a row of H values:
//   d  = dout + r2 w~2 dnext - out c,   c = r2^3 S1 / H,   S1 = sum w~2 dnext out
//   dx = a d;   dg = s'(g) d y r w~ (summed over the row for a gate per token)
//   dy = r w~ s d - y r^3 M / H,   M = sum w~ s y d = S2 - c S3,
//        S2 = sum w~ s y (dout + r2 w~2 dnext),   S3 = sum w~ s y out
//   dw = sum over rows of s d y r;   dw2 = sum over rows of dnext out r2
// Splitting M into S2 - c S3 makes the three sums independent of one another,
// so a row costs one reduction instead of two.
//
// Nothing is used twice but the weights, so every form is bound by HBM: each
// tensor is read or written once.  A CTA takes one row at a time, thread i the
// 8-value vectors i, i + blockDim, ...: a row's values stay in registers
// between the sums and their use, and the next row's are loaded while the
// current row is reduced.  The weight gradients are summed over a CTA's rows
// in shared memory (each thread its own columns, so no barrier), written as
// one partial row per CTA, and added in a fixed order by a second kernel:
// results do not depend on scheduling.

#include "common.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int MAX_WARPS = 32;

// Eight consecutive values of a row.  `full` (whole, 16-byte aligned vectors)
// holds for the entire matrix when H % 8 == 0; otherwise rows start anywhere
// and the last vector is partial, so values go one by one.
struct F8 {
  float v[8];
};

template <bool F32>
struct Raw;  // a vector as it lies in memory
template <>
struct Raw<false> {
  uint4 q;
};
template <>
struct Raw<true> {
  uint4 q, r;
};

template <bool F32>
__device__ __forceinline__ Raw<F32> raw_zero() {
  Raw<F32> o;
  o.q = make_uint4(0, 0, 0, 0);
  if constexpr (F32) o.r = o.q;
  return o;
}

template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void* row, int col, int H, bool full) {
  Raw<F32> o = raw_zero<F32>();
  if (col >= H) return o;
  if constexpr (F32) {
    const float* p = static_cast<const float*>(row) + col;
    if (full) {
      o.q = __ldcs(reinterpret_cast<const uint4*>(p));
      o.r = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
    } else {
      uint32_t t[8] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < H) t[i] = __float_as_uint(p[i]);
      o.q = make_uint4(t[0], t[1], t[2], t[3]);
      o.r = make_uint4(t[4], t[5], t[6], t[7]);
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + col;
    if (full) {
      o.q = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
      uint32_t t[4] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < H) t[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
      o.q = make_uint4(t[0], t[1], t[2], t[3]);
    }
  }
  return o;
}

template <bool F32>
__device__ __forceinline__ F8 widen(const Raw<F32>& a) {
  F8 o;
  if constexpr (F32) {
    const uint32_t t[8] = {a.q.x, a.q.y, a.q.z, a.q.w, a.r.x, a.r.y, a.r.z, a.r.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __uint_as_float(t[i]);
  } else {
    const uint32_t t[4] = {a.q.x, a.q.y, a.q.z, a.q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[2 * i] = bf16_lo(t[i]);
      o.v[2 * i + 1] = bf16_hi(t[i]);
    }
  }
  return o;
}

// Rounds once to the tensor's type (nearest even).
template <bool F32>
__device__ __forceinline__ Raw<F32> narrow(const F8& a) {
  Raw<F32> o;
  if constexpr (F32) {
    o.q = make_uint4(__float_as_uint(a.v[0]), __float_as_uint(a.v[1]), __float_as_uint(a.v[2]), __float_as_uint(a.v[3]));
    o.r = make_uint4(__float_as_uint(a.v[4]), __float_as_uint(a.v[5]), __float_as_uint(a.v[6]), __float_as_uint(a.v[7]));
  } else {
    o.q = make_uint4(pack_bf16x2(a.v[0], a.v[1]), pack_bf16x2(a.v[2], a.v[3]), pack_bf16x2(a.v[4], a.v[5]),
                     pack_bf16x2(a.v[6], a.v[7]));
  }
  return o;
}

template <bool F32>
__device__ __forceinline__ void store_raw(void* row, int col, int H, bool full, const Raw<F32>& a) {
  if (col >= H) return;
  if constexpr (F32) {
    float* p = static_cast<float*>(row) + col;
    if (full) {
      reinterpret_cast<uint4*>(p)[0] = a.q;
      reinterpret_cast<uint4*>(p)[1] = a.r;
    } else {
      const uint32_t t[8] = {a.q.x, a.q.y, a.q.z, a.q.w, a.r.x, a.r.y, a.r.z, a.r.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < H) p[i] = __uint_as_float(t[i]);
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(row) + col;
    if (full) {
      *reinterpret_cast<uint4*>(p) = a.q;
    } else {
      const uint32_t t[4] = {a.q.x, a.q.y, a.q.z, a.q.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < H) p[i] = static_cast<uint16_t>(t[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// Weights and element gates: bf16 or fp32 by a flag that is the same for the
// whole launch.
__device__ __forceinline__ F8 load_either(const void* row, int f32, int col, int H, bool full) {
  return f32 ? widen(load_raw<true>(row, col, H, full)) : widen(load_raw<false>(row, col, H, full));
}

__device__ __forceinline__ const void* row_of(const void* p, long long row, int H, int f32) {
  return static_cast<const char*>(p) + row * H * (f32 ? 4 : 2);
}
__device__ __forceinline__ void* row_of(void* p, long long row, int H, int f32) {
  return static_cast<char*>(p) + row * H * (f32 ? 4 : 2);
}

// Sums N values over the CTA; every thread gets the totals.  The two halves of
// `red` alternate, so one barrier a call is enough: a warp can reach its
// next write of a half only after a barrier that follows every read of it.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float (*red)[MAX_WARPS][4], int& phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(FULL_MASK, v[k], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[phase][threadIdx.x >> 5][k] = v[k];
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lane < warps ? red[phase][lane][k] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(FULL_MASK, v[k], o);
  phase ^= 1;
}

// The gate's factor s and ds/dg.  From e = exp(-|g|), which cannot overflow:
// s = 1 / (1 + e) or e / (1 + e), and ds/dg = e / (1 + e)^2 on both sides,
// without the cancellation of 1 - s where s is near 1.
struct Gate {
  float s, slope;
};
__device__ __forceinline__ Gate gate_of(float g, int sigmoid) {
  if (!sigmoid) return {g, 1.0f};
  const float e = __expf(-fabsf(g)), inv = 1.0f / (1.0f + e);
  return {g >= 0.f ? inv : e * inv, e * inv * inv};
}

__device__ __forceinline__ float load_scalar(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) norm_forward_kernel(const NormArgs a) {
  __shared__ float red[2][MAX_WARPS][4];
  griddep_launch_dependents();
  griddep_wait();
  const int H = a.H;
  const bool full = (H & 7) == 0;
  const float inv_h = 1.0f / static_cast<float>(H);
  int phase = 0, col[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) col[j] = 8 * (threadIdx.x + j * blockDim.x);

  Raw<XF32> x[NV];
  Raw<false> y[NV];
  auto load = [&](long long t) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = load_raw<XF32>(row_of(a.x, t, H, XF32), col[j], H, full);
      if constexpr (HAS_Y) y[j] = load_raw<false>(row_of(a.y, t, H, 0), col[j], H, full);
    }
  };
  // up to two vectors a thread: the weights stay in registers and the next
  // row is loaded ahead; more would not fit
  constexpr bool KEEP = NV <= 2;
  long long t = blockIdx.x;
  if (KEEP && t < a.T) load(t);
  F8 wk[KEEP ? NV : 1] = {}, w2k[KEEP ? NV : 1] = {};
#pragma unroll
  for (int j = 0; KEEP && j < NV; ++j) {
    if constexpr (HAS_Y) wk[j] = load_either(a.w, a.w_f32, col[j], H, full);
    if constexpr (HAS_NEXT) w2k[j] = load_either(a.w2, a.w_f32, col[j], H, full);
  }
  for (; t < a.T; t += gridDim.x) {
    if constexpr (!KEEP) load(t);
    F8 xs[NV];
    Raw<false> ys[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xs[j] = widen(x[j]);
      if constexpr (HAS_Y) ys[j] = y[j];
    }
    float s = 1.0f;
    if constexpr (HAS_Y)
      if (a.gate_kind == MOE_GATE_TOKEN) s = gate_of(load_scalar(a.gate, t, a.gate_f32), a.sigmoid).s;
    if (KEEP && t + gridDim.x < a.T) load(t + gridDim.x);
    if constexpr (HAS_Y) {
      float sum[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const F8 f = widen(ys[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] += f.v[i] * f.v[i];
      }
      cta_sum(sum, red, phase);
      const float r = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
      if (a.rstd && threadIdx.x == 0) a.rstd[t] = r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const F8 f = widen(ys[j]);
        const F8 w = KEEP ? wk[j % (KEEP ? NV : 1)] : load_either(a.w, a.w_f32, col[j], H, full);
        F8 g;
        if (a.gate_kind == MOE_GATE_ELEMENT) {
          g = load_either(row_of(a.gate, t, H, a.gate_f32), a.gate_f32, col[j], H, full);
#pragma unroll
          for (int i = 0; i < 8; ++i) g.v[i] = gate_of(g.v[i], a.sigmoid).s;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) g.v[i] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          xs[j].v[i] = a.residual_scale * xs[j].v[i] + g.v[i] * (f.v[i] * r * (a.offset + w.v[i]));
        const Raw<XF32> o = narrow<XF32>(xs[j]);
        store_raw<XF32>(row_of(a.out, t, H, XF32), col[j], H, full, o);
        xs[j] = widen(o);  // the stream as it is held
      }
    }
    if constexpr (HAS_NEXT) {
      float sum[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col[j] + i < H) sum[0] += xs[j].v[i] * xs[j].v[i];
      cta_sum(sum, red, phase);
      const float r = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
      if (a.rstd2 && threadIdx.x == 0) a.rstd2[t] = r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const F8 w = KEEP ? w2k[j % (KEEP ? NV : 1)] : load_either(a.w2, a.w_f32, col[j], H, full);
#pragma unroll
        for (int i = 0; i < 8; ++i) xs[j].v[i] = xs[j].v[i] * r * (a.offset + w.v[i]);
        store_raw<false>(row_of(a.next, t, H, 0), col[j], H, full, narrow<false>(xs[j]));
      }
    }
  }
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT, int NV>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackwardArgs a) {
  __shared__ float red[2][MAX_WARPS][4];
  extern __shared__ float4 acc[];  // [(HAS_Y + HAS_NEXT) * NV * 2][blockDim.x]
  griddep_launch_dependents();
  griddep_wait();
  const int H = a.H;
  const bool full = (H & 7) == 0;
  const float inv_h = 1.0f / static_cast<float>(H);
  int phase = 0, col[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) col[j] = 8 * (threadIdx.x + j * blockDim.x);
  constexpr int ACC = (HAS_Y ? 1 : 0) + (HAS_NEXT ? 1 : 0);
#pragma unroll
  for (int k = 0; k < ACC * NV * 2; ++k) acc[k * blockDim.x + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto accumulate = [&](int which, int j, const F8& v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4* p = acc + ((which * NV + j) * 2 + h) * blockDim.x + threadIdx.x;
      float4 q = *p;
      q.x += v.v[4 * h];
      q.y += v.v[4 * h + 1];
      q.z += v.v[4 * h + 2];
      q.w += v.v[4 * h + 3];
      *p = q;
    }
  };

  // a row's tensors; with one vector a thread the next row's are loaded ahead
  struct Row {
    Raw<XF32> dout[NV], out[NV];
    Raw<false> dnext[NV], y[NV];
  };
  auto load = [&](Row& q, long long t) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      q.dout[j] = a.dout ? load_raw<XF32>(row_of(a.dout, t, H, XF32), col[j], H, full) : raw_zero<XF32>();
      if constexpr (HAS_NEXT) {
        q.dnext[j] = load_raw<false>(row_of(a.dnext, t, H, 0), col[j], H, full);
        q.out[j] = load_raw<XF32>(row_of(a.out, t, H, XF32), col[j], H, full);
      }
      if constexpr (HAS_Y) q.y[j] = load_raw<false>(row_of(a.y, t, H, 0), col[j], H, full);
    }
  };
  constexpr bool AHEAD = NV == 1;
  Row next_row;
  long long t = blockIdx.x;
  if (AHEAD && t < a.T) load(next_row, t);
  F8 wk[1] = {}, w2k[1] = {};
  if constexpr (AHEAD) {
    if constexpr (HAS_Y) wk[0] = load_either(a.w, a.w_f32, col[0], H, full);
    if constexpr (HAS_NEXT) w2k[0] = load_either(a.w2, a.w_f32, col[0], H, full);
  }
  auto weight = [&](int j) {
    F8 o = AHEAD ? wk[0] : load_either(a.w, a.w_f32, col[j], H, full);
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] += a.offset;
    return o;
  };
  auto weight2 = [&](int j) {
    F8 o = AHEAD ? w2k[0] : load_either(a.w2, a.w_f32, col[j], H, full);
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] += a.offset;
    return o;
  };

  for (; t < a.T; t += gridDim.x) {
    Row q;
    if constexpr (AHEAD) q = next_row; else load(q, t);
    const float r = HAS_Y ? a.rstd[t] : 0.f;
    const float r2 = HAS_NEXT ? a.rstd2[t] : 0.f;
    Gate gate = {1.0f, 1.0f};
    if constexpr (HAS_Y)
      if (a.gate_kind == MOE_GATE_TOKEN) gate = gate_of(load_scalar(a.gate, t, a.gate_f32), a.sigmoid);
    const float s = gate.s;
    auto element_gate = [&](int j) { return load_either(row_of(a.gate, t, H, a.gate_f32), a.gate_f32, col[j], H, full); };
    if (AHEAD && t + gridDim.x < a.T) load(next_row, t + gridDim.x);

    // S1, S2, S3: a gate per token stays outside of the sums
    constexpr int N = HAS_Y && HAS_NEXT ? 3 : 1, S1 = 0, S2 = HAS_NEXT ? 1 : 0, S3 = 2;
    float sum[N] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      F8 d = widen(q.dout[j]), o, dn;
      if constexpr (HAS_NEXT) {
        o = widen(q.out[j]);
        dn = widen(q.dnext[j]);
        const F8 w2 = weight2(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = w2.v[i] * dn.v[i];
          sum[S1] += e * o.v[i];
          d.v[i] += r2 * e;
        }
      }
      if constexpr (HAS_Y) {
        const F8 y = widen(q.y[j]), w = weight(j);
        F8 g;
        if (a.gate_kind == MOE_GATE_ELEMENT) g = element_gate(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e = w.v[i] * y.v[i];
          if (a.gate_kind == MOE_GATE_ELEMENT) e *= gate_of(g.v[i], a.sigmoid).s;
          sum[S2] += e * d.v[i];
          if constexpr (HAS_NEXT) sum[S3] += e * o.v[i];
        }
      }
    }
    cta_sum(sum, red, phase);
    const float c = HAS_NEXT ? r2 * r2 * r2 * (sum[S1] * inv_h) : 0.f;
    float m = HAS_Y ? sum[N == 3 ? S2 : 0] : 0.f;  // sum of w y d (times s where it is per element)
    if constexpr (N == 3) m -= c * sum[S3];
    const float k = r * r * r * (s * m * inv_h);
    if constexpr (HAS_Y)
      if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && threadIdx.x == 0) {
        const float dg = gate.slope * r * m;
        if (a.gate_f32) static_cast<float*>(a.dgate)[t] = dg;
        else static_cast<uint16_t*>(a.dgate)[t] = static_cast<uint16_t>(pack_bf16x2(dg, 0.f));
      }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      F8 d = widen(q.dout[j]);
      if constexpr (HAS_NEXT) {
        const F8 o = widen(q.out[j]), dn = widen(q.dnext[j]), w2 = weight2(j);
        F8 e;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d.v[i] += r2 * (w2.v[i] * dn.v[i]) - o.v[i] * c;
          e.v[i] = dn.v[i] * (o.v[i] * r2);
        }
        accumulate(HAS_Y ? 1 : 0, j, e);
      }
      F8 dx;
#pragma unroll
      for (int i = 0; i < 8; ++i) dx.v[i] = HAS_Y ? a.residual_scale * d.v[i] : d.v[i];
      store_raw<XF32>(row_of(a.dx, t, H, XF32), col[j], H, full, narrow<XF32>(dx));
      if constexpr (HAS_Y) {
        const F8 y = widen(q.y[j]), w = weight(j);
        F8 g, e, dy;
        if (a.gate_kind == MOE_GATE_ELEMENT) g = element_gate(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const Gate gi = a.gate_kind == MOE_GATE_ELEMENT ? gate_of(g.v[i], a.sigmoid) : gate;
          const float sd = gi.s * d.v[i], yr = y.v[i] * r;
          e.v[i] = sd * yr;
          dy.v[i] = r * (w.v[i] * sd) - y.v[i] * k;
          if (a.gate_kind == MOE_GATE_ELEMENT) g.v[i] = gi.slope * (d.v[i] * (yr * w.v[i]));
        }
        accumulate(0, j, e);
        store_raw<false>(row_of(a.dy, t, H, 0), col[j], H, full, narrow<false>(dy));
        if (a.gate_kind == MOE_GATE_ELEMENT && a.dgate) {
          void* dst = row_of(a.dgate, t, H, a.gate_f32);
          if (a.gate_f32) store_raw<true>(dst, col[j], H, full, narrow<true>(g));
          else store_raw<false>(dst, col[j], H, full, narrow<false>(g));
        }
      }
    }
  }

  // this CTA's sums: one row of [ACC, H] partials, or the result when it is alone
#pragma unroll
  for (int which = 0; which < ACC; ++which) {
    float* dst = a.partials + (static_cast<long long>(blockIdx.x) * ACC + which) * H;
    if (gridDim.x == 1) dst = which == 0 && HAS_Y ? a.dw : a.dw2;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = acc[((which * NV + j) * 2 + h) * blockDim.x + threadIdx.x];
        const int c = col[j] + 4 * h;
        if (full) {
          if (c < H) *reinterpret_cast<float4*>(dst + c) = v;
        } else {
          const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < H) dst[c + i] = f[i];
        }
      }
  }
}

// Adds the partial rows [rows, cols] of the weight gradients (columns
// [0, split) go to d0, the others to d1).  A CTA takes 32 columns, its 32
// warps every 32nd row each; the warps' sums are added in warp order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ partials, int rows, int cols,
                                                           int split, float* __restrict__ d0,
                                                           float* __restrict__ d1) {
  __shared__ float part[32][33];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < cols)
    for (int r = warp; r < rows; r += 32) v += partials[static_cast<long long>(r) * cols + c];
  part[warp][lane] = v;
  __syncthreads();
  v = part[lane][warp];  // warp w now holds column w's 32 sums, one per lane
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  const int oc = blockIdx.x * 32 + warp;
  if (lane == 0 && oc < cols) {
    if (oc < split) d0[oc] = v; else d1[oc - split] = v;
  }
}

int vectors(int H) { return (H + 7) / 8; }
int round_warp(int n) { return (n + 31) / 32 * 32; }

// Vectors a thread: one while that leaves a CTA of at most 256 threads, or
// while there are too few rows for two CTAs on every SM (then a row is spread
// over as many threads as it can use: what counts is the latency of one row).
int forward_nv(long long T, int H) {
  const int v = vectors(H);
  if (v <= 256 || (T < 2LL * sm_count() && v <= 1024)) return 1;
  return v <= 1024 ? 2 : 4;
}

int backward_nv(int H) {
  const int v = vectors(H);
  return v <= 512 ? 1 : v <= 1024 ? 2 : 4;
}

template <typename Kernel, typename Args>
cudaError_t launch_rows(Kernel kernel, long long T, int threads, int per_sm, size_t smem, const Args& a,
                        cudaStream_t s, int grid_limit = 1 << 30) {
  long long grid = static_cast<long long>(sm_count()) * per_sm;
  if (grid > T) grid = T;
  if (grid > grid_limit) grid = grid_limit;
  return launch_dependent(kernel, static_cast<unsigned>(grid), threads, smem, s, a);
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT>
cudaError_t forward(const NormArgs& a, cudaStream_t s) {
  const int nv = forward_nv(a.T, a.H);
  const int threads = round_warp((vectors(a.H) + nv - 1) / nv);
  const int per_sm = threads >= 512 ? 2 : threads >= 256 ? 4 : threads >= 128 ? 8 : 16;
  if (nv == 1) return launch_rows(norm_forward_kernel<XF32, HAS_Y, HAS_NEXT, 1>, a.T, threads, per_sm, 0, a, s);
  if (nv == 2) return launch_rows(norm_forward_kernel<XF32, HAS_Y, HAS_NEXT, 2>, a.T, threads, per_sm, 0, a, s);
  return launch_rows(norm_forward_kernel<XF32, HAS_Y, HAS_NEXT, 4>, a.T, threads, per_sm, 0, a, s);
}

int backward_per_sm(int H) {
  const int threads = round_warp((vectors(H) + backward_nv(H) - 1) / backward_nv(H));
  return threads > 256 ? 1 : threads > 128 ? 2 : threads > 64 ? 4 : 8;
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT, int NV>
cudaError_t backward_nv_launch(const NormBackwardArgs& a, int threads, cudaStream_t s) {
  constexpr int ACC = (HAS_Y ? 1 : 0) + (HAS_NEXT ? 1 : 0);
  auto kernel = norm_backward_kernel<XF32, HAS_Y, HAS_NEXT, NV>;
  const size_t smem = static_cast<size_t>(ACC) * NV * 2 * threads * sizeof(float4);
  if (smem > 48 * 1024) {
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
  }
  return launch_rows(kernel, a.T, threads, backward_per_sm(a.H), smem, a, s);
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT>
cudaError_t backward(const NormBackwardArgs& a, cudaStream_t s) {
  constexpr int ACC = (HAS_Y ? 1 : 0) + (HAS_NEXT ? 1 : 0);
  const long long most = static_cast<long long>(sm_count()) * backward_per_sm(a.H);
  const int grid = static_cast<int>(a.T < most ? a.T : most);
  if (grid > 0) {
    const int nv = backward_nv(a.H);
    const int threads = round_warp((vectors(a.H) + nv - 1) / nv);
    const cudaError_t err = nv == 1   ? backward_nv_launch<XF32, HAS_Y, HAS_NEXT, 1>(a, threads, s)
                            : nv == 2 ? backward_nv_launch<XF32, HAS_Y, HAS_NEXT, 2>(a, threads, s)
                                      : backward_nv_launch<XF32, HAS_Y, HAS_NEXT, 4>(a, threads, s);
    if (err != cudaSuccess || grid == 1) return err;
  }
  const int cols = ACC * a.H;
  return launch_dependent(norm_reduce_kernel, (cols + 31) / 32, 1024, 0, s, a.partials, grid, cols,
                          HAS_Y ? a.H : 0, a.dw, a.dw2);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (a.x_f32) {
    if (!a.y) return forward<true, false, true>(a, s);
    return a.next ? forward<true, true, true>(a, s) : forward<true, true, false>(a, s);
  }
  if (!a.y) return forward<false, false, true>(a, s);
  return a.next ? forward<false, true, true>(a, s) : forward<false, true, false>(a, s);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& a, cudaStream_t s) {
  if (a.x_f32) {
    if (!a.has_y) return backward<true, false, true>(a, s);
    return a.has_next ? backward<true, true, true>(a, s) : backward<true, true, false>(a, s);
  }
  if (!a.has_y) return backward<false, false, true>(a, s);
  return a.has_next ? backward<false, true, true>(a, s) : backward<false, true, false>(a, s);
}

size_t norm_backward_workspace(long long T, int H) {
  const long long most = static_cast<long long>(sm_count()) * backward_per_sm(H);
  return static_cast<size_t>(T < most ? T : most) * 2 * H * sizeof(float);
}

}  // namespace moe
