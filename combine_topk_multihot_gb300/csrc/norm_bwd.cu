// The backward of the norms before and after a block (norm.cu has the forward
// and the notation).
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
// Each tensor is read or written once: bound by HBM.  A row's values stay in
// registers between the sums and their use, while bulk copies bring the next
// row to shared memory.  The weight gradients are summed over a group's rows in
// shared memory (each thread its own columns, so no barrier), written as one
// partial row per CTA, and added in a fixed order by a second kernel: results
// do not depend on scheduling.

#include "norm.cuh"

namespace moe {

using namespace norm;

namespace {

// One row in flight a group besides the current one: a second slot takes the
// room in L1 that the weights need (183 against 240 us at T = 16384, H = 4096).
constexpr int SLOTS = 1;

// A CTA's threads form groups of `row_threads`, each with a row of its own and
// its own accumulators; they are added up before the CTA's partial row is
// written, so that there are few of those.
// PIPE: rows arrive through shared memory (H a multiple of 8).  THIRD: CTAs of
// up to 256 threads, three an SM.
template <bool XF32, bool HAS_Y, bool HAS_NEXT, bool ELEM, int NV, bool PIPE, bool THIRD = false>
__global__ void __launch_bounds__(THIRD ? 256 : 512, THIRD ? 3 : 1)
    norm_backward_kernel(const NormBackwardArgs a, int row_threads) {
  __shared__ float red[2][MAX_WARPS][4];
  __shared__ uint64_t s_bar[MAX_GROUPS][SLOTS];
  __shared__ int s_abort;
  extern __shared__ __align__(128) float4 acc[];  // [(HAS_Y + HAS_NEXT) * NV * 2][blockDim.x], then the groups' slots
  const int H = a.H;
  const bool full = PIPE || (H & 7) == 0;
  const float inv_h = 1.0f / static_cast<float>(H);
  const int group = threadIdx.x / row_threads, in_row = threadIdx.x - group * row_threads;
  const int groups = blockDim.x / row_threads;
  constexpr uint32_t XB = XF32 ? 4 : 2;
  const uint32_t bytes[5] = {a.dout ? H * XB : 0u, HAS_NEXT ? H * XB : 0u, HAS_NEXT ? 2u * H : 0u, HAS_Y ? 2u * H : 0u,
                             ELEM && !a.gate_f32 ? 2u * H : 0u};  // (an fp32 gate is read from memory)
  RowPipe<SLOTS> pipe = {};
  if constexpr (PIPE) {
    pipe.slot_bytes = (bytes[0] + bytes[1] + bytes[2] + bytes[3] + bytes[4] + 127u) & ~127u;
    pipe.base = smem_u32(acc) + ((HAS_Y ? 1 : 0) + (HAS_NEXT ? 1 : 0)) * NV * 32 * blockDim.x +
                group * SLOTS * pipe.slot_bytes;
    pipe.bars = smem_u32(&s_bar[group][0]);
    if (in_row < SLOTS) mbar_init(pipe.bars + 8 * in_row, 1);
    if (threadIdx.x == 0) s_abort = 0;
    mbar_fence_init();
    __syncthreads();
  }
  griddep_launch_dependents();
  griddep_wait();
  auto issue = [&](long long row, int slot) {
    const char* const src[5] = {a.dout ? static_cast<const char*>(row_of(a.dout, row, H, XF32)) : nullptr,
                                HAS_NEXT ? static_cast<const char*>(row_of(a.out, row, H, XF32)) : nullptr,
                                HAS_NEXT ? static_cast<const char*>(row_of(a.dnext, row, H, 0)) : nullptr,
                                HAS_Y ? static_cast<const char*>(row_of(a.y, row, H, 0)) : nullptr,
                                ELEM && !a.gate_f32 ? static_cast<const char*>(row_of(a.gate, row, H, 0)) : nullptr};
    pipe_issue(pipe.base + slot * pipe.slot_bytes, pipe.bars + 8 * slot, src, bytes);
  };
  int phase = 0;
  auto col = [&](int j) { return 8 * (in_row + j * row_threads); };
  constexpr int ACC = (HAS_Y ? 1 : 0) + (HAS_NEXT ? 1 : 0);
#pragma unroll
  for (int k = 0; k < ACC * NV * 2; ++k) acc[k * blockDim.x + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto accumulate = [&](int which, int j, const F8& p, const F8& q) {  // += p q
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4* at = acc + ((which * NV + j) * 2 + h) * blockDim.x + threadIdx.x;
      float4 v = *at;
      v.x += p.v[4 * h] * q.v[4 * h];
      v.y += p.v[4 * h + 1] * q.v[4 * h + 1];
      v.z += p.v[4 * h + 2] * q.v[4 * h + 2];
      v.w += p.v[4 * h + 3] * q.v[4 * h + 3];
      *at = v;
    }
  };

  const long long stride = static_cast<long long>(gridDim.x) * groups;
  long long t = static_cast<long long>(blockIdx.x) * groups + group;
  if (PIPE && in_row == 0)
    for (int i = 0; i < SLOTS; ++i)
      if (t + i * stride < a.load_T) issue(t + i * stride, i);
  for (; t < a.T; t += stride) {
    Raw<XF32> dout[NV], out[NV];
    Raw<false> dnext[NV], y[NV], gates[ELEM && PIPE ? NV : 1];
    if constexpr (PIPE) {
      const bool here = mbar_wait(pipe.bar(), pipe.phase, &s_abort);
      uint32_t slot = pipe.slot();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        dout[j] = a.dout ? read_slot<XF32>(slot, col(j), H) : raw_zero<XF32>();
        if constexpr (HAS_NEXT) {
          out[j] = read_slot<XF32>(slot + bytes[0], col(j), H);
          dnext[j] = read_slot<false>(slot + bytes[0] + bytes[1], col(j), H);
        }
        if constexpr (HAS_Y) y[j] = read_slot<false>(slot + bytes[0] + bytes[1] + bytes[2], col(j), H);
        if constexpr (ELEM)
          if (!a.gate_f32) gates[j] = read_slot<false>(slot + bytes[0] + bytes[1] + bytes[2] + bytes[3], col(j), H);
      }
      if (!group_all(here, row_threads, group)) {  // (also: every read of the slot is done)
        pipe_drain(pipe, t, stride, a.load_T);
#pragma unroll 1
        for (; t < a.T; t += stride) {
          spoil_row<XF32>(a.dx, t, H, in_row, row_threads);
          if constexpr (HAS_Y) {
            spoil_row<false>(a.dy, t, H, in_row, row_threads);
            const int per_row = ELEM ? H : a.gate_kind == MOE_GATE_TOKEN ? 1 : 0;
            if (a.gate_f32) spoil_row<true>(a.dgate, t, per_row, in_row, row_threads);
            else spoil_row<false>(a.dgate, t, per_row, in_row, row_threads);
          }
        }
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll 1
        for (int k = 0; k < ACC * NV * 2; ++k) acc[k * blockDim.x + threadIdx.x] = make_float4(nan, nan, nan, nan);
        break;
      }
      if (in_row == 0 && t + SLOTS * stride < a.load_T) issue(t + SLOTS * stride, pipe.at);
      pipe.next();
    }
#pragma unroll
    for (int j = 0; j < NV && !PIPE; ++j) {
      dout[j] = a.dout ? load_raw<XF32>(row_of(a.dout, t, H, XF32), col(j), H, full) : raw_zero<XF32>();
      if constexpr (HAS_NEXT) {
        dnext[j] = load_raw<false>(row_of(a.dnext, t, H, 0), col(j), H, full);
        out[j] = load_raw<XF32>(row_of(a.out, t, H, XF32), col(j), H, full);
      }
      if constexpr (HAS_Y) y[j] = load_raw<false>(row_of(a.y, t, H, 0), col(j), H, full);
    }
    const float r = HAS_Y ? a.rstd[t] : 0.f;
    const float r2 = HAS_NEXT ? a.rstd2[t] : 0.f;
    Gate gate = {1.0f, 1.0f};
    if constexpr (HAS_Y && !ELEM)
      if (a.gate_kind == MOE_GATE_TOKEN) gate = gate_of(load_scalar(a.gate, t, a.gate_f32), a.sigmoid);
    auto element_gate = [&](int j) {
      return PIPE && !a.gate_f32 ? widen(gates[ELEM && PIPE ? j : 0])
                                 : load_either(row_of(a.gate, t, H, a.gate_f32), a.gate_f32, col(j), H, full);
    };

    // S1, S2, S3 (a gate per token stays outside of them), and what needs none
    // of them: dw2, and d without its last term, which is kept in fp32 with w
    constexpr int N = HAS_Y && HAS_NEXT ? 3 : 1, S1 = 0, S2 = HAS_NEXT ? 1 : 0, S3 = 2;
    float sum[N] = {};
    F8 d[NV], w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      d[j] = widen(dout[j]);
      F8 o;
      if constexpr (HAS_NEXT) {
        o = widen(out[j]);
        const F8 w2 = load_weight(a.w2, a.w_f32, a.offset, col(j), H, full);
        F8 dn = widen(dnext[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dn.v[i] *= r2;
          const float e = w2.v[i] * dn.v[i];
          sum[S1] += e * o.v[i];
          d[j].v[i] += e;
        }
        accumulate(HAS_Y ? 1 : 0, j, dn, o);
      }
      if constexpr (HAS_Y) {
        const F8 f = widen(y[j]);
        w[j] = load_weight(a.w, a.w_f32, a.offset, col(j), H, full);
        F8 g;
        if constexpr (ELEM) g = element_gate(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e = w[j].v[i] * f.v[i];
          if constexpr (ELEM) e *= gate_of(g.v[i], a.sigmoid).s;
          sum[S2] += e * d[j].v[i];
          if constexpr (HAS_NEXT) sum[S3] += e * o.v[i];
        }
      }
    }
    group_sum(sum, red, row_threads, group, phase);
    const float c = HAS_NEXT ? r2 * r2 * (sum[S1] * inv_h) : 0.f;  // S1 has one factor r2 already
    float m = HAS_Y ? sum[N == 3 ? S2 : 0] : 0.f;  // sum of w y d (times s where it is per element)
    if constexpr (N == 3) m -= c * sum[S3];
    const float k = r * r * r * (gate.s * m * inv_h), rs = r * gate.s;
    if constexpr (HAS_Y && !ELEM)
      if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && in_row == 0) {
        const float dg = gate.slope * r * m;
        if (a.gate_f32) static_cast<float*>(a.dgate)[t] = dg;
        else static_cast<uint16_t*>(a.dgate)[t] = static_cast<uint16_t>(pack_bf16x2(dg, 0.f));
      }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (HAS_NEXT) {
        const F8 o = widen(out[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[j].v[i] -= o.v[i] * c;
      }
      F8 dx;
#pragma unroll
      for (int i = 0; i < 8; ++i) dx.v[i] = HAS_Y ? a.residual_scale * d[j].v[i] : d[j].v[i];
      store_raw<XF32>(row_of(a.dx, t, H, XF32), col(j), H, full, narrow<XF32>(dx));
      if constexpr (HAS_Y) {
        const F8 f = widen(y[j]);
        F8 dy, sd;  // sd: r s d
        if constexpr (ELEM) {
          F8 g = element_gate(j);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const Gate gi = gate_of(g.v[i], a.sigmoid);
            const float rd = r * d[j].v[i];
            sd.v[i] = gi.s * rd;
            g.v[i] = gi.slope * (rd * (f.v[i] * w[j].v[i]));
          }
          if (a.dgate) {
            void* dst = row_of(a.dgate, t, H, a.gate_f32);
            if (a.gate_f32) store_raw<true>(dst, col(j), H, full, narrow<true>(g));
            else store_raw<false>(dst, col(j), H, full, narrow<false>(g));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) sd.v[i] = rs * d[j].v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dy.v[i] = w[j].v[i] * sd.v[i] - f.v[i] * k;
        accumulate(0, j, sd, f);
        store_raw<false>(row_of(a.dy, t, H, 0), col(j), H, full, narrow<false>(dy));
      }
    }
  }
  __syncthreads();

  // this CTA's sums: one row of [ACC, H] partials, or the result when it is
  // alone; the groups are added in order
  if (group == 0) {
#pragma unroll
    for (int which = 0; which < ACC; ++which) {
      float* dst = a.partials + (static_cast<long long>(blockIdx.x) * ACC + which) * H;
      if (gridDim.x == 1) dst = which == 0 && HAS_Y ? a.dw : a.dw2;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4* at = acc + ((which * NV + j) * 2 + h) * blockDim.x + threadIdx.x;
          float4 v = at[0];
          for (int g = 1; g < groups; ++g) {
            const float4 u = at[g * row_threads];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
          }
          const int c = col(j) + 4 * h;
          if (full) {
            if (c < H) *reinterpret_cast<float4*>(dst + c) = v;
          } else {
            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (const int at_col = ragged_col(col(j), 4 * h + i); at_col < H) dst[at_col] = f[i];
          }
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

constexpr size_t SMEM_PER_SM = 228 * 1024;

// Vectors a thread: one while there are too few rows to fill the SMs (then the
// latency of one counts) or rows are short or ragged, else two, which keep the
// tensors of a row in 128 registers; four above 8192 values a row, where
// up to 472 bytes a thread spill (4096 x 16384, bf16: before a block 90 us for 60 at the copy
// rate, after one with the next norm 230 for 119; two vectors would be 1024 threads of 64 registers).
struct BackwardShape {
  int nv, row_threads, groups, per_sm, grid;
  bool pipe, third;
};
BackwardShape backward_shape(long long T, int H, bool lean) {
  const int v = vectors(H);
  BackwardShape b = {};
  b.nv = (v <= 32 || T < 4LL * sm_count() || H % 8) && v <= 512 ? 1 : v <= 1024 && H % 8 == 0 ? 2 : 4;
  b.row_threads = threads_of(H, b.nv);
  b.pipe = b.nv > 1 && H % 8 == 0;
  b.groups = T > sm_count() && b.row_threads <= 128 ? 256 / b.row_threads : 1;
  if (b.groups > MAX_GROUPS) b.groups = MAX_GROUPS;
  const int threads = b.row_threads * b.groups;
  // A lean form's row tensors (no element gate, no second norm) fit 80
  // registers, for a third CTA, which pays from a dozen rows a group on (before a
  // block, 16384 x 4096 bf16: 98 -> 89 us; below, its partial sums and the
  // smaller register file cost more: 4096 x 2048 fp32 26 -> 29).
  b.third = lean && b.nv == 2 && threads == 256 && T >= 12LL * b.groups * 3 * sm_count();
  b.per_sm = threads > 256 ? 1 : b.third ? 3 : 512 / threads > 4 ? 4 : 512 / threads;
  const long long need = (T + b.groups - 1) / b.groups, most = static_cast<long long>(sm_count()) * b.per_sm;
  b.grid = static_cast<int>(need < most ? need : most);
  return b;
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT>
size_t slot_bytes(const NormBackwardArgs& a) {
  const size_t row = (a.dout ? (XF32 ? 4 : 2) : 0) + (HAS_NEXT ? (XF32 ? 4 : 2) + 2 : 0) + (HAS_Y ? 2 : 0) +
                     (a.gate_kind == MOE_GATE_ELEMENT && !a.gate_f32 ? 2 : 0);
  return (row * a.H + 127) / 128 * 128;
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT, bool ELEM, int NV, bool PIPE, bool THIRD = false>
cudaError_t backward_launch(const NormBackwardArgs& a, const BackwardShape& b, cudaStream_t s) {
  constexpr int ACC = (HAS_Y ? 1 : 0) + (HAS_NEXT ? 1 : 0);
  auto kernel = norm_backward_kernel<XF32, HAS_Y, HAS_NEXT, ELEM, NV, PIPE, THIRD>;
  const int threads = b.row_threads * b.groups;
  size_t smem = static_cast<size_t>(ACC) * NV * 2 * threads * sizeof(float4);
  if (PIPE) smem += slot_bytes<XF32, HAS_Y, HAS_NEXT>(a) * b.groups * SLOTS;
  if (smem > 32 * 1024) {  // (with the static part, above 48 KiB needs leave)
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
  }
  return launch_dependent(kernel, static_cast<unsigned>(b.grid), threads, smem, s, a, b.row_threads);
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT, bool ELEM>
cudaError_t backward(const NormBackwardArgs& a, cudaStream_t s) {
  constexpr int ACC = (HAS_Y ? 1 : 0) + (HAS_NEXT ? 1 : 0);
  constexpr bool LEAN = !ELEM && !(HAS_Y && HAS_NEXT);
  BackwardShape b = backward_shape(a.T, a.H, LEAN);
  // The slots have to fit beside the sums, if need be with one CTA an SM; else
  // (wide rows) the rows are loaded directly.
  const size_t sums = static_cast<size_t>(ACC) * b.nv * 2 * b.row_threads * b.groups * sizeof(float4);
  const size_t all = sums + slot_bytes<XF32, HAS_Y, HAS_NEXT>(a) * b.groups * SLOTS;
  if (b.pipe && all > SMEM_PER_SM - 3072) b.pipe = false;
  if (b.pipe && all > SMEM_PER_SM / b.per_sm - 3072 && b.grid > sm_count()) b.grid = sm_count();
  if (b.grid > 0) {
    const cudaError_t err = b.nv == 1   ? backward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 1, false>(a, b, s)
                            : b.third   ? backward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 2, true, LEAN>(a, b, s)
                            : b.nv == 2 ? backward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 2, true>(a, b, s)  // fits: H <= 8192
                            : b.pipe    ? backward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 4, true>(a, b, s)
                                        : backward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 4, false>(a, b, s);
    if (err != cudaSuccess || b.grid == 1) return err;
  }
  const int cols = ACC * a.H;
  return launch_dependent(norm_reduce_kernel, (cols + 31) / 32, 1024, 0, s, a.partials, b.grid, cols,
                          HAS_Y ? a.H : 0, a.dw, a.dw2);
}

// The three forms, each with and without a gate per element.
template <bool XF32>
cudaError_t backward_any(const NormBackwardArgs& a, cudaStream_t s) {
  const bool elem = a.gate_kind == MOE_GATE_ELEMENT;
  if (!a.has_y) return backward<XF32, false, true, false>(a, s);
  if (a.has_next) return elem ? backward<XF32, true, true, true>(a, s) : backward<XF32, true, true, false>(a, s);
  return elem ? backward<XF32, true, false, true>(a, s) : backward<XF32, true, false, false>(a, s);
}

}  // namespace

cudaError_t launch_norm_backward(const NormBackwardArgs& a, cudaStream_t s) {
  return a.x_f32 ? backward_any<true>(a, s) : backward_any<false>(a, s);
}

size_t norm_backward_workspace(long long T, int H) {
  const int lean = backward_shape(T, H, true).grid, full = backward_shape(T, H, false).grid;
  return static_cast<size_t>(lean > full ? lean : full) * 2 * H * sizeof(float);  // (whichever form is called)
}

}  // namespace moe
