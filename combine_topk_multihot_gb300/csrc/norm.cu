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
// Nothing is used twice but the weights, so every form is bound by HBM: each
// tensor is read or written once.  A row's values stay in registers between
// the sums and their use.

#include "norm.cuh"

namespace moe {

using namespace norm;

namespace {

// Rows in flight a group: with the weights in registers two; with the weights
// in L1 one, which leaves them the room.
template <int NV>
constexpr int SLOTS_OF = NV <= 2 ? 2 : 1;

// CTAs an SM with rows through shared memory: as many as the registers of the
// form allow (T = 16384, bf16: after a block with the next norm, H = 2048 48 us
// with three, 54 with two, 56 with four; before a block 21 with four, 24 with
// three; of rows of 8192 values 46 with three, 51 with two).
template <bool HAS_Y, bool ELEM, int NV>
constexpr int PIPE_CTAS = ELEM ? 2 : NV == 2 ? (HAS_Y ? 3 : 4) : HAS_Y ? 2 : 3;

// A group of `row_threads` threads takes one row at a time.  With up to two
// vectors a thread the weights stay in registers; else they come from L1 at
// each use.  PIPE: rows arrive through
// shared memory (H a multiple of 8).
template <bool XF32, bool HAS_Y, bool HAS_NEXT, bool ELEM, int NV, bool PIPE>
__global__ void __launch_bounds__(NV == 1 ? 1024 : PIPE ? 256 : 512,
                                  !PIPE ? (NV == 4 && !HAS_Y ? 2 : 1) : PIPE_CTAS<HAS_Y, ELEM, NV>)
    norm_forward_kernel(const NormArgs a, int row_threads) {
  __shared__ float red[2][MAX_WARPS][4];
  constexpr int SLOTS = SLOTS_OF<NV>;
  __shared__ uint64_t s_bar[MAX_GROUPS][SLOTS];
  __shared__ int s_abort;
  extern __shared__ __align__(128) uint8_t s_rows[];
  const int H = a.H;
  const bool full = PIPE || (H & 7) == 0;
  const int group = threadIdx.x / row_threads, in_row = threadIdx.x - group * row_threads;
  const int groups = blockDim.x / row_threads;
  const uint32_t bytes[3] = {HAS_Y ? 2u * H : 0u, H * (XF32 ? 4u : 2u), ELEM && !a.gate_f32 ? 2u * H : 0u};
  RowPipe<SLOTS> pipe = {};
  if constexpr (PIPE) {
    pipe.slot_bytes = (bytes[0] + bytes[1] + bytes[2] + 127u) & ~127u;
    pipe.base = smem_u32(s_rows) + group * SLOTS * pipe.slot_bytes;
    pipe.bars = smem_u32(&s_bar[group][0]);
    if (in_row < SLOTS) mbar_init(pipe.bars + 8 * in_row, 1);
    if (threadIdx.x == 0) s_abort = 0;
    mbar_fence_init();
    __syncthreads();
  }
  griddep_launch_dependents();
  griddep_wait();
  const long long stride = static_cast<long long>(gridDim.x) * groups;
  long long t = static_cast<long long>(blockIdx.x) * groups + group;
  auto issue = [&](long long row, int slot) {
    const char* const src[3] = {HAS_Y ? static_cast<const char*>(row_of(a.y, row, H, 0)) : nullptr,
                                static_cast<const char*>(row_of(a.x, row, H, XF32)),
                                ELEM && !a.gate_f32 ? static_cast<const char*>(row_of(a.gate, row, H, 0)) : nullptr};
    pipe_issue(pipe.base + slot * pipe.slot_bytes, pipe.bars + 8 * slot, src, bytes);
  };
  if (PIPE && in_row == 0)
    for (int i = 0; i < SLOTS; ++i)
      if (t + i * stride < a.load_T) issue(t + i * stride, i);
  const float inv_h = 1.0f / static_cast<float>(H);
  int phase = 0;
  auto col = [&](int j) { return 8 * (in_row + j * row_threads); };
  constexpr bool KEEP = NV <= 2;
  F8 wk[KEEP ? NV : 1] = {}, w2k[KEEP ? NV : 1] = {};
#pragma unroll
  for (int j = 0; KEEP && j < NV; ++j) {
    if constexpr (HAS_Y) wk[j] = load_weight(a.w, a.w_f32, a.offset, col(j), H, full);
    if constexpr (HAS_NEXT) w2k[j] = load_weight(a.w2, a.w_f32, a.offset, col(j), H, full);
  }
  for (; t < a.T; t += stride) {
    Raw<XF32> x[NV];
    Raw<false> y[NV];
    Raw<false> gates[ELEM && PIPE ? NV : 1];  // an fp32 gate is read from memory again: registers
    if constexpr (PIPE) {
      const bool here = mbar_wait(pipe.bar(), pipe.phase, &s_abort);
      const uint32_t slot = pipe.slot();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if constexpr (HAS_Y) y[j] = read_slot<false>(slot, col(j), H);
        x[j] = read_slot<XF32>(slot + bytes[0], col(j), H);
        if constexpr (ELEM)
          if (!a.gate_f32) gates[j] = read_slot<false>(slot + bytes[0] + bytes[1], col(j), H);
      }
      if (!group_all(here, row_threads, group)) {  // (also: every read of the slot is done)
        pipe_drain(pipe, t, stride, a.load_T);
#pragma unroll 1
        for (; t < a.T; t += stride) {
          if (in_row == 0) {
            if (HAS_Y && a.rstd) a.rstd[t] = __uint_as_float(0x7fc00000u);
            if (HAS_NEXT && a.rstd2) a.rstd2[t] = __uint_as_float(0x7fc00000u);
          }
          if constexpr (HAS_Y) spoil_row<XF32>(a.out, t, H, in_row, row_threads);
          if constexpr (HAS_NEXT) spoil_row<false>(a.next, t, H, in_row, row_threads);
        }
        break;
      }
      if (in_row == 0 && t + SLOTS * stride < a.load_T) issue(t + SLOTS * stride, pipe.at);
      pipe.next();
    } else {
      const void* xr = row_of(a.x, t, H, XF32);
      const void* yr = HAS_Y ? row_of(a.y, t, H, 0) : nullptr;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if constexpr (HAS_Y) y[j] = load_raw<false>(yr, col(j), H, full);
        x[j] = load_raw<XF32>(xr, col(j), H, full);
      }
    }
    float sum[1] = {0.f};
    if constexpr (HAS_Y) {
      float s = 1.0f;
      if (!ELEM && a.gate_kind == MOE_GATE_TOKEN) s = gate_of(load_scalar(a.gate, t, a.gate_f32), a.sigmoid).s;
      float ms[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const F8 f = widen(y[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ms[0] += f.v[i] * f.v[i];
      }
      group_sum(ms, red, row_threads, group, phase);
      const float r = 1.0f / sqrtf(ms[0] * inv_h + a.eps);
      if (a.rstd && in_row == 0) a.rstd[t] = r;
      const float sr = s * r;
      void* out = row_of(a.out, t, H, XF32);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const F8 f = widen(y[j]), w = KEEP ? wk[KEEP ? j : 0] : load_weight(a.w, a.w_f32, a.offset, col(j), H, full);
        F8 o = widen(x[j]);
        if constexpr (ELEM) {
          const F8 g = PIPE && !a.gate_f32 ? widen(gates[PIPE ? j : 0])
                                           : load_either(row_of(a.gate, t, H, a.gate_f32), a.gate_f32, col(j), H, full);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            o.v[i] = a.residual_scale * o.v[i] + gate_of(g.v[i], a.sigmoid).s * (f.v[i] * r * w.v[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o.v[i] = a.residual_scale * o.v[i] + f.v[i] * sr * w.v[i];
        }
        x[j] = narrow<XF32>(o);  // the stream as it is held
        store_raw<XF32>(out, col(j), H, full, x[j]);
      }
    }
    if constexpr (HAS_NEXT) {
      // (values past H are zero here: their x, y and products were)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const F8 o = widen(x[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] += o.v[i] * o.v[i];
      }
      group_sum(sum, red, row_threads, group, phase);
      const float r = 1.0f / sqrtf(sum[0] * inv_h + a.eps);
      if (a.rstd2 && in_row == 0) a.rstd2[t] = r;
      void* next = row_of(a.next, t, H, 0);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const F8 w = KEEP ? w2k[KEEP ? j : 0] : load_weight(a.w2, a.w_f32, a.offset, col(j), H, full);
        F8 o = widen(x[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[i] = o.v[i] * r * w.v[i];
        store_raw<false>(next, col(j), H, full, narrow<false>(o));
      }
    }
  }
}

// Vectors a thread.  Each row costs a thread about 100 instructions besides
// its elements' (sums, addresses), so with rows enough to fill the SMs a
// thread takes two vectors, with the weights in registers, or four where a row
// is longer than 4096 (T = 16384, H = 2048, bf16 with the next norm: 64 us with
// one vector, 53 with two, 59 with eight and the weights in L1); with fewer than four rows an SM a row is
// spread over as many threads as it can use: what counts then is the latency
// of one.
struct ForwardShape {
  int nv, row_threads, groups, per_sm;  // (per_sm: of the direct form)
  bool pipe;
};
ForwardShape forward_shape(long long T, int H) {
  const int v = vectors(H);
  ForwardShape f = {};
  const bool direct = T < 4LL * sm_count() || v <= 32 || H % 8;
  f.nv = direct && v <= 1024 ? 1 : v <= 512 ? 2 : 4;
  f.row_threads = threads_of(H, f.nv);
  f.pipe = f.nv > 1 && H % 8 == 0 && f.row_threads <= 256;
  f.groups = !f.pipe ? 1 : 256 / f.row_threads > MAX_GROUPS ? MAX_GROUPS : 256 / f.row_threads;
  f.per_sm = f.row_threads >= 512 ? 2 : 1024 / f.row_threads > 16 ? 16 : 1024 / f.row_threads;
  return f;
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT, bool ELEM, int NV, bool PIPE>
cudaError_t forward_launch(const NormArgs& a, const ForwardShape& f, cudaStream_t s) {
  auto kernel = norm_forward_kernel<XF32, HAS_Y, HAS_NEXT, ELEM, NV, PIPE>;
  long long grid = static_cast<long long>(sm_count()) * (PIPE ? PIPE_CTAS<HAS_Y, ELEM, NV> : f.per_sm);
  const long long need = (a.T + f.groups - 1) / f.groups;
  if (grid > need) grid = need;
  size_t smem = 0;
  if (PIPE) {
    const size_t row = (HAS_Y ? 2 : 0) + (XF32 ? 4 : 2) + (ELEM && !a.gate_f32 ? 2 : 0);
    smem = (row * a.H + 127) / 128 * 128 * f.groups * SLOTS_OF<NV>;
    if (smem > 32 * 1024) {  // (with the static part, above 48 KiB needs leave)
      const cudaError_t err =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (err != cudaSuccess) return err;
    }
  }
  return launch_dependent(kernel, static_cast<unsigned>(grid), f.row_threads * f.groups, smem, s, a, f.row_threads);
}

template <bool XF32, bool HAS_Y, bool HAS_NEXT, bool ELEM>
cudaError_t forward(const NormArgs& a, cudaStream_t s) {
  const ForwardShape f = forward_shape(a.T, a.H);
  if (f.nv == 1) return forward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 1, false>(a, f, s);
  if (!f.pipe) return forward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 4, false>(a, f, s);
  if (f.nv == 2) return forward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 2, true>(a, f, s);
  return forward_launch<XF32, HAS_Y, HAS_NEXT, ELEM, 4, true>(a, f, s);
}

// The three forms, each with and without a gate per element.
template <bool XF32>
cudaError_t forward_any(const NormArgs& a, cudaStream_t s) {
  const bool elem = a.gate_kind == MOE_GATE_ELEMENT;
  if (!a.y) return forward<XF32, false, true, false>(a, s);
  if (a.next) return elem ? forward<XF32, true, true, true>(a, s) : forward<XF32, true, true, false>(a, s);
  return elem ? forward<XF32, true, false, true>(a, s) : forward<XF32, true, false, false>(a, s);
}

// The self-test's limit of the rows that are loaded, for this host thread's launches.
thread_local long long tls_load_rows = -1;

}  // namespace

void selftest_norm_load_rows(long long rows) { tls_load_rows = rows; }
long long norm_load_rows(long long T) { return tls_load_rows >= 0 && tls_load_rows < T ? tls_load_rows : T; }

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return a.x_f32 ? forward_any<true>(a, s) : forward_any<false>(a, s);
}

}  // namespace moe
