// A whole MoE layer for at most 8 tokens, in two launches.
//
//   logits = x R^T;  e_k, w_k: the K largest of a token and their softmax
//   h_k = silu(x Wg[e_k]^T) * (x Wu[e_k]^T)         (rounded to bf16)
//   out = sum_k w_k (h_k W2[e_k]^T)
//
// With so few rows the layer is a stream over the active experts' weights, read
// once: 3 H I numbers each.  The first launch makes the logits, a CTA an expert.
// The second is one persistent cooperative kernel, a CTA an SM, that has one
// grid barrier, between h and the second product:
//   * every CTA picks the experts itself (T K values), so that the weights can be
//     asked for without another launch or barrier;
//   * the active experts' h columns are numbered through and cut into equal runs,
//     one a CTA, and so are the rows of the output: each CTA sums its rows over
//     all active experts, so no partial sums leave it and every order is fixed;
//   * warp 8 asks for the rows of both products in one go, in bulk copies to a
//     ring of shared memory; the second product's rows arrive while h is being
//     finished and while the CTAs meet at the barrier;
//   * warps 0..7 multiply with mma.sync, 16 weight rows (8 gate and their 8 up
//     rows, or 16 rows of W2) by the 8 tokens, each warp a slice of K, joined
//     in shared memory in a fixed order.  A token's column is computed for every
//     expert and used for its own.
//
// Weights are bf16, e4m3 with a scale per 128 x 128, or e2m1 with a scale per 32
// of a row.  For the codes the tokens (and h) are held as the sum of two e4m3 numbers
// in units of a power of two for each 128 values: x = s (hi + lo), hi of 4
// significant bits, lo of the 4 below; exact for bf16 values down to 2^-10 of
// their block's largest, and within 2^-18 of that below it.  So the products of codes
// run on the same instruction, twice, without rounding the activations to 8 bits.

#include "common.cuh"
#include "fp4.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int TOK = FEW_TOKENS;        // 8: one mma operand
constexpr int MAX_K = FEW_TOP_K;       // 16
constexpr int PAIRS = TOK * MAX_K;
constexpr int CONSUMERS = 8;           // warps
constexpr int THREADS = 32 * (CONSUMERS + 1);
constexpr int MAX_STAGES = 16;
constexpr int SMEM_LIMIT = 232448;

template <int FMT>
struct Form {
  // bytes of a row in a stage, and from row to row: 64 (bf16, e4m3: a quarter
  // warp reads 16 bytes of each of two rows' 64) or 16 more (e2m1: a warp reads
  // 16 bytes of each of eight rows) keep the rows' banks apart
  static constexpr int CHUNK = FMT == FEW_FP4 ? 512 : 1024;
  static constexpr int PITCH = FMT == FEW_FP4 ? CHUNK + 16 : CHUNK + 64;
  static constexpr int SCALES = FMT == FEW_BF16 ? 0 : 16 * 32;  // 8 words of each row: a word per 128 columns
  static constexpr int STAGE = 16 * PITCH + SCALES;
  __host__ __device__ static constexpr int row_bytes(int K) { return FMT == FEW_BF16 ? 2 * K : FMT == FEW_FP8 ? K : K / 2; }
};

__host__ __device__ constexpr int token_pitch(int K) { return 2 * K + 64; }

struct Smem {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  int abort;
  int ok;
  int active;
  int expert[PAIRS];         // ascending
  int first[PAIRS + 1];      // pairs before each
  uint8_t tokens[PAIRS];     // a bit for each token
  float weight[PAIRS][TOK];
  int chosen[TOK][MAX_K];
  float prob[TOK][MAX_K];
  int mask[1024];            // tokens of each expert, then its place in the list
  float part[2][CONSUMERS][4][32];
};

struct FewArgs {
  const uint16_t* x;
  const float* logits;       // [T, E]; NULL: the routing is given
  const int64_t* topk_idx;
  const float* topk_probs;
  const uint8_t *W1, *W2;
  const void *S1, *S2;
  int T, E, K, H, I;
  int stages, cap;           // ring stages; rows of h that shared memory holds
  int region;                // bytes of the tokens' rows and their scales
  uint16_t* h;               // [T K, I]
  unsigned* barrier;
  uint16_t* out;
  int64_t* idx_out;
  float* probs_out;
  int* status;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * CONSUMERS) : "memory"); }

__device__ __forceinline__ void mma_bf16_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- logits
// A CTA an expert: its row of the router against every token, in fp32.  The
// first CTA also clears the other kernel's barrier.
constexpr int LOGIT_THREADS = 128;
template <bool F32>
__global__ void __launch_bounds__(LOGIT_THREADS) few_logits_kernel(const uint16_t* __restrict__ x, const void* __restrict__ router,
                                                                   int T, int E, int H, float* __restrict__ logits,
                                                                   unsigned* __restrict__ barrier) {
  __shared__ float s_sum[LOGIT_THREADS / 32][TOK];
  griddep_launch_dependents();
  griddep_wait();
  const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (e == 0 && threadIdx.x == 0) *barrier = 0u;
  if (logits == nullptr) return;
  float acc[TOK] = {};
  for (int k = threadIdx.x * 8; k < H; k += LOGIT_THREADS * 8) {
    float r[8];
    if constexpr (F32) {
      const float4* at = reinterpret_cast<const float4*>(static_cast<const float*>(router) + static_cast<long long>(e) * H + k);
      const float4 a = __ldg(at), b = __ldg(at + 1);
      r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    } else {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(router) + static_cast<long long>(e) * H + k));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) r[2 * i] = bf16_lo(w[i]), r[2 * i + 1] = bf16_hi(w[i]);
    }
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      if (t < T) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(x + static_cast<long long>(t) * H + k));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t] = fmaf(bf16_hi(w[i]), r[2 * i + 1], fmaf(bf16_lo(w[i]), r[2 * i], acc[t]));
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TOK; ++t)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(FULL_MASK, acc[t], o);
  if (lane == 0)
#pragma unroll
    for (int t = 0; t < TOK; ++t) s_sum[warp][t] = acc[t];
  __syncthreads();
  if (threadIdx.x < T) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < LOGIT_THREADS / 32; ++w) v += s_sum[w][threadIdx.x];
    logits[static_cast<long long>(threadIdx.x) * E + e] = v;
  }
}

// ---------------------------------------------------------------- routing
// An order-preserving map of floats to integers above 0 (NaN as -infinity).
__device__ __forceinline__ uint32_t sort_key(float v) {
  const uint32_t u = __float_as_uint(v != v ? -INFINITY : v);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

// One token's K largest logits by one warp, in descending order, equal ones by
// ascending index, as moe_router_topk has them, and their softmax.  A lane keeps
// the best of its logits and looks again only when that was taken.
__device__ __forceinline__ void pick_experts(const float* logits, uint32_t* keys, int E, int K, int lane, int* chosen, float* prob) {
  uint32_t best = 0;
  int at = 0x7fffffff;
  for (int e = lane; e < E; e += 32) {
    const uint32_t k = sort_key(__ldcg(logits + e));
    keys[e] = k;
    if (k > best) best = k, at = e;
  }
  int mine = 0;
  float l = -INFINITY;
  for (int k = 0; k < K; ++k) {
    const uint32_t top = __reduce_max_sync(FULL_MASK, best);
    const int e = static_cast<int>(__reduce_min_sync(FULL_MASK, best == top ? static_cast<uint32_t>(at) : 0x7fffffffu));
    if (lane == k) mine = e, l = of_key(top);
    if (at == e) {
      keys[e] = 0;
      best = 0;
      at = 0x7fffffff;
      for (int o = lane; o < E; o += 32)
        if (keys[o] > best) best = keys[o], at = o;
    }
    __syncwarp();
  }
  const float l0 = __shfl_sync(FULL_MASK, l, 0);
  const float ex = lane < K ? expf(l - l0) : 0.f;
  float sum = ex;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
  if (lane < K) chosen[lane] = mine, prob[lane] = ex / sum;
}

// ---------------------------------------------------------------- rows of tokens
// `rows` rows of K bf16 values (row r from src + r K) into shared memory, as the
// products read them, with a scale for each 128 of a row.  All consumers.
template <int FMT>
__device__ __forceinline__ void stage_rows(const uint16_t* src, int rows, int K, uint8_t* dst, float* scales) {
  const int pitch = token_pitch(K);
  if constexpr (FMT == FEW_BF16) {
    const int nv = K >> 3;
    for (int i = threadIdx.x; i < rows * nv; i += 32 * CONSUMERS) {
      const int r = i / nv, v = i - r * nv;
      *reinterpret_cast<uint4*>(dst + r * pitch + v * 16) = __ldcg(reinterpret_cast<const uint4*>(src + static_cast<long long>(r) * K) + v);
    }
  } else {
    const int kb = K >> 7;
    // 16 threads a block of 128; two blocks at a time, so that their loads overlap
    for (int u0 = threadIdx.x >> 4; u0 < rows * kb; u0 += 4 * CONSUMERS) {
      uint4 q[2];
      uint32_t top[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int u = u0 + j * 2 * CONSUMERS;
        q[j] = u < rows * kb ? __ldcg(reinterpret_cast<const uint4*>(src + static_cast<long long>(u) * 128) + (threadIdx.x & 15))
                             : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned half = 0xffffu << (threadIdx.x & 16);
        top[j] = bf16x2_abs_max(bf16x2_abs_max(q[j].x, q[j].y), bf16x2_abs_max(q[j].z, q[j].w));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top[j] = bf16x2_abs_max(top[j], __shfl_xor_sync(half, top[j], o));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int u = u0 + j * 2 * CONSUMERS;
        if (u >= rows * kb) break;
        const int r = u / kb, b = u - r * kb;
        const uint32_t bits = __float_as_uint(max_nan(bf16_lo(top[j]), bf16_hi(top[j])));
        const bool bad = bits >= 0x7f800000u;
        // s = 2^(floor(log2 amax) - 7), at least 2^-126: values up to 256
        const uint32_t e = bits >> 23 > 8u ? (bits >> 23) - 7u : 1u;
        const float inv = bad ? 0.f : __uint_as_float((254u - e) << 23);
        const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bad ? 0.f : bf16_lo(w[i]) * inv, v[2 * i + 1] = bad ? 0.f : bf16_hi(w[i]) * inv;
        // the order in which the weights' codes meet them: as they come, or (e2m1) the even ones first
        constexpr int P[8] = {0, FMT == FEW_FP4 ? 2 : 1, FMT == FEW_FP4 ? 4 : 2, FMT == FEW_FP4 ? 6 : 3,
                              FMT == FEW_FP4 ? 1 : 4, FMT == FEW_FP4 ? 3 : 5, FMT == FEW_FP4 ? 5 : 6, 7};
        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = v[P[2 * i]], c = v[P[2 * i + 1]];
          const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(make_float2(a, c), __NV_SATFINITE, __NV_E4M3);
          const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
          const __nv_fp8x2_storage_t l = __nv_cvt_float2_to_fp8x2(make_float2(a - f.x, c - f.y), __NV_SATFINITE, __NV_E4M3);
          hi[i >> 1] |= static_cast<uint32_t>(h) << (16 * (i & 1));
          lo[i >> 1] |= static_cast<uint32_t>(l) << (16 * (i & 1));
        }
        const int c0 = (threadIdx.x & 15) * 8;  // of the block
        uint8_t* at = dst + r * pitch + b * 256;
        if constexpr (FMT == FEW_FP8) {  // of each 64: their hi codes, then their lo codes
          *reinterpret_cast<uint2*>(at + (c0 >> 6) * 128 + (c0 & 63)) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(at + (c0 >> 6) * 128 + 64 + (c0 & 63)) = make_uint2(lo[0], lo[1]);
        } else {  // a lane's eight of each 32, hi and lo
          *reinterpret_cast<uint4*>(at + c0 * 2) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
        }
        // (e2m1 codes are multiplied as 2^-6 times their values)
        if ((threadIdx.x & 15) == 0)
          scales[u] = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float((FMT == FEW_FP4 ? e + 6u : e) << 23);
      }
    }
  }
}

// ---------------------------------------------------------------- products
// d[16 rows x 8 tokens] += a stage's rows times the tokens' rows, this warp's
// pieces of 64 bytes of a weight row.  `token`: the row of token lane / 4 (0:
// none, zeros), s0 and s1 the scales of tokens 2 (lane % 4) and the next; `byte0`: where in the weight row the stage begins.
template <int FMT>
__device__ __forceinline__ void multiply(float (&d)[4], uint32_t stage, int bytes, int byte0, int warp, int lane, uint32_t token,
                                         const float* s0, const float* s1) {
  using F = Form<FMT>;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t lo = stage + g * F::PITCH, hi = lo + 8 * F::PITCH;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < F::CHUNK / 64 / CONSUMERS; ++i) {
    const int at = (warp + CONSUMERS * i) * 64;
    if (at >= bytes) break;
    if constexpr (FMT == FEW_BF16) {
      const uint4 a = lds128(lo + at + 16 * t), c = lds128(hi + at + 16 * t);
      const uint4 b = token ? lds128(token + byte0 + at + 16 * t) : zero;
      mma_bf16_16x8x16(d, a.x, c.x, a.y, c.y, b.x, b.y);
      mma_bf16_16x8x16(d, a.z, c.z, a.w, c.w, b.z, b.w);
    } else if constexpr (FMT == FEW_FP8) {
      const uint4 a = lds128(lo + at + 16 * t), c = lds128(hi + at + 16 * t);
      const uint32_t from = token + 2 * (byte0 + at) + 16 * t;
      const uint4 bh = token ? lds128(from) : zero, bl = token ? lds128(from + 64) : zero;
      float p[4] = {0.f, 0.f, 0.f, 0.f};
      mma_e4m3_16x8x32(p, a.x, c.x, a.y, c.y, bh.x, bh.y);
      mma_e4m3_16x8x32(p, a.z, c.z, a.w, c.w, bh.z, bh.w);
      mma_e4m3_16x8x32(p, a.x, c.x, a.y, c.y, bl.x, bl.y);
      mma_e4m3_16x8x32(p, a.z, c.z, a.w, c.w, bl.z, bl.w);
      const int kb = (byte0 + at) >> 7;
      const uint32_t sc = stage + 16 * F::PITCH + (at >> 7) * 4;
      const float w0 = __uint_as_float(lds32(sc + g * 32)), w1 = __uint_as_float(lds32(sc + (g + 8) * 32));
      const float x0 = s0[kb], x1 = s1[kb];
      d[0] = fmaf(p[0], w0 * x0, d[0]);
      d[1] = fmaf(p[1], w0 * x1, d[1]);
      d[2] = fmaf(p[2], w1 * x0, d[2]);
      d[3] = fmaf(p[3], w1 * x1, d[3]);
    } else {
      const int kb = (byte0 + at) >> 6;
      const uint32_t sc = stage + 16 * F::PITCH + (at >> 6) * 4;
      const uint32_t e0 = lds32(sc + g * 32), e1 = lds32(sc + (g + 8) * 32);
      float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = lds32(lo + at + 16 * j + 4 * t), c = lds32(hi + at + 16 * j + 4 * t);
        const uint4 b = token ? lds128(token + kb * 256 + j * 64 + 16 * t) : zero;
        const uint32_t ae = e4m3_of_even(a), ao = e4m3_of_odd(a), ce = e4m3_of_even(c), co = e4m3_of_odd(c);
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        mma_e4m3_16x8x32(p, ae, ce, ao, co, b.x, b.y);
        mma_e4m3_16x8x32(p, ae, ce, ao, co, b.z, b.w);
        const float w0 = e8m0_value((e0 >> (8 * j)) & 255u), w1 = e8m0_value((e1 >> (8 * j)) & 255u);
        q[0] = fmaf(p[0], w0, q[0]);
        q[1] = fmaf(p[1], w0, q[1]);
        q[2] = fmaf(p[2], w1, q[2]);
        q[3] = fmaf(p[3], w1, q[3]);
      }
      const float x0 = s0[kb], x1 = s1[kb];
      d[0] = fmaf(q[0], x0, d[0]);
      d[1] = fmaf(q[1], x1, d[1]);
      d[2] = fmaf(q[2], x0, d[2]);
      d[3] = fmaf(q[3], x1, d[3]);
    }
  }
}

// ---------------------------------------------------------------- the layer
template <int FMT>
__global__ void __launch_bounds__(THREADS, 1) few_layer_kernel(const FewArgs args) {
  using F = Form<FMT>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* region = smem + args.stages * F::STAGE;
  Smem& s = *reinterpret_cast<Smem*>(region + args.region);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = args.T, E = args.E, K = args.K, H = args.H, I = args.I, stages = args.stages;
  volatile int* abort_flag = &s.abort;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(smem_u32(&s.full[i]), FMT == FEW_BF16 ? 1 : 33);
      mbar_init(smem_u32(&s.empty[i]), CONSUMERS);
    }
    s.abort = 0;
    s.ok = 1;
    mbar_fence_init();
  }
  for (int e = threadIdx.x; e < E; e += THREADS) s.mask[e] = 0;
  for (int i = threadIdx.x; i < PAIRS * TOK; i += THREADS) s.weight[0][i] = 0.f;
  griddep_wait();
  __syncthreads();

  // the routing: a warp a token
  if (warp < T) {
    if (args.logits) {  // (the ring is not in use yet)
      pick_experts(args.logits + static_cast<long long>(warp) * E, reinterpret_cast<uint32_t*>(smem) + warp * 1024, E, K, lane,
                   s.chosen[warp], s.prob[warp]);
    } else if (lane < K) {
      long long e = args.topk_idx[warp * K + lane];
      if (e < -1 || e >= E) {
        if (blockIdx.x == 0) report(args.status, MOE_DEVERR_BAD_INDEX);
        e = -1;
      }
      s.chosen[warp][lane] = static_cast<int>(e);
      s.prob[warp][lane] = args.topk_probs[warp * K + lane];
    }
    fence_proxy_async_shared();  // the bulk copies to the ring come after its use here
    __syncwarp();
    if (lane < K) {
      const int e = s.chosen[warp][lane];
      if (e >= 0) atomicOr(&s.mask[e], 1 << warp);
      if (blockIdx.x == 0 && args.idx_out) {
        args.idx_out[warp * K + lane] = e;
        args.probs_out[warp * K + lane] = s.prob[warp][lane];
      }
    }
  }
  __syncthreads();
  if (warp == 0) {  // the experts with tokens, ascending
    int n = 0, pairs = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int m = e0 + lane < E ? s.mask[e0 + lane] : 0;
      const unsigned any = __ballot_sync(FULL_MASK, m != 0);
      const int mine = __popc(m);
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, upto, o);
        if (lane >= o) upto += v;
      }
      if (m) {
        const int a = n + __popc(any & ((1u << lane) - 1u));
        s.expert[a] = e0 + lane;
        s.tokens[a] = static_cast<uint8_t>(m);
        s.first[a] = pairs + upto - mine;
        s.mask[e0 + lane] = a;
      }
      n += __popc(any);
      pairs += __shfl_sync(FULL_MASK, upto, 31);
    }
    if (lane == 0) {
      s.active = n;
      s.first[n] = pairs;
    }
    __syncwarp();
    if (lane < T)  // of an expert that is named twice the last slot counts
      for (int k = 0; k < K; ++k)
        if (s.chosen[lane][k] >= 0) s.weight[s.mask[s.chosen[lane][k]]][lane] = s.prob[lane][k];
  }
  __syncthreads();

  const int active = s.active;
  const long long G = gridDim.x, b = blockIdx.x;
  const long long cols = static_cast<long long>(active) * I;
  const long long f0 = b * cols / G, f1 = (b + 1) * cols / G;   // this CTA's columns of h
  const int r0 = static_cast<int>(b * H / G), r1 = static_cast<int>((b + 1) * H / G);  // and rows of the output
  const int bytes1 = F::row_bytes(H), bytes2 = F::row_bytes(I);
  const int chunks1 = (bytes1 + F::CHUNK - 1) / F::CHUNK, chunks2 = (bytes2 + F::CHUNK - 1) / F::CHUNK;
  const uint32_t ring = smem_u32(smem);

  if (warp == CONSUMERS) {
    // ================= all weights, in the order of their use =================
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    // rows of a stage: lane r's from `row` (NULL: none), n in all; scale words from `scale_of(r, word)`
    auto load = [&](const uint8_t* row, int n, int row_bytes, int c, auto scale_of) {
      const bool ready = mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, abort_flag);
      if (!__all_sync(FULL_MASK, ready)) return false;
      const uint32_t full = smem_u32(&s.full[stage]), dst = ring + stage * F::STAGE;
      const int bytes = min(F::CHUNK, row_bytes - c * F::CHUNK);
      if (lane == 0) mbar_arrive_expect_tx(full, n * bytes);
      __syncwarp();
      if (row) bulk_load(dst + lane * F::PITCH, row + c * F::CHUNK, bytes, full);
      if constexpr (FMT != FEW_BF16) {
        const int words = bytes / (FMT == FEW_FP8 ? 128 : 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (lane >> 3) + 4 * i, w = lane & 7;
          const bool there = __shfl_sync(FULL_MASK, row != nullptr ? 1 : 0, r) != 0;
          if (there && w < words) cp_async_4(dst + 16 * F::PITCH + r * 32 + w * 4, scale_of(r, c * (F::CHUNK / (FMT == FEW_FP8 ? 128 : 64)) + w));
        }
        cp_async_mbar_arrive_noinc(full);
      }
      ++issued;
      if (++stage == stages) { stage = 0; phase ^= 1u; }
      return true;
    };
    // the four bytes of scales of row `row` of matrix `e` ([rows, K]) and columns [128 kb, 128 kb + 128)
    auto scale_at = [&](const void* base, int e, int rows, int K, int row, int kb) -> const void* {
      const int kbs = K >> 7;
      if constexpr (FMT == FEW_FP8)
        return static_cast<const float*>(base) + (static_cast<long long>(e) * (rows >> 7) + (row >> 7)) * kbs + kb;
      return static_cast<const uint8_t*>(base) + static_cast<long long>(e) * (rows >> 7) * kbs * SCALE_TILE + scale_word(row, kb, kbs);
    };
    for (long long f = f0; f < f1 && ok;) {
      const int a = static_cast<int>(f / I), j0 = static_cast<int>(f - static_cast<long long>(a) * I);
      const int n = static_cast<int>(min(8ll, min(f1 - f, static_cast<long long>(I - j0))));
      const int e = s.expert[a];
      const int i = lane & 7;
      const uint8_t* row = lane < 16 && i < n
                               ? args.W1 + (static_cast<long long>(e) * 2 * I + (lane < 8 ? 0 : I) + j0 + i) * bytes1 : nullptr;
      for (int c = 0; c < chunks1 && ok; ++c)
        ok = load(row, 2 * n, bytes1, c,
                  [&](int r, int kb) { return scale_at(args.S1, e, 2 * I, H, (r < 8 ? 0 : I) + j0 + (r & 7), kb); });
      f += n;
    }
    for (int m0 = r0; m0 < r1 && ok; m0 += 16) {
      const int n = min(16, r1 - m0);
      for (int a = 0; a < active && ok; ++a) {
        const int e = s.expert[a];
        const uint8_t* row = lane < n ? args.W2 + (static_cast<long long>(e) * H + m0 + lane) * bytes2 : nullptr;
        for (int c = 0; c < chunks2 && ok; ++c)
          ok = load(row, n, bytes2, c, [&](int r, int kb) { return scale_at(args.S2, e, H, I, m0 + r, kb); });
      }
    }
    if (!ok) {  // wait for the copies of the last (up to `stages`) issued stages
      if (FMT != FEW_BF16) cp_async_wait_all();
      if (lane == 0) {
        for (int i = 0; i < stages && i < issued; ++i) {
          if (--stage < 0) { stage = stages - 1; phase ^= 1u; }
          mbar_wait_drain(smem_u32(&s.full[stage]), phase);
        }
      }
      __syncwarp();
    }
  } else {
    // ================= products =================
    const int g = lane >> 2, t = lane & 3;
    int stage = 0;
    uint32_t phase = 0;
    int par = 0;
    bool ok = true;
    float* s_scale = reinterpret_cast<float*>(region + T * token_pitch(H));
    stage_rows<FMT>(args.x, T, H, region, s_scale);
    consumers_sync();
    const uint32_t rows_u32 = smem_u32(region);
    auto next = [&](float (&d)[4], int row_bytes, int c, uint32_t token, const float* s0, const float* s1) {
      const bool ready = mbar_wait(smem_u32(&s.full[stage]), phase, abort_flag);
      if (!__all_sync(FULL_MASK, ready)) return false;
      multiply<FMT>(d, ring + stage * F::STAGE, min(F::CHUNK, row_bytes - c * F::CHUNK), c * F::CHUNK, warp, lane, token, s0, s1);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.empty[stage]));
      if (++stage == stages) { stage = 0; phase ^= 1u; }
      return true;
    };
    {
      const uint32_t token = g < T ? rows_u32 + g * token_pitch(H) : 0u;
      const float* s0 = s_scale + min(2 * t, T - 1) * (H >> 7);
      const float* s1 = s_scale + min(2 * t + 1, T - 1) * (H >> 7);
      for (long long f = f0; f < f1 && ok;) {
        const int a = static_cast<int>(f / I), j0 = static_cast<int>(f - static_cast<long long>(a) * I);
        const int n = static_cast<int>(min(8ll, min(f1 - f, static_cast<long long>(I - j0))));
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < chunks1 && ok; ++c) ok = next(d, bytes1, c, token, s0, s1);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) s.part[par][warp][i][lane] = d[i];
        // one meeting a tile: this parity's sums are written again after the next
        // tile's, which follows their reading here
        consumers_sync();
        if (threadIdx.x < 64) {
          const int j = threadIdx.x >> 3, tok = threadIdx.x & 7;
          const int m = s.tokens[a];
          if (j < n && ((m >> tok) & 1)) {
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < CONSUMERS; ++w) {
              gate += s.part[par][w][tok & 1][j * 4 + (tok >> 1)];
              up += s.part[par][w][2 + (tok & 1)][j * 4 + (tok >> 1)];
            }
            const int pair = s.first[a] + __popc(m & ((1 << tok) - 1));
            args.h[static_cast<long long>(pair) * I + j0 + j] =
                __bfloat16_as_ushort(__float2bfloat16_rn(gate / (1.0f + expf(-gate)) * up));
          }
        }
        par ^= 1;
        f += n;
      }
    }
    // h is whole once every CTA has been here (one whose waits ran out does not
    // come, so that no other takes its part of h for a result)
    if (!ok) *abort_flag = 1;
    __threadfence();
    consumers_sync();
    if (threadIdx.x == 0) {
      int met = !*abort_flag;
      if (met) {
        atomicAdd(args.barrier, 1u);
        const unsigned long long t0 = global_timer_ns();
        while (*reinterpret_cast<volatile unsigned*>(args.barrier) < gridDim.x) {
          if (global_timer_ns() - t0 > WAIT_LIMIT_NS) {
            met = 0;
            break;
          }
        }
      }
      __threadfence();
      s.ok = met;
      if (!met) *abort_flag = 1;
    }
    consumers_sync();
    ok = ok && s.ok && !*abort_flag;

    const int hp = token_pitch(I);
    float* h_scale = reinterpret_cast<float*>(region + args.cap * hp);
    int m0 = r0;
    for (; m0 < r1 && ok; m0 += 16) {
      const int n = min(16, r1 - m0);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      int sa = 0, sb = 0;  // experts whose rows of h are in shared memory
      if (m0 > r0 && s.first[active] <= args.cap) sb = active;  // all, from the 16 rows before
      for (int a = 0; a < active && ok; ++a) {
        if (a == sb) {
          sa = a;
          while (sb < active && s.first[sb + 1] - s.first[sa] <= args.cap) ++sb;
          consumers_sync();
          stage_rows<FMT>(args.h + static_cast<long long>(s.first[sa]) * I, s.first[sb] - s.first[sa], I, region, h_scale);
          consumers_sync();
        }
        const int m = s.tokens[a], at = s.first[a] - s.first[sa];
        auto place = [&](int tok) { return at + __popc(m & ((1 << tok) - 1)); };
        const uint32_t token = (m >> g) & 1 ? rows_u32 + place(g) * hp : 0u;
        const bool u0 = (m >> (2 * t)) & 1, u1 = (m >> (2 * t + 1)) & 1;
        const float* s0 = h_scale + (u0 ? place(2 * t) : at) * (I >> 7);
        const float* s1 = h_scale + (u1 ? place(2 * t + 1) : at) * (I >> 7);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < chunks2 && ok; ++c) ok = next(d, bytes2, c, token, s0, s1);
        if (u0) {
          const float w = s.weight[a][2 * t];
          acc[0] = fmaf(w, d[0], acc[0]);
          acc[2] = fmaf(w, d[2], acc[2]);
        }
        if (u1) {
          const float w = s.weight[a][2 * t + 1];
          acc[1] = fmaf(w, d[1], acc[1]);
          acc[3] = fmaf(w, d[3], acc[3]);
        }
      }
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) s.part[par][warp][i][lane] = acc[i];
      consumers_sync();
      if (threadIdx.x < 128) {  // rows fastest
        const int r = threadIdx.x & 15, tok = threadIdx.x >> 4;
        if (r < n && tok < T) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < CONSUMERS; ++w) v += s.part[par][w][(r >> 3) * 2 + (tok & 1)][(r & 7) * 4 + (tok >> 1)];
          args.out[static_cast<long long>(tok) * H + m0 + r] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
      }
      par ^= 1;
    }
    if (!ok) *abort_flag = 1;
  }
  __syncthreads();
  if (s.abort) {  // a wait ran out: this CTA's rows are no result
    for (int i = threadIdx.x; i < T * (r1 - r0); i += THREADS)
      args.out[static_cast<long long>(i / (r1 - r0)) * H + r0 + i % (r1 - r0)] = 0x7fc0;
    if (threadIdx.x == 0) report(args.status, MOE_DEVERR_TIMEOUT);
  }
}

constexpr int FIXED = sizeof(Smem) + 128;

template <int FMT>
bool plan(FewArgs& g, size_t* smem) {
  const int x_row = token_pitch(g.H) + 4 * (g.H / 128), h_row = token_pitch(g.I) + 4 * (g.I / 128);
  // all rows of h where they fit in 64 KiB, else as many as are there for the tokens
  const int need = g.T * (x_row > h_row ? x_row : h_row);
  int room = g.T * g.K * h_row;
  if (room > 64 * 1024) room = 64 * 1024;
  if (room < need) room = need;
  g.cap = room / h_row < g.T * g.K ? room / h_row : g.T * g.K;
  g.region = (room + 127) / 128 * 128;
  const int left = SMEM_LIMIT - FIXED - g.region;
  g.stages = left < 0 ? 0 : left / Form<FMT>::STAGE;
  if (g.stages > MAX_STAGES) g.stages = MAX_STAGES;
  // (the routing borrows 4 KiB a token)
  if (g.stages < 3 || g.stages * Form<FMT>::STAGE < g.T * 4096) return false;
  *smem = static_cast<size_t>(g.stages) * Form<FMT>::STAGE + g.region + FIXED;
  return true;
}

template <int FMT>
cudaError_t launch(FewArgs g, const void* router, bool router_f32, float* logits, cudaStream_t s) {
  size_t smem = 0;
  if (!plan<FMT>(g, &smem)) return cudaErrorInvalidValue;
  auto first = router_f32 ? few_logits_kernel<true> : few_logits_kernel<false>;
  cudaError_t err = launch_dependent(first, router ? g.E : 1, LOGIT_THREADS, 0, s, g.x, router, g.T, g.E, g.H,
                                     router ? logits : static_cast<float*>(nullptr), g.barrier);
  if (err != cudaSuccess) return err;
  g.logits = router ? logits : nullptr;
  auto kernel = few_layer_kernel<FMT>;
  if ((err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT)) != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sm_count());
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, g);
}

}  // namespace

bool few_layer_fits(int format, int T, int K, int H, int I) {
  FewArgs g{};
  g.T = T, g.K = K, g.H = H, g.I = I;
  size_t smem;
  return format == FEW_BF16 ? plan<FEW_BF16>(g, &smem) : format == FEW_FP8 ? plan<FEW_FP8>(g, &smem) : plan<FEW_FP4>(g, &smem);
}

cudaError_t launch_few_layer(const FewLayer& f, cudaStream_t s) {
  FewArgs g{};
  g.x = f.x;
  g.topk_idx = f.topk_idx;
  g.topk_probs = f.topk_probs;
  g.W1 = static_cast<const uint8_t*>(f.W1);
  g.W2 = static_cast<const uint8_t*>(f.W2);
  g.S1 = f.S1;
  g.S2 = f.S2;
  g.T = f.T, g.E = f.E, g.K = f.K, g.H = f.H, g.I = f.I;
  g.h = f.h;
  g.barrier = f.barrier;
  g.out = f.out;
  g.idx_out = f.idx_out;
  g.probs_out = f.probs_out;
  g.status = f.status;
  return f.format == FEW_BF16  ? launch<FEW_BF16>(g, f.router, f.router_f32, f.logits, s)
         : f.format == FEW_FP8 ? launch<FEW_FP8>(g, f.router, f.router_f32, f.logits, s)
                               : launch<FEW_FP4>(g, f.router, f.router_f32, f.logits, s);
}

}  // namespace moe
