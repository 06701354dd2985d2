// A whole MoE layer for at most 8 tokens, in two launches.
//
//   logits = x R^T;  e_k, w_k: the K largest of a token and their softmax
//   h_k = silu(x Wg[e_k]^T) * (x Wu[e_k]^T)
//   out = sum_k w_k (h_k W2[e_k]^T)
//
// With so few rows the layer is a stream over the active experts' weights, read
// once: 3 H I numbers each.  The first launch makes the logits, a CTA an expert and a
// token.  The second is one persistent cooperative kernel, a CTA an SM, that has
// one grid barrier, between h and the second product:
//   * every CTA picks the experts itself (T K values), so that the weights can be
//     asked for without another launch or barrier;
//   * the active experts' h columns are numbered through and cut into equal runs,
//     one a CTA, and so are the rows of the output: each CTA sums its rows over
//     all active experts, so no partial sums leave it and every order is fixed;
//   * a warp brings its own weights to its own slots of shared memory (cp.async,
//     pieces of 16 rows x 128 bytes, several on their way), the second
//     product's behind the first's: those arrive while h is being finished and
//     while the CTAs meet at the barrier;
//   * it multiplies with mma.sync, 16 weight rows (8 gate and their 8 up rows, or 16
//     rows of W2) by the 8 tokens.  Four warps share a tile of the first product,
//     each a slice of K, all sixteen one of the second; their sums are joined in
//     shared memory in a fixed order.  A token's column is computed for
//     every expert and used for its own.
// What bounds it, at H = 2048, I = 768 and 8 of E = 128 experts a token: HBM for 8
// tokens in bf16 (86 us, 70.6 of them the bytes of 51 experts); for the codes (e4m3 54.6,
// bytes 35.4; e2m1 43.4, bytes 18.8) the instructions that make f16 numbers of them, 250
// to 330 for a piece; for one token (22.2, 17.7 and 14.0) the way from launch to launch: the logits
// 2 us, the list of experts 3, both products' first bytes, the meeting 1.5 to 2, h 1.5.
//
// Tried and slower: a ring of TMA boxes shared by all warps and filled by one (8 tokens: 167 us
// in bf16, 113 in e4m3, 144 in e2m1: what a warp does for a stage, the wait for it included,
// is a chain of a thousand cycles, and each stage took all of them); clusters of two CTAs that
// share rows of the output and split the experts (1.2 us more a launch, 49.9 us for 49.5);
// scales by loads of words that are stored to their slots a piece later, for cp.async (47.9 for 46.6).
//
// Weights are bf16, e4m3 with a scale per 128 x 128, or e2m1 with a scale per 32
// of a row.  Codes are multiplied as f16 numbers, which they are exactly, by tokens and h
// in f16 with a power of two for each row: exact for values down to 2^-28 of the row's
// largest (a bf16 token: 2^-31), and within 2^-38 of that below it.  (mma.sync on e4m3
// operands takes 28 cycles an SM quarter here, on f16 12 for half of K, and converting a pair
// of codes 2.3.)  h goes through memory as f16 with a power of two for eight columns:
// its rounding, 2^-11 at the most, is an eighth of the output's, and half the bytes of fp32 have to reach
// every SM (in fp32 8 tokens took 0.9 to 2.3 us more).  With bf16 weights it is multiplied as
// the sum of two bf16 numbers, which is exact: rounded to one it would add as much error as
// the output's rounding.

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int TOK = FEW_TOKENS;        // 8: one mma operand
constexpr int MAX_K = FEW_TOP_K;       // 16
constexpr int PAIRS = TOK * MAX_K;
constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;
constexpr int TEAM = 4;                // warps that share a tile of the first product
constexpr int MAX_SLOTS = 6;           // of a warp
constexpr int PIECE = 128;             // bytes of a weight row in a slot
// Bytes from row to row in a slot, whose rows' banks are kept apart: 16 more for
// e2m1 (a warp reads 16 bytes of each of eight rows), else by turning the parts
// (a quarter warp reads 64 bytes of each of two rows).
template <int FMT>
__host__ __device__ constexpr int slot_pitch() { return FMT == FEW_FP4 ? PIECE + 16 : PIECE; }
template <int FMT>
__host__ __device__ constexpr int slot_bytes() { return 16 * slot_pitch<FMT>() + 128; }  // and a word or two of scales of each row
constexpr int SMEM_LIMIT = 232448;

template <int FMT>
__host__ __device__ constexpr int row_bytes(int K) { return FMT == FEW_BF16 ? 2 * K : FMT == FEW_FP8 ? K : K / 2; }

// bytes from row to row of tokens, and of h, in shared memory
__host__ __device__ constexpr int token_pitch(int K) { return 2 * K + 64; }
template <int FMT>
__host__ __device__ constexpr int h_pitch(int K) { return (FMT == FEW_BF16 ? 4 : 2) * K + 64; }

struct Smem {
  int ok;
  int expert[PAIRS];          // ascending
  int first[PAIRS + 1];       // pairs before each: its first row of h
  float weight[PAIRS];        // of each row of h
  int8_t row[PAIRS][TOK];     // of h, of each token; -1: none
  uint32_t seen[32];          // a bit for each expert with tokens
  uint32_t tokens[1024 / 4];  // the tokens of each expert, a bit each, four experts a word
  float part[WARPS][4][32];   // the second product's sums; the first's are behind the tokens
};
constexpr int FRONT_PARTS = 2 * WARPS * 4 * 32 * 4;
// bytes of T tokens' rows, and their scales
__host__ __device__ constexpr int front_bytes(int T, int H) { return T * token_pitch(H) + 64; }

struct FewArgs {
  const uint16_t* x;
  const float* logits;       // [T, E]; NULL: the routing is given
  const int64_t* topk_idx;
  const float* topk_probs;
  const uint8_t *W1, *W2;
  const void *S1, *S2;
  int T, E, K, H, I;
  int slots, cap;            // of a warp; rows of h that shared memory holds
  int region;                // bytes of the tokens' rows and their scales
  uint16_t* h;               // [T K, I] in f16, eight columns of a row to a power of two,
  uint8_t* h_exp;            // [T K, I / 8], as the exponent of an fp32 number; 255: NaN
  unsigned* barrier;
  uint16_t* out;
  int64_t* idx_out;
  float* probs_out;
  int* status;
  int ctas;                  // that come to the barrier: all, but in the self-test
};

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// until at most n of this thread's groups are on their way
__device__ __forceinline__ void cp_async_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}
// (not volatile, so that loads of a piece run ahead of its products; the "memory"
// operands keep them behind the waits)
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  return *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  return *reinterpret_cast<const uint32_t*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ void team_sync(int team) { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TEAM) : "memory"); }

__device__ __forceinline__ void mma_bf16_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- logits
// A CTA an expert and a token: their rows' product in fp32.  The first CTA also
// clears the other kernel's barrier.  The latency of its loads bounds it, so that
// all are on their way at once (H = 2048; longer rows in a few steps): an expert's 8
// tokens in one CTA of 128 threads, which read the router's rows once, took 3 to 4 us more
// with 128 experts; with 1024, where the rows come from L2 eight times, 2 us less.
constexpr int LOGIT_THREADS = 256;
template <bool F32>
__global__ void __launch_bounds__(LOGIT_THREADS) few_logits_kernel(const uint16_t* __restrict__ x, const void* __restrict__ router,
                                                                   int E, int H, float* __restrict__ logits,
                                                                   unsigned* __restrict__ barrier) {
  __shared__ float s_sum[LOGIT_THREADS / 32];
  griddep_launch_dependents();
  const int e = blockIdx.x, t = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (logits && t == 0)  // (only a hint, so it may come before the wait for earlier kernels)
    for (int k = threadIdx.x * 128; k < H * (F32 ? 4 : 2); k += LOGIT_THREADS * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(router) + static_cast<long long>(e) * H * (F32 ? 4 : 2) + k));
  griddep_wait();
  if (e == 0 && t == 0 && threadIdx.x == 0) *barrier = 0u;
  if (logits == nullptr) return;
  float acc = 0.f;
#pragma unroll 4
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
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(x + static_cast<long long>(t) * H + k));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = fmaf(bf16_hi(w[i]), r[2 * i + 1], fmaf(bf16_lo(w[i]), r[2 * i], acc));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(FULL_MASK, acc, o);
  if (lane == 0) s_sum[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < LOGIT_THREADS / 32; ++w) v += s_sum[w];
    logits[static_cast<long long>(t) * E + e] = v;
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
// ascending index, as moe_router_topk has them: lane k's slot k.  Lane l keeps logits
// J l .. J l + J - 1 in registers, and the first of the best of those: of lanes with
// the same best the first has the lowest index.
template <int J>
__device__ __forceinline__ void pick_experts(const float* logits, int E, int K, int lane, int& chosen, float& logit) {
  uint32_t key[J];
#pragma unroll
  for (int j = 0; j < J; ++j) key[j] = lane * J + j < E ? sort_key(__ldcg(logits + lane * J + j)) : 0u;
  int mine = 0;
  uint32_t won = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < J; ++j)
      if (key[j] > best) best = key[j], at = j;
    const uint32_t top = __reduce_max_sync(FULL_MASK, best);
    const int src = __ffs(__ballot_sync(FULL_MASK, best == top)) - 1;
    const int e = src * J + __shfl_sync(FULL_MASK, at, src);
    if (lane == k) mine = e, won = top;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane == src && j == at) key[j] = 0u;
  }
  if (lane < K) chosen = mine, logit = of_key(won);
}
// and their softmax
__device__ __forceinline__ float softmax_of(float logit, int K, int lane) {
  const float top = __shfl_sync(FULL_MASK, logit, 0);
  const float ex = lane < K ? expf(logit - top) : 0.f;
  float sum = ex;
#pragma unroll
  for (int o = MAX_K / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
  return ex / sum;
}

// ---------------------------------------------------------------- rows of tokens
// The power of two by which a row is divided to become f16: 2^(floor(log2 amax) -
// 14), at least 2^-126, so that values are below 2^15; NaN for a row with a NaN or
// an infinity.  `inv`: its reciprocal.
__device__ __forceinline__ float row_scale_f16(float amax, float& inv) {
  const uint32_t bits = __float_as_uint(amax);
  const uint32_t e = bits >> 23 > 15u ? (bits >> 23) - 14u : 1u;
  inv = __uint_as_float((254u - e) << 23);
  return bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
}
__device__ __forceinline__ uint4 f16x8(const float (&v)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 h = __floats2half2_rn(v[2 * k] * inv, v[2 * k + 1] * inv);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where the 16 bytes of values [8 v, 8 v + 8) of a row lie: in their place, or for e4m3 of
// each 64 first the first 8 of every 16, then the others, as a lane's codes meet them.
template <int FMT>
__device__ __forceinline__ int place_of(int v) {
  return FMT == FEW_FP8 ? (v & ~7) | (v & 1) << 2 | (v & 7) >> 1 : v;
}

// `rows` rows of K bf16 values into shared memory as the products read them, `warps`
// warps of which this is number `warp`, a row each.  For codes: f16 with a scale for each row.
template <int FMT>
__device__ __forceinline__ void stage_tokens(const uint16_t* src, int rows, int K, int pitch, uint8_t* dst, float* scales, int warp, int warps) {
  constexpr int V = 8;  // eights of a lane at a time
  const int per_row = K >> 3, lane = threadIdx.x & 31;
  uint4 q[V];
  auto load = [&](int r, int v0) {
    const uint4* row = reinterpret_cast<const uint4*>(src + static_cast<long long>(r) * K);
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] = v0 + 32 * j < per_row ? __ldcg(row + v0 + 32 * j) : make_uint4(0, 0, 0, 0);
  };
  auto values = [&](const uint4& of, float (&f)[8]) {
    const uint32_t w[4] = {of.x, of.y, of.z, of.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
  };
  for (int r = warp; r < rows; r += warps) {
    float f[8], inv = 1.f;
    if constexpr (FMT != FEW_BF16) {
      float top = 0.f;
      for (int v0 = lane; v0 < per_row; v0 += 32 * V) {
        load(r, v0);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          values(q[j], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(f[k]));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(FULL_MASK, top, o));
      const float scale = row_scale_f16(top, inv);
      if (lane == 0) scales[r] = scale;
    }
    for (int v0 = lane; v0 < per_row; v0 += 32 * V) {
      if (FMT == FEW_BF16 || per_row > 32 * V) load(r, v0);  // (else they are still here)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = v0 + 32 * j;
        if (v >= per_row) break;
        uint4 to = q[j];
        if constexpr (FMT != FEW_BF16) {
          values(q[j], f);
          to = f16x8(f, inv);
        }
        *reinterpret_cast<uint4*>(dst + r * pitch + place_of<FMT>(v) * 16) = to;
      }
    }
  }
}

__device__ __forceinline__ float scale_of_exp(uint32_t e) { return __uint_as_float(e == 255u ? 0x7fc00000u : e << 23); }

// `rows` rows of h, from row r0, in the same way, two of a warp on their way at a time.
// For codes: f16 to the largest of its powers of two.  For bf16 weights: the nearest
// bf16 numbers and, 2 I bytes on, what those leave (11 bits are the sum of two numbers of 8).
template <int FMT>
__device__ __forceinline__ void stage_h(const FewArgs& args, int r0, int rows, int pitch, uint8_t* dst, float* scales, int warp) {
  constexpr int V = 4, AT = 2;  // eights of a lane and rows of a warp at a time
  const int per_row = args.I >> 3, lane = threadIdx.x & 31;
  const uint4* codes = reinterpret_cast<const uint4*>(args.h) + r0 * per_row + lane;
  const uint8_t* exps = args.h_exp + r0 * per_row + lane;
  dst += place_of<FMT>(lane) * 16;
  uint4 q[AT][V];
  uint32_t e[AT][V];
  auto load = [&](int n, int r, int v0) {  // eights v0 + lane + 32 j
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool there = r < rows && v0 + lane + 32 * j < per_row;
      e[n][j] = there ? __ldcg(exps + r * per_row + v0 + 32 * j) : 0u;
      if (there) q[n][j] = __ldcg(codes + r * per_row + v0 + 32 * j);
    }
  };
  auto largest = [&](int n) { return max(max(e[n][0], e[n][1]), max(e[n][2], e[n][3])); };
  auto store = [&](int n, int r, int v0, uint32_t top) {
    uint8_t* to = dst + r * pitch + v0 * 16;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (v0 + lane + 32 * j >= per_row) break;
      const uint32_t w[4] = {q[n][j].x, q[n][j].y, q[n][j].z, q[n][j].w};
      uint32_t hi[4], lo[4];
      if constexpr (FMT == FEW_BF16) {
        const float scale = scale_of_exp(e[n][j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          f.x *= scale, f.y *= scale;
          hi[k] = pack_bf16x2(f.x, f.y);
          lo[k] = pack_bf16x2(f.x - bf16_lo(hi[k]), f.y - bf16_hi(hi[k]));
        }
        *reinterpret_cast<uint4*>(to + 512 * j + 2 * args.I) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      } else {
        // 2^-24 is the least f16: what is further below the row's largest goes down in two steps
        const uint32_t down = top - e[n][j];
        const __half2 scale = __float2half2_rn(__uint_as_float((127u - min(down, 24u)) << 23));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 f = __hmul2(*reinterpret_cast<const __half2*>(&w[k]), scale);
          hi[k] = *reinterpret_cast<const uint32_t*>(&f);
        }
        if (down > 24u) {
          const __half2 rest = __float2half2_rn(__uint_as_float((127u - min(down - 24u, 24u)) << 23));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 f = __hmul2(*reinterpret_cast<const __half2*>(&hi[k]), rest);
            hi[k] = *reinterpret_cast<const uint32_t*>(&f);
          }
        }
      }
      *reinterpret_cast<uint4*>(to + 512 * j) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
  };
  auto scale_row = [&](int r, uint32_t top) {
    top = __reduce_max_sync(FULL_MASK, top);
    if (lane == 0) scales[r] = scale_of_exp(top);
    return top;
  };
  if (per_row <= 32 * V) {
#pragma unroll
    for (int n = 0; n < AT; ++n) load(n, warp + n * WARPS, 0);
    for (int i = warp; i < rows; i += AT * WARPS) {
#pragma unroll
      for (int n = 0; n < AT; ++n) {
        const int r = i + n * WARPS;
        if (r >= rows) break;
        uint32_t top = 0;
        if constexpr (FMT != FEW_BF16) top = scale_row(r, largest(n));
        store(n, r, 0, top);
        load(n, r + AT * WARPS, 0);
      }
    }
    return;
  }
  for (int r = warp; r < rows; r += WARPS) {  // a row in pieces
    uint32_t top = 0;
    if constexpr (FMT != FEW_BF16) {
      for (int v0 = 0; v0 < per_row; v0 += 32 * V) {
        load(0, r, v0);
        top = max(top, largest(0));
      }
      top = scale_row(r, top);
    }
    for (int v0 = 0; v0 < per_row; v0 += 32 * V) {
      load(0, r, v0);
      store(0, r, v0, top);
    }
  }
}

// ---------------------------------------------------------------- pieces of weights
// A warp's weights in the order of their use: its pieces of the first product's
// tiles (8 gate rows and their 8 up rows; every fourth tile is its team's, every
// fourth piece of it its own), then of the second's (16 rows, every
// sixteenth piece of all experts' rows).
template <int FMT>
struct Cursor {
  const Smem& s;
  const int active, warp, lane, I;
  const int bytes1, bytes2, steps1, steps2;  // bytes and pieces of a row
  int a, j0, left;           // first product: expert (place in the list), column, columns to come
  int m0, left2;             // second product: row of the output, rows to come
  int st, steps;             // piece, pieces of a row
  bool first;
  int n_lo, n_hi, rb;        // rows of the tile's halves, bytes of a row
  const uint32_t part;       // where this lane's 16 bytes of rows lane / 8 go in a slot
  // this lane's 16 bytes of the piece: in row lane / 8 of the expert's rows, of the tile's halves
  const uint8_t *base, *lo, *hi;
  long long stride;          // bytes of an expert
  // fp8, fp4: the first word of row lane % 16, in the expert's scales and the tile's
  const uint8_t *scale_base, *scale;
  long long scale_stride;
  const FewArgs& args;

  __device__ __forceinline__ Cursor(const FewArgs& args_, const Smem& s_, int active_, int warp_, int lane_, int a_, int j0_, int cols, int r0, int rows)
      : s(s_), active(active_), warp(warp_), lane(lane_), I(args_.I), bytes1(row_bytes<FMT>(args_.H)), bytes2(row_bytes<FMT>(args_.I)),
        steps1((bytes1 + PIECE - 1) / PIECE), steps2((bytes2 + PIECE - 1) / PIECE), a(a_), j0(j0_), left(cols), m0(r0), left2(rows),
        st(warp_ % TEAM), steps(steps1), first(true), rb(bytes1),
        part((lane_ >> 3) * slot_pitch<FMT>() + (((lane_ & 7) ^ (FMT == FEW_FP4 ? 0 : ((lane_ >> 3) & 1) * 4 + (lane_ >> 4))) << 4)),
        args(args_) {
    for (int i = 0; i < warp / TEAM; ++i) skip_tile();
    if (st >= steps1) left = 0;  // no piece for this warp
    base = args.W1 + static_cast<long long>(lane >> 3) * bytes1 + (lane & 7) * 16;
    stride = 2ll * I * bytes1;
    if constexpr (FMT != FEW_BF16) scale_stride = scales(2 * I, args.H);
    if (left > 0) aim1(); else second();
  }
  // scales of a matrix of [rows, K], and of the 128 rows with row r in it
  __device__ __forceinline__ long long scales(int rows, int K) const {
    return static_cast<long long>(rows >> 7) * (K >> 7) * (FMT == FEW_FP8 ? 4 : SCALE_TILE);
  }
  __device__ __forceinline__ const uint8_t* row_scales(const uint8_t* of, int K, int r) const {
    of += scales(r, K);
    return FMT == FEW_FP8 ? of : of + (r & 31) * 16 + ((r >> 5) & 3) * 4;
  }
  __device__ __forceinline__ void skip_tile() {
    left -= 8;
    j0 += 8;
    if (j0 == I) j0 = 0, ++a;
  }
  __device__ __forceinline__ bool more() const { return left2 > 0; }  // (every CTA has rows of the output)
  __device__ __forceinline__ void aim1() {
    n_lo = n_hi = 8;
    const int e = s.expert[a];
    lo = base + e * stride + static_cast<long long>(j0) * bytes1;
    hi = lo + static_cast<long long>(I) * bytes1;
    if constexpr (FMT != FEW_BF16)
      scale = row_scales(static_cast<const uint8_t*>(args.S1) + e * scale_stride, args.H,
                         j0 + (lane & 7) + (lane & 8 ? I : 0));
  }
  // the 16 rows of the output from m0
  __device__ __forceinline__ void rows_at() {
    base = args.W2 + static_cast<long long>(m0 + (lane >> 3)) * bytes2 + (lane & 7) * 16;
    const int n = min(16, left2);
    n_lo = min(n, 8);
    n_hi = n - n_lo;
    if constexpr (FMT != FEW_BF16) scale_base = row_scales(static_cast<const uint8_t*>(args.S2), I, m0 + min(lane & 15, n - 1));
    a = 0;
    st = warp;
  }
  __device__ __forceinline__ void second() {
    first = false;
    steps = steps2;
    rb = bytes2;
    stride = static_cast<long long>(args.H) * bytes2;
    if constexpr (FMT != FEW_BF16) scale_stride = scales(args.H, I);
    if (active == 0) left2 = 0;
    if (left2 <= 0) return;
    rows_at();
    aim2();
  }
  __device__ __forceinline__ void aim2() {
    while (st >= steps2) {
      st -= steps2;
      if (++a == active) {
        m0 += 16;
        left2 -= 16;
        if (left2 <= 0) return;
        rows_at();
      }
    }
    const int e = s.expert[a];
    lo = base + e * stride;
    hi = lo + 8ll * bytes2;
    if constexpr (FMT != FEW_BF16) scale = scale_base + e * scale_stride;
  }
  // Asks for the piece and goes on to the next.  Unless rows are 16 bytes apart
  // more (e2m1), row r's 16-byte part c goes to part c ^ (r % 2 * 4 + r / 2 % 4).
  __device__ __forceinline__ void issue(uint32_t slot) {
    constexpr int PITCH = slot_pitch<FMT>();
    if (more()) {
      const int row = lane >> 3, at = st * PIECE;
      if (at + (lane & 7) * 16 < rb) {
        const uint32_t dst = slot + part, dst4 = slot + ((part + 4 * PITCH) ^ (FMT == FEW_FP4 ? 0 : 32));
        const uint8_t *p = lo + at, *q = hi + at;
        if (row < n_lo) cp_async_16(dst, p);
        if (row + 4 < n_lo) cp_async_16(dst4, p + 4 * rb);
        if (row < n_hi) cp_async_16(dst + 8 * PITCH, q);
        if (row + 4 < n_hi) cp_async_16(dst4 + 8 * PITCH, q + 4 * rb);
      }
      if constexpr (FMT == FEW_FP8) {
        if (lane < 16) cp_async_4(slot + 16 * PITCH + lane * 4, scale + st * 4);
      } else if constexpr (FMT == FEW_FP4) {
        const int kb = 2 * st + (lane >> 4);
        if (kb * 64 < rb) cp_async_4(slot + 16 * PITCH + lane * 4, scale + kb * SCALE_TILE);
      }
      st += first ? TEAM : WARPS;
      if (st >= steps) {
        if (first) {
          st = warp % TEAM;
          for (int i = 0; i < WARPS / TEAM; ++i) skip_tile();
          if (left > 0) aim1(); else second();
        } else {
          aim2();
        }
      }
    }
    cp_async_commit();
  }
};

// ---------------------------------------------------------------- products
// d[16 rows x 8 tokens] += a slot's rows times the tokens' rows.  `token`: the row
// of token lane / 4 (any row where there is none: its column is no one's), `st` the
// piece, `bytes` those of a weight row.  With SUM (bf16) a token's row is followed by
// what it was rounded from.
template <int FMT, bool SUM>
__device__ __forceinline__ void multiply(float (&d)[4], uint32_t slot, int st, int bytes, int lane, uint32_t token) {
  constexpr int PITCH = slot_pitch<FMT>();
  const int g = lane >> 2, t = lane & 3;
  // part c of the row: at lo ^ (c << 4) (rows are 128 bytes at multiples of 128), or at lo + 16 c
  const uint32_t turn = FMT == FEW_FP4 ? 4 * t : (((g & 1) * 4 + (g >> 1)) ^ t) << 4;
  const uint32_t lo = slot + g * PITCH + turn, hi = lo + 8 * PITCH;
  const uint32_t sc = slot + 16 * PITCH + g * 4;
  token += 16 * t;
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // halves of 64 bytes
    if (st * PIECE + h * 64 >= bytes) break;
    if constexpr (FMT == FEW_BF16) {
      const uint4 a = lds128(lo ^ (h * 64)), c = lds128(hi ^ (h * 64));
      const uint4 b = lds128(token + st * PIECE + h * 64);
      mma_bf16_16x8x16(d, a.x, c.x, a.y, c.y, b.x, b.y);
      mma_bf16_16x8x16(d, a.z, c.z, a.w, c.w, b.z, b.w);
      if constexpr (SUM) {
        const uint4 r = lds128(token + bytes + st * PIECE + h * 64);
        mma_bf16_16x8x16(d, a.x, c.x, a.y, c.y, r.x, r.y);
        mma_bf16_16x8x16(d, a.z, c.z, a.w, c.w, r.z, r.w);
      }
    } else if constexpr (FMT == FEW_FP8) {
      const uint4 a = lds128(lo ^ (h * 64)), c = lds128(hi ^ (h * 64));
      const uint32_t from = token + (2 * st + h) * 128;
      const uint4 b0 = lds128(from), b1 = lds128(from + 64);
      float p[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
      const uint32_t wb[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t ha[2], hc[2];
        f16_of_e4m3x4(wa[i], ha);
        f16_of_e4m3x4(wc[i], hc);
        mma_f16_16x8x16(i & 1 ? q : p, ha[0], hc[0], ha[1], hc[1], wb[2 * i], wb[2 * i + 1]);
      }
      const float w0 = __uint_as_float(lds32(sc)), w1 = __uint_as_float(lds32(sc + 32));
      d[0] = fmaf(p[0] + q[0], w0, d[0]);
      d[1] = fmaf(p[1] + q[1], w0, d[1]);
      d[2] = fmaf(p[2] + q[2], w1, d[2]);
      d[3] = fmaf(p[3] + q[3], w1, d[3]);
    } else {
      uint32_t f0[2], f1[2];
      bf16_of_e8m0x4(lds32(sc + h * 64), f0);
      bf16_of_e8m0x4(lds32(sc + h * 64 + 32), f1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = lds32(lo + (h * 4 + j) * 16), c = lds32(hi + (h * 4 + j) * 16);
        const uint4 b = lds128(token + st * 512 + (h * 4 + j) * 64);
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t ha[4], hc[4];
        f16_of_e2m1x8(a, ha);
        f16_of_e2m1x8(c, hc);
        mma_f16_16x8x16(p, ha[0], hc[0], ha[1], hc[1], b.x, b.y);
        mma_f16_16x8x16(p, ha[2], hc[2], ha[3], hc[3], b.z, b.w);
        const float w0 = j & 1 ? bf16_hi(f0[j >> 1]) : bf16_lo(f0[j >> 1]), w1 = j & 1 ? bf16_hi(f1[j >> 1]) : bf16_lo(f1[j >> 1]);
        d[0] = fmaf(p[0], w0, d[0]);
        d[1] = fmaf(p[1], w0, d[1]);
        d[2] = fmaf(p[2], w1, d[2]);
        d[3] = fmaf(p[3], w1, d[3]);
      }
    }
  }
}

// ---------------------------------------------------------------- the layer
template <int FMT>
__global__ void __launch_bounds__(THREADS, 1) few_layer_kernel(const FewArgs args) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int SLOT = slot_bytes<FMT>();
  uint8_t* region = smem + args.slots * WARPS * SLOT;
  Smem& s = *reinterpret_cast<Smem*>(region + args.region);
  // (a number that the compiler knows to be the warp's)
  const int warp = __shfl_sync(FULL_MASK, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int T = args.T, E = args.E, K = args.K, H = args.H, I = args.I;
  // (no griddep_launch_dependents(): CTAs of the next kernel that wait beside this
  // one's cost it 1.2 us)
  if (static_cast<int>(threadIdx.x) * 4 < E) s.tokens[threadIdx.x] = 0;
  if (threadIdx.x < 32) s.seen[threadIdx.x] = 0;
  __syncthreads();
  griddep_wait();

  // the routing, a warp a token; the other warps bring the tokens
  float* s_scale = reinterpret_cast<float*>(region + T * token_pitch(H));
  int chosen = -1;
  float prob = 0.f;  // its logit, until there is time for the softmax
  if (warp >= TOK) {
    stage_tokens<FMT>(args.x, T, H, token_pitch(H), region, s_scale, warp - TOK, WARPS - TOK);
  } else if (warp < T) {
    if (args.logits) {
      const float* l = args.logits + warp * E;
      if (E <= 128) pick_experts<4>(l, E, K, lane, chosen, prob);
      else pick_experts<32>(l, E, K, lane, chosen, prob);
    } else if (lane < K) {
      const long long e = args.topk_idx[warp * K + lane];
      prob = args.topk_probs[warp * K + lane];
      if (e >= 0 && e < E) chosen = static_cast<int>(e);
      else if (e != -1 && blockIdx.x == 0) report(args.status, MOE_DEVERR_BAD_INDEX);
    }
    if (chosen >= 0) {
      atomicOr(&s.seen[chosen >> 5], 1u << (chosen & 31));
      atomicOr(&s.tokens[chosen >> 2], 1u << ((chosen & 3) * 8 + warp));
    }
  }
  __syncthreads();
  // the experts with tokens, ascending: each warp counts those before each 32
  const uint32_t bits = s.seen[lane];
  int upto = __popc(bits);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL_MASK, upto, o);
    if (lane >= o) upto += v;
  }
  for (int w = warp; w * 32 < E; w += WARPS) {
    const uint32_t there = __shfl_sync(FULL_MASK, bits, w);
    const int before = __shfl_sync(FULL_MASK, upto, w) - __popc(there);
    if ((there >> lane) & 1) s.expert[before + __popc(there & ((1u << lane) - 1u))] = w * 32 + lane;
  }
  __syncthreads();
  const int active = __shfl_sync(FULL_MASK, upto, 31);

  const uint32_t G = gridDim.x, b = blockIdx.x;
  // this CTA's columns of h, numbered through the experts, and rows of the output
  const uint32_t tiles = static_cast<uint32_t>(active) * (I >> 3);
  const int f0 = b * tiles / G * 8, my_cols = (b + 1) * tiles / G * 8 - f0;
  const int first_a = f0 / I, first_j = f0 - first_a * I;
  const int r0 = b * static_cast<uint32_t>(H) / G, r1 = (b + 1) * static_cast<uint32_t>(H) / G;
  const int bytes1 = row_bytes<FMT>(H), bytes2 = row_bytes<FMT>(I);
  const uint32_t slots = smem_u32(smem) + warp * args.slots * SLOT;
  Cursor<FMT> cursor(args, s, active, warp, lane, first_a, first_j, my_cols, r0, r1 - r0);
  for (int i = 0; i < args.slots; ++i) cursor.issue(slots + i * SLOT);
  if (warp == TOK) {  // the experts' rows of h
    int row = 0;
    for (int a0 = 0; a0 < active; a0 += 32) {
      const int e = a0 + lane < active ? s.expert[a0 + lane] : 0;
      const int m = a0 + lane < active ? (s.tokens[e >> 2] >> ((e & 3) * 8)) & 0xff : 0;
      int n = __popc(m);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, n, o);
        if (lane >= o) n += v;
      }
      if (a0 + lane < active) {
        int r = row + n - __popc(m);
        s.first[a0 + lane] = r;
#pragma unroll
        for (int t = 0; t < TOK; ++t) s.row[a0 + lane][t] = static_cast<int8_t>((m >> t) & 1 ? r++ : -1);
      }
      row += __shfl_sync(FULL_MASK, n, 31);
    }
    if (lane == 0) s.first[active] = row;
  }
  __syncthreads();
  int slot = 0;
  auto next = [&](auto sum, float (&d)[4], int st, int bytes, uint32_t token) {
    cp_async_wait(args.slots - 1);
    __syncwarp();
    multiply<FMT, decltype(sum)::value>(d, slots + slot * SLOT, st, bytes, lane, token);
    __syncwarp();
    cursor.issue(slots + slot * SLOT);
    if (++slot == args.slots) slot = 0;
  };

  // ---- h
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rows_u32 = smem_u32(region);
  {
    const uint32_t token = rows_u32 + min(g, T - 1) * token_pitch(H);
    auto* parts = reinterpret_cast<float (*)[WARPS][4][32]>(region + front_bytes(T, H));
    const int team = warp / TEAM, tid = threadIdx.x % (32 * TEAM);
    int par = 0, a = first_a, j = first_j, turn = 0;
    for (int left = my_cols; left > 0; left -= 8) {
      if (j == I) j = 0, ++a;
      const int j0 = j;
      j += 8;
      const bool mine = turn == team;
      if (++turn == WARPS / TEAM) turn = 0;
      if (!mine) continue;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      for (int st = warp % TEAM; st * PIECE < bytes1; st += TEAM) next(std::false_type{}, d, st, bytes1, token);
#pragma unroll
      for (int i = 0; i < 4; ++i) parts[par][warp][i][lane] = d[i];
      // one meeting a tile: this parity's sums are written again after the next
      // tile's, which follows their reading here
      team_sync(team);
      if (tid >> 6 == par) {  // two of the team's warps, the others at the next tile
        const int tok = (tid >> 3) & 7, i = tid & 7;
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < TEAM; ++w) {
          gate += parts[par][team * TEAM + w][tok & 1][i * 4 + (tok >> 1)];
          up += parts[par][team * TEAM + w][2 + (tok & 1)][i * 4 + (tok >> 1)];
        }
        if constexpr (FMT != FEW_BF16) gate *= s_scale[min(tok, T - 1)], up *= s_scale[min(tok, T - 1)];
        const float v = gate / (1.0f + expf(-gate)) * up;
        float top = fabsf(v), inv;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max_nan(top, __shfl_xor_sync(FULL_MASK, top, o));
        const float scale = row_scale_f16(top, inv);
        const int row = s.row[a][tok];
        if (row >= 0) {
          args.h[static_cast<long long>(row) * I + j0 + i] = __half_as_ushort(__float2half_rn(v * inv));
          if (i == 0) args.h_exp[static_cast<long long>(row) * (I >> 3) + (j0 >> 3)] = static_cast<uint8_t>(__float_as_uint(scale) >> 23);
        }
      }
      par ^= 1;
    }
  }
  // h is whole once every CTA has been here
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 32 * TOK) {
    int met = 1;
    if (static_cast<int>(blockIdx.x) < args.ctas) atomicAdd(args.barrier, 1u);
    const unsigned long long t0 = global_timer_ns();
    while (*reinterpret_cast<volatile unsigned*>(args.barrier) < gridDim.x) {
      if (global_timer_ns() - t0 > WAIT_LIMIT_NS) {
        met = 0;
        break;
      }
    }
    __threadfence();
    s.ok = met;
  }
  // meanwhile, the weights of the rows of h (of an expert that a token names twice the last slot counts)
  if (warp < T) {
    if (args.logits) prob = softmax_of(prob, K, lane);
    if (lane < K && blockIdx.x == 0 && args.idx_out) {
      args.idx_out[warp * K + lane] = chosen;
      args.probs_out[warp * K + lane] = prob;
    }
    const int word = max(chosen, 0) >> 5;
    const uint32_t same = __match_any_sync(FULL_MASK, chosen), there = __shfl_sync(FULL_MASK, bits, word);
    const int before = __shfl_sync(FULL_MASK, upto, word) - __popc(there);
    if (chosen >= 0 && lane == 31 - __clz(same)) s.weight[s.row[before + __popc(there & ((1u << (chosen & 31)) - 1u))][warp]] = prob;
  }
  __syncthreads();
  if (!s.ok) {  // the wait ran out: this CTA's rows are no result
    cp_async_wait(0);
    for (int i = threadIdx.x; i < T * (r1 - r0); i += THREADS)
      args.out[static_cast<long long>(i / (r1 - r0)) * H + r0 + i % (r1 - r0)] = 0x7fc0;
    if (threadIdx.x == 0) report(args.status, MOE_DEVERR_TIMEOUT);
    return;
  }

  // ---- out
  const int hp = h_pitch<FMT>(I), steps2 = (bytes2 + PIECE - 1) / PIECE;
  float* h_scale = reinterpret_cast<float*>(region + args.cap * hp);
  const bool whole = s.first[active] <= args.cap;  // all rows of h at once
  for (int m0 = r0; m0 < r1; m0 += 16) {
    const int n = min(16, r1 - m0);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int a = 0, st = warp;  // this warp's next piece
    for (int sa = 0, sb = 0; sa < active; sa = sb) {  // experts whose rows of h are in shared memory
      while (sb < active && s.first[sb + 1] - s.first[sa] <= args.cap) ++sb;
      if (!whole || m0 == r0) {
        __syncthreads();
        stage_h<FMT>(args, s.first[sa], s.first[sb] - s.first[sa], hp, region, h_scale, warp);
        __syncthreads();
      }
      while (true) {
        while (a < sb && st >= steps2) st -= steps2, ++a;
        if (a >= sb) break;
        const int base = s.first[sa], mine = s.row[a][g], row0 = s.row[a][2 * t], row1 = s.row[a][2 * t + 1];
        const uint32_t token = rows_u32 + max(mine - base, 0) * hp;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        next(std::bool_constant<FMT == FEW_BF16>{}, d, st, bytes2, token);
        if (row0 >= 0) {
          float w = s.weight[row0];
          if constexpr (FMT != FEW_BF16) w *= h_scale[row0 - base];
          acc[0] = fmaf(w, d[0], acc[0]);
          acc[2] = fmaf(w, d[2], acc[2]);
        }
        if (row1 >= 0) {
          float w = s.weight[row1];
          if constexpr (FMT != FEW_BF16) w *= h_scale[row1 - base];
          acc[1] = fmaf(w, d[1], acc[1]);
          acc[3] = fmaf(w, d[3], acc[3]);
        }
        st += WARPS;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s.part[warp][i][lane] = acc[i];
    __syncthreads();
    if (threadIdx.x < 128) {  // rows fastest
      const int r = threadIdx.x & 15, tok = threadIdx.x >> 4;
      if (r < n && tok < T) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += s.part[w][(r >> 3) * 2 + (tok & 1)][(r & 7) * 4 + (tok >> 1)];
        args.out[static_cast<long long>(tok) * H + m0 + r] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
      }
    }
    if (m0 + 16 < r1) __syncthreads();
  }
}

constexpr int FIXED = sizeof(Smem);

// The self-test's limit of the CTAs that come to the barrier, for this host thread's launches.
thread_local int tls_ctas = 0x7fffffff;

template <int FMT>
bool plan(FewArgs& g, size_t* smem) {
  constexpr int SLOT = slot_bytes<FMT>();
  if (g.H > 1 << 20 || g.I > 1 << 20) return false;  // no row fits, and the sizes below pass 32 bits
  const long long h_row = h_pitch<FMT>(g.I) + 4, front = front_bytes(g.T, g.H) + FRONT_PARTS;
  // all rows of h where they leave three slots a warp, else as many as there are tokens
  const long long need = g.T * h_row > front ? g.T * h_row : front, most = SMEM_LIMIT - FIXED - 128 - 3 * WARPS * SLOT;
  long long room = g.T * g.K * h_row;
  if (room > most) room = most;
  if (room < need) room = need;
  if (room > SMEM_LIMIT - FIXED - 128) return false;
  g.cap = static_cast<int>(room / h_row < g.T * g.K ? room / h_row : g.T * g.K);
  g.region = static_cast<int>((room + 127) / 128 * 128);
  g.slots = (SMEM_LIMIT - FIXED - g.region) / (WARPS * SLOT);
  if (g.slots > MAX_SLOTS) g.slots = MAX_SLOTS;
  if (g.slots < 2) return false;
  *smem = static_cast<size_t>(g.slots) * WARPS * SLOT + g.region + FIXED;
  return true;
}

template <int FMT>
cudaError_t launch(FewArgs g, const void* router, bool router_f32, float* logits, cudaStream_t s) {
  size_t smem = 0;
  if (!plan<FMT>(g, &smem)) return cudaErrorInvalidValue;
  auto first = router_f32 ? few_logits_kernel<true> : few_logits_kernel<false>;
  cudaError_t err = launch_dependent(first, router ? dim3(g.E, g.T) : dim3(1), LOGIT_THREADS, 0, s, g.x, router, g.E, g.H,
                                     router ? logits : static_cast<float*>(nullptr), g.barrier);
  if (err != cudaSuccess) return err;
  g.logits = router ? logits : nullptr;
  g.ctas = tls_ctas;
  auto kernel = few_layer_kernel<FMT>;
  if ((err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT)) != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  // No more CTAs than rows of the output: the cursor asks for nothing once it has no row left, so that
  // a CTA with columns of h alone would multiply what it never loaded.  (H is 256 at the least.)
  cfg.gridDim = dim3(g.H < sm_count() ? g.H : sm_count());
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

void selftest_few_ctas(int ctas) { tls_ctas = ctas; }

bool few_layer_fits(int format, int T, int K, int H, int I, int* rows, int* slots) {
  FewArgs g{};
  g.T = T, g.K = K, g.H = H, g.I = I;
  size_t smem;
  const bool fits = format == FEW_BF16 ? plan<FEW_BF16>(g, &smem) : format == FEW_FP8 ? plan<FEW_FP8>(g, &smem) : plan<FEW_FP4>(g, &smem);
  if (rows) *rows = fits ? g.cap : 0;
  if (slots) *slots = fits ? g.slots : 0;
  return fits;
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
  g.h_exp = reinterpret_cast<uint8_t*>(f.h + static_cast<size_t>(f.T) * f.K * f.I);
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
