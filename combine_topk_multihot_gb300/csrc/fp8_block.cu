// e4m3 codes with a scale for each block of 128: quantisation, and the
// products with few rows.
//
// Codes and scales: scale = max|v| / 448 over a block (1 for a block of
// zeros), code = e4m3(v / scale) to nearest even; a block is 128 columns of
// one row (activations) or 128 x 128 (weights).  Both kernels read their input
// once and are bound by HBM.
//
// With at most 8 rows (per expert; one operand of the instruction) the product is a stream over the weights:
// every weight is used at most 8 times.  A 128-row tile of the tensor-core
// kernel would be empty for the most part, and its tiles too few to keep all
// SMs loading (8 rows here against 9 there, N x K: 4096 x 2048 10.2 us for
// 12.3, 1024 x 8192 14.3 for 22.5, 8192 x 8192 24.6 for 27 to 35).  Here a warp takes 16 weight rows and a slice of K, loads them
// straight into registers in 16-byte pieces (64 consecutive bytes of a row
// per four lanes), and multiplies with mma.sync: the weights are its 16-row
// operand, the 8 rows the other, both with the same permutation of K (a
// lane's 16 bytes are 16 consecutive codes of one row in either operand, so
// that no shuffle is needed).  Products of codes are exact; the
// instruction adds 32 of them in fp32 (measured: beside 2^17.6 what is 2^-6
// or more is kept, 24 bits); after the four of a block, its scales are applied in fp32.
// The slices of K are joined in shared memory in a fixed order.
//
// For the experts each CTA makes the codes of its group's rows itself, from
// bf16 rows or from the fp32 gate/up rows, while its first weights are on their
// way: a few KB read again by every CTA, from L2, in place of a launch before
// each product (T = 1, E = 128, H = 2048, I = 768: 28 -> 18 us).

#include "common.cuh"
#include "fp8_quant.cuh"
#include "launch.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- quantisation

// A warp takes up to four 256-column pieces (two blocks each) of one row:
// lane l holds 8 values, 16 lanes a block.  blockIdx.y picks the pieces.
// Bound by HBM and, close behind, by instructions: 48 registers, so that 40
// warps an SM overlap one's loads with another's arithmetic (32768 x 2048:
// 37.9 us, 5.4 TB/s; with 53 registers and 32 warps 39.5; 2 or 8 pieces 47).
constexpr int PIECES = 4;
__global__ void __launch_bounds__(256, 5) quantize_row_blocks_kernel(const uint16_t* __restrict__ src, long long rows,
                                                                  int cols, uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales,
                                                                  const int* __restrict__ row_token) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int blocks = (cols + 127) >> 7;
  const int col0 = blockIdx.y * (PIECES * 256) + lane * 8;
  const long long nwarps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long r = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows;
       r += nwarps) {
    if (row_token && __ldg(row_token + r) < 0) continue;
    uint4 q[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int c = col0 + 256 * p;
      q[p] = c < cols ? __ldcs(reinterpret_cast<const uint4*>(src + r * cols + c)) : make_uint4(0, 0, 0, 0);
    }
    uint32_t top[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
      top[p] = bf16x2_abs_max(bf16x2_abs_max(q[p].x, q[p].y), bf16x2_abs_max(q[p].z, q[p].w));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int p = 0; p < PIECES; ++p) top[p] = bf16x2_abs_max(top[p], __shfl_xor_sync(FULL_MASK, top[p], o));
    float mine = 0.f;  // lane i (and i + 16, ...): the scale of piece i / 2's block i % 2
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const float scale = block_scale(max_nan(bf16_lo(top[p]), bf16_hi(top[p])));
      const uint32_t w[4] = {q[p].x, q[p].y, q[p].z, q[p].w};
      const int c = col0 + 256 * p;
      if (c < cols) *reinterpret_cast<uint2*>(codes + r * cols + c) = BlockDivide(scale).codes(w);
      const float s = __shfl_sync(FULL_MASK, scale, (lane & 1) * 16);
      if ((lane >> 1) == p) mine = s;
    }
    const int b = blockIdx.y * (2 * PIECES) + lane;
    if (lane < 2 * PIECES && b < blocks) scales[r * blocks + b] = mine;
  }
}

// A CTA takes one 128 x 128 block: thread t holds 8 columns of rows t / 16 +
// 16 i.  Rows and columns past the matrix count as zeros.  (403 M weights: 212
// us, 5.7 TB/s; with two CTAs an SM 245, with four 226.)
__global__ void __launch_bounds__(256, 3) quantize_square_blocks_kernel(const uint16_t* __restrict__ src, int rows,
                                                                     int cols, uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales) {
  __shared__ float s_top[8];
  griddep_launch_dependents();
  griddep_wait();
  const int nr = (rows + 127) >> 7, nc = (cols + 127) >> 7;
  const long long block = blockIdx.x;
  const long long mat = block / (static_cast<long long>(nr) * nc);
  const int rem = static_cast<int>(block - mat * nr * nc);
  const int br = rem / nc, bc = rem - br * nc;
  const int c = bc * 128 + (threadIdx.x & 15) * 8;
  const int r0 = br * 128 + (threadIdx.x >> 4);
  const long long base = mat * rows * cols;
  uint4 q[8];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    q[i] = r < rows && c < cols ? __ldcs(reinterpret_cast<const uint4*>(src + base + static_cast<long long>(r) * cols + c))
                                : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max_nan(top, max_nan(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(FULL_MASK, top, o));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, s_top[i]);
  const float scale = block_scale(top);
  const BlockDivide by(scale);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (r < rows && c < cols) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      *reinterpret_cast<uint2*>(codes + base + static_cast<long long>(r) * cols + c) = by.codes(w);
    }
  }
  if (threadIdx.x == 0) scales[block] = scale;
}

// ---------------------------------------------------------------- few rows

__device__ __forceinline__ void mma_e4m3_16x8x32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

enum StreamMode { STREAM_BF16 = 0, STREAM_WEIGHTED = 1, STREAM_F32 = 2 };
// Where a group's rows come from: codes and scales, bf16 rows to quantise, or
// the fp32 gate/up rows whose SwiGLU is quantised.
enum StreamSource { FROM_CODES = 0, FROM_BF16 = 1, FROM_GATE_UP = 2 };

struct StreamArgs {
  const int* counts;   // [E]; NULL: one group of `rows` rows
  const int* offsets;  // [E + 1]
  int rows, E;
  int N, K, k_blocks;  // weight rows per expert, codes per row
  int n_blocks;        // scale rows per expert
  int split;           // slices of K a CTA's warps are divided into (1, 2, 4 or 8)
  const void* a;       // the rows, by StreamSource
  const float* a_scale;
  const uint8_t* w;
  const float* w_scale;
  const float* row_weight;
  void* out;  // [rows, N] bf16, or fp32
};

constexpr int CTAS = 3;                   // an SM
constexpr int ROWS = BLOCK_STREAM_ROWS;  // 8: one mma operand
// Bytes from one row of codes to the next in shared memory: 64 more than a
// multiple of 128, so that a quarter warp's 16-byte reads of two rows meet
// different banks.
__host__ __device__ constexpr int row_pitch(int K) { return (K + 127) / 128 * 128 + 64; }
constexpr size_t stream_smem(int K, int E) {  // (codes that come as they are take none)
  return E == 0 ? 0 : static_cast<size_t>(ROWS) * row_pitch(K) + ROWS * ((K + 127) / 128) * sizeof(float) + E * sizeof(int);
}

// The experts with rows, ascending, into list (all counts are loaded at once,
// at most 1024, then placed by ballots); returns how many.  All 256 threads.
__device__ __forceinline__ int active_list(const int* counts, int E, int* list) {
  __shared__ int s_found[32];  // experts with rows in each 32
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool has[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) has[i] = threadIdx.x + 256 * i < E && counts[threadIdx.x + 256 * i] > 0;
  unsigned m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = __ballot_sync(FULL_MASK, has[i]);
    if (lane == 0) s_found[8 * i + warp] = __popc(m[i]);
  }
  __syncthreads();
  int upto = s_found[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL_MASK, upto, o);
    if (lane >= o) upto += v;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int before = __shfl_sync(FULL_MASK, upto, 8 * i + warp) - __popc(m[i]);
    if (has[i]) list[before + __popc(m[i] & ((1u << lane) - 1u))] = threadIdx.x + 256 * i;
  }
  __syncthreads();
  return __shfl_sync(FULL_MASK, upto, 31);
}

// An expert's rows as codes and scales in shared memory; rows from cnt to ROWS
// and columns from K to the block's end are zeros.  All 256 threads; a unit is
// a block of 128 codes, 16 threads of 8 codes each.
template <int SRC>
__device__ __forceinline__ void stage_rows(const StreamArgs& args, long long row0, int cnt, uint8_t* codes, float* scales) {
  const int pitch = row_pitch(args.K), kb = args.k_blocks;
  for (int unit = threadIdx.x >> 4; unit < ROWS * kb; unit += 16) {
    const int r = unit / kb, b = unit - r * kb;
    const int c = b * 128 + (threadIdx.x & 15) * 8;
    uint2 q = make_uint2(0, 0);
    float scale = 0.f;
    if (r < cnt) {  // (the same for a unit's 16 threads, as in the shuffles below)
      const long long row = row0 + r;
      const unsigned half = 0xffffu << (threadIdx.x & 16);
      if constexpr (SRC == FROM_BF16) {
        const uint4 v = c < args.K ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(args.a) + row * args.K + c))
                                   : make_uint4(0, 0, 0, 0);
        uint32_t top = bf16x2_abs_max(bf16x2_abs_max(v.x, v.y), bf16x2_abs_max(v.z, v.w));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = bf16x2_abs_max(top, __shfl_xor_sync(half, top, o));
        scale = block_scale(max_nan(bf16_lo(top), bf16_hi(top)));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        q = BlockDivide(scale).codes(w);
      } else {
        const float* gu = static_cast<const float*>(args.a) + row * 2 * args.K + c;
        float h[8] = {};
        float top = 0.f;
        if (c < args.K) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 g = __ldg(reinterpret_cast<const float4*>(gu) + i);
            const float4 u = __ldg(reinterpret_cast<const float4*>(gu + args.K) + i);
            h[4 * i] = silu_mul(g.x, u.x);
            h[4 * i + 1] = silu_mul(g.y, u.y);
            h[4 * i + 2] = silu_mul(g.z, u.z);
            h[4 * i + 3] = silu_mul(g.w, u.w);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(h[i]));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(half, top, o));
        scale = block_scale(top);
        const float y = __fdiv_rn(1.0f, scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] *= y;
        q = make_uint2(e4m3x4(h[0], h[1], h[2], h[3]), e4m3x4(h[4], h[5], h[6], h[7]));
      }
    }
    *reinterpret_cast<uint2*>(codes + r * pitch + c) = q;
    if ((threadIdx.x & 15) == 0) scales[r * kb + b] = scale;
  }
}

// Items are (group with rows, 16-row slabs of its weights, 8 / split of them at
// a time), in that order; a CTA takes a run of them, so that it stages a
// group's rows once, and asks for an item's first weights before it joins the
// sums of the item before.
template <int SRC, int MODE>
__global__ void __launch_bounds__(256, CTAS) stream_kernel(const StreamArgs args) {
  extern __shared__ __align__(128) uint8_t s_codes[];  // [ROWS][pitch], the scales, the list
  __shared__ float s_part[8][4][32];                   // [warp][register][lane]
  float* s_scale = reinterpret_cast<float*>(s_codes + ROWS * row_pitch(args.K));
  int* s_list = reinterpret_cast<int*>(s_scale + ROWS * args.k_blocks);
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int active = args.counts ? active_list(args.counts, args.E, s_list) : 1;
  const int split = args.split, slabs = 8 / split;
  const int ks = warp % split, slab = warp / split;
  const int per_group = ((args.N + 15) / 16 + slabs - 1) / slabs;
  const int items = active * per_group;
  const int per_slice = (args.k_blocks + split - 1) / split;
  const int kb0 = ks * per_slice, kb1 = min(kb0 + per_slice, args.k_blocks);
  const int g = lane >> 2, t = lane & 3;
  const int pitch = row_pitch(args.K);
  const int share = items / gridDim.x, more = items % gridDim.x;
  const int first = blockIdx.x * share + min(static_cast<int>(blockIdx.x), more);
  const int end = first + share + (static_cast<int>(blockIdx.x) < more ? 1 : 0);
  auto expert_of = [&](int item) { return args.counts ? s_list[item / per_group] : 0; };
  auto slab_of = [&](int item) { return (item % per_group) * slabs; };

  const uint8_t *w_lo = nullptr, *w_hi = nullptr;
  const float* sb = nullptr;
  auto aim = [&](int item) {
    const int e = expert_of(item), n0 = (slab_of(item) + slab) * 16;
    // weight rows past N repeat the last one; their sums are not stored
    const uint8_t* w = args.w + static_cast<long long>(e) * args.N * args.K + 16 * t;
    w_lo = w + static_cast<long long>(min(n0 + g, args.N - 1)) * args.K;
    w_hi = w + static_cast<long long>(min(n0 + g + 8, args.N - 1)) * args.K;
    sb = args.w_scale + (static_cast<long long>(e) * args.n_blocks + min(n0 >> 7, args.n_blocks - 1)) * args.k_blocks;
  };
  uint4 wl[2], wh[2], rows[2];  // rows: codes that come as they are are read along with the weights
  float sbk = 0.f, sak[2] = {0.f, 0.f};
  auto load = [&](int kb) {
    if constexpr (SRC == FROM_CODES) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = kb * 128 + 64 * j + 16 * t;
        rows[j] = g < args.rows && k < args.K
                      ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(args.a) +
                                                             static_cast<long long>(g) * args.K + k))
                      : make_uint4(0, 0, 0, 0);
        sak[j] = 2 * t + j < args.rows ? __ldg(args.a_scale + static_cast<long long>(2 * t + j) * args.k_blocks + kb) : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // 64 codes of each row
      const int k = kb * 128 + 64 * j;
      const bool in = k + 16 * t < args.K;
      wl[j] = in ? __ldcs(reinterpret_cast<const uint4*>(w_lo + k)) : make_uint4(0, 0, 0, 0);
      wh[j] = in ? __ldcs(reinterpret_cast<const uint4*>(w_hi + k)) : make_uint4(0, 0, 0, 0);
    }
    sbk = __ldg(sb + kb);
  };
  int staged = -1, cnt = 0;
  long long row0 = 0;
  if (first < end) {
    aim(first);
    if (kb0 < kb1) load(kb0);
  }
  for (int item = first; item < end; ++item) {
    const int e = expert_of(item);
    if (SRC == FROM_CODES) {
      cnt = args.rows;
    } else if (e != staged) {
      // an expert has at most T <= ROWS rows: a token names it at most once
      cnt = min(args.counts ? args.counts[e] : args.rows, ROWS);
      row0 = args.counts ? args.offsets[e] : 0;
      stage_rows<SRC>(args, row0, cnt, s_codes, s_scale);
      staged = e;
      __syncthreads();
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int kb = kb0; kb < kb1; ++kb) {
      const uint4 cl[2] = {wl[0], wl[1]}, ch[2] = {wh[0], wh[1]}, cb[2] = {rows[0], rows[1]};
      const float cs = sbk, ca[2] = {sak[0], sak[1]};
      if (kb + 1 < kb1) {
        load(kb + 1);
      } else if (item + 1 < end) {
        aim(item + 1);
        load(kb0);
      }
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 b = SRC == FROM_CODES
                            ? cb[j] : *reinterpret_cast<const uint4*>(s_codes + g * pitch + kb * 128 + 64 * j + 16 * t);
        const uint32_t a0[4] = {cl[j].x, ch[j].x, cl[j].y, ch[j].y};
        const uint32_t a1[4] = {cl[j].z, ch[j].z, cl[j].w, ch[j].w};
        mma_e4m3_16x8x32(d, a0, b.x, b.y);
        mma_e4m3_16x8x32(d, a1, b.z, b.w);
      }
      // this lane's sums are those of rows 2t and 2t + 1
      const float s0 = (SRC == FROM_CODES ? ca[0] : s_scale[2 * t * args.k_blocks + kb]) * cs;
      const float s1 = (SRC == FROM_CODES ? ca[1] : s_scale[(2 * t + 1) * args.k_blocks + kb]) * cs;
      acc[0] = fmaf(d[0], s0, acc[0]);
      acc[1] = fmaf(d[1], s1, acc[1]);
      acc[2] = fmaf(d[2], s0, acc[2]);
      acc[3] = fmaf(d[3], s1, acc[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[warp][i][lane] = acc[i];
    __syncthreads();  // (also: the staged rows may be replaced)
    // outputs (slab, row, weight row), weight rows fastest
    const int outs = slabs * cnt * 16;
    for (int i = threadIdx.x; i < outs; i += blockDim.x) {
      const int r = i & 15, st = i >> 4;
      const int sl = st / cnt, tok = st - sl * cnt;
      const int n = (slab_of(item) + sl) * 16 + r;
      if (n >= args.N) continue;
      const int ln = (r & 7) * 4 + (tok >> 1), reg = (r >> 3) * 2 + (tok & 1);
      float v = 0.f;
      for (int k = 0; k < split; ++k) v += s_part[sl * split + k][reg][ln];
      const long long row = row0 + tok;
      if constexpr (MODE == STREAM_F32) {
        static_cast<float*>(args.out)[row * args.N + n] = v;
      } else {
        if constexpr (MODE == STREAM_WEIGHTED) v *= args.row_weight[row];
        static_cast<uint16_t*>(args.out)[row * args.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
      }
    }
    __syncthreads();
  }
}

template <int SRC, int MODE>
cudaError_t launch_stream(StreamArgs g, long long groups, cudaStream_t s) {
  // as many slices of K as leave a warp two blocks or more
  g.split = g.k_blocks >= 16 ? 8 : g.k_blocks >= 8 ? 4 : g.k_blocks >= 4 ? 2 : 1;
  const int slabs = 8 / g.split;
  const long long items = groups * (((g.N + 15) / 16 + slabs - 1) / slabs);
  const long long most = static_cast<long long>(CTAS) * sm_count();
  const size_t smem = stream_smem(g.K, SRC == FROM_CODES ? 0 : g.E);
  auto kernel = stream_kernel<SRC, MODE>;
  if (smem > 32 * 1024) {  // (with the static part, above 48 KiB needs leave)
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
  }
  return launch_dependent(kernel, static_cast<unsigned>(items < most ? items : most), 256, smem, s, g);
}

}  // namespace

cudaError_t launch_quantize_block(const uint16_t* src, long long batch, long long rows, int cols, int block_rows,
                                  uint8_t* codes, float* scales, const int* row_token, cudaStream_t s) {
  if (batch == 0 || rows == 0) return cudaSuccess;
  if (block_rows == 1) {
    const long long all = batch * rows;
    const int y = (cols + PIECES * 256 - 1) / (PIECES * 256);
    // a CTA per 8 rows and 1024 columns: the SMs overlap one CTA's loads with
    // another's arithmetic (CTAs that loop, 8 an SM, took a fifth longer)
    const long long need = (all + 7) / 8, most = 1 << 20;
    const dim3 grid(static_cast<unsigned>(need < most ? need : most), y);
    return launch_dependent(quantize_row_blocks_kernel, grid, 256, 0, s, src, all, cols, codes, scales, row_token);
  }
  const long long blocks = batch * ((rows + 127) / 128) * ((cols + 127) / 128);
  return launch_dependent(quantize_square_blocks_kernel, static_cast<unsigned>(blocks), 256, 0, s, src,
                          static_cast<int>(rows), cols, codes, scales);
}

bool block_stream_fits(int rows, int K, int E) {
  return rows <= BLOCK_STREAM_ROWS && stream_smem(K, E) <= 200 * 1024;
}

cudaError_t launch_block_matmul_stream(const uint8_t* a, const float* a_scale, int M, const uint8_t* b,
                                       const float* b_scale, int N, int K, uint16_t* out, cudaStream_t s) {
  StreamArgs g{};
  g.rows = M;
  g.N = N;
  g.K = K;
  g.k_blocks = (K + 127) / 128;
  g.n_blocks = (N + 127) / 128;
  g.a = a;
  g.a_scale = a_scale;
  g.w = b;
  g.w_scale = b_scale;
  g.out = out;
  return launch_stream<FROM_CODES, STREAM_BF16>(g, 1, s);
}

cudaError_t launch_block_experts_stream(const uint16_t* x_disp, const moe_layout& L, int H, int I, const uint8_t* W1,
                                        const float* W1_scale, const uint8_t* W2, const float* W2_scale, float* gu,
                                        uint16_t* y, cudaStream_t s) {
  const long long pairs = static_cast<long long>(L.T) * L.K;
  const long long active = pairs < L.E ? pairs : L.E;
  if (active == 0) return cudaSuccess;
  StreamArgs g{};
  g.counts = L.tokens_per_expert;
  g.offsets = L.offsets;
  g.E = L.E;
  g.N = 2 * I;
  g.K = H;
  g.k_blocks = H / 128;
  g.n_blocks = 2 * I / 128;
  g.a = x_disp;
  g.w = W1;
  g.w_scale = W1_scale;
  g.out = gu;
  const cudaError_t err = launch_stream<FROM_BF16, STREAM_F32>(g, active, s);
  if (err != cudaSuccess) return err;
  g.N = H;
  g.K = I;
  g.k_blocks = I / 128;
  g.n_blocks = H / 128;
  g.a = gu;
  g.w = W2;
  g.w_scale = W2_scale;
  g.row_weight = L.row_weight;
  g.out = y;
  return launch_stream<FROM_GATE_UP, STREAM_WEIGHTED>(g, active, s);
}

}  // namespace moe
