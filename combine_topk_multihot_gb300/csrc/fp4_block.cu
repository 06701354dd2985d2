// Microscaled 4-bit floating point: quantisation, the way back, and the dense
// product with few rows.  The format is in fp4.cuh.

#include <cuda_fp16.h>

#include "fp4.cuh"
#include "launch.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- quantisation

// A warp takes 256 columns of four rows that lie 32 apart, whose scale words are
// neighbours in their tile; lane l holds 8 values of each, 4 lanes a block, 16
// lanes a scale word.  Rows up to the next multiple of 128 have scales only,
// zeros.  Every quotient is a product with a power of two, so codes are functions
// of the input alone.  403 M bf16 weights take 189 us, 5.4 TB/s (a row a warp: 217),
// which the instructions bound as much as HBM: the issue slots are 79 % busy, the integer
// pipe, which compares and packs, 66 %, HBM 60 % by the profiler's peak.
constexpr int PIECES = 4;
template <bool F32>
__global__ void __launch_bounds__(256, F32 ? 4 : 5) quantize_fp4_kernel(const void* __restrict__ src, long long all, int rows,
                                                                       int row_tiles, int cols, uint8_t* __restrict__ codes,
                                                                       uint8_t* __restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int kts = (cols + 127) >> 7;
  const int c = blockIdx.y * 256 + lane * 8, kt = c >> 7;
  const long long nwarps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long i = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < all; i += nwarps) {
    const long long tile = i >> 5;  // of all matrices' row tiles
    const long long mat = all == 32ll * row_tiles ? 0 : tile / row_tiles;
    const int row0 = static_cast<int>(tile - mat * row_tiles) * 128 + static_cast<int>(i & 31);
    uint4 q[PIECES][F32 ? 2 : 1];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const bool in = row0 + 32 * p < rows && c < cols;
      const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) +
                                                       ((mat * rows + row0 + 32 * p) * cols + c) * (F32 ? 4 : 2));
#pragma unroll
      for (int k = 0; k < (F32 ? 2 : 1); ++k) q[p][k] = in ? __ldcs(at + k) : make_uint4(0, 0, 0, 0);
    }
    uint32_t words[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      float v[8], top;
      if constexpr (F32) {
        top = 0.f;
        const uint32_t w[8] = {q[p][0].x, q[p][0].y, q[p][0].z, q[p][0].w, q[p][1].x, q[p][1].y, q[p][1].z, q[p][1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] = __uint_as_float(w[k]);
          top = max_nan(top, fabsf(v[k]));
        }
        top = max_nan(top, __shfl_xor_sync(FULL_MASK, top, 1));
        top = max_nan(top, __shfl_xor_sync(FULL_MASK, top, 2));
      } else {
        const uint32_t w[4] = {q[p][0].x, q[p][0].y, q[p][0].z, q[p][0].w};
        uint32_t t = bf16x2_abs_max(bf16x2_abs_max(w[0], w[1]), bf16x2_abs_max(w[2], w[3]));
        t = bf16x2_abs_max(t, __shfl_xor_sync(FULL_MASK, t, 1));
        t = bf16x2_abs_max(t, __shfl_xor_sync(FULL_MASK, t, 2));
        top = max_nan(bf16_lo(t), bf16_hi(t));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(w[k]), v[2 * k + 1] = bf16_hi(w[k]);
      }
      const uint32_t e = e8m0_of(top);
      const float f = e8m0_inverse(e);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= f;
      const uint32_t code = e == 255u ? 0u : e2m1x8(v);
      if (row0 + 32 * p < rows && c < cols) *reinterpret_cast<uint32_t*>(codes + ((mat * rows + row0 + 32 * p) * cols + c) / 2) = code;
      uint32_t s = e << (8 * ((lane >> 2) & 3));
      s |= __shfl_xor_sync(FULL_MASK, s, 4);
      words[p] = s | __shfl_xor_sync(FULL_MASK, s, 8);
    }
    if ((lane & 15) == 0 && kt < kts)
      *reinterpret_cast<uint4*>(scales + (tile * kts + kt) * SCALE_TILE + (i & 31) * 16) =
          make_uint4(words[0], words[1], words[2], words[3]);
  }
}

// The way back: exact in either type, a code has two significant bits.  A warp takes
// up to four 256-column pieces of one row; blockIdx.y picks the pieces.  Bound by
// HBM: 403 M bf16 weights take 146 us, 7.0 TB/s.
template <bool F32>
__global__ void __launch_bounds__(256) dequantize_fp4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                             long long all, int rows, int cols, void* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int kts = (cols + 127) >> 7;
  const long long tiles = static_cast<long long>((rows + 127) >> 7) * kts * SCALE_TILE;
  const int col0 = blockIdx.y * (PIECES * 256) + lane * 8;
  const long long nwarps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long r = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); r < all; r += nwarps) {
    const long long mat = all == rows ? 0 : r / rows;
    const uint8_t* sc = scales + mat * tiles + scale_word(r - mat * rows, 0, kts);
    uint32_t c[PIECES], e[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int col = col0 + 256 * p;
      c[p] = col < cols ? __ldcs(reinterpret_cast<const uint32_t*>(codes + (r * cols + col) / 2)) : 0u;
      e[p] = col < cols ? __ldg(sc + static_cast<long long>(col >> 7) * SCALE_TILE + ((col >> 5) & 3)) : 0u;
    }
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int col = col0 + 256 * p;
      if (col >= cols) break;
      const float f = e8m0_value(e[p]);
      uint32_t halves[4];
      f16_of_e2m1x8(c[p], halves);
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&halves[k]));
        v[2 * k] = t.x * f, v[2 * k + 1] = t.y * f;
      }
      if constexpr (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + r * cols + col);
        __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
      } else {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + r * cols + col),
               make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
      }
    }
  }
}

// ---------------------------------------------------------------- few rows

// The product with at most 8 rows is a stream over the weights: a warp takes 16
// of their rows and a slice of K, and multiplies with mma.sync, the 8 rows as its
// other operand.  Codes become f16 numbers (exact) in registers; lane t of a row's
// four takes word t of each block of 32, so that two instructions' 32 products
// share their scales, which are applied to the sums.  The slices of K are joined in
// shared memory in a fixed order.  It takes the calls of few tiles (8 rows by 1024
// columns at the most), where the tensor cores' kernel leaves SMs idle and is bound by its
// start and end (8 x 1024 x 8192: 8.8 us here, 11.3 there); with more columns that one is
// faster at the larger depths (8 x 16384 x 4096: 12 us for 23 here).
// 2^(ea + eb - 254) as two factors: their product may leave fp32's range where
// the value does not.
struct Scale2 {
  float f1, f2;
  __device__ __forceinline__ Scale2(uint32_t ea, uint32_t eb) {
    const int s = static_cast<int>(ea + eb) - 254, h = s >> 1;
    const bool nan = ea == 255u || eb == 255u;
    f1 = nan ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(min(h, 127) + 127) << 23);
    f2 = __uint_as_float(static_cast<uint32_t>(min(s - h, 127) + 127) << 23);
  }
};

struct StreamArgs {
  const uint8_t *a, *a_scale, *w, *w_scale;
  int rows, N, K, split;
  uint16_t* out;
};

__global__ void __launch_bounds__(256, 3) fp4_stream_kernel(const StreamArgs args) {
  __shared__ float s_part[8][4][32];  // [warp][register][lane]
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int split = args.split, slabs = 8 / split;
  const int ks = warp % split, slab = warp / split;
  const int items = ((args.N + 15) / 16 + slabs - 1) / slabs;
  const int kts = (args.K + 127) >> 7;
  const int per_slice = (kts + split - 1) / split;
  const int kt0 = ks * per_slice, kt1 = min(kt0 + per_slice, kts);
  const int g = lane >> 2, t = lane & 3;
  const int row_bytes = args.K >> 1;
  uint32_t wl[4], wh[4], rw[4], sl = 0, sh = 0, sr[2] = {0, 0};
  auto load = [&](int item, int kt) {
    const int n0 = (item * slabs + slab) * 16;
    // weight rows past N repeat the last one; their sums are not stored
    const long long lo = min(n0 + g, args.N - 1), hi = min(n0 + g + 8, args.N - 1);
    const int at = kt * 64 + 4 * t;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = at + 16 * j < row_bytes;
      wl[j] = in ? __ldg(reinterpret_cast<const uint32_t*>(args.w + lo * row_bytes + at + 16 * j)) : 0u;
      wh[j] = in ? __ldg(reinterpret_cast<const uint32_t*>(args.w + hi * row_bytes + at + 16 * j)) : 0u;
      rw[j] = in && g < args.rows ? __ldg(reinterpret_cast<const uint32_t*>(args.a + static_cast<long long>(g) * row_bytes + at + 16 * j)) : 0u;
    }
    sl = __ldg(reinterpret_cast<const uint32_t*>(args.w_scale + scale_word(lo, kt, kts)));
    sh = __ldg(reinterpret_cast<const uint32_t*>(args.w_scale + scale_word(hi, kt, kts)));
#pragma unroll
    for (int j = 0; j < 2; ++j) sr[j] = 2 * t + j < args.rows ? __ldg(reinterpret_cast<const uint32_t*>(args.a_scale + scale_word(2 * t + j, kt, kts))) : 0u;
  };
  if (blockIdx.x < items && kt0 < kt1) load(blockIdx.x, kt0);
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int kt = kt0; kt < kt1; ++kt) {
      uint32_t cl[4], ch[4], cr[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) cl[j] = wl[j], ch[j] = wh[j], cr[j] = rw[j];
      const uint32_t el = sl, eh = sh, er[2] = {sr[0], sr[1]};
      if (kt + 1 < kt1) load(item, kt + 1);
      else if (item + static_cast<int>(gridDim.x) < items) load(item + gridDim.x, kt0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kt * 4 + j >= args.K / FP4_BLOCK) break;  // past the last block: its scales are no one's
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t lo[4], hi[4], row[4];
        f16_of_e2m1x8(cl[j], lo);
        f16_of_e2m1x8(ch[j], hi);
        f16_of_e2m1x8(cr[j], row);
        mma_f16_16x8x16(d, lo[0], hi[0], lo[1], hi[1], row[0], row[1]);
        mma_f16_16x8x16(d, lo[2], hi[2], lo[3], hi[3], row[2], row[3]);
        // this lane's sums are those of rows 2t and 2t + 1, weight rows g and g + 8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Scale2 f((er[i & 1] >> (8 * j)) & 255u, ((i < 2 ? el : eh) >> (8 * j)) & 255u);
          acc[i] = fmaf(d[i] * f.f1, f.f2, acc[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[warp][i][lane] = acc[i];
    __syncthreads();
    // outputs (slab, row, weight row), weight rows fastest
    const int outs = slabs * args.rows * 16;
    for (int i = threadIdx.x; i < outs; i += blockDim.x) {
      const int r = i & 15, st = i >> 4;
      const int sb = st / args.rows, tok = st - sb * args.rows;
      const int n = (item * slabs + sb) * 16 + r;
      if (n >= args.N) continue;
      const int ln = (r & 7) * 4 + (tok >> 1), reg = (r >> 3) * 2 + (tok & 1);
      float v = 0.f;
      for (int k = 0; k < split; ++k) v += s_part[sb * split + k][reg][ln];
      args.out[static_cast<long long>(tok) * args.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* src, bool f32, long long batch, long long rows, int cols, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s) {
  const int row_tiles = static_cast<int>((rows + 127) / 128);
  const long long all = batch * row_tiles * 32;
  if (all == 0) return cudaSuccess;
  const long long need = (all + 7) / 8, most = 1 << 20;
  const dim3 grid(static_cast<unsigned>(need < most ? need : most), (cols + 255) / 256);
  return launch_dependent(f32 ? quantize_fp4_kernel<true> : quantize_fp4_kernel<false>, grid, 256, 0, s, src, all,
                          static_cast<int>(rows), row_tiles, cols, codes, scales);
}

cudaError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, long long batch, long long rows, int cols, bool f32,
                                  void* out, cudaStream_t s) {
  const long long all = batch * rows;
  if (all == 0) return cudaSuccess;
  const int y = (cols + PIECES * 256 - 1) / (PIECES * 256);
  const long long need = (all + 7) / 8, most = 1 << 20;
  const dim3 grid(static_cast<unsigned>(need < most ? need : most), y);
  return launch_dependent(f32 ? dequantize_fp4_kernel<true> : dequantize_fp4_kernel<false>, grid, 256, 0, s, codes, scales, all,
                          static_cast<int>(rows), cols, out);
}

cudaError_t launch_fp4_matmul_stream(const uint8_t* a, const uint8_t* a_scale, int M, const uint8_t* b, const uint8_t* b_scale, int N,
                                     int K, uint16_t* out, cudaStream_t s) {
  StreamArgs g{a, a_scale, b, b_scale, M, N, K, 0, out};
  const int kts = (K + 127) / 128;
  g.split = kts >= 8 ? 8 : kts >= 4 ? 4 : kts >= 2 ? 2 : 1;
  const int slabs = 8 / g.split;
  const int items = ((N + 15) / 16 + slabs - 1) / slabs, most = 3 * sm_count();
  return launch_dependent(fp4_stream_kernel, items < most ? items : most, 256, 0, s, g);
}

}  // namespace moe
