// Products of e2m1 codes with a scale for each 32 of a row, on the 5th-
// generation tensor cores.
//
//   C[m, n] = sum_b sa[m, b] sb[n, b] sum_{k in block b} a[m, k] b[n, k]
//
// The tensor cores apply these scales themselves (tcgen05.mma kind::mxf4, 64
// codes an instruction): they are read from tensor memory, where tcgen05.cp puts
// each tile of 128 rows' scales, 512 bytes, from shared memory.
//   * warp 0 stages codes by TMA (128-byte swizzle, 256 codes a stage) and
//     scales by bulk copies, warp 1 copies a stage's scales to its own columns of
//     tensor memory and issues its MMAs, warps 4..11 take the finished tile out:
//     bf16, through shared memory and TMA stores;
//   * a stage's scale columns are written again only after the MMAs that read
//     them have finished (the same barrier that frees its shared memory).
// One persistent CTA per SM; every wait is bounded, and a wait that runs out
// sets MOE_DEVERR_TIMEOUT, drains and leaves NaN in the tiles not reached.

#include "common.cuh"
#include "fp4.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int BM = 128;
constexpr int BKC = 256;  // codes a stage: 128 bytes of a row
constexpr int MAX_STAGES = 8;
constexpr int SMEM_LIMIT = 232448;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (4 + EPI_WARPS);
constexpr int STAGING_BYTES = EPI_WARPS * 2048;

template <int BN>
struct Shape {
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int B_TILES = (BN + 127) / 128;  // of scales
  static constexpr int SF_BYTES = 2 * SCALE_TILE * (1 + B_TILES);
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 5 : 7;
  static constexpr int BUFS = BN == 256 ? 1 : 2;
  static constexpr int SF_COLS = 8 * (1 + B_TILES);  // of a stage
  static constexpr int TMEM_COLS = 512;
  static_assert(BN * BUFS + STAGES * SF_COLS <= TMEM_COLS, "accumulators and scales fit in tensor memory");
};

struct Smem {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int BN>
constexpr size_t smem_bytes() {
  return 1024 + static_cast<size_t>(Shape<BN>::STAGES) * Shape<BN>::STAGE_BYTES + STAGING_BYTES + sizeof(Smem);
}

struct Args {
  const uint8_t *a_scale, *b_scale;
  int M, N, K;
  int k_steps;   // stages of a tile
  int kts;       // block tiles of a scale row
  int n_tiles, tiles;
  uint16_t* out;
  int out_staged;
  int* status;
};

// untiled copy of whole 16 bytes into shared memory
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// A tile of scales: 32 rows of 16 bytes to four columns of each 32-lane quarter.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);  // no swizzle
  d |= static_cast<uint64_t>(128 >> 4) << 32;                   // 8 rows x 16 B to the next 8 rows
  d |= static_cast<uint64_t>(1) << 46;                          // descriptor version
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// e2m1 x e2m1 with e8m0 scales, fp32 accumulator, M x N tile; `id`: the first of
// the two scale bytes in each column word (0 or 2).
__device__ __forceinline__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t id) {
  return (id << 4)                                  // B's scale bytes
         | (1u << 7)                                // A format: e2m1
         | (1u << 10)                               // B format: e2m1
         | (static_cast<uint32_t>(N >> 3) << 17)    // N / 8
         | (1u << 23)                               // scales: e8m0
         | (static_cast<uint32_t>(M >> 4) << 24)    // M / 16
         | (id << 29);                              // A's scale bytes
}

template <int BN>
__global__ void __launch_bounds__(THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmOut, const Args args) {
  using S = Shape<BN>;
  constexpr int STAGES = S::STAGES, BUFS = S::BUFS, COLS = BN / 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* tiles = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(tiles + STAGES * S::STAGE_BYTES + STAGING_BYTES);
  const uint32_t tiles_u32 = smem_u32(tiles);
  // codes of all stages, then their scales, then the output's staging
  const uint32_t sf_u32 = tiles_u32 + STAGES * (S::A_BYTES + S::B_BYTES);
  const uint32_t staging_u32 = tiles_u32 + STAGES * S::STAGE_BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(smem_u32(&s.tfull[i]), 1);
      mbar_init(smem_u32(&s.tempty[i]), EPI_WARPS);
    }
    mbar_init(smem_u32(&s.drain), 1);
    s.abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (args.out_staged) tma_prefetch_desc(&tmOut);
  }
  if (warp == 1) tmem_alloc(smem_u32(&s.tmem_base), S::TMEM_COLS);
  griddep_wait();  // the codes and scales come from earlier kernels
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = s.tmem_base;
  volatile int* abort_flag = &s.abort;

  if (warp == 0 && lane == 0) {
    // ================= TMA producer =================
    const int b_row_tiles = (args.N + 127) >> 7;
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < args.tiles && ok; tile += gridDim.x) {
      const int mt = tile / args.n_tiles, n0 = (tile - mt * args.n_tiles) * BN;
      for (int ks = 0; ks < args.k_steps; ++ks) {
        if (!mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t full = smem_u32(&s.full[stage]);
        const uint32_t a_dst = tiles_u32 + stage * (S::A_BYTES + S::B_BYTES);
        const uint32_t sf = sf_u32 + stage * S::SF_BYTES;
        const uint32_t bytes = min(2, args.kts - 2 * ks) * SCALE_TILE;  // a last half stage has one tile a row
        int b_tiles = 0;
#pragma unroll
        for (int i = 0; i < S::B_TILES; ++i) b_tiles += (n0 >> 7) + i < b_row_tiles;
        mbar_arrive_expect_tx(full, S::A_BYTES + S::B_BYTES + bytes * (1 + b_tiles));
        tma_load_2d(a_dst, &tmA, ks * 128, mt * BM, full);
        tma_load_2d(a_dst + S::A_BYTES, &tmB, ks * 128, n0, full);
        if constexpr (BN == 256) tma_load_2d(a_dst + S::A_BYTES + S::B_BYTES / 2, &tmB, ks * 128, n0 + 128, full);
        bulk_load(sf, args.a_scale + (static_cast<long long>(mt) * args.kts + 2 * ks) * SCALE_TILE, bytes, full);
#pragma unroll
        for (int i = 0; i < S::B_TILES; ++i)
          if (i < b_tiles)
            bulk_load(sf + (1 + i) * 2 * SCALE_TILE,
                      args.b_scale + (static_cast<long long>((n0 >> 7) + i) * args.kts + 2 * ks) * SCALE_TILE, bytes, full);
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok) {  // wait for the loads of the last (up to STAGES) issued stages
      for (int i = 0; i < STAGES && i < issued; ++i) {
        if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
        mbar_wait_drain(smem_u32(&s.full[stage]), phase);
      }
    }
  } else if (warp == 1 && lane == 0) {
    // ================= scales and MMAs =================
    int stage = 0, buf = 0;
    uint32_t phase = 0, use = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < args.tiles && ok; tile += gridDim.x) {
      const int n0 = tile % args.n_tiles * BN;
      if (!mbar_wait(smem_u32(&s.tempty[buf]), use ^ 1u, abort_flag)) break;
      tc_fence_after();
      for (int ks = 0; ks < args.k_steps; ++ks) {
        if (!mbar_wait(smem_u32(&s.full[stage]), phase, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sf = sf_u32 + stage * S::SF_BYTES;
        const uint32_t tsa = tmem_base + BN * BUFS + stage * S::SF_COLS, tsb = tsa + 8;
        const int left = args.K - ks * BKC;  // codes from here on
        // columns: A's scales of each 128 codes (4), then B's (4 for each 128 rows)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          if (kt * 128 >= left) break;
          tc_copy_scales(tsa + kt * 4, sf + kt * SCALE_TILE);
#pragma unroll
          for (int i = 0; i < S::B_TILES; ++i)
            tc_copy_scales(tsb + (kt * S::B_TILES + i) * 4, sf + ((1 + i) * 2 + kt) * SCALE_TILE);
        }
        const uint32_t a_addr = tiles_u32 + stage * (S::A_BYTES + S::B_BYTES);
        const uint64_t a_desc = sdesc_k_sw128(a_addr);
        const uint64_t b_desc = sdesc_k_sw128(a_addr + S::A_BYTES);
        const uint32_t skew = BN == 64 ? (n0 & 64) >> 5 : 0;  // rows 64.. of a tile of scales
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk * 64 >= left) break;
          tc_mma_mxf4(tmem_base + buf * BN, a_desc + 2 * kk, b_desc + 2 * kk, kk & 1 ? idesc_mxf4(BM, BN, 2) : idesc_mxf4(BM, BN, 0),
                      tsa + (kk >> 1) * 4, tsb + (kk >> 1) * 4 * S::B_TILES + skew, ks != 0 || kk != 0);
        }
        tc_commit(smem_u32(&s.empty[stage]));
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      tc_commit(smem_u32(&s.tfull[buf]));
      if (++buf == BUFS) { buf = 0; use ^= 1u; }
    }
    // every operation this thread issued has finished before anyone frees memory
    tc_commit(smem_u32(&s.drain));
    if (!mbar_wait_drain(smem_u32(&s.drain), 0)) *abort_flag = 1;
  } else if (warp >= 4) {
    // ================= epilogue =================
    // lane quarter q = warp % 4 of tensor memory; column half = (warp - 4) / 4
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t staging = staging_u32 + (warp - 4) * 2048;
    int buf = 0;
    uint32_t use = 0;
    int tile = blockIdx.x;
    for (; tile < args.tiles; tile += gridDim.x) {
      const bool ready = mbar_wait(smem_u32(&s.tfull[buf]), use, abort_flag);
      if (!__all_sync(FULL_MASK, ready)) break;
      tc_fence_after();
      const int mt = tile / args.n_tiles, nt = tile - mt * args.n_tiles;
      const int row0 = mt * BM + q * 32, col0 = nt * BN + half * COLS;
      const int rows = min(args.M - row0, 32);
      const uint32_t tb = tmem_base + buf * BN + half * COLS + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < COLS; c += 32) {
        uint32_t p[32];
        tmem_ld32(tb + c, p);
        tmem_ld_wait();
        if (c + 32 >= COLS) {  // all of this warp's reads have landed
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.tempty[buf]));
        }
        if (col0 + c >= args.N || rows <= 0) continue;
        if (lane == 0) tma_store_wait_read<0>();  // the box before
        __syncwarp();
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = pack_bf16x2(__uint_as_float(p[2 * k]), __uint_as_float(p[2 * k + 1]));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(staging + staged_chunk(lane, i)), "r"(v[4 * i]),
                       "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                       : "memory");
        if (args.out_staged) {  // rows and columns past the matrix are clipped by the tensor map
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, staging, col0 + c, row0);
            tma_store_commit();
          }
        } else {  // rows that do not start on 16 bytes: the warp writes 32 neighbours of a row at a time
          __syncwarp();
          uint16_t* dst = args.out + static_cast<long long>(row0) * args.N + col0 + c + lane;
          const bool there = col0 + c + lane < args.N;
#pragma unroll 4
          for (int r = 0; r < rows; ++r, dst += args.N) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(staging + staged_chunk(r, lane >> 3) + 2 * (lane & 7)) : "memory");
            if (there) *dst = h;
          }
          __syncwarp();
        }
      }
      if (++buf == BUFS) { buf = 0; use ^= 1u; }
    }
    // after a wait that ran out: this warp's part of the tiles not reached
    for (; tile < args.tiles; tile += gridDim.x) {
      const int mt = tile / args.n_tiles, nt = tile - mt * args.n_tiles;
      const int row0 = mt * BM + q * 32, col0 = nt * BN + half * COLS;
      const int rows = min(args.M - row0, 32), cols = min(args.N - col0, COLS);
#pragma unroll 1
      for (int r = 0; r < rows; ++r)
#pragma unroll 1
        for (int c = lane; c < cols; c += 32) args.out[static_cast<long long>(row0 + r) * args.N + col0 + c] = 0x7fc0;
    }
    if (lane == 0) tma_store_wait_all();
  }
  __syncwarp();

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, S::TMEM_COLS);
  if (threadIdx.x == 0 && s.abort) report(args.status, MOE_DEVERR_TIMEOUT);
}

template <int BN>
cudaError_t launch(const void* a, const void* b, Args args, cudaStream_t s) {
  args.n_tiles = (args.N + BN - 1) / BN;
  args.tiles = (args.M + BM - 1) / BM * args.n_tiles;
  CUtensorMap ma, mb, mo;
  if (!make_tma_2d_u8(&ma, a, args.M, args.K / 2, BM) || !make_tma_2d_u8(&mb, b, args.N, args.K / 2, BN == 256 ? 128 : BN))
    return cudaErrorInvalidValue;
  if (args.out_staged && !make_tma_store_2d_bf16(&mo, args.out, args.M, args.N)) return cudaErrorInvalidValue;
  if (!args.out_staged) mo = ma;  // not used
  auto kernel = fp4_gemm_kernel<BN>;
  static_assert(smem_bytes<BN>() <= SMEM_LIMIT, "fits");
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<BN>());
  if (err != cudaSuccess) return err;
  const int sms = sm_count();
  return launch_dependent(kernel, args.tiles < sms ? args.tiles : sms, THREADS, smem_bytes<BN>(), s, ma, mb, mo, args);
}

}  // namespace

cudaError_t launch_fp4_matmul_tc(const uint8_t* a, const uint8_t* a_scale, int M, const uint8_t* b, const uint8_t* b_scale, int N,
                                 int K, uint16_t* out, int* status, cudaStream_t s) {
  Args g{};
  g.a_scale = a_scale;
  g.b_scale = b_scale;
  g.M = M;
  g.N = N;
  g.K = K;
  g.k_steps = (K + BKC - 1) / BKC;
  g.kts = (K + 127) / 128;
  g.out = out;
  g.out_staged = N % 8 == 0;
  g.status = status;
  const long long mt = (M + BM - 1) / BM;
  const int sms = sm_count();
  auto rounds = [&](int bn) { return (mt * ((N + bn - 1) / bn) + sms - 1) / sms * bn; };
  const long long r64 = rounds(64), r128 = rounds(128), r256 = rounds(256);
  if (r256 <= r128 && r256 <= r64) return launch<256>(a, b, g, s);
  if (r128 <= r64) return launch<128>(a, b, g, s);
  return launch<64>(a, b, g, s);
}

}  // namespace moe
