// Products of e2m1 codes with a scale for each 32 of a row, on the 5th-
// generation tensor cores.
//
//   C[m, n] = sum_b sa[m, b] sb[n, b] sum_{k in block b} a[m, k] b[n, k]
//
// The tensor cores apply these scales themselves (tcgen05.mma kind::mxf4, 64
// codes an instruction): they are read from tensor memory, where tcgen05.cp puts
// each tile of 128 rows' scales, 512 bytes, from shared memory.
//   * warps 0 and 3 stage codes (128-byte swizzle, 256 codes a stage) and scales by
//     TMA, warp 2 copies a stage's scales to its own columns of tensor memory while
//     warp 1 issues the MMAs of the stage before, warps 4..11 take the finished tile out: to bf16 in
//     registers, which frees the accumulator, then through shared memory and TMA
//     stores;
//   * a stage's scale columns are written again only after the MMAs that read
//     them have finished (the same barrier that frees its shared memory);
//   * above 128 rows two CTAs on two SMs share a tile of 256 rows (cta_group::2): each
//     holds 128 rows of a, half of b's, and the scales of its rows of a and of all
//     of b's.  What bounds a tile of one CTA is L2: 384 rows arrive for
//     128 x 256 of output, 256 for as much of a pair's.
// One persistent CTA per SM; every wait is bounded, and a wait that runs out
// sets MOE_DEVERR_TIMEOUT, drains and leaves NaN in the tiles not reached.
//
// 8192 x 8192 x 4096 takes 82.5 us (6.7 PFLOP/s; the tensor pipe is busy 70 % of the
// time), 8192 x 8192 x 8192 151 (7.3), 4097 x 4096 x 4096 25.1, 333 x 4097 x 2080 7.3.
// What is left is the way out of a tile of 256 columns, for which tensor memory beside
// the scales has one accumulator (1 us a tile), and the operands' way from L2.  What carries it: a
// warp issues as a whole with an elected lane (MMAs and loads issued from a branch of one
// lane take 80 to 200 cycles each: 208 us), loads by two warps and the scales' copies
// by a third (88 us).  Slower: K split over clusters, fewer or more stages.

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
constexpr int STAGING_BYTES = EPI_WARPS * 4096;

template <int BN, bool PAIR>
struct Shape {
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;  // of this CTA
  static constexpr int B_BYTES = B_ROWS * 128;
  static constexpr int B_TILES = (BN + 127) / 128;  // of scales
  static constexpr int SF_BYTES = 2 * SCALE_TILE * (1 + B_TILES);
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;
  static constexpr int BUFS = BN == 256 ? 1 : 2;
  static constexpr int SF_COLS = 8 * (1 + B_TILES);  // of a stage
  static constexpr int TMEM_COLS = 512;
  // as many stages as shared memory and the scales' tensor memory hold
  static constexpr int IN_SMEM = (SMEM_LIMIT - 1024 - STAGING_BYTES - 512) / STAGE_BYTES, IN_TMEM = (TMEM_COLS - BN * BUFS) / SF_COLS;
  static constexpr int MOST = IN_SMEM < IN_TMEM ? IN_SMEM : IN_TMEM;
  static constexpr int STAGES = MOST < MAX_STAGES ? MOST : MAX_STAGES;
  static_assert(BN * BUFS + STAGES * SF_COLS <= TMEM_COLS, "accumulators and scales fit in tensor memory");
};

struct Smem {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t scaled[MAX_STAGES];  // the stage's scales are in tensor memory
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
  uint32_t issued;    // of the odd CTA's stages
};

template <int BN, bool PAIR>
constexpr size_t smem_bytes() {
  return 1024 + static_cast<size_t>(Shape<BN, PAIR>::STAGES) * Shape<BN, PAIR>::STAGE_BYTES + STAGING_BYTES + sizeof(Smem);
}

struct Args {
  int M, N, K;
  int k_steps;   // stages of a tile
  int n_tiles, tiles;
  uint16_t* out;
  int out_staged;
  int* status;
  int load_tiles;  // tiles a CTA loads operands for: all, but in the self-test
  unsigned long long pair_wait_ns;
};

// Loads whose arrival is counted on this CTA's barrier, or on the even CTA's.
template <bool PAIR>
__device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (PAIR) tma_load_2d_pair(dst, map, x, y, bar);
  else tma_load_2d(dst, map, x, y, bar);
}

// A tile of scales: 32 rows of 16 bytes to four columns of each 32-lane quarter
// (of a pair: each CTA's from its own shared memory).
template <bool PAIR>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);  // no swizzle
  d |= static_cast<uint64_t>(128 >> 4) << 32;                   // 8 rows x 16 B to the next 8 rows
  d |= static_cast<uint64_t>(1) << 46;                          // descriptor version
  if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// One lane of a warp that runs as a whole, always the same: what such a lane
// issues has its operands in uniform registers already (in a branch for lane 0
// each MMA or load took 80 to 200 cycles to issue).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// A barrier's wait by the whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(FULL_MASK, mbar_wait(bar, parity, abort_flag));
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (PAIR) tc_commit_pair(bar);
  else tc_commit(bar);
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

template <int BN, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmOut, const Args args) {
  using S = Shape<BN, PAIR>;
  constexpr int STAGES = S::STAGES, BUFS = S::BUFS, COLS = BN / 2, CTAS = PAIR ? 2 : 1;
  constexpr uint32_t IDESC0 = idesc_mxf4(CTAS * BM, BN, 0), IDESC2 = idesc_mxf4(CTAS * BM, BN, 2);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* tiles = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(tiles + STAGES * S::STAGE_BYTES + STAGING_BYTES);
  const uint32_t tiles_u32 = smem_u32(tiles);
  // codes of all stages, then their scales, then the output's staging
  const uint32_t sf_u32 = tiles_u32 + STAGES * (S::A_BYTES + S::B_BYTES);
  const uint32_t staging_u32 = tiles_u32 + STAGES * S::STAGE_BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;  // the even CTA of a pair issues the MMAs
  const int tile0 = blockIdx.x / CTAS, step = gridDim.x / CTAS;
  griddep_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
      mbar_init(smem_u32(&s.scaled[i]), 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(smem_u32(&s.tfull[i]), 1);
      mbar_init(smem_u32(&s.tempty[i]), CTAS * EPI_WARPS);
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&s.drain[i]), 1);
    s.abort = 0;
    s.issued = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    if (args.out_staged) tma_prefetch_desc(&tmOut);
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(smem_u32(&s.tmem_base), S::TMEM_COLS);
    else tmem_alloc(smem_u32(&s.tmem_base), S::TMEM_COLS);
  }
  griddep_wait();  // the codes and scales come from earlier kernels
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers are there before either signals the other's
  tc_fence_after();

  const uint32_t tmem_base = s.tmem_base;
  volatile int* abort_flag = &s.abort;

  if (warp == 0 || warp == 3) {
    // ================= TMA producers: a and its scales, b and its scales =================
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    int left = args.load_tiles;
    for (int tile = tile0; tile < args.tiles && ok && left > 0; tile += step, --left) {
      const int mt = tile / args.n_tiles, n0 = (tile - mt * args.n_tiles) * BN;
      const int row_tile = mt * CTAS + rank;  // this CTA's 128 rows of a
      for (int ks = 0; ks < args.k_steps; ++ks) {
        if (!warp_wait(smem_u32(&s.empty[stage]), phase ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t full = smem_u32(&s.full[stage]), full0 = PAIR ? mapa_shared(full, 0) : full;
        const uint32_t a_dst = tiles_u32 + stage * (S::A_BYTES + S::B_BYTES);
        const uint32_t sf = sf_u32 + stage * S::SF_BYTES;
        if (elect_one()) {  // (what lies past a matrix arrives as zeros)
          if (warp == 0) {
            if (rank == 0) mbar_arrive_expect_tx(full, CTAS * S::STAGE_BYTES);
            else *const_cast<volatile uint32_t*>(&s.issued) = static_cast<uint32_t>(issued) + 1;
            load<PAIR>(a_dst, &tmA, ks * 128, row_tile * BM, full0);
            load<PAIR>(sf, &tmSA, ks * 256, row_tile, full0);
          } else {
            load<PAIR>(a_dst + S::A_BYTES, &tmB, ks * 128, n0 + rank * S::B_ROWS, full0);
            load<PAIR>(sf + 2 * SCALE_TILE, &tmSB, ks * 256, n0 >> 7, full0);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && rank == 0) {  // wait for the loads of the last (up to STAGES) issued stages
      for (int i = 0; i < STAGES && i < issued; ++i) {
        if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
        mbar_wait_drain(smem_u32(&s.full[stage]), phase);
      }
    }
  } else if (warp < 3 && rank != 0) {
    // the odd CTA issues nothing; it waits until the even CTA's last operations,
    // which write its tensor memory, have finished: as long as its own loads go on
    if (!mbar_wait_working(smem_u32(&s.drain[warp - 1]), 0, &s.issued, args.pair_wait_ns)) *abort_flag = 1;
  } else if (warp == 2) {
    // ================= scales to tensor memory =================
    int stage = 0;
    uint32_t phase = 0;
    const int my_tiles = tile0 < args.tiles ? (args.tiles - 1 - tile0) / step + 1 : 0;
    for (long long i = static_cast<long long>(my_tiles) * args.k_steps; i > 0; --i) {
      if (!warp_wait(smem_u32(&s.full[stage]), phase, abort_flag)) break;
      tc_fence_after();
      const uint32_t sf = sf_u32 + stage * S::SF_BYTES;
      const uint32_t tsa = tmem_base + BN * BUFS + stage * S::SF_COLS, tsb = tsa + 8;
      if (elect_one()) {
        // columns: A's scales of each 128 codes (4), then B's (4 for each 128 rows)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          tc_copy_scales<PAIR>(tsa + kt * 4, sf + kt * SCALE_TILE);
#pragma unroll
          for (int i = 0; i < S::B_TILES; ++i)
            tc_copy_scales<PAIR>(tsb + (kt * S::B_TILES + i) * 4, sf + ((1 + i) * 2 + kt) * SCALE_TILE);
        }
        commit<PAIR>(smem_u32(&s.scaled[stage]));
      }
      __syncwarp();
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    }
    if (elect_one()) commit<PAIR>(smem_u32(&s.drain[1]));
    if (!mbar_wait_drain(smem_u32(&s.drain[1]), 0)) *abort_flag = 1;
  } else if (warp == 1) {
    // ================= MMAs =================
    int stage = 0, buf = 0;
    uint32_t phase = 0, use = 0;
    bool ok = true;
    for (int tile = tile0; tile < args.tiles && ok; tile += step) {
      const int n0 = tile % args.n_tiles * BN;
      const uint32_t skew = BN % 128 ? (n0 & 64) >> 5 : 0;  // rows from 64 of a tile of scales on
      if (!warp_wait(smem_u32(&s.tempty[buf]), use ^ 1u, abort_flag)) break;
      for (int ks = 0; ks < args.k_steps; ++ks) {
        // (the scales were copied after the stage's arrival: one wait for both)
        if (!warp_wait(smem_u32(&s.scaled[stage]), phase, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tsa = tmem_base + BN * BUFS + stage * S::SF_COLS, tsb = tsa + 8;
        const int left = args.K - ks * BKC;  // codes from here on
        const uint32_t a_addr = tiles_u32 + stage * (S::A_BYTES + S::B_BYTES);
        const uint64_t a_desc = sdesc_k_sw128(a_addr);
        const uint64_t b_desc = sdesc_k_sw128(a_addr + S::A_BYTES);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk * 64 >= left) break;
            tc_mma_mxf4<PAIR>(tmem_base + buf * BN, a_desc + 2 * kk, b_desc + 2 * kk, kk & 1 ? IDESC2 : IDESC0,
                              tsa + (kk >> 1) * 4, tsb + (kk >> 1) * 4 * S::B_TILES + skew, ks != 0 || kk != 0);
          }
          commit<PAIR>(smem_u32(&s.empty[stage]));
          if (ks + 1 == args.k_steps) commit<PAIR>(smem_u32(&s.tfull[buf]));
        }
        __syncwarp();
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if (++buf == BUFS) { buf = 0; use ^= 1u; }
    }
    // every operation this warp issued has finished before anyone frees memory
    if (elect_one()) commit<PAIR>(smem_u32(&s.drain[0]));
    if (!mbar_wait_drain(smem_u32(&s.drain[0]), 0)) *abort_flag = 1;
  } else if (warp >= 4) {
    // ================= epilogue =================
    // lane quarter q = warp % 4 of tensor memory; column half = (warp - 4) / 4
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t staging = staging_u32 + (warp - 4) * 4096;
    int buf = 0;
    uint32_t use = 0, box = 0;
    int tile = tile0;
    for (; tile < args.tiles; tile += step) {
      const bool ready = mbar_wait(smem_u32(&s.tfull[buf]), use, abort_flag);
      if (!__all_sync(FULL_MASK, ready)) break;
      tc_fence_after();
      const int mt = tile / args.n_tiles, nt = tile - mt * args.n_tiles;
      const int row0 = (mt * CTAS + rank) * BM + q * 32, col0 = nt * BN + half * COLS;
      const int rows = min(args.M - row0, 32);
      const uint32_t tb = tmem_base + buf * BN + half * COLS + (static_cast<uint32_t>(q * 32) << 16);
      // all columns first, so that the accumulator is free as soon as may be
      uint32_t p[COLS / 32][32];
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) tmem_ld32(tb + 32 * c, p[c]);
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) tmem_ld_wait32(p[c]);
      tc_fence_before();  // all of this warp's reads have landed
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&s.tempty[buf]), 0));
        else mbar_arrive(smem_u32(&s.tempty[buf]));
      }
#pragma unroll
      for (int c = 0; c < COLS; c += 32) {
        if (col0 + c >= args.N || rows <= 0) break;
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = pack_bf16x2(__uint_as_float(p[c / 32][2 * k]), __uint_as_float(p[c / 32][2 * k + 1]));
        const uint32_t dst = staging + box * 2048;
        box ^= 1u;
        if (lane == 0) tma_store_wait_read<1>();  // the box before the last
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + staged_chunk(lane, i)), "r"(v[4 * i]),
                       "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                       : "memory");
        if (args.out_staged) {  // rows and columns past the matrix are clipped by the tensor map
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, dst, col0 + c, row0);
            tma_store_commit();
          }
        } else {  // rows that do not start on 16 bytes: the warp writes 32 neighbours of a row at a time
          __syncwarp();
          uint16_t* out = args.out + static_cast<long long>(row0) * args.N + col0 + c + lane;
          const bool there = col0 + c + lane < args.N;
#pragma unroll 4
          for (int r = 0; r < rows; ++r, out += args.N) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(dst + staged_chunk(r, lane >> 3) + 2 * (lane & 7)) : "memory");
            if (there) *out = h;
          }
          __syncwarp();
        }
      }
      if (++buf == BUFS) { buf = 0; use ^= 1u; }
    }
    // after a wait that ran out: this warp's part of the tiles not reached
    for (; tile < args.tiles; tile += step) {
      const int mt = tile / args.n_tiles, nt = tile - mt * args.n_tiles;
      const int row0 = (mt * CTAS + rank) * BM + q * 32, col0 = nt * BN + half * COLS;
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
  // neither CTA of a pair frees its tensor memory or leaves while MMAs, loads or
  // signals may still reach it
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, S::TMEM_COLS);
    else tmem_dealloc(tmem_base, S::TMEM_COLS);
  }
  if (threadIdx.x == 0 && s.abort) report(args.status, MOE_DEVERR_TIMEOUT);
}

// CTA pairs that can be resident at once (a pair needs two SMs of one GPC).
template <typename Kernel>
int resident_pairs(Kernel kernel, cudaLaunchConfig_t cfg, int& cache) {
  if (cache == 0) {
    int pairs = 0;
    cfg.gridDim = dim3(sm_count() & ~1);
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs < 1) pairs = sm_count() / 2;
    cache = pairs < sm_count() / 2 ? pairs : sm_count() / 2;
  }
  return cache;
}

template <int BN, bool PAIR>
cudaError_t launch(const uint8_t* a, const uint8_t* a_scale, const uint8_t* b, const uint8_t* b_scale, Args args, cudaStream_t s) {
  constexpr int CTAS = PAIR ? 2 : 1;
  const int kts = (args.K + 127) / 128;
  args.n_tiles = (args.N + BN - 1) / BN;
  args.tiles = (args.M + CTAS * BM - 1) / (CTAS * BM) * args.n_tiles;
  CUtensorMap ma, mb, msa, msb, mo;
  if (!make_tma_2d_u8(&ma, a, args.M, args.K / 2, BM) || !make_tma_2d_u8(&mb, b, args.N, args.K / 2, Shape<BN, PAIR>::B_ROWS) ||
      !make_tma_scale_tiles(&msa, a_scale, (args.M + 127) / 128, kts, 1) ||
      !make_tma_scale_tiles(&msb, b_scale, (args.N + 127) / 128, kts, Shape<BN, PAIR>::B_TILES))
    return cudaErrorInvalidValue;
  if (args.out_staged && !make_tma_store_2d_bf16(&mo, args.out, args.M, args.N)) return cudaErrorInvalidValue;
  if (!args.out_staged) mo = ma;  // not used
  auto kernel = fp4_gemm_kernel<BN, PAIR>;
  constexpr size_t smem = smem_bytes<BN, PAIR>();
  static_assert(smem <= SMEM_LIMIT, "fits");
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  if constexpr (!PAIR) {
    const int sms = sm_count();
    return launch_dependent(kernel, args.tiles < sms ? args.tiles : sms, THREADS, smem, s, ma, mb, msa, msb, mo, args);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  static int cache[64] = {};
  int dev = 0, none = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) dev = 64;
  const int pairs = resident_pairs(kernel, cfg, dev < 64 ? cache[dev] : none);
  cfg.gridDim = dim3(2 * (args.tiles < pairs ? args.tiles : pairs));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, msa, msb, mo, args);
}

}  // namespace

cudaError_t launch_fp4_matmul_tc(const uint8_t* a, const uint8_t* a_scale, int M, const uint8_t* b, const uint8_t* b_scale, int N,
                                 int K, uint16_t* out, int* status, cudaStream_t s) {
  Args g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.k_steps = (K + BKC - 1) / BKC;
  g.out = out;
  g.out_staged = N % 8 == 0;
  g.status = status;
  g.load_tiles = block_load_tiles();
  g.pair_wait_ns = pair_wait_ns();
  const bool pair = M > BM;
  const long long mt = pair ? (static_cast<long long>(M) + 2 * BM - 1) / (2 * BM) : 1;
  const int at_once = pair ? sm_count() / 2 : sm_count();
  // The width with the shortest rounds of tiles in all.  In pairs a stage of 128, 192
  // or 256 columns takes about 240, 270 and 305 ns and a tile 0.3, 0.45 and 1.0 us
  // more (8192 x 8192 x 4096: 120, 93 and 82 us; 333 x 4096 x 2048: 5.9, 6.1 and 6.5;
  // 64 columns take as long a stage as 128: 239 and 7.8 us).  A single CTA's tiles are few: the fewest
  // rounds, then the narrowest.
  auto rounds = [&](int bn) { return (mt * ((N + bn - 1) / bn) + at_once - 1) / at_once; };
  int bn = 256;
  if (pair) {
    auto cost = [&](int width, int stage, int tile) { return rounds(width) * (static_cast<long long>(g.k_steps) * stage + tile); };
    long long best = cost(256, 305, 1000);
    auto look = [&](int width, int stage, int tile) {
      const long long c = cost(width, stage, tile);
      if (c < best) best = c, bn = width;
    };
    look(192, 270, 450);
    look(128, 240, 300);
  } else {
    bn = rounds(64) <= rounds(256) ? 64 : rounds(128) <= rounds(256) ? 128 : 256;
  }
  if (pair)
    return bn == 256   ? launch<256, true>(a, a_scale, b, b_scale, g, s)
           : bn == 192 ? launch<192, true>(a, a_scale, b, b_scale, g, s)
                       : launch<128, true>(a, a_scale, b, b_scale, g, s);
  return bn == 256   ? launch<256, false>(a, a_scale, b, b_scale, g, s)
         : bn == 128 ? launch<128, false>(a, a_scale, b, b_scale, g, s)
                     : launch<64, false>(a, a_scale, b, b_scale, g, s);
}

}  // namespace moe
