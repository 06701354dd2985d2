// Products of e4m3 codes with a scale for each block of 128, on the 5th-
// generation tensor cores.
//
//   C[m, n] = sum_kb sa[m, kb] sb[n / 128, kb] sum_{k in block kb} a[m, k] b[n, k]
//
// a [M, K] has a scale per row and 128 columns, b [N, K] one per 128 x 128
// block (for the grouped form each expert's matrix has its own).  The tensor
// cores sum one block of 128 products as they stand (codes times codes, exact
// products, fp32 accumulation in tensor memory: measured, beside 2^17.6 what is
// 2^-6 or more is kept, within one instruction's 32 three bits more); the scales differ from block to
// block, so each block's partial sums are read back, scaled and added in fp32
// registers.  That promotion is what the kernel is built around:
//   * warp 0 stages operands by TMA (128-byte swizzle, one K block of 128
//     codes per stage), warps 1 and 2 issue four tcgen05.mma of K = 32 per
//     block into one of the accumulators in tensor memory (two of 256
//     columns, or four narrower ones), warps 4..11 read it back, free it and
//     add it to their registers while the next blocks are multiplied;
//   * a lane of a promoting warp owns a row of C; warp 3 multiplies each
//     block's scales out for it, one number per row and 128 columns.
//
// What bounds it, at 8192 x 8192 x 4096 (216 us, 2.5 PFLOP/s): the MMAs alone
// run at 4.4 PFLOP/s (547 cycles a block of 128 x 256 x 128); with operands
// arriving and accumulators handed over, but not read, 183 us; the rest is the
// accumulators' reading.  A block's products can be replaced only when all
// eight warps have read theirs, and two blocks fill tensor memory.  Tried
// without gain: CTA pairs with half of B each (224 us), halves of 128 columns
// with an accumulator pair each (250), packed fused multiply-adds (240), longer
// and shorter pieces, reading into the next block.
//
// Three epilogues: bf16 of C; bf16 of w_row C (the experts' down product);
// and SwiGLU with requantisation (the experts' gate/up product): the tile
// pairs 128 gate with 128 up columns, h = silu(g) u stays in fp32 until it is
// e4m3 codes with a scale per row and 128 columns.  (Through bf16 first, one
// code in thirty would move by a step.)
//
// As in the bf16 experts, the tile list is built on the device from the
// layout's counts, one persistent CTA per SM; every wait is bounded, and a
// wait that runs out sets MOE_DEVERR_TIMEOUT, drains and leaves NaN in the
// tiles that the CTA does not reach (NaN codes of h, which make the second
// product's rows NaN), so that the call cannot pass for a finished one.

#include "common.cuh"
#include "fp8_quant.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int BM = 128;
constexpr int BKB = 128;  // codes per block and stage
constexpr int MAX_STAGES = 8;
constexpr int MAX_BUFS = 4;
constexpr int SMEM_LIMIT = 232448;

enum Mode { OUT_PLAIN = 0, OUT_WEIGHTED = 1, OUT_SWIGLU = 2 };

// Warps 0..3 are the producer, the issuers and the scales; eight more promote,
// two for each lane quarter of tensor memory, half of the tile's columns each.
// Such a thread holds up to 128 accumulators, more registers than an even
// share: the first warpgroup passes some of its own on.  (Sixteen promoting
// warps of 64 accumulators took longer to meet in each block: 247 against 216 us
// at 8192 x 8192 x 4096.)
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (4 + EPI_WARPS);
constexpr int LAUNCH_REGS = 168, FEW_REGS = 56, MANY_REGS = 224;
static_assert(128 * FEW_REGS + 32 * EPI_WARPS * MANY_REGS <= THREADS * LAUNCH_REGS, "registers are only passed on");

template <int BN>
struct Shape {
  static constexpr int A_BYTES = BM * BKB;
  static constexpr int B_BYTES = BN * BKB;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // What is left beside the staged output (two bytes a value, the whole tile)
  static constexpr int STAGES = BN == 256 ? 3 : BN == 128 ? 5 : 7;
  static constexpr int STAGING_BYTES = BM * BN * 2;
  static constexpr int BUFS = BN == 256 ? 2 : 4;
  static constexpr int TMEM_COLS = BN * BUFS;
  static constexpr int COLS = BN / 2;  // accumulators of a promoting thread
};

struct Smem {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tfull[MAX_BUFS];
  uint64_t tempty[MAX_BUFS];
  uint64_t drain[2];
  uint64_t meet[4];   // SwiGLU: the two warps of a lane quarter, once a tile
  uint32_t tmem_base;
  int abort;
  int total_tiles;
  float scale[MAX_BUFS][2][BM];  // of each row, for the two blocks of 128 columns (or gate and up)
};

template <int BN>
constexpr size_t smem_bytes(int E) {
  using S = Shape<BN>;
  return 1024 + static_cast<size_t>(S::STAGES) * S::STAGE_BYTES + S::STAGING_BYTES + sizeof(Smem) + static_cast<size_t>(3 * E + 2) * sizeof(int);
}

struct Args {
  const int* counts;   // [E] rows of each expert; NULL: one group of `rows` rows
  const int* offsets;  // [E + 1]
  int rows;
  int E;
  int K, k_blocks;
  int N;               // columns of C (OUT_SWIGLU: of h, half of b's rows)
  int n_tiles;
  int b_rows;          // rows of b per expert
  int b_scale_rows;    // scale rows of b per expert
  const float* a_scale;    // [rows, k_blocks]
  const float* b_scale;    // [E, b_scale_rows, k_blocks]
  const float* row_weight; // OUT_WEIGHTED
  uint16_t* out;           // bf16 [rows, N]
  int out_staged;          // tmOut describes the output (its rows are 16-byte aligned)
  uint8_t* out_q;          // OUT_SWIGLU: codes [rows, N] and scales [rows, N / 128]
  float* out_scale;
  int* status;
  int load_tiles;          // tiles a CTA loads operands for: all, but in the self-test
};

struct Tile {
  int e, mt, nt;
};

__device__ __forceinline__ Tile decode_tile(const int* tile_prefix, int E, int n_tiles, int tile) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_prefix[mid] <= tile) lo = mid; else hi = mid;
  }
  const int local = tile - tile_prefix[lo];
  Tile t;
  t.e = lo;
  t.mt = local / n_tiles;
  t.nt = local - t.mt * n_tiles;
  return t;
}

template <int MODE, int BN>
__global__ void __launch_bounds__(THREADS, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmOut, const Args args) {
  using S = Shape<BN>;
  static_assert(MODE != OUT_SWIGLU || BN == 256, "a tile of h is one scale block wide, 64 columns a warp");
  constexpr int STAGES = S::STAGES, BUFS = S::BUFS, COLS = S::COLS;
  constexpr uint32_t IDESC = idesc_e4m3_f32(BM, BN);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* tiles = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(tiles + STAGES * S::STAGE_BYTES + S::STAGING_BYTES);
  int* s_off = reinterpret_cast<int*>(&s + 1);  // [E+1]
  int* s_cnt = s_off + args.E + 1;              // [E]
  int* s_pre = s_cnt + args.E;                  // [E+1] tile prefix
  const uint32_t tiles_u32 = smem_u32(tiles);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = args.E;
  griddep_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(smem_u32(&s.tfull[i]), 2);  // the products and their scales
      mbar_init(smem_u32(&s.tempty[i]), EPI_WARPS);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.meet[i]), 2);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&s.drain[i]), 1);
    s.abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (args.out_staged) tma_prefetch_desc(&tmOut);
  }
  if (warp == 1) tmem_alloc(smem_u32(&s.tmem_base), S::TMEM_COLS);
  griddep_wait();  // the codes, the scales and the layout come from earlier kernels
  if (args.counts) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) s_off[e] = args.offsets[e];
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_cnt[e] = args.counts[e];
  } else if (threadIdx.x == 0) {
    s_off[0] = 0;
    s_off[1] = s_cnt[0] = args.rows;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive scan of per-expert tile counts
    int running = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < E ? ((s_cnt[e] + BM - 1) / BM) * args.n_tiles : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < E) s_pre[e] = running + incl - n;
      running += __shfl_sync(FULL_MASK, incl, 31);
    }
    if (lane == 0) {
      s_pre[E] = running;
      s.total_tiles = running;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const int total = s.total_tiles;
  const uint32_t tmem_base = s.tmem_base;
  volatile int* abort_flag = &s.abort;
  const int k_blocks = args.k_blocks;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
    // ================= TMA producer =================
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      int left = args.load_tiles;
      for (int tile = blockIdx.x; tile < total && ok && left > 0; tile += gridDim.x, --left) {
        const Tile t = decode_tile(s_pre, E, args.n_tiles, tile);
        const int a_row = s_off[t.e] + t.mt * BM;
        const int b_row = t.e * args.b_rows + t.nt * (MODE == OUT_SWIGLU ? BN / 2 : BN);
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t full = smem_u32(&s.full[stage]);
          const uint32_t a_dst = tiles_u32 + stage * S::STAGE_BYTES;
          const uint32_t b_dst = a_dst + S::A_BYTES;
          mbar_arrive_expect_tx(full, S::STAGE_BYTES);
          tma_load_2d(a_dst, &tmA, kb * BKB, a_row, full);
          tma_load_2d(b_dst, &tmB, kb * BKB, b_row, full);
          if constexpr (BN == 256)  // the up rows, or the tile's second half
            tma_load_2d(b_dst + S::B_BYTES / 2, &tmB, kb * BKB, b_row + (MODE == OUT_SWIGLU ? args.N : BN / 2), full);
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
    }
    // ================= MMA issuers =================
    // Two warps take turns, one K block each.  A block's four instructions
    // are accepted only as the ones before them finish, so a single issuer
    // would spend the time of its next waits and commits (about 300 cycles)
    // with an idle tensor pipe; the accumulators of neighbouring blocks are
    // different ones, so their order does not matter.
    if ((warp == 1 || warp == 2) && lane == 0) {
      const int w = warp - 1;
      const int my_tiles = total > static_cast<int>(blockIdx.x) ? (total - 1 - blockIdx.x) / gridDim.x + 1 : 0;
      const long long blocks = static_cast<long long>(my_tiles) * k_blocks;
      int stage = w, buf = w;
      uint32_t phase = 0, use = 0;
      for (long long it = w; it < blocks; it += 2) {
        if (!mbar_wait(smem_u32(&s.tempty[buf]), use ^ 1u, abort_flag) ||
            !mbar_wait(smem_u32(&s.full[stage]), phase, abort_flag))
          break;
        tc_fence_after();
        const uint32_t a_addr = tiles_u32 + stage * S::STAGE_BYTES;
        const uint64_t a_desc = sdesc_k_sw128(a_addr);
        const uint64_t b_desc = sdesc_k_sw128(a_addr + S::A_BYTES);
#pragma unroll
        for (int kk = 0; kk < BKB / 32; ++kk)  // 32 codes = 32 bytes of the swizzled row a step
          tc_mma_e4m3(tmem_base + buf * BN, a_desc + 2 * kk, b_desc + 2 * kk, IDESC, kk != 0);
        tc_commit(smem_u32(&s.empty[stage]));
        tc_commit(smem_u32(&s.tfull[buf]));
        if ((stage += 2) >= STAGES) { stage -= STAGES; phase ^= 1u; }
        if ((buf += 2) >= BUFS) { buf -= BUFS; use ^= 1u; }
      }
      // every MMA this thread issued has finished before anyone frees memory
      tc_commit(smem_u32(&s.drain[w]));
      if (!mbar_wait_drain(smem_u32(&s.drain[w]), 0)) *abort_flag = 1;
    }
    // ================= scales =================
    // Warp 3 multiplies the scales of each K block out for the promotion: for
    // every row of the tile its own times that of each 128 columns.
    if (warp == 3) {
      int buf = 0;
      uint32_t use = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const Tile t = decode_tile(s_pre, E, args.n_tiles, tile);
        const float* sa = args.a_scale + static_cast<long long>(s_off[t.e] + t.mt * BM) * k_blocks;
        const int last = s_cnt[t.e] - 1 - t.mt * BM;  // rows past the group repeat its last one
        // columns past N read the last block's scale and are not stored
        const int b0 = MODE == OUT_SWIGLU ? t.nt : min(t.nt * BN >> 7, args.b_scale_rows - 1);
        const int b1 = MODE == OUT_SWIGLU ? t.nt + (args.N >> 7) : min((t.nt * BN + BN - 1) >> 7, args.b_scale_rows - 1);
        const float* sb = args.b_scale + static_cast<long long>(t.e) * args.b_scale_rows * k_blocks;
        float v[4], f0, f1;
        auto fetch = [&](int kb) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __ldg(sa + min(lane + 32 * i, last) * k_blocks + kb);
          f0 = __ldg(sb + b0 * k_blocks + kb);
          f1 = __ldg(sb + b1 * k_blocks + kb);
        };
        fetch(0);
        for (int kb = 0; kb < k_blocks; ++kb) {
          const bool ready = mbar_wait(smem_u32(&s.tempty[buf]), use ^ 1u, abort_flag);
          if (!__all_sync(FULL_MASK, ready)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s.scale[buf][0][lane + 32 * i] = v[i] * f0;
            s.scale[buf][1][lane + 32 * i] = v[i] * f1;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.tfull[buf]));
          if (kb + 1 < k_blocks) fetch(kb + 1);
          if (++buf == BUFS) { buf = 0; use ^= 1u; }
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
    // ================= promotion and epilogue =================
    // lane quarter q = warp % 4 of tensor memory; column half = (warp - 4) / 4.
    // OUT_SWIGLU: 64 gate columns, then their 64 up columns.
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int r_in_tile = q * 32 + lane;
    const uint32_t staging = tiles_u32 + STAGES * S::STAGE_BYTES + (warp - 4) * (S::STAGING_BYTES / EPI_WARPS);
    // SwiGLU: [tile parity][column half][row] largest |h| of a row, in parts of
    // the staging that codes leave free (they take 2 KiB of each warp's 8)
    auto amax = [&](int par, int part) -> float& {
      return reinterpret_cast<float*>(tiles + STAGES * S::STAGE_BYTES + 4096)[(par * 2 + part) * 2048 + r_in_tile];
    };
    auto column = [&](int c) {  // tensor-memory column of this thread's accumulator c
      return MODE == OUT_SWIGLU ? (c < 64 ? half * 64 + c : 128 + half * 64 + c - 64) : half * COLS + c;
    };
    int buf = 0;
    uint32_t use = 0, parity = 0;
    bool ok = true;
    int tile = blockIdx.x;
    for (; tile < total && ok; tile += gridDim.x, parity ^= 1u) {
      float acc[COLS];
#pragma unroll
      for (int i = 0; i < COLS; ++i) acc[i] = 0.f;
      for (int kb = 0; kb < k_blocks; ++kb) {
        const bool ready = mbar_wait(smem_u32(&s.tfull[buf]), use, abort_flag);
        if (!__all_sync(FULL_MASK, ready)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tmem_base + buf * BN + (static_cast<uint32_t>(q * 32) << 16);
        const float scale = s.scale[buf][MODE == OUT_SWIGLU || BN < 256 ? 0 : (half * COLS) >> 7][r_in_tile];
        const float scale_up = MODE == OUT_SWIGLU ? s.scale[buf][1][r_in_tile] : 0.f;
        // the next 32 columns are read while these are added
        uint32_t p[COLS > 32 ? 2 : 1][32];
        tmem_ld32(tb + column(0), p[0]);
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          uint32_t(&now)[32] = p[COLS > 32 ? (c >> 5) & 1 : 0];
          tmem_ld_wait32(now);
          if (c + 32 < COLS) {
            tmem_ld32(tb + column(c + 32), p[COLS > 32 ? ((c >> 5) & 1) ^ 1 : 0]);
          } else {  // all of this warp's reads have landed
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.tempty[buf]));
          }
          const float f = MODE == OUT_SWIGLU && c >= 64 ? scale_up : scale;
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c + i] = fmaf(__uint_as_float(now[i]), f, acc[c + i]);
        }
        if (++buf == BUFS) { buf = 0; use ^= 1u; }
      }
      if (!ok) break;
      // Output: a warp whose 32 rows all exist writes them to its staging
      // boxes (32 rows, of 64 bytes swizzled or of 32 bytes) and stores those
      // by TMA, which goes on while the next tile is multiplied; else rows one
      // by one.  Rows past a dense matrix are clipped by the tensor map.
      const Tile t = decode_tile(s_pre, E, args.n_tiles, tile);
      const bool valid = t.mt * BM + r_in_tile < s_cnt[t.e];
      const int row0 = s_off[t.e] + t.mt * BM + q * 32;
      const bool staged = args.out_staged && (!args.counts || __all_sync(FULL_MASK, valid));
      const long long row = static_cast<long long>(row0) + lane;
      if (staged) {
        if (lane == 0) tma_store_wait_read<0>();  // the last tile's boxes
        __syncwarp();
      }
      auto put = [&](uint32_t dst, int x) {  // x: column in units of 2 bytes
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmOut, dst, x, row0);
          tma_store_commit();
        }
      };
      if constexpr (MODE == OUT_SWIGLU) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          acc[i] = silu_mul(acc[i], acc[64 + i]);
          top = max_nan(top, fabsf(acc[i]));
        }
        // The two warps of a lane quarter exchange their maxima.  One meeting a
        // tile is enough: this parity's slots are written again two tiles
        // on, after the next tile's meeting, which follows both reads here.
        amax(parity, half) = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.meet[q]));
        const bool met = mbar_wait(smem_u32(&s.meet[q]), parity, abort_flag);
        if (!__all_sync(FULL_MASK, met)) break;
        const float scale = block_scale(max_nan(amax(parity, 0), amax(parity, 1)));
        const float y = __fdiv_rn(1.0f, scale);
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          v[k] = e4m3x4(y * acc[4 * k], y * acc[4 * k + 1], y * acc[4 * k + 2], y * acc[4 * k + 3]);
        if (staged) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(staging + staged_chunk(lane, i)), "r"(v[4 * i]),
                         "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                         : "memory");
          put(staging, t.nt * 64 + half * 32);
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(args.out_q + row * args.N + t.nt * 128 + half * 64);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        if (valid && half == 0) args.out_scale[row * (args.N >> 7) + t.nt] = scale;
      } else {
        const float w = MODE == OUT_WEIGHTED && valid ? __ldg(args.row_weight + row) : 1.0f;
        const int col0 = t.nt * BN + half * COLS;
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          if (col0 + c >= args.N) break;
          uint32_t v[32 / 2];
#pragma unroll
          for (int k = 0; k < 32 / 2; ++k) v[k] = pack_bf16x2(w * acc[c + 2 * k], w * acc[c + 2 * k + 1]);
          if (staged) {
            const uint32_t dst = staging + (c >> 5) * 2048;
#pragma unroll
            for (int i = 0; i < 32 / 8; ++i)
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + staged_chunk(lane, i)), "r"(v[4 * i]),
                           "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                           : "memory");
            put(dst, col0 + c);
          } else if (MODE == OUT_PLAIN) {
            // rows that do not start on 16 bytes: turned in the staging box, so
            // that the warp writes 32 neighbours of a row at a time (4097 x 4097 x
            // 4096: 74 us; each lane its own row 204)
#pragma unroll
            for (int i = 0; i < 32 / 8; ++i)
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(staging + staged_chunk(lane, i)),
                           "r"(v[4 * i]), "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                           : "memory");
            __syncwarp();
            const int rows = min(s_cnt[t.e] - t.mt * BM - q * 32, 32);
            uint16_t* dst = args.out + static_cast<long long>(row0) * args.N + col0 + c + lane;
            const bool there = col0 + c + lane < args.N;
#pragma unroll 4
            for (int r = 0; r < rows; ++r, dst += args.N) {
              uint16_t h;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(staging + staged_chunk(r, lane >> 3) + 2 * (lane & 7)) : "memory");
              if (there) *dst = h;
            }
            __syncwarp();
          } else if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(args.out + row * args.N + col0 + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (col0 + c + 8 * i < args.N) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
      }
    }
    // after a wait that ran out: this warp's part of the tiles not reached
    for (; tile < total; tile += gridDim.x) {
      const Tile t = decode_tile(s_pre, E, args.n_tiles, tile);
      const int first = t.mt * BM + q * 32, rows = min(s_cnt[t.e] - first, 32);
      const long long row0 = s_off[t.e] + first;
      const int col0 = MODE == OUT_SWIGLU ? t.nt * 128 + half * 64 : t.nt * BN + half * COLS;
      const int cols = min(args.N - col0, MODE == OUT_SWIGLU ? 64 : COLS);
#pragma unroll 1
      for (int r = 0; r < rows; ++r)
#pragma unroll 1
        for (int c = lane; c < cols; c += 32) {
          const long long at = (row0 + r) * args.N + col0 + c;
          if constexpr (MODE == OUT_SWIGLU) args.out_q[at] = 0x7f;
          else args.out[at] = 0x7fc0;
        }
    }
    if (lane == 0) tma_store_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, S::TMEM_COLS);
  if (threadIdx.x == 0 && s.abort) report(args.status, MOE_DEVERR_TIMEOUT);
}

// The self-test's limit of the tiles that a CTA loads, for this host thread's launches.
thread_local int tls_load_tiles = 0x7fffffff;

template <int MODE, int BN>
cudaError_t launch(const void* a, uint64_t a_rows, const void* b, uint64_t b_rows, Args args, int grid,
                   cudaStream_t s) {
  args.load_tiles = tls_load_tiles;
  CUtensorMap ma, mb, mo;
  if (!make_tma_2d_u8(&ma, a, a_rows, args.K, BM) || !make_tma_2d_u8(&mb, b, b_rows, args.K, BN == 256 ? 128 : BN))
    return cudaErrorInvalidValue;
  // codes are stored as pairs of bytes
  const bool staged = args.out_staged;
  if (staged && !(MODE == OUT_SWIGLU ? make_tma_store_2d_bf16(&mo, args.out_q, a_rows, args.N / 2)
                                     : make_tma_store_2d_bf16(&mo, args.out, a_rows, args.N)))
    return cudaErrorInvalidValue;
  if (!staged) mo = ma;  // not used
  auto kernel = block_gemm_kernel<MODE, BN>;
  static_assert(smem_bytes<BN>(1024) <= SMEM_LIMIT, "fits for every E");
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT);
  if (err != cudaSuccess) return err;
  return launch_dependent(kernel, grid, THREADS, smem_bytes<BN>(args.E), s, ma, mb, mo, args);
}

}  // namespace

void selftest_block_load_tiles(int tiles) { tls_load_tiles = tiles; }
int block_load_tiles() { return tls_load_tiles; }

cudaError_t launch_block_matmul_tc(const uint8_t* a, const float* a_scale, int M, const uint8_t* b,
                                   const float* b_scale, int N, int K, uint16_t* out, int* status,
                                   cudaStream_t s) {
  Args g{};
  g.rows = M;
  g.E = 1;
  g.K = K;
  g.k_blocks = (K + BKB - 1) / BKB;
  g.N = N;
  g.b_rows = N;
  g.b_scale_rows = (N + 127) / 128;
  g.a_scale = a_scale;
  g.b_scale = b_scale;
  g.out = out;
  g.out_staged = N % 8 == 0;
  g.status = status;
  const long long mt = (static_cast<long long>(M) + BM - 1) / BM;
  auto tiles = [&](int bn) { return mt * ((N + bn - 1) / bn); };
  const int sms = sm_count();
  // The tile width with the shortest rounds in all: a K block of 64, 128 or 256
  // columns takes about 250, 310 and 450 ns.
  auto cost = [&](int bn, int per_block) { return (tiles(bn) + sms - 1) / sms * per_block; };
  const long long c64 = cost(64, 25), c128 = cost(128, 31), c256 = cost(256, 45);
  const int bn = c256 <= c128 && c256 <= c64 ? 256 : c128 <= c64 ? 128 : 64;
  g.n_tiles = (N + bn - 1) / bn;
  const int grid = static_cast<int>(tiles(bn) < sms ? tiles(bn) : sms);
  if (bn == 256) return launch<OUT_PLAIN, 256>(a, M, b, N, g, grid, s);
  if (bn == 128) return launch<OUT_PLAIN, 128>(a, M, b, N, g, grid, s);
  return launch<OUT_PLAIN, 64>(a, M, b, N, g, grid, s);
}

cudaError_t launch_block_experts_tc(const uint8_t* x_q, const float* x_scale, const moe_layout& L, int H, int I,
                                    const uint8_t* W1, const float* W1_scale, const uint8_t* W2,
                                    const float* W2_scale, uint8_t* h_q, float* h_scale, uint16_t* y,
                                    cudaStream_t s) {
  Args g{};
  g.counts = L.tokens_per_expert;
  g.offsets = L.offsets;
  g.E = L.E;
  g.status = L.status;
  g.K = H;
  g.k_blocks = (H + BKB - 1) / BKB;
  g.N = I;
  g.n_tiles = I / 128;
  g.b_rows = 2 * I;
  g.b_scale_rows = 2 * I / 128;
  g.a_scale = x_scale;
  g.b_scale = W1_scale;
  g.out_q = h_q;
  g.out_staged = 1;
  g.out_scale = h_scale;
  const uint64_t C = static_cast<uint64_t>(L.capacity), E = static_cast<uint64_t>(L.E);
  cudaError_t err = launch<OUT_SWIGLU, 256>(x_q, C, W1, E * 2 * I, g, sm_count(), s);
  if (err != cudaSuccess) return err;
  g.K = I;
  g.k_blocks = I / BKB;
  g.N = H;
  g.n_tiles = H / 256;
  g.b_rows = H;
  g.b_scale_rows = H / 128;
  g.a_scale = h_scale;
  g.b_scale = W2_scale;
  g.row_weight = L.row_weight;
  g.out = y;
  return launch<OUT_WEIGHTED, 256>(h_q, C, W2, E * H, g, sm_count(), s);
}

}  // namespace moe
