// What the forward and the backward of the norms around a block share: rows
// as vectors of eight values, sums over a row, the gate, and the copies that
// bring a row to shared memory.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace moe {

namespace norm {

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

// Rows that do not start on 16 bytes: value by value, out of line (the fast
// path's code would drown in it).  There the 256 values of a warp's 32 vectors
// are dealt out one by one, so that each access is to 32 neighbours
// (T = 16384, H = 2049, before a block: 66 us, 8 neighbours a lane 111); a sum
// over the row does not mind.  `col` is a multiple of 8, col / 8 of a warp's
// first lane one of 32.
__device__ __forceinline__ int ragged_col(int col, int i) {
  const int v = col >> 3;
  return ((v & ~31) << 3) + 32 * i + (v & 31);
}

template <bool F32>
__device__ __noinline__ Raw<F32> load_ragged(const void* row, int col, int H) {
  Raw<F32> o = raw_zero<F32>();
  if constexpr (F32) {
    const float* p = static_cast<const float*>(row);
    uint32_t t[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (const int c = ragged_col(col, i); c < H) t[i] = __float_as_uint(p[c]);
    o.q = make_uint4(t[0], t[1], t[2], t[3]);
    o.r = make_uint4(t[4], t[5], t[6], t[7]);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row);
    uint32_t t[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (const int c = ragged_col(col, i); c < H) t[i >> 1] |= static_cast<uint32_t>(p[c]) << (16 * (i & 1));
    o.q = make_uint4(t[0], t[1], t[2], t[3]);
  }
  return o;
}

// KEEP: a tensor that every row reads again (the weights) stays in L1; the
// others pass through it once.
template <bool F32, bool KEEP = false>
__device__ __forceinline__ Raw<F32> load_raw(const void* row, int col, int H, bool full) {
  if (!full) return load_ragged<F32>(row, col, H);
  Raw<F32> o = raw_zero<F32>();
  if (col >= H) return o;
  auto get = [](const uint4* p) { return KEEP ? __ldg(p) : __ldcs(p); };
  if constexpr (F32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + col);
    o.q = get(p);
    o.r = get(p + 1);
  } else {
    o.q = get(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + col));
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
__device__ __noinline__ void store_ragged(void* row, int col, int H, const Raw<F32> a) {
  if constexpr (F32) {
    float* p = static_cast<float*>(row);
    const uint32_t t[8] = {a.q.x, a.q.y, a.q.z, a.q.w, a.r.x, a.r.y, a.r.z, a.r.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (const int c = ragged_col(col, i); c < H) p[c] = __uint_as_float(t[i]);
  } else {
    uint16_t* p = static_cast<uint16_t*>(row);
    const uint32_t t[4] = {a.q.x, a.q.y, a.q.z, a.q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (const int c = ragged_col(col, i); c < H) p[c] = static_cast<uint16_t>(t[i >> 1] >> (16 * (i & 1)));
  }
}

template <bool F32>
__device__ __forceinline__ void store_raw(void* row, int col, int H, bool full, const Raw<F32>& a) {
  if (!full) {
    store_ragged<F32>(row, col, H, a);
    return;
  }
  if (col >= H) return;
  if constexpr (F32) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(row) + col);
    p[0] = a.q;
    p[1] = a.r;
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + col) = a.q;
  }
}

// Weights and element gates: bf16 or fp32 by a flag that is the same for the
// whole launch.
template <bool KEEP = false>
__device__ __forceinline__ F8 load_either(const void* row, int f32, int col, int H, bool full) {
  return f32 ? widen(load_raw<true, KEEP>(row, col, H, full)) : widen(load_raw<false, KEEP>(row, col, H, full));
}

__device__ __forceinline__ const void* row_of(const void* p, long long row, int H, int f32) {
  return static_cast<const char*>(p) + row * H * (f32 ? 4 : 2);
}
__device__ __forceinline__ void* row_of(void* p, long long row, int H, int f32) {
  return static_cast<char*>(p) + row * H * (f32 ? 4 : 2);
}

// Sums N values over a group of `threads` threads (a multiple of 32); every
// thread gets the totals.  The two halves of `red` (this group's) alternate,
// so one barrier a call is enough: a warp can reach its next write of a half
// only after a barrier that follows every read of it.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*red)[MAX_WARPS][4], int threads, int group,
                                          int& phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(FULL_MASK, v[k], o);
  if (threads == 32) return;
  const int warps = threads >> 5, first = group * warps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[phase][warp][k] = v[k];
  }
  if (threads == blockDim.x) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
  // the warps' sums lie in every 2^n lanes, so that all lanes end with the total
  const int span = 2 << (31 - __clz(warps - 1)), mine = lane & (span - 1);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = mine < warps ? red[phase][first + mine][k] : 0.f;
  for (int o = 1; o < span; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(FULL_MASK, v[k], o);
  phase ^= 1;
}

// The gate's factor s and ds/dg.  From e = exp(-|g|), which cannot overflow:
// s = 1 / (1 + e) or e / (1 + e), and ds/dg = e / (1 + e)^2 on both sides,
// without the cancellation of 1 - s where s is near 1.  The fast exponential
// is off by up to 2 + 1.2 |g| ulp, so s by 2^-18 of itself at |g| = 16 at the
// worst, and less where s is near 1: below half a bf16 ulp by far, and of an fp32
// stream it is one term.  (With expf and a rounded reciprocal a gate per
// element costs half as much time again: 16384 x 2048, bf16, backward 131 us for 86,
// forward 70 for 49.)
struct Gate {
  float s, slope;
};
__device__ __forceinline__ Gate gate_of(float g, int sigmoid) {
  if (!sigmoid) return {g, 1.0f};
  // 1 + e lies in [1, 2]: the fast division is within 2 ulp there
  const float e = __expf(-fabsf(g)), inv = __fdividef(1.0f, 1.0f + e);
  return {g >= 0.f ? inv : e * inv, e * inv * inv};
}

__device__ __forceinline__ float load_scalar(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

// The weight of the norm: offset + w.
__device__ __forceinline__ F8 load_weight(const void* w, int f32, float offset, int col, int H, bool full) {
  F8 o = load_either<true>(w, f32, col, H, full);
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] += offset;
  return o;
}

// ---------------------------------------------------------------- rows through shared memory
// A group of threads brings its next rows' tensors to shared memory with bulk
// copies while it works on the current one from registers: a row leaves its
// slot for the registers as a whole, so the group's SLOTS slots are all in
// flight while it computes.
constexpr int MAX_GROUPS = 8;
template <int SLOTS>
struct RowPipe {
  uint32_t base, slot_bytes, bars;  // shared-memory addresses of the group's slots and barriers
  int at;                           // the slot of the current row
  uint32_t phase;
  __device__ __forceinline__ uint32_t slot() const { return base + at * slot_bytes; }
  __device__ __forceinline__ uint32_t bar() const { return bars + 8 * at; }
  __device__ __forceinline__ void next() {
    if (++at == SLOTS) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// One thread: the copies of `bytes` (a multiple of 16) each from src[0 .. n)
// to the slot, one after the other; null sources are left out.
template <int N>
__device__ __forceinline__ void pipe_issue(uint32_t slot, uint32_t bar, const char* const (&src)[N], const uint32_t (&bytes)[N]) {
  uint32_t total = 0;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (src[k]) total += bytes[k];
  mbar_arrive_expect_tx(bar, total);
  uint32_t at = slot;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (src[k])
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(at),
                   "l"(src[k]), "r"(bytes[k]), "r"(bar)
                   : "memory");
    at += bytes[k];
  }
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <bool F32>
__device__ __forceinline__ Raw<F32> read_slot(uint32_t row, int col, int H) {
  Raw<F32> o = raw_zero<F32>();
  if (col >= H) return o;
  if constexpr (F32) {
    o.q = ld_shared_v4(row + col * 4);
    o.r = ld_shared_v4(row + col * 4 + 16);
  } else {
    o.q = ld_shared_v4(row + col * 2);
  }
  return o;
}

// All threads of the group (named barrier 1 + group) agree whether all of them
// saw their row arrive, and have read what they read of the slot: it may be
// filled again.  (A vote alone orders no memory.)
__device__ __forceinline__ bool group_all(bool ok, int threads, int group) {
  if (threads == 32) {
    const bool all = __all_sync(FULL_MASK, ok);
    __syncwarp();
    return all;
  }
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(ok)), "r"(1 + group), "r"(threads)
      : "memory");
  return r != 0;
}

// Before a group leaves early: its copies in flight, from the current slot on
// (a bounded wait as well), since they write to this CTA's shared memory.
template <int SLOTS>
__device__ __forceinline__ void pipe_drain(RowPipe<SLOTS> pipe, long long t, long long stride, long long T) {
#pragma unroll 1
  for (int i = 0; i < SLOTS && t + i * stride < T; ++i, pipe.next()) mbar_wait_drain(pipe.bar(), pipe.phase);
}

// A group whose wait for a row ran out leaves NaN in the rows that it does not
// reach, so that the call cannot pass for a finished one.
template <bool F32>
__device__ __forceinline__ void spoil_row(void* base, long long row, int H, int in_row, int row_threads) {
  if (!base) return;
#pragma unroll 1
  for (int c = in_row; c < H; c += row_threads) {
    if constexpr (F32) static_cast<uint32_t*>(base)[row * H + c] = 0x7fc00000u;
    else static_cast<uint16_t*>(base)[row * H + c] = 0x7fc0u;
  }
}

inline int vectors(int H) { return (H + 7) / 8; }
inline int threads_of(int H, int nv) { return ((vectors(H) + nv - 1) / nv + 31) / 32 * 32; }

}  // namespace norm

}  // namespace moe
