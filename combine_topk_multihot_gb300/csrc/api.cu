// The C ABI declared in include/moe.h: argument validation on the host, then
// the launches.  No allocation, no global state besides per-device caches of
// immutable device properties and the thread-local error text.

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <atomic>
#include <chrono>
#include <cmath>
#include <mutex>
#include <new>

#include "common.cuh"
#include "launch.h"

namespace moe {

namespace {

thread_local char g_last_error[512] = "";

moe_status fail(moe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

moe_status cuda_fail(cudaError_t err, const char* where) {
  return fail(MOE_ERR_CUDA, "%s: %s", where, cudaGetErrorString(err));
}

constexpr int MAX_DEVICES = 64;
int g_cc_ok[MAX_DEVICES];    // 0 unknown, 1 compute capability 10.3, -1 other
int g_sms[MAX_DEVICES];

// The host-synced dispatch reads R, N and the status word from 16 bytes of
// mapped pinned host memory that the layout kernel writes directly, so the
// readback needs no copy engine and cannot queue behind bulk copies on other
// streams.  One buffer per device, made on first use; the mutex is held from
// the launch until the kernel can no longer write to it, so concurrent
// host-synced calls take turns.
std::mutex g_rb_mu;
// The host polls the mapped buffer for this long before it falls back to a
// stream synchronisation (the layout kernel's own waits give up after 2 s).
constexpr int READBACK_POLL_LIMIT_S = 10;
int* g_rb_host[MAX_DEVICES];
int* g_rb_dev[MAX_DEVICES];

bool readback_buffer(int dev, int** host, int** dev_ptr) {
  if (dev < 0 || dev >= MAX_DEVICES) return false;
  if (!g_rb_host[dev]) {
    void* h = nullptr;
    void* d = nullptr;
    if (cudaHostAlloc(&h, 16, cudaHostAllocMapped) != cudaSuccess) return false;
    if (cudaHostGetDevicePointer(&d, h, 0) != cudaSuccess) {
      cudaFreeHost(h);
      return false;
    }
    g_rb_host[dev] = static_cast<int*>(h);
    g_rb_dev[dev] = static_cast<int*>(d);
  }
  *host = g_rb_host[dev];
  *dev_ptr = g_rb_dev[dev];
  return true;
}

moe_status check_device() {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return cuda_fail(err, "cudaGetDevice");
  if (dev < 0 || dev >= MAX_DEVICES) return fail(MOE_ERR_DEVICE, "device ordinal %d unsupported", dev);
  if (g_cc_ok[dev] == 0) {
    int major = 0, minor = 0, sms = 0;
    if ((err = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(err, "cudaDeviceGetAttribute");
    g_sms[dev] = sms;
    g_cc_ok[dev] = (major == 10 && minor == 3) ? 1 : -1;
    if (g_cc_ok[dev] < 0) {
      return fail(MOE_ERR_DEVICE, "device %d has compute capability %d.%d; this library is built for 10.3 (sm_103a)",
                  dev, major, minor);
    }
  }
  if (g_cc_ok[dev] < 0) return fail(MOE_ERR_DEVICE, "device %d is not compute capability 10.3", dev);
  return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define MOE_REQUIRE(cond, st, ...) \
  do {                             \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

moe_status check_routing_shape(int32_t T, int32_t K, int32_t E) {
  MOE_REQUIRE(T >= 0, MOE_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
  MOE_REQUIRE(E >= 1 && E <= 1024, MOE_ERR_UNSUPPORTED_SHAPE, "E must be in [1, 1024] (got %d)", E);
  MOE_REQUIRE(E % 4 == 0, MOE_ERR_UNSUPPORTED_SHAPE, "E must be a multiple of 4 (got %d)", E);
  MOE_REQUIRE(K >= 1 && K <= E && K <= 127, MOE_ERR_UNSUPPORTED_SHAPE,
              "K must be in [1, min(E, 127)] (got K=%d, E=%d)", K, E);
  return MOE_OK;
}

moe_status check_hidden(int32_t H) {
  MOE_REQUIRE(H > 0 && H % 256 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "the hidden size must be a positive multiple of 256 (got %d)", H);
  return MOE_OK;
}

moe_status check_layout(const moe_layout* L) {
  MOE_REQUIRE(L != nullptr, MOE_ERR_INVALID_ARG, "layout is NULL");
  moe_status st = check_routing_shape(L->T, L->K, L->E);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(L->pad_multiple >= 1, MOE_ERR_INVALID_ARG, "pad_multiple must be >= 1 (got %d)",
              L->pad_multiple);
  MOE_REQUIRE(L->capacity >= 0, MOE_ERR_INVALID_ARG, "capacity must be >= 0");
  const int64_t worst = static_cast<int64_t>(L->T) * L->K +
                        static_cast<int64_t>(L->E) * (L->pad_multiple - 1);
  MOE_REQUIRE(worst < (int64_t(1) << 31) && L->capacity < (int64_t(1) << 31),
              MOE_ERR_UNSUPPORTED_SHAPE, "row counts must fit in int32");
  MOE_REQUIRE(L->tokens_per_expert && L->offsets && L->totals && L->status && L->workspace,
              MOE_ERR_INVALID_ARG, "layout has a NULL count/offset/total/status/workspace pointer");
  MOE_REQUIRE(L->capacity == 0 || (L->row_token && L->row_expert && L->row_weight),
              MOE_ERR_INVALID_ARG, "layout has a NULL row buffer");
  MOE_REQUIRE(L->T == 0 || L->token_row, MOE_ERR_INVALID_ARG, "layout has a NULL token_row");
  MOE_REQUIRE(aligned16(L->workspace), MOE_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return MOE_OK;
}

}  // namespace

moe_status set_last_error(moe_status st, const char* text) { return fail(st, "%s", text); }

int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return 148;
  if (g_sms[dev] == 0) {
    int sms = 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    g_sms[dev] = sms > 0 ? sms : 148;
  }
  return g_sms[dev];
}

}  // namespace moe

using namespace moe;

extern "C" {

const char* moe_status_string(moe_status status) {
  switch (status) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
    case MOE_ERR_UNSUPPORTED_SHAPE: return "MOE_ERR_UNSUPPORTED_SHAPE";
    case MOE_ERR_CAPACITY: return "MOE_ERR_CAPACITY";
    case MOE_ERR_BAD_INDEX: return "MOE_ERR_BAD_INDEX";
    case MOE_ERR_TIMEOUT: return "MOE_ERR_TIMEOUT";
    case MOE_ERR_DEVICE: return "MOE_ERR_DEVICE";
    case MOE_ERR_CUDA: return "MOE_ERR_CUDA";
  }
  return "MOE_ERR_UNKNOWN";
}

const char* moe_last_error(void) { return g_last_error; }

moe_status moe_device_check(void) { return check_device(); }

uint32_t moe_build_flags(void) {
#ifdef MOE_DEBUG_BOUNDS
  return MOE_BUILD_BOUNDS_CHECKS;
#else
  return 0u;
#endif
}

int64_t moe_worst_case_rows(int32_t T, int32_t E, int32_t K, int32_t pad_multiple) {
  if (T < 0 || E < 1 || K < 1 || pad_multiple < 1) return -1;
  return static_cast<int64_t>(T) * K + static_cast<int64_t>(E) * (pad_multiple - 1);
}

moe_status moe_layout_workspace_bytes(int32_t T, int32_t E, size_t* bytes) {
  MOE_REQUIRE(bytes != nullptr, MOE_ERR_INVALID_ARG, "bytes is NULL");
  MOE_REQUIRE(T >= 0 && E >= 1, MOE_ERR_INVALID_ARG, "bad T/E");
  *bytes = dispatch_workspace_bytes(T, E);
  return MOE_OK;
}

moe_status moe_route_to_multihot(const int64_t* topk_idx, const float* topk_probs, int32_t T,
                                 int32_t K, int32_t E, uint8_t* routing_map, float* probs,
                                 int8_t* winner_slot, int32_t* status, moe_stream_t stream) {
  moe_status st = check_routing_shape(T, K, E);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(T == 0 || (topk_idx && topk_probs && routing_map && probs && winner_slot && status),
              MOE_ERR_INVALID_ARG, "moe_route_to_multihot: NULL pointer");
  MOE_REQUIRE(aligned16(routing_map) && aligned16(probs) && aligned16(winner_slot),
              MOE_ERR_INVALID_ARG, "moe_route_to_multihot: outputs must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_multihot(topk_idx, topk_probs, T, K, E, routing_map, probs, winner_slot,
                                    status, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_route_to_multihot launch");
}

}  // extern "C"

namespace {

// moe_dispatch and moe_dispatch_fp8: the layout (host-synced or sync-free),
// then the rows, in bf16 (x_disp) or as e4m3 codes with per-row scales.
// With topk_idx non-NULL the input is the top-k choices, and routing_map /
// probs / winner are outputs (the multihot step fused into the dispatch).
moe_status dispatch_impl(const char* who, const moe_bf16* x, const uint8_t* routing_map,
                         const float* probs, int32_t H, const moe_layout* L, moe_bf16* x_disp,
                         uint8_t* x_q, float* x_scale, int64_t* rows_host, moe_stream_t stream,
                         bool layout_only = false, const int64_t* topk_idx = nullptr,
                         const float* topk_probs = nullptr, int8_t* winner = nullptr) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if (layout_only) H = 256;  // no rows are copied; any valid hidden size will do
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(L->T == 0 || ((x || layout_only) && routing_map && probs), MOE_ERR_INVALID_ARG,
              "%s: NULL input", who);
  MOE_REQUIRE(!topk_idx || L->T == 0 || (topk_probs && winner), MOE_ERR_INVALID_ARG,
              "%s: NULL top-k input or multihot output", who);
  MOE_REQUIRE(aligned16(probs) && aligned16(winner), MOE_ERR_INVALID_ARG,
              "%s: probs and winner_slot must be 16-byte aligned", who);
  MOE_REQUIRE(L->capacity == 0 || layout_only || x_disp || (x_q && x_scale), MOE_ERR_INVALID_ARG,
              "%s: NULL output rows", who);
  MOE_REQUIRE(aligned16(x) && aligned16(x_disp) && aligned16(x_q) && aligned16(routing_map),
              MOE_ERR_INVALID_ARG, "%s: x, the output rows and routing_map must be 16-byte aligned",
              who);
  const int64_t worst = moe_worst_case_rows(L->T, L->E, L->K, L->pad_multiple);
  if (!rows_host && L->capacity < worst)
    return fail(MOE_ERR_CAPACITY,
                "sync-free dispatch needs capacity >= T*K + E*(pad_multiple-1) = %lld rows (got %lld)",
                static_cast<long long>(worst), static_cast<long long>(L->capacity));
  if ((st = check_device()) != MOE_OK) return st;

  // Host-synced callers get R, N and the status word through mapped pinned
  // memory that the layout kernel writes as soon as the offsets are known.
  int *rb_host = nullptr, *rb_dev = nullptr;
  std::unique_lock<std::mutex> rb_lock(g_rb_mu, std::defer_lock);
  bool mapped = false;
  if (rows_host) {
    int dev = 0;
    rb_lock.lock();
    mapped = cudaGetDevice(&dev) == cudaSuccess && readback_buffer(dev, &rb_host, &rb_dev);
    if (mapped) {
      volatile int* rb = rb_host;
      rb[0] = rb[1] = rb[2] = -1;  // overwritten by the layout kernel
    } else {
      rb_lock.unlock();
    }
  }
  // The layout, then the rows (or, for the layout alone, just the pad and
  // spare rows' metadata), queued at once in both modes.  When the rows do
  // not fit (host-synced, R > capacity) both kernels write nothing.
  cudaError_t err;
  bool rows_done = false;  // the layout kernel did the row pass itself
  const bool bf16_rows = x_disp || layout_only;
  const bool fp8_rows = !bf16_rows && x_q != nullptr;
  const bool fused = (bf16_rows || fp8_rows) && dispatch_fused_fits(*L);
  const uint16_t* x16 = reinterpret_cast<const uint16_t*>(x);
  uint16_t* xd16 = reinterpret_cast<uint16_t*>(x_disp);
  int* rb_kernel = mapped ? rb_dev : nullptr;
  if (topk_idx && !fused) {
    // small layers: the multihot step first, then the layout from its map
    if ((err = launch_multihot(topk_idx, topk_probs, L->T, L->K, L->E, const_cast<uint8_t*>(routing_map),
                               const_cast<float*>(probs), winner, L->status, stream)) != cudaSuccess) {
      if (mapped) rb_lock.unlock();
      return cuda_fail(err, "dispatch: multihot");
    }
  }
  if (fused) {
    if (topk_idx)
      err = fp8_rows ? launch_dispatch_fused_topk_fp8(topk_idx, topk_probs, const_cast<uint8_t*>(routing_map),
                                                      const_cast<float*>(probs), winner, *L, H, x16, x_q, x_scale,
                                                      rb_kernel, stream)
                     : launch_dispatch_fused_topk(topk_idx, topk_probs, const_cast<uint8_t*>(routing_map),
                                                  const_cast<float*>(probs), winner, *L, H, x16, xd16, rb_kernel,
                                                  stream);
    else
      err = fp8_rows ? launch_dispatch_fused_map_fp8(routing_map, probs, *L, H, x16, x_q, x_scale, rb_kernel, stream)
                     : launch_dispatch_fused_map(routing_map, probs, *L, H, x16, xd16, rb_kernel, stream);
    if (err != cudaSuccess) {
      if (mapped) cudaStreamSynchronize(stream);  // the kernel may still write the readback buffer
      return cuda_fail(err, "dispatch: fused layout and rows");
    }
    rows_done = true;
  } else if ((err = launch_layout(routing_map, probs, *L, L->workspace, stream, rb_kernel, x16, xd16, H,
                                  bf16_rows ? &rows_done : nullptr)) != cudaSuccess) {
    return cuda_fail(err, "dispatch: layout");
  }
  if (!rows_done) {
    err = bf16_rows ? launch_row_gather(x, *L, H, x_disp, true, nullptr, nullptr, stream)
                    : launch_row_gather_fp8(x, *L, H, x_q, x_scale, stream);
    if (err != cudaSuccess) {
      // the layout kernel may still write the readback buffer: let it finish
      // before the buffer goes to the next caller
      if (mapped) cudaStreamSynchronize(stream);
      return cuda_fail(err, "dispatch: rows");
    }
  }
  if (!rows_host) return MOE_OK;

  // Host-synced: wait for the counts.  With the mapped buffer, until the
  // layout kernel publishes R (the kernels behind it keep running), or until
  // the stream is idle without it (the kernel gave up: read the device
  // copies).
  int32_t tot[2] = {0, 0}, dev_status = 0;
  volatile int* rb = rb_host;
  bool published = false;
  if (mapped) {
    const auto t0 = std::chrono::steady_clock::now();
    for (unsigned spin = 0;; ++spin) {
      if (rb[0] >= 0) {
        published = true;
        break;
      }
      if ((spin & 255u) != 255u) continue;
      const cudaError_t q = cudaStreamQuery(stream);
      if (q == cudaSuccess) {
        published = rb[0] >= 0;
        break;
      }
      if (q != cudaErrorNotReady) {
        cudaStreamSynchronize(stream);  // as above: nothing may write the buffer afterwards
        return cuda_fail(q, "dispatch: waiting for the row counts");
      }
      if (std::chrono::steady_clock::now() - t0 > std::chrono::seconds(READBACK_POLL_LIMIT_S)) break;
    }
  }
  if (published) {
    std::atomic_thread_fence(std::memory_order_acquire);
    tot[0] = rb[0];
    tot[1] = rb[1];
    dev_status = rb[2];
  } else if ((err = cudaStreamSynchronize(stream)) != cudaSuccess ||
             (err = cudaMemcpy(tot, L->totals, sizeof(tot), cudaMemcpyDeviceToHost)) != cudaSuccess ||
             (err = cudaMemcpy(&dev_status, L->status, sizeof(int32_t), cudaMemcpyDeviceToHost)) != cudaSuccess) {
    return cuda_fail(err, "dispatch: reading the row counts");
  }
  if (rb_lock.owns_lock()) rb_lock.unlock();
  rows_host[0] = tot[0];
  rows_host[1] = tot[1];
  if (dev_status & MOE_DEVERR_TIMEOUT)
    return fail(MOE_ERR_TIMEOUT, "the layout kernel's grid barrier timed out");
  if (dev_status & MOE_DEVERR_BAD_INDEX)
    return fail(MOE_ERR_BAD_INDEX, "an expert index outside [-1, E) was seen");
  if (tot[0] > L->capacity)
    return fail(MOE_ERR_CAPACITY, "the layout needs %d rows, capacity is %lld", tot[0],
                static_cast<long long>(L->capacity));
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_dispatch(const moe_bf16* x, const uint8_t* routing_map, const float* probs,
                        int32_t H, const moe_layout* L, moe_bf16* x_disp, int64_t* rows_host,
                        moe_stream_t stream) {
  MOE_REQUIRE(L == nullptr || L->capacity == 0 || x_disp, MOE_ERR_INVALID_ARG,
              "moe_dispatch: NULL x_disp");
  return dispatch_impl("moe_dispatch", x, routing_map, probs, H, L, x_disp, nullptr, nullptr,
                       rows_host, stream);
}

moe_status moe_dispatch_topk(const moe_bf16* x, const int64_t* topk_idx, const float* topk_probs,
                             int32_t H, const moe_layout* L, uint8_t* routing_map, float* probs,
                             int8_t* winner_slot, moe_bf16* x_disp, int64_t* rows_host,
                             moe_stream_t stream) {
  MOE_REQUIRE(L == nullptr || L->capacity == 0 || x_disp, MOE_ERR_INVALID_ARG,
              "moe_dispatch_topk: NULL x_disp");
  MOE_REQUIRE(L == nullptr || L->T == 0 || (topk_idx && topk_probs), MOE_ERR_INVALID_ARG,
              "moe_dispatch_topk: NULL top-k input");
  static const int64_t no_slots = 0;  // T == 0: marks the top-k input without reading it
  return dispatch_impl("moe_dispatch_topk", x, routing_map, probs, H, L, x_disp, nullptr, nullptr,
                       rows_host, stream, false, topk_idx ? topk_idx : &no_slots, topk_probs,
                       winner_slot);
}

moe_status moe_dispatch_topk_fp8(const moe_bf16* x, const int64_t* topk_idx, const float* topk_probs,
                                 int32_t H, const moe_layout* L, uint8_t* routing_map, float* probs,
                                 int8_t* winner_slot, uint8_t* x_disp_q, float* x_disp_scale, int64_t* rows_host,
                                 moe_stream_t stream) {
  MOE_REQUIRE(L == nullptr || L->capacity == 0 || (x_disp_q && x_disp_scale), MOE_ERR_INVALID_ARG,
              "moe_dispatch_topk_fp8: NULL x_disp_q or x_disp_scale");
  MOE_REQUIRE(L == nullptr || L->T == 0 || (topk_idx && topk_probs), MOE_ERR_INVALID_ARG,
              "moe_dispatch_topk_fp8: NULL top-k input");
  static const int64_t no_slots = 0;  // T == 0: marks the top-k input without reading it
  return dispatch_impl("moe_dispatch_topk_fp8", x, routing_map, probs, H, L, nullptr, x_disp_q, x_disp_scale,
                       rows_host, stream, false, topk_idx ? topk_idx : &no_slots, topk_probs, winner_slot);
}

moe_status moe_dispatch_fp8(const moe_bf16* x, const uint8_t* routing_map, const float* probs,
                            int32_t H, const moe_layout* L, uint8_t* x_disp_q, float* x_disp_scale,
                            int64_t* rows_host, moe_stream_t stream) {
  MOE_REQUIRE(L == nullptr || L->capacity == 0 || (x_disp_q && x_disp_scale), MOE_ERR_INVALID_ARG,
              "moe_dispatch_fp8: NULL x_disp_q or x_disp_scale");
  return dispatch_impl("moe_dispatch_fp8", x, routing_map, probs, H, L, nullptr, x_disp_q,
                       x_disp_scale, rows_host, stream);
}

moe_status moe_dispatch_layout(const uint8_t* routing_map, const float* probs, const moe_layout* L,
                               int64_t* rows_host, moe_stream_t stream) {
  return dispatch_impl("moe_dispatch_layout", nullptr, routing_map, probs, 256, L, nullptr, nullptr,
                       nullptr, rows_host, stream, /*layout_only=*/true);
}

moe_status moe_grouped_experts_gather(const moe_bf16* x, const moe_layout* L, int32_t H, int32_t I,
                                      const moe_bf16* W1, const moe_bf16* W2, moe_bf16* h,
                                      moe_bf16* y_disp, moe_bf16* o_save, moe_bf16* gu_save,
                                      moe_stream_t stream) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(I > 0 && I % 128 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "the intermediate size must be a positive multiple of 128 (got %d)", I);
  MOE_REQUIRE(L->capacity == 0 || ((x || L->T == 0) && W1 && W2 && h && y_disp), MOE_ERR_INVALID_ARG,
              "moe_grouped_experts_gather: NULL pointer");
  MOE_REQUIRE(aligned16(x) && aligned16(W1) && aligned16(W2) && aligned16(h) && aligned16(y_disp) &&
                  aligned16(o_save) && aligned16(gu_save),
              MOE_ERR_INVALID_ARG, "moe_grouped_experts_gather: pointers must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_experts_forward_gather(x, *L, H, I, W1, W2, h, y_disp, o_save, gu_save, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_grouped_experts_gather launch");
}

moe_status moe_quantize_fp8(const moe_bf16* src, int64_t rows, int32_t cols, uint8_t* codes,
                            float* scales, moe_stream_t stream) {
  MOE_REQUIRE(rows >= 0, MOE_ERR_INVALID_ARG, "moe_quantize_fp8: rows must be >= 0");
  MOE_REQUIRE(cols > 0 && cols % 256 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "moe_quantize_fp8: cols must be a positive multiple of 256 (got %d)", cols);
  MOE_REQUIRE(rows == 0 || (src && codes && scales), MOE_ERR_INVALID_ARG,
              "moe_quantize_fp8: NULL pointer");
  MOE_REQUIRE(aligned16(src) && aligned16(codes), MOE_ERR_INVALID_ARG,
              "moe_quantize_fp8: src and codes must be 16-byte aligned");
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  cudaError_t err = launch_quantize_rows_fp8(src, rows, cols, codes, scales, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_quantize_fp8 launch");
}

moe_status moe_grouped_experts_fp8(const uint8_t* x_disp_q, const float* x_disp_scale,
                                   const moe_layout* L, int32_t H, int32_t I, const uint8_t* W1_q,
                                   const float* W1_scale, const moe_bf16* W2, moe_bf16* h,
                                   moe_bf16* y_disp, moe_stream_t stream) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(I > 0 && I % 128 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "the intermediate size must be a positive multiple of 128 (got %d)", I);
  MOE_REQUIRE(L->capacity == 0 || (x_disp_q && x_disp_scale && W1_q && W1_scale && W2 && h && y_disp),
              MOE_ERR_INVALID_ARG, "moe_grouped_experts_fp8: NULL pointer");
  MOE_REQUIRE(aligned16(x_disp_q) && aligned16(W1_q) && aligned16(W2) && aligned16(h) &&
                  aligned16(y_disp),
              MOE_ERR_INVALID_ARG, "moe_grouped_experts_fp8: pointers must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_experts_forward_fp8(x_disp_q, x_disp_scale, *L, H, I, W1_q, W1_scale, W2,
                                               h, y_disp, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_grouped_experts_fp8 launch");
}

moe_status moe_grouped_experts(const moe_bf16* x_disp, const moe_layout* L, int32_t H, int32_t I,
                               const moe_bf16* W1, const moe_bf16* W2, moe_bf16* h,
                               moe_bf16* y_disp, moe_bf16* o_save, moe_bf16* gu_save,
                               moe_stream_t stream) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(I > 0 && I % 128 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "the intermediate size must be a positive multiple of 128 (got %d)", I);
  MOE_REQUIRE(L->capacity == 0 || (x_disp && W1 && W2 && h && y_disp), MOE_ERR_INVALID_ARG,
              "moe_grouped_experts: NULL pointer");
  MOE_REQUIRE(aligned16(x_disp) && aligned16(W1) && aligned16(W2) && aligned16(h) &&
                  aligned16(y_disp) && aligned16(o_save) && aligned16(gu_save),
              MOE_ERR_INVALID_ARG, "moe_grouped_experts: pointers must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_experts_forward(x_disp, *L, H, I, W1, W2, h, y_disp, o_save, gu_save, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_grouped_experts launch");
}

moe_status moe_combine(const moe_bf16* y_disp, const moe_layout* L, int32_t H, moe_bf16* out,
                       moe_stream_t stream) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(L->T == 0 || (y_disp && out), MOE_ERR_INVALID_ARG, "moe_combine: NULL pointer");
  MOE_REQUIRE(aligned16(y_disp) && aligned16(out), MOE_ERR_INVALID_ARG,
              "moe_combine: pointers must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_combine(y_disp, *L, H, out, nullptr, nullptr, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_combine launch");
}

}  // extern "C"

namespace {

moe_status combine_backward_impl(const char* who, const moe_bf16* grad_out, const moe_bf16* o_save,
                                 const moe_layout* L, int32_t H, moe_bf16* grad_y, float* grad_w,
                                 moe_stream_t stream, bool scale) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(L->capacity == 0 || (grad_out && grad_y), MOE_ERR_INVALID_ARG, "%s: NULL pointer", who);
  MOE_REQUIRE(!grad_w || o_save, MOE_ERR_INVALID_ARG, "%s: grad_w needs o_save", who);
  MOE_REQUIRE(aligned16(grad_out) && aligned16(grad_y) && aligned16(o_save), MOE_ERR_INVALID_ARG,
              "%s: pointers must be 16-byte aligned", who);
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_row_gather(grad_out, *L, H, grad_y, false, o_save, grad_w, stream, scale);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, who);
}

moe_status experts_backward_impl(const char* who, const moe_bf16* grad_y, const moe_bf16* x_disp,
                                 const moe_bf16* h, const moe_bf16* gu_save, const moe_layout* L,
                                 int32_t H, int32_t I, const moe_bf16* W1, const moe_bf16* W2,
                                 moe_bf16* grad_x_disp, float* dW1, float* dW2, void* workspace,
                                 moe_stream_t stream, bool g_o_given) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(I > 0 && I % 128 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "the intermediate size must be a positive multiple of 128 (got %d)", I);
  MOE_REQUIRE(W1 && W2 && workspace, MOE_ERR_INVALID_ARG, "%s: NULL weight or workspace pointer", who);
  MOE_REQUIRE(L->capacity == 0 || (grad_y && x_disp && h && gu_save && grad_x_disp),
              MOE_ERR_INVALID_ARG, "%s: NULL row buffer", who);
  MOE_REQUIRE(aligned16(grad_y) && aligned16(x_disp) && aligned16(h) && aligned16(gu_save) &&
                  aligned16(W1) && aligned16(W2) && aligned16(grad_x_disp) && aligned16(dW1) &&
                  aligned16(dW2),
              MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_experts_backward(grad_y, x_disp, h, gu_save, *L, H, I, W1, W2, grad_x_disp,
                                            dW1, dW2, workspace, stream, g_o_given);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, who);
}

}  // namespace

extern "C" {

moe_status moe_combine_backward_scaled(const moe_bf16* grad_out, const moe_bf16* o_save,
                                       const moe_layout* L, int32_t H, moe_bf16* g_o, float* grad_w,
                                       moe_stream_t stream) {
  return combine_backward_impl("moe_combine_backward_scaled", grad_out, o_save, L, H, g_o, grad_w, stream,
                               true);
}

moe_status moe_grouped_experts_backward_scaled(const moe_bf16* g_o, const moe_bf16* x_disp,
                                               const moe_bf16* h, const moe_bf16* gu_save,
                                               const moe_layout* L, int32_t H, int32_t I,
                                               const moe_bf16* W1, const moe_bf16* W2,
                                               moe_bf16* grad_x_disp, float* dW1, float* dW2,
                                               void* workspace, moe_stream_t stream) {
  return experts_backward_impl("moe_grouped_experts_backward_scaled", g_o, x_disp, h, gu_save, L, H, I, W1,
                               W2, grad_x_disp, dW1, dW2, workspace, stream, true);
}

moe_status moe_combine_backward(const moe_bf16* grad_out, const moe_bf16* o_save,
                                const moe_layout* L, int32_t H, moe_bf16* grad_y, float* grad_w,
                                moe_stream_t stream) {
  return combine_backward_impl("moe_combine_backward", grad_out, o_save, L, H, grad_y, grad_w, stream,
                               false);
}


moe_status moe_dispatch_backward(const moe_bf16* grad_x_disp, const float* grad_w,
                                 const moe_layout* L, int32_t H, moe_bf16* grad_x,
                                 float* grad_probs, moe_stream_t stream) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(L->T == 0 || (grad_x_disp && grad_x), MOE_ERR_INVALID_ARG,
              "moe_dispatch_backward: NULL pointer");
  MOE_REQUIRE(aligned16(grad_x_disp) && aligned16(grad_x) && aligned16(grad_probs),
              MOE_ERR_INVALID_ARG, "moe_dispatch_backward: pointers must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_combine(grad_x_disp, *L, H, grad_x, grad_w, grad_probs, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_dispatch_backward launch");
}

moe_status moe_router_topk(const float* logits, int32_t T, int32_t E, int32_t K, int64_t* topk_idx,
                           float* topk_probs, uint8_t* routing_map, float* probs,
                           int8_t* winner_slot, moe_stream_t stream) {
  moe_status st = check_routing_shape(T, K, E);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(T == 0 || (logits && topk_idx && topk_probs), MOE_ERR_INVALID_ARG,
              "moe_router_topk: NULL logits or top-k output");
  const bool mh = routing_map || probs || winner_slot;
  MOE_REQUIRE(!mh || (routing_map && probs && winner_slot), MOE_ERR_INVALID_ARG,
              "moe_router_topk: give all three multihot outputs or none");
  MOE_REQUIRE(aligned16(routing_map) && aligned16(probs) && aligned16(winner_slot),
              MOE_ERR_INVALID_ARG, "moe_router_topk: multihot outputs must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_router_topk(logits, T, K, E, topk_idx, topk_probs,
                                       mh ? routing_map : nullptr, probs, winner_slot, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_router_topk launch");
}

moe_status moe_router_topk_backward(const float* grad_topk_probs, const float* topk_probs,
                                    const int64_t* topk_idx, int32_t T, int32_t E, int32_t K,
                                    float* grad_logits, moe_stream_t stream) {
  moe_status st = check_routing_shape(T, K, E);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(T == 0 || (grad_topk_probs && topk_probs && topk_idx && grad_logits),
              MOE_ERR_INVALID_ARG, "moe_router_topk_backward: NULL pointer");
  MOE_REQUIRE(aligned16(grad_logits), MOE_ERR_INVALID_ARG,
              "moe_router_topk_backward: grad_logits must be 16-byte aligned");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_router_topk_backward(grad_topk_probs, topk_probs, topk_idx, T, K, E,
                                                grad_logits, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_router_topk_backward launch");
}

moe_status moe_route_to_multihot_backward(const float* grad_probs, const int64_t* topk_idx,
                                          const int8_t* winner_slot, int32_t T, int32_t K,
                                          int32_t E, float* grad_topk_probs, moe_stream_t stream) {
  moe_status st = check_routing_shape(T, K, E);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(T == 0 || (grad_probs && topk_idx && winner_slot && grad_topk_probs),
              MOE_ERR_INVALID_ARG, "moe_route_to_multihot_backward: NULL pointer");
  if ((st = check_device()) != MOE_OK) return st;
  cudaError_t err = launch_multihot_backward(grad_probs, topk_idx, winner_slot, T, K, E,
                                             grad_topk_probs, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_route_to_multihot_backward launch");
}

moe_status moe_experts_backward_workspace_bytes(int64_t capacity, int32_t H, int32_t I,
                                                size_t* bytes) {
  MOE_REQUIRE(bytes != nullptr, MOE_ERR_INVALID_ARG, "bytes is NULL");
  MOE_REQUIRE(capacity >= 0 && H > 0 && I > 0, MOE_ERR_INVALID_ARG, "bad capacity / H / I");
  *bytes = experts_backward_workspace(capacity, H, I);
  return MOE_OK;
}

moe_status moe_grouped_experts_backward(const moe_bf16* grad_y, const moe_bf16* x_disp,
                                        const moe_bf16* h, const moe_bf16* gu_save,
                                        const moe_layout* L, int32_t H, int32_t I,
                                        const moe_bf16* W1, const moe_bf16* W2,
                                        moe_bf16* grad_x_disp, float* dW1, float* dW2,
                                        void* workspace, moe_stream_t stream) {
  return experts_backward_impl("moe_grouped_experts_backward", grad_y, x_disp, h, gu_save, L, H, I, W1, W2,
                               grad_x_disp, dW1, dW2, workspace, stream, false);
}

}  // extern "C"

namespace {

bool is_dtype(int32_t d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }

moe_status check_norm(const char* who, const moe_norm* n) {
  MOE_REQUIRE(n != nullptr, MOE_ERR_INVALID_ARG, "%s: NULL moe_norm", who);
  MOE_REQUIRE(n->T >= 0, MOE_ERR_INVALID_ARG, "%s: T must be >= 0 (got %lld)", who,
              static_cast<long long>(n->T));
  MOE_REQUIRE(n->H >= 1 && n->H <= 16384, MOE_ERR_UNSUPPORTED_SHAPE, "%s: H must be in [1, 16384] (got %d)", who,
              n->H);
  MOE_REQUIRE(is_dtype(n->x_dtype) && is_dtype(n->weight_dtype) && is_dtype(n->gate_dtype), MOE_ERR_INVALID_ARG,
              "%s: unknown element type", who);
  MOE_REQUIRE(n->gate_kind >= MOE_GATE_NONE && n->gate_kind <= MOE_GATE_ELEMENT, MOE_ERR_INVALID_ARG,
              "%s: unknown gate kind %d", who, n->gate_kind);
  MOE_REQUIRE(std::isfinite(n->eps) && n->eps >= 0.f && std::isfinite(n->residual_scale) &&
                  std::isfinite(n->weight_offset),
              MOE_ERR_INVALID_ARG, "%s: eps must be finite and >= 0, the scale and the offset finite", who);
  return MOE_OK;
}

bool aligned_to(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename... P>
bool all_aligned(uintptr_t bytes, P... p) {
  return (aligned_to(p, bytes) && ...);
}

uintptr_t bytes_of(int32_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Rows of a multiple of 8 values are read in pieces of 16 bytes, others value by value.
uintptr_t row_bytes(const moe_norm* n, int32_t dtype) { return n->H % 8 == 0 ? 16 : bytes_of(dtype); }

// A gate of one value a token is read value by value.
uintptr_t gate_bytes(const moe_norm* n) {
  return n->gate_kind == MOE_GATE_ELEMENT ? row_bytes(n, n->gate_dtype) : bytes_of(n->gate_dtype);
}

NormArgs norm_args(const moe_norm* n) {
  NormArgs a{};
  a.T = n->T;
  a.load_T = norm_load_rows(n->T);
  a.H = n->H;
  a.x_f32 = n->x_dtype == MOE_DTYPE_F32;
  a.w_f32 = n->weight_dtype == MOE_DTYPE_F32;
  a.gate_f32 = n->gate_dtype == MOE_DTYPE_F32;
  a.gate_kind = n->gate_kind;
  a.sigmoid = n->gate_sigmoid != 0;
  a.residual_scale = n->residual_scale;
  a.eps = n->eps;
  a.offset = n->weight_offset;
  return a;
}

NormBackwardArgs norm_backward_args(const moe_norm* n) {
  NormBackwardArgs a{};
  a.T = n->T;
  a.load_T = norm_load_rows(n->T);
  a.H = n->H;
  a.x_f32 = n->x_dtype == MOE_DTYPE_F32;
  a.w_f32 = n->weight_dtype == MOE_DTYPE_F32;
  a.gate_f32 = n->gate_dtype == MOE_DTYPE_F32;
  a.gate_kind = n->gate_kind;
  a.sigmoid = n->gate_sigmoid != 0;
  a.residual_scale = n->residual_scale;
  a.offset = n->weight_offset;
  return a;
}

}  // namespace

extern "C" {

moe_status moe_norm_in(const moe_norm* n, const void* x, const void* weight, moe_bf16* norm, float* rstd,
                       moe_stream_t stream) {
  moe_status st = check_norm("moe_norm_in", n);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(n->T == 0 || (x && weight && norm), MOE_ERR_INVALID_ARG, "moe_norm_in: NULL pointer");
  MOE_REQUIRE(all_aligned(row_bytes(n, n->x_dtype), x) && all_aligned(row_bytes(n, n->weight_dtype), weight) &&
                  all_aligned(row_bytes(n, MOE_DTYPE_BF16), norm) && all_aligned(4, rstd),
              MOE_ERR_INVALID_ARG,
              "moe_norm_in: rows and weights must be 16-byte aligned (H % 8 == 0), others by their type");
  if ((st = check_device()) != MOE_OK) return st;
  NormArgs a = norm_args(n);
  a.gate_kind = MOE_GATE_NONE;
  a.x = x;
  a.w2 = weight;
  a.next = norm;
  a.rstd2 = rstd;
  cudaError_t err = launch_norm_forward(a, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_norm_in launch");
}

moe_status moe_norm_backward_workspace_bytes(int64_t T, int32_t H, size_t* bytes) {
  MOE_REQUIRE(bytes != nullptr, MOE_ERR_INVALID_ARG, "bytes is NULL");
  MOE_REQUIRE(T >= 0 && H >= 1 && H <= 16384, MOE_ERR_INVALID_ARG, "bad T / H");
  *bytes = norm_backward_workspace(T, H);
  return MOE_OK;
}

moe_status moe_norm_in_backward(const moe_norm* n, const moe_bf16* grad_norm, const void* x, const void* weight,
                                const float* rstd, const void* grad_res, void* grad_x, float* grad_weight,
                                void* workspace, moe_stream_t stream) {
  moe_status st = check_norm("moe_norm_in_backward", n);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(grad_weight && (n->T == 0 || (grad_norm && x && weight && rstd && grad_x && workspace)),
              MOE_ERR_INVALID_ARG, "moe_norm_in_backward: NULL pointer");
  MOE_REQUIRE(all_aligned(row_bytes(n, MOE_DTYPE_BF16), grad_norm) &&
                  all_aligned(row_bytes(n, n->x_dtype), x, grad_res, grad_x) &&
                  all_aligned(row_bytes(n, n->weight_dtype), weight) &&
                  all_aligned(row_bytes(n, MOE_DTYPE_F32), grad_weight) && all_aligned(4, rstd) && aligned16(workspace),
              MOE_ERR_INVALID_ARG,
              "moe_norm_in_backward: rows and weights must be 16-byte aligned (H % 8 == 0), others by their type");
  if ((st = check_device()) != MOE_OK) return st;
  NormBackwardArgs a = norm_backward_args(n);
  a.gate_kind = MOE_GATE_NONE;
  a.has_next = 1;
  a.dout = grad_res;
  a.dnext = grad_norm;
  a.out = x;
  a.w2 = weight;
  a.rstd2 = rstd;
  a.dx = grad_x;
  a.dw2 = grad_weight;
  a.partials = static_cast<float*>(workspace);
  cudaError_t err = launch_norm_backward(a, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_norm_in_backward launch");
}

moe_status moe_norm_out(const moe_norm* n, const void* x, const moe_bf16* y, const void* weight, const void* gate,
                        void* out, float* rstd, const void* next_weight, moe_bf16* next, float* next_rstd,
                        moe_stream_t stream) {
  moe_status st = check_norm("moe_norm_out", n);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(n->T == 0 || (x && y && weight && out), MOE_ERR_INVALID_ARG, "moe_norm_out: NULL pointer");
  MOE_REQUIRE((n->gate_kind == MOE_GATE_NONE) ? !gate : (gate || n->T == 0), MOE_ERR_INVALID_ARG,
              "moe_norm_out: give gate exactly when gate_kind is not MOE_GATE_NONE");
  MOE_REQUIRE((next_weight != nullptr) == (next != nullptr) || n->T == 0, MOE_ERR_INVALID_ARG,
              "moe_norm_out: give next_weight and next, or neither");
  MOE_REQUIRE(next_weight || !next_rstd, MOE_ERR_INVALID_ARG, "moe_norm_out: next_rstd without next_weight");
  MOE_REQUIRE(all_aligned(row_bytes(n, n->x_dtype), x, out) && all_aligned(row_bytes(n, MOE_DTYPE_BF16), y, next) &&
                  all_aligned(row_bytes(n, n->weight_dtype), weight, next_weight) && all_aligned(gate_bytes(n), gate) &&
                  all_aligned(4, rstd, next_rstd),
              MOE_ERR_INVALID_ARG,
              "moe_norm_out: rows and weights must be 16-byte aligned (H % 8 == 0), others by their type");
  if ((st = check_device()) != MOE_OK) return st;
  NormArgs a = norm_args(n);
  a.x = x;
  a.y = y;
  a.w = weight;
  a.gate = gate;
  a.w2 = next_weight;
  a.out = out;
  a.next = next;
  a.rstd = rstd;
  a.rstd2 = next_rstd;
  cudaError_t err = launch_norm_forward(a, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_norm_out launch");
}

moe_status moe_norm_out_backward(const moe_norm* n, const void* grad_out, const moe_bf16* grad_next,
                                 const void* out, const moe_bf16* y, const void* weight, const void* gate,
                                 const float* rstd, const void* next_weight, const float* next_rstd, void* grad_x,
                                 moe_bf16* grad_y, void* grad_gate, float* grad_weight, float* grad_next_weight,
                                 void* workspace, moe_stream_t stream) {
  moe_status st = check_norm("moe_norm_out_backward", n);
  if (st != MOE_OK) return st;
  // which of the two there are, told by a pointer that is there for T = 0 too
  const bool has_next = grad_next_weight != nullptr;
  MOE_REQUIRE(grad_weight, MOE_ERR_INVALID_ARG, "moe_norm_out_backward: NULL grad_weight");
  MOE_REQUIRE(n->T == 0 || (y && weight && rstd && grad_x && grad_y && workspace && (grad_out || has_next)),
              MOE_ERR_INVALID_ARG, "moe_norm_out_backward: NULL pointer");
  MOE_REQUIRE(has_next ? (n->T == 0 || (grad_next && out && next_weight && next_rstd))
                       : (!grad_next && !next_weight && !next_rstd),
              MOE_ERR_INVALID_ARG,
              "moe_norm_out_backward: give grad_next, out, next_weight, next_rstd and grad_next_weight, or none");
  MOE_REQUIRE((n->gate_kind == MOE_GATE_NONE) ? (!gate && !grad_gate) : (gate || n->T == 0), MOE_ERR_INVALID_ARG,
              "moe_norm_out_backward: give gate exactly when gate_kind is not MOE_GATE_NONE");
  MOE_REQUIRE(all_aligned(row_bytes(n, n->x_dtype), grad_out, out, grad_x) &&
                  all_aligned(row_bytes(n, MOE_DTYPE_BF16), grad_next, y, grad_y) &&
                  all_aligned(row_bytes(n, n->weight_dtype), weight, next_weight) &&
                  all_aligned(row_bytes(n, MOE_DTYPE_F32), grad_weight, grad_next_weight) &&
                  all_aligned(gate_bytes(n), gate, grad_gate) && all_aligned(4, rstd, next_rstd) && aligned16(workspace),
              MOE_ERR_INVALID_ARG,
              "moe_norm_out_backward: rows and weights must be 16-byte aligned (H % 8 == 0), others by their type");
  if ((st = check_device()) != MOE_OK) return st;
  NormBackwardArgs a = norm_backward_args(n);
  a.has_y = 1;
  a.has_next = has_next;
  a.dout = grad_out;
  a.dnext = grad_next;
  a.out = out;
  a.y = y;
  a.w = weight;
  a.gate = gate;
  a.w2 = next_weight;
  a.rstd = rstd;
  a.rstd2 = next_rstd;
  a.dx = grad_x;
  a.dy = grad_y;
  a.dgate = grad_gate;
  a.dw = grad_weight;
  a.dw2 = grad_next_weight;
  a.partials = static_cast<float*>(workspace);
  cudaError_t err = launch_norm_backward(a, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_norm_out_backward launch");
}

}  // extern "C"

extern "C" {

moe_status moe_adamw_step(const moe_adamw* h, const moe_adamw_tensor* tensors, int32_t count, moe_stream_t stream) {
  MOE_REQUIRE(h && (tensors || count == 0) && count >= 0, MOE_ERR_INVALID_ARG,
              "moe_adamw_step: NULL argument or negative count");
  MOE_REQUIRE(h->state_bits == 8 || h->state_bits == 32, MOE_ERR_INVALID_ARG,
              "moe_adamw_step: state_bits must be 8 or 32 (got %d)", h->state_bits);
  MOE_REQUIRE(h->step >= 1, MOE_ERR_INVALID_ARG, "moe_adamw_step: step must be >= 1 (got %lld)",
              static_cast<long long>(h->step));
  MOE_REQUIRE(h->beta1 >= 0 && h->beta1 < 1 && h->beta2 >= 0 && h->beta2 < 1, MOE_ERR_INVALID_ARG,
              "moe_adamw_step: betas must be in [0, 1)");
  // (below 1e30: what the update divides by stays in its division's range)
  MOE_REQUIRE(std::isfinite(h->lr) && h->lr >= 0 && h->eps >= 0 && h->eps < 1e30, MOE_ERR_INVALID_ARG,
              "moe_adamw_step: lr must be finite and >= 0, eps in [0, 1e30)");
  MOE_REQUIRE(aligned_to(h->grad_scale, 4) && aligned_to(h->skip, 4) && aligned_to(h->step_dev, 8),
              MOE_ERR_INVALID_ARG, "moe_adamw_step: misaligned grad_scale, skip or step_dev");
  const bool eight = h->state_bits == 8;
  AdamWTensor* list = new (std::nothrow) AdamWTensor[count > 0 ? count : 1];
  MOE_REQUIRE(list, MOE_ERR_INVALID_ARG, "moe_adamw_step: no host memory for %d tensors", count);
  struct Free {
    AdamWTensor* p;
    ~Free() { delete[] p; }
  } release{list};
  int64_t blocks = 0;
  for (int32_t k = 0; k < count; ++k) {
    const moe_adamw_tensor& t = tensors[k];
    MOE_REQUIRE(t.n >= 0, MOE_ERR_INVALID_ARG, "moe_adamw_step: tensor %d has n < 0", k);
    MOE_REQUIRE(is_dtype(t.param_dtype) && is_dtype(t.grad_dtype), MOE_ERR_INVALID_ARG,
                "moe_adamw_step: tensor %d has an unknown element type", k);
    MOE_REQUIRE(std::isfinite(t.weight_decay) && t.weight_decay >= 0, MOE_ERR_INVALID_ARG,
                "moe_adamw_step: tensor %d: weight_decay must be finite and >= 0", k);
    MOE_REQUIRE(!t.master || t.param_dtype == MOE_DTYPE_BF16, MOE_ERR_INVALID_ARG,
                "moe_adamw_step: tensor %d has a master beside an fp32 param", k);
    MOE_REQUIRE(t.n == 0 || (t.param && t.grad && t.exp_avg && t.exp_avg_sq &&
                             (!eight || (t.exp_avg_scale && t.exp_avg_sq_scale))),
                MOE_ERR_INVALID_ARG, "moe_adamw_step: tensor %d has a NULL pointer", k);
    const uintptr_t pb = t.param_dtype == MOE_DTYPE_F32 ? 4 : 2, gb = t.grad_dtype == MOE_DTYPE_F32 ? 4 : 2,
                    sb = eight ? 1 : 4;
    MOE_REQUIRE(aligned_to(t.param, pb) && aligned_to(t.grad, gb) && aligned_to(t.master, 4) &&
                    aligned_to(t.exp_avg, sb) && aligned_to(t.exp_avg_sq, sb) && aligned_to(t.exp_avg_scale, 4) &&
                    aligned_to(t.exp_avg_sq_scale, 4),
                MOE_ERR_INVALID_ARG, "moe_adamw_step: tensor %d has a pointer misaligned for its type", k);
    // 2^31 blocks a launch; n is checked first so that the sum cannot overflow
    MOE_REQUIRE(t.n <= (int64_t(1) << 39) &&
                    (blocks = (k % ADAMW_BATCH ? blocks : 0) + (t.n + ADAMW_STATE_BLOCK - 1) / ADAMW_STATE_BLOCK) <=
                        0x7fffffffLL,
                MOE_ERR_UNSUPPORTED_SHAPE, "moe_adamw_step: more than 2^31 - 1 blocks of 256 elements in a launch");
    AdamWTensor& o = list[k];
    o = {t.param, t.grad, t.master, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale, t.n};
    o.kind = (t.param_dtype == MOE_DTYPE_F32 ? 0 : t.master ? 2 : 1) + (t.grad_dtype == MOE_DTYPE_F32 ? 3 : 0);
    o.wide = aligned_to(t.param, 4 * pb) && aligned_to(t.grad, 4 * gb) && aligned_to(t.master, 16) &&
             aligned_to(t.exp_avg, 4 * sb) && aligned_to(t.exp_avg_sq, 4 * sb);
    o.decay = static_cast<float>(1.0 - h->lr * t.weight_decay);
    o.key = adamw_key(h->seed, static_cast<uint32_t>(k));
  }
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  AdamWStep a{};
  a.lr = h->lr;
  a.beta1 = h->beta1;
  a.beta2 = h->beta2;
  a.eps = h->eps;
  a.step = h->step;
  a.step_size = static_cast<float>(h->lr / (1.0 - std::pow(h->beta1, static_cast<double>(h->step))));
  a.root_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h->beta2, static_cast<double>(h->step))));
  a.grad_scale = h->grad_scale;
  a.skip = h->skip;
  a.step_dev = reinterpret_cast<const long long*>(h->step_dev);
  cudaError_t err = launch_adamw(list, count, a, eight, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_adamw_step launch");
}

}  // extern "C"

namespace {

// The experts' scratch: x's codes and scales and h's, or for few rows the fp32
// gate/up rows; each from a 256-byte boundary.
struct BlockWorkspace {
  size_t x_q, x_scale, h_q, h_scale, gu, total;
};

bool experts_stream(int32_t T, int32_t E, int32_t H, int32_t I) {
  return block_stream_fits(T, H > I ? H : I, E);
}

BlockWorkspace block_workspace(int64_t C, bool stream, int32_t H, int32_t I) {
  const size_t c = static_cast<size_t>(C);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  BlockWorkspace w{};
  if (stream) {
    w.gu = take(c * 2 * I * sizeof(float));
  } else {
    w.x_q = take(c * H);
    w.x_scale = take(c * ((H + 127) / 128) * sizeof(float));
    w.h_q = take(c * I);
    w.h_scale = take(c * ((I + 127) / 128) * sizeof(float));
  }
  w.total = at;
  return w;
}

moe_status check_fp4(const char* who, const void* values, int32_t dtype, int64_t batch, int64_t rows, int32_t cols,
                     const uint8_t* codes, const uint8_t* scales) {
  MOE_REQUIRE(batch >= 0 && rows >= 0, MOE_ERR_INVALID_ARG, "%s: batch and rows must be >= 0", who);
  MOE_REQUIRE(dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F32, MOE_ERR_INVALID_ARG, "%s: unknown type %d", who, dtype);
  MOE_REQUIRE(cols >= 32 && cols % 32 == 0 && cols < (1 << 24) - 256, MOE_ERR_UNSUPPORTED_SHAPE,
              "%s: cols must be a positive multiple of 32 below 2^24 - 256 (got %d)", who, cols);
  MOE_REQUIRE(rows < (int64_t(1) << 31) - 128 && (batch == 0 || rows < (int64_t(1) << 47) / cols / batch), MOE_ERR_UNSUPPORTED_SHAPE,
              "%s: too many rows", who);
  MOE_REQUIRE(batch == 0 || rows == 0 || (values && codes && scales), MOE_ERR_INVALID_ARG, "%s: NULL pointer", who);
  MOE_REQUIRE(all_aligned(16, values, codes, scales), MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_quantize_fp8_block(const moe_bf16* src, int64_t batch, int64_t rows, int32_t cols, int32_t block_rows,
                                  uint8_t* codes, float* scales, moe_stream_t stream) {
  MOE_REQUIRE(batch >= 0 && rows >= 0, MOE_ERR_INVALID_ARG, "moe_quantize_fp8_block: batch and rows must be >= 0");
  MOE_REQUIRE(cols > 0 && cols % 16 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "moe_quantize_fp8_block: cols must be a positive multiple of 16 (got %d)", cols);
  MOE_REQUIRE(block_rows == 1 || block_rows == 128, MOE_ERR_INVALID_ARG,
              "moe_quantize_fp8_block: block_rows must be 1 or 128 (got %d)", block_rows);
  MOE_REQUIRE(rows < (int64_t(1) << 31) && batch < (int64_t(1) << 31) &&
                  batch * ((rows + block_rows - 1) / block_rows) < (int64_t(1) << 31) / ((cols + 127) / 128),
              MOE_ERR_UNSUPPORTED_SHAPE, "moe_quantize_fp8_block: 2^31 blocks or more");
  MOE_REQUIRE(batch == 0 || rows == 0 || (src && codes && scales), MOE_ERR_INVALID_ARG,
              "moe_quantize_fp8_block: NULL pointer");
  MOE_REQUIRE(aligned16(src) && aligned16(codes) && aligned_to(scales, 4), MOE_ERR_INVALID_ARG,
              "moe_quantize_fp8_block: src and codes must be 16-byte aligned, scales by their type");
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  cudaError_t err = launch_quantize_block(src, batch, rows, cols, block_rows, codes, scales, nullptr, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_quantize_fp8_block launch");
}

moe_status moe_matmul_fp8_block(const uint8_t* a_q, const float* a_scale, int32_t M, const uint8_t* b_q,
                                const float* b_scale, int32_t N, int32_t K, moe_bf16* out, int32_t* status,
                                moe_stream_t stream) {
  MOE_REQUIRE(M >= 0 && N >= 1, MOE_ERR_INVALID_ARG, "moe_matmul_fp8_block: M must be >= 0 and N >= 1 (got %d, %d)", M,
              N);
  constexpr int32_t most_k = (int64_t(1) << 31) - 256;  // (rounded up to whole blocks it stays within 32 bits)
  MOE_REQUIRE(K >= 16 && K % 16 == 0 && K <= most_k, MOE_ERR_UNSUPPORTED_SHAPE,
              "moe_matmul_fp8_block: K must be a positive multiple of 16 up to 2^31 - 256 (got %d)", K);
  MOE_REQUIRE(M == 0 || (a_q && a_scale && b_q && b_scale && out), MOE_ERR_INVALID_ARG,
              "moe_matmul_fp8_block: NULL pointer");
  MOE_REQUIRE(aligned16(a_q) && aligned16(b_q) && all_aligned(4, a_scale, b_scale) && aligned_to(out, N % 8 == 0 ? 16 : 2),
              MOE_ERR_INVALID_ARG,
              "moe_matmul_fp8_block: codes and (N % 8 == 0) out must be 16-byte aligned, others by their type");
  MOE_REQUIRE((static_cast<int64_t>(M) + 127) / 128 * ((N + 63) / 64) < (int64_t(1) << 31), MOE_ERR_UNSUPPORTED_SHAPE,
              "moe_matmul_fp8_block: too many tiles");
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  cudaError_t err = M <= BLOCK_STREAM_ROWS
                        ? launch_block_matmul_stream(a_q, a_scale, M, b_q, b_scale, N, K, out, stream)
                        : launch_block_matmul_tc(a_q, a_scale, M, b_q, b_scale, N, K, out, status, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_matmul_fp8_block launch");
}

moe_status moe_quantize_fp4_block(const void* src, int32_t src_dtype, int64_t batch, int64_t rows, int32_t cols, uint8_t* codes,
                                  uint8_t* scales, moe_stream_t stream) {
  moe_status st = check_fp4("moe_quantize_fp4_block", src, src_dtype, batch, rows, cols, codes, scales);
  if (st != MOE_OK) return st;
  if ((st = check_device()) != MOE_OK) return st;
  const cudaError_t err = launch_quantize_fp4(src, src_dtype == MOE_DTYPE_F32, batch, rows, cols, codes, scales, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_quantize_fp4_block launch");
}

moe_status moe_dequantize_fp4_block(const uint8_t* codes, const uint8_t* scales, int64_t batch, int64_t rows, int32_t cols,
                                    int32_t out_dtype, void* out, moe_stream_t stream) {
  moe_status st = check_fp4("moe_dequantize_fp4_block", out, out_dtype, batch, rows, cols, codes, scales);
  if (st != MOE_OK) return st;
  if ((st = check_device()) != MOE_OK) return st;
  const cudaError_t err = launch_dequantize_fp4(codes, scales, batch, rows, cols, out_dtype == MOE_DTYPE_F32, out, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_dequantize_fp4_block launch");
}

moe_status moe_matmul_fp4_block(const uint8_t* a_q, const uint8_t* a_scale, int32_t M, const uint8_t* b_q, const uint8_t* b_scale,
                                int32_t N, int32_t K, moe_bf16* out, int32_t* status, moe_stream_t stream) {
  MOE_REQUIRE(M >= 0 && N >= 1, MOE_ERR_INVALID_ARG, "moe_matmul_fp4_block: M must be >= 0 and N >= 1 (got %d, %d)", M, N);
  // (a tile's 2^21 steps of K take less than the limit of a wait, and no count of them passes 32 bits)
  MOE_REQUIRE(K >= 32 && K % 32 == 0 && K <= 1 << 29, MOE_ERR_UNSUPPORTED_SHAPE,
              "moe_matmul_fp4_block: K must be a positive multiple of 32 up to 2^29 (got %d)", K);
  MOE_REQUIRE(M == 0 || (a_q && a_scale && b_q && b_scale && out), MOE_ERR_INVALID_ARG, "moe_matmul_fp4_block: NULL pointer");
  MOE_REQUIRE(all_aligned(16, a_q, a_scale, b_q, b_scale) && aligned_to(out, N % 8 == 0 ? 16 : 2) && aligned_to(status, 4),
              MOE_ERR_INVALID_ARG,
              "moe_matmul_fp4_block: codes, scales and (N a multiple of 8) out must be 16-byte aligned, others by their type");
  constexpr int32_t most = (int64_t(1) << 31) - 256;
  MOE_REQUIRE(M < most && N < most && (static_cast<int64_t>(M) + 127) / 128 * ((N + 63) / 64) < most, MOE_ERR_UNSUPPORTED_SHAPE,
              "moe_matmul_fp4_block: too many tiles");
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  // Few rows by few weight rows leave the tensor cores' tiles too few to keep all SMs
  // loading (8 x N x K, stream against tiles: 1024 x 8192 8.8 us and 11.3, 256 x 512
  // 2.7 and 2.8; 2048 x 768 3.7 and 3.4, 4096 x 2048 6.6 and 5.1, 16384 x 4096 23 and 12).
  const bool few = M <= FP4_STREAM_ROWS && N <= 1024;
  const cudaError_t err = few ? launch_fp4_matmul_stream(a_q, a_scale, M, b_q, b_scale, N, K, out, stream)
                              : launch_fp4_matmul_tc(a_q, a_scale, M, b_q, b_scale, N, K, out, status, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_matmul_fp4_block launch");
}

moe_status moe_experts_fp8_block_workspace_bytes(int64_t capacity, int32_t T, int32_t E, int32_t H, int32_t I,
                                                 size_t* bytes) {
  MOE_REQUIRE(bytes != nullptr, MOE_ERR_INVALID_ARG, "bytes is NULL");
  MOE_REQUIRE(capacity >= 0 && T >= 0 && E > 0 && H > 0 && I > 0, MOE_ERR_INVALID_ARG, "bad capacity / T / E / H / I");
  *bytes = block_workspace(capacity, experts_stream(T, E, H, I), H, I).total;
  return MOE_OK;
}

moe_status moe_grouped_experts_fp8_block(const moe_bf16* x_disp, const moe_layout* L, int32_t H, int32_t I,
                                         const uint8_t* W1_q, const float* W1_scale, const uint8_t* W2_q,
                                         const float* W2_scale, moe_bf16* y_disp, void* workspace,
                                         moe_stream_t stream) {
  moe_status st = check_layout(L);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(I > 0 && I % 128 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "the intermediate size must be a positive multiple of 128 (got %d)", I);
  MOE_REQUIRE(L->capacity == 0 || (x_disp && W1_q && W1_scale && W2_q && W2_scale && y_disp && workspace),
              MOE_ERR_INVALID_ARG, "moe_grouped_experts_fp8_block: NULL pointer");
  MOE_REQUIRE(all_aligned(16, x_disp, W1_q, W2_q, y_disp, workspace) && all_aligned(4, W1_scale, W2_scale),
              MOE_ERR_INVALID_ARG,
              "moe_grouped_experts_fp8_block: rows and codes must be 16-byte aligned, scales by their type");
  if ((st = check_device()) != MOE_OK) return st;
  if (L->capacity == 0 || L->T == 0) return MOE_OK;
  const bool stream_form = experts_stream(L->T, L->E, H, I);
  const BlockWorkspace w = block_workspace(L->capacity, stream_form, H, I);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  cudaError_t err;
  if (stream_form) {
    err = launch_block_experts_stream(x_disp, *L, H, I, W1_q, W1_scale, W2_q, W2_scale,
                                      reinterpret_cast<float*>(base + w.gu), y_disp, stream);
  } else {
    uint8_t* x_q = base + w.x_q;
    float* x_scale = reinterpret_cast<float*>(base + w.x_scale);
    err = launch_quantize_block(x_disp, 1, L->capacity, H, 1, x_q, x_scale, L->row_token, stream);
    if (err == cudaSuccess)
      err = launch_block_experts_tc(x_q, x_scale, *L, H, I, W1_q, W1_scale, W2_q, W2_scale, base + w.h_q,
                                    reinterpret_cast<float*>(base + w.h_scale), y_disp, stream);
  }
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_grouped_experts_fp8_block launch");
}

}  // extern "C"

namespace {

struct FewWorkspace {
  size_t logits, h, total;
};

FewWorkspace few_workspace(int32_t T, int32_t E, int32_t K, int32_t I) {
  auto up = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
  FewWorkspace w{};
  w.logits = 256;  // behind the barrier's word
  w.h = w.logits + up(static_cast<size_t>(T) * E * sizeof(float));
  w.total = w.h + up(static_cast<size_t>(T) * K * I / 8 * 17);  // 2 bytes a number and 1 for eight
  return w;
}

moe_status check_few(int32_t T, int32_t E, int32_t K, int32_t I) {
  MOE_REQUIRE(T >= 0, MOE_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
  MOE_REQUIRE(T <= MOE_FEW_TOKENS, MOE_ERR_UNSUPPORTED_SHAPE, "moe_layer_few takes at most %d tokens (got %d)", MOE_FEW_TOKENS, T);
  MOE_REQUIRE(E >= 1 && E <= 1024, MOE_ERR_UNSUPPORTED_SHAPE, "E must be in [1, 1024] (got %d)", E);
  MOE_REQUIRE(K >= 1 && K <= E && K <= MOE_FEW_TOP_K, MOE_ERR_UNSUPPORTED_SHAPE,
              "K must be in [1, min(E, %d)] (got K=%d, E=%d)", MOE_FEW_TOP_K, K, E);
  MOE_REQUIRE(I > 0 && I % 128 == 0, MOE_ERR_UNSUPPORTED_SHAPE,
              "the intermediate size must be a positive multiple of 128 (got %d)", I);
  return MOE_OK;
}

moe_status check_few_all(int32_t T, int32_t E, int32_t K, int32_t H, int32_t I, int32_t weights) {
  moe_status st = check_few(T, E, K, I);
  if (st != MOE_OK) return st;
  if ((st = check_hidden(H)) != MOE_OK) return st;
  MOE_REQUIRE(H <= 1 << 20 && I <= 1 << 20, MOE_ERR_UNSUPPORTED_SHAPE, "moe_layer_few: H and I must be at most 2^20 (got %d, %d)", H, I);
  static_assert(FEW_TOKENS == MOE_FEW_TOKENS && FEW_TOP_K == MOE_FEW_TOP_K && int(FEW_FP8) == int(MOE_WEIGHTS_FP8_BLOCK) &&
                int(FEW_FP4) == int(MOE_WEIGHTS_FP4_BLOCK), "one set of constants");
  MOE_REQUIRE(weights >= MOE_WEIGHTS_BF16 && weights <= MOE_WEIGHTS_FP4_BLOCK, MOE_ERR_INVALID_ARG,
              "moe_layer_few: unknown weight format %d", weights);
  MOE_REQUIRE(few_layer_fits(weights, T, K, H, I), MOE_ERR_UNSUPPORTED_SHAPE,
              "moe_layer_few: the rows of %d tokens of H=%d and I=%d do not fit in shared memory", T, H, I);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_layer_few_workspace_bytes(int32_t T, int32_t E, int32_t K, int32_t I, size_t* bytes) {
  MOE_REQUIRE(bytes != nullptr, MOE_ERR_INVALID_ARG, "bytes is NULL");
  const moe_status st = check_few(T, E, K, I);
  if (st != MOE_OK) return st;
  *bytes = few_workspace(T, E, K, I).total;
  return MOE_OK;
}

int32_t moe_layer_few_fits(int32_t T, int32_t E, int32_t K, int32_t H, int32_t I, int32_t weights) {
  return check_few_all(T, E, K, H, I, weights) == MOE_OK;
}

moe_status moe_layer_few(const moe_few* f, moe_stream_t stream) {
  MOE_REQUIRE(f != nullptr, MOE_ERR_INVALID_ARG, "moe_layer_few: NULL pointer");
  moe_status st = check_few_all(f->T, f->E, f->K, f->H, f->I, f->weights);
  if (st != MOE_OK) return st;
  MOE_REQUIRE(f->router_dtype == MOE_DTYPE_BF16 || f->router_dtype == MOE_DTYPE_F32, MOE_ERR_INVALID_ARG,
              "moe_layer_few: unknown type %d", f->router_dtype);
  const bool coded = f->weights != MOE_WEIGHTS_BF16;
  MOE_REQUIRE(f->T == 0 || (f->x && f->W1 && f->W2 && f->out && f->workspace && (!coded || (f->W1_scale && f->W2_scale))),
              MOE_ERR_INVALID_ARG, "moe_layer_few: NULL pointer");
  MOE_REQUIRE(f->T == 0 || (f->router ? !f->topk_idx && !f->topk_probs : f->topk_idx && f->topk_probs), MOE_ERR_INVALID_ARG,
              "moe_layer_few: give the router, or topk_idx and topk_probs");
  MOE_REQUIRE((f->idx_out == nullptr) == (f->probs_out == nullptr), MOE_ERR_INVALID_ARG,
              "moe_layer_few: give idx_out and probs_out, or neither");
  MOE_REQUIRE(all_aligned(16, f->x, f->router, f->W1, f->W2, f->workspace) && all_aligned(8, f->topk_idx, f->idx_out) &&
                  all_aligned(4, f->topk_probs, f->probs_out, f->W1_scale, f->W2_scale, f->status) && aligned_to(f->out, 2),
              MOE_ERR_INVALID_ARG, "moe_layer_few: x, router, weights and workspace must be 16-byte aligned, others by their type");
  if ((st = check_device()) != MOE_OK) return st;
  if (f->T == 0) return MOE_OK;
  const FewWorkspace w = few_workspace(f->T, f->E, f->K, f->I);
  uint8_t* base = static_cast<uint8_t*>(f->workspace);
  FewLayer g{};
  g.x = f->x;
  g.router = f->router;
  g.router_f32 = f->router_dtype == MOE_DTYPE_F32;
  g.topk_idx = f->topk_idx;
  g.topk_probs = f->topk_probs;
  g.format = f->weights;
  g.W1 = f->W1;
  g.S1 = f->W1_scale;
  g.W2 = f->W2;
  g.S2 = f->W2_scale;
  g.T = f->T, g.E = f->E, g.K = f->K, g.H = f->H, g.I = f->I;
  g.barrier = reinterpret_cast<unsigned*>(base);
  g.logits = reinterpret_cast<float*>(base + w.logits);
  g.h = reinterpret_cast<uint16_t*>(base + w.h);
  g.out = f->out;
  g.idx_out = f->idx_out;
  g.probs_out = f->probs_out;
  g.status = f->status;
  const cudaError_t err = launch_few_layer(g, stream);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err, "moe_layer_few launch");
}

}  // extern "C"
