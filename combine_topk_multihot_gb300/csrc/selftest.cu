// Self-tests of the bounded device waits that every pipelined kernel here uses.
//
// One CTA initialises an mbarrier that nothing will ever arrive on and waits
// for it with the same helper the grouped GEMMs use, under a caller-chosen
// limit.  The wait must give up, raise the CTA's abort flag and report
// MOE_DEVERR_TIMEOUT through the status word; the kernel then returns
// normally, so the context stays usable.  Nothing traps or spins forever.

#include "common.cuh"
#include "launch.h"

namespace moe {

namespace {

__global__ void wait_timeout_kernel(int* status, unsigned long long limit_ns,
                                    unsigned long long* waited_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned long long t0 = global_timer_ns();
    const bool ok = mbar_wait(smem_u32(&bar), 0, &abort_flag, limit_ns);
    if (waited_ns) *waited_ns = global_timer_ns() - t0;
    if (!ok) report(status, MOE_DEVERR_TIMEOUT);
  }
}

thread_local unsigned long long tls_pair_wait_ns = WAIT_LIMIT_NS;

}  // namespace

unsigned long long pair_wait_ns() { return tls_pair_wait_ns; }

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_selftest_wait_timeout(int32_t* status, int64_t limit_ns,
                                                uint64_t* waited_ns, moe_stream_t stream) {
  if (!status || limit_ns <= 0 || limit_ns > 1000000000LL)
    return set_last_error(MOE_ERR_INVALID_ARG,
                          "moe_selftest_wait_timeout: needs a status word and 0 < limit_ns <= 1e9");
  const moe_status st = moe_device_check();
  if (st != MOE_OK) return st;
  wait_timeout_kernel<<<1, 32, 0, stream>>>(status, static_cast<unsigned long long>(limit_ns),
                                            reinterpret_cast<unsigned long long*>(waited_ns));
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return set_last_error(MOE_ERR_CUDA, cudaGetErrorString(err));
  return MOE_OK;
}

extern "C" moe_status moe_selftest_pair_wait(int64_t limit_ns) {
  if (limit_ns < -1 || limit_ns == 0 || limit_ns > static_cast<int64_t>(WAIT_LIMIT_NS))
    return set_last_error(MOE_ERR_INVALID_ARG, "moe_selftest_pair_wait: needs 0 < limit_ns <= 2e9, or -1 for the usual limit");
  tls_pair_wait_ns = limit_ns < 0 ? WAIT_LIMIT_NS : static_cast<unsigned long long>(limit_ns);
  return MOE_OK;
}

extern "C" moe_status moe_selftest_few_ctas(int32_t ctas) {
  if (ctas < -1) return set_last_error(MOE_ERR_INVALID_ARG, "moe_selftest_few_ctas: ctas must be >= 0, or -1 for all");
  selftest_few_ctas(ctas < 0 ? 0x7fffffff : ctas);
  return MOE_OK;
}

extern "C" moe_status moe_selftest_few_plan(int32_t T, int32_t K, int32_t H, int32_t I, int32_t weights, int32_t* rows,
                                            int32_t* slots) {
  if (!rows || !slots || !moe_layer_few_fits(T, MOE_FEW_TOP_K, K, H, I, weights))
    return set_last_error(MOE_ERR_INVALID_ARG, "moe_selftest_few_plan: needs rows, slots and a layer that fits");
  few_layer_fits(weights, T, K, H, I, rows, slots);
  return MOE_OK;
}

extern "C" moe_status moe_selftest_block_product_tiles(int32_t tiles) {
  if (tiles < -1)
    return set_last_error(MOE_ERR_INVALID_ARG, "moe_selftest_block_product_tiles: tiles must be >= 0, or -1 for all");
  selftest_block_load_tiles(tiles < 0 ? 0x7fffffff : tiles);
  return MOE_OK;
}

extern "C" moe_status moe_selftest_norm_rows(int64_t rows) {
  if (rows < -1) return set_last_error(MOE_ERR_INVALID_ARG, "moe_selftest_norm_rows: rows must be >= 0, or -1 for all");
  selftest_norm_load_rows(rows);
  return MOE_OK;
}
