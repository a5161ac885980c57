// Self-test of the bounded-wait path every kernel relies on: a one-CTA kernel
// waits on an mbarrier that nothing ever arrives at, with a short limit, and
// must come back with the timeout recorded in its status word instead of
// hanging.  Used by the failure-detection test; it faults nothing and leaves
// the context usable.
#include <cuda_runtime.h>

#include "fa2.h"
#include "ptx.cuh"

namespace fa2 {
namespace {

__device__ int g_selftest_status;

__global__ void wait_timeout_kernel(unsigned long long timeout_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);  // expects one arrival that never comes
    fence_mbar_init();
  }
  __syncthreads();
  mbar_wait(&bar, 0, &g_selftest_status, timeout_ns);
}

// Warp 0 waits for a phase that a lane of warp 1 completes after `late_ns`:
// first with limits that are over by then in the even lanes only, then for a
// second phase with long limits everywhere.  out: the lanes that were told
// "in time", of both waits.
__global__ void warp_wait_kernel(unsigned long long late_ns, unsigned* out) {
  __shared__ __align__(8) uint64_t bar[2];
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x >= 32) {
    if (lane == 0) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < late_ns) {
      }
      mbar_arrive(&bar[0]);
      mbar_arrive(&bar[1]);
    }
    return;
  }
  // (the even lanes' time-outs are meant: the status word is not looked at)
  const uint64_t limit = lane & 1 ? late_ns + FA2_WAIT_TIMEOUT_NS : late_ns / 8;
  const bool first = mbar_wait_warp(&bar[0], 0, &g_selftest_status, limit);
  const unsigned a = __ballot_sync(0xffffffffu, first);
  const bool second = mbar_wait_warp(&bar[1], 0, &g_selftest_status, late_ns + FA2_WAIT_TIMEOUT_NS);
  const unsigned b = __ballot_sync(0xffffffffu, second);
  if (lane == 0) out[0] = a, out[1] = b;
}

__device__ unsigned g_warp_wait_lanes[2];

}  // namespace
}  // namespace fa2

extern "C" int fa2_check_wait_timeout(int timeout_us, int* status_out) {
  if (!status_out) return FA2_ERR_NULL;
  if (timeout_us < 1 || timeout_us > 5000000) return FA2_ERR_SHAPE;
  const int zero = 0;
  if (cudaMemcpyToSymbol(fa2::g_selftest_status, &zero, sizeof(int)) != cudaSuccess) return FA2_ERR_CUDA;
  fa2::wait_timeout_kernel<<<1, 32>>>(static_cast<unsigned long long>(timeout_us) * 1000ull);
  if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return FA2_ERR_CUDA;
  if (cudaMemcpyFromSymbol(status_out, fa2::g_selftest_status, sizeof(int)) != cudaSuccess) return FA2_ERR_CUDA;
  return FA2_OK;
}

extern "C" int fa2_check_warp_wait(int late_us, unsigned* lanes_out) {
  if (!lanes_out) return FA2_ERR_NULL;
  if (late_us < 100 || late_us > 1000000) return FA2_ERR_SHAPE;
  void* lanes = nullptr;
  if (cudaGetSymbolAddress(&lanes, fa2::g_warp_wait_lanes) != cudaSuccess) return FA2_ERR_CUDA;
  fa2::warp_wait_kernel<<<1, 64>>>(static_cast<unsigned long long>(late_us) * 1000ull, static_cast<unsigned*>(lanes));
  if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return FA2_ERR_CUDA;
  if (cudaMemcpyFromSymbol(lanes_out, fa2::g_warp_wait_lanes, 2 * sizeof(unsigned)) != cudaSuccess) return FA2_ERR_CUDA;
  return FA2_OK;
}
