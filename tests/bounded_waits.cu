// Eight warps that take items together, as the prefill's softmax warps do (test_kernel_barriers.py):
// each waits for an item, they agree whether all of them have it, and meet once more in it.
#include "ptx.cuh"
#include "rcp.h"

namespace {
constexpr int kItems = 8, kThreads = 256;

__global__ void __launch_bounds__(kThreads) items_kernel(int items, int missing, unsigned late,
                                                         int* taken, uint32_t* err) {
  __shared__ uint64_t full[kItems], never;
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kItems; ++i) rcp::mbar_init(&full[i], 1);
    rcp::mbar_init(&never, 1);
    *abort_flag = 0;
    rcp::fence_mbar_init();
    for (int i = 0; i < kItems; ++i) rcp::mbar_arrive(&full[i]);
  }
  __syncthreads();
  int n = 0;
  for (int it = 0; it < items && it < kItems; ++it) {
    const bool lost = it == missing && (late >> warp & 1u);
    bool ok = rcp::mbar_wait(lost ? &never : &full[it], 0, abort_flag, err);
    ok = rcp::named_bar_and(1, kThreads, ok);
    if (!ok) break;
    rcp::named_bar_sync(2, kThreads);
    ++n;
  }
  taken[threadIdx.x] = n;
}
}  // namespace

extern "C" int run(int items, int missing, unsigned late, int* taken, uint32_t* err) {
  items_kernel<<<1, kThreads>>>(items, missing, late, taken, err);
  const cudaError_t e = cudaGetLastError();
  return static_cast<int>(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
