// Small kernels around device functions of the paged cache's attention, for
// tests/test_gpu_paged_device.py: each runs one function and returns what it did.
#include <cuda_runtime.h>

#include "../../bit_decode_selective_b200/csrc/kvp_wait.cuh"

using namespace sf;

namespace {

// A barrier that one arrival completes.  mode 0: it arrives; the warps drain.
// 1: nothing arrives; the warps drain.  2: nothing arrives; they wait.  3: nothing
// arrives, a wait has given up before: they wait and then drain.
__global__ void wait_kernel(int mode, unsigned int* counts, int* gave_up, unsigned long long* ns) {
  __shared__ uint64_t bar;
  __shared__ volatile int given_up;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    given_up = mode == 3;
  }
  __syncthreads();
  if (mode == 0 && threadIdx.x == 0) mbar_arrive(&bar);
  const unsigned long long t0 = now_ns();
  if (mode >= 2) mbar_wait(&bar, 0, &given_up, &counts[0]);
  const unsigned long long t1 = now_ns();
  __syncwarp();
  if (mode != 2) mbar_drain(&bar, 0, &counts[1]);
  const unsigned long long t2 = now_ns();
  __syncthreads();
  if (threadIdx.x == 0) *gave_up = given_up, ns[0] = t1 - t0, ns[1] = t2 - t1;
}

}  // namespace

#define CHECK extern "C" __attribute__((visibility("default"))) int

CHECK kvp_check_wait(int mode, unsigned int* counts, int* gave_up, unsigned long long* ns) {
  wait_kernel<<<1, 64>>>(mode, counts, gave_up, ns);
  return (int)cudaDeviceSynchronize();
}
