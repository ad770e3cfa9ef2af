// Small kernels around device functions of the paged cache's attention, for
// tests/test_gpu_paged_device.py: each runs one function and returns what it did.
#include <cuda_runtime.h>

#include "../../bit_decode_selective_b200/csrc/kvp_attend.cuh"
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

// What a CTA finds out about its range of the work: 12 numbers per CTA.
template <int ROWS, int STEP, int EXTRA, bool FEW, int THREADS>
__global__ void __launch_bounds__(THREADS) range_kernel(KvpAttendArgs a, int min_steps, long* out) {
  using Item = KvpItem<ROWS, STEP, EXTRA, FEW>;
  __shared__ KvpRangeShared<Item> sh;
  Item it;
  const KvpRange r = kvp_range<THREADS, !FEW>(a, min_steps, sh, it);
  long* o = out + 12 * blockIdx.x;
  const bool some = r.u0 < r.u1;
  if (threadIdx.x == THREADS - 1) {
    o[0] = r.u0, o[1] = r.u1;
    if (some) {
      o[2] = r.at, o[3] = it.b, o[4] = it.rt, o[5] = it.g, o[6] = it.steps, o[7] = it.seq.q0, o[8] = it.seq.n, o[9] = it.seq.len;
      o[10] = r.cta_of(r.u0), o[11] = r.cta_of(r.u1 - 1);
    }
  }
}

}  // namespace

#define CHECK extern "C" __attribute__((visibility("default"))) int

CHECK kvp_check_wait(int mode, unsigned int* counts, int* gave_up, unsigned long long* ns) {
  wait_kernel<<<1, 64>>>(mode, counts, gave_up, ns);
  return (int)cudaDeviceSynchronize();
}

// few: the few-row kernel's items, else the many-row kernel's; out [ctas][12], zeroed.
CHECK kvp_check_range(int few, int ctas, int batch, int h_kv, int group, int n_q, const int* cu_q, const int* lens,
                      int max_pages, int page_shift, int window, int sinks, int min_steps, long* out) {
  KvpAttendArgs a = {};
  a.h_kv = h_kv, a.group = group, a.h_q = h_kv * group, a.n_q = n_q, a.cu_q = cu_q, a.lens = lens, a.batch = batch;
  a.max_pages = max_pages, a.page_shift = page_shift, a.window = window, a.sinks = sinks, a.few_rows = 64;
  kvp_divisor((uint32_t)group, a.group_mul, a.group_shift);
  if (few)
    range_kernel<8, 2, 8, true, 128><<<ctas, 128>>>(a, min_steps, out);
  else
    range_kernel<256, 8, 4, false, 640><<<ctas, 640>>>(a, min_steps, out);
  return (int)cudaDeviceSynchronize();
}
