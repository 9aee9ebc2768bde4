// The sparse attention forward's launches (the kernel: prefill_kernel.cuh).
#include "prefill_kernel.cuh"

namespace msa {

int device_sm_count() {
  static int cache[128] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 1;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 1;
    cache[dev] = n;
  }
  return cache[dev];
}

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t s) { return launch_attention<false>(a, s); }

}  // namespace msa
