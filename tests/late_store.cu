// Test helper: a launch that lets the next one on its stream start at once, and
// stores the list that the next one reads only some time later (bounded, and
// without waiting for anything). What a kernel reads before its dependency wait
// is then the list as it was.
#include <cuda_runtime.h>
#include <stdint.h>

namespace {

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__global__ void late_store_kernel(int32_t* dst, const int32_t* src, int n, uint64_t delay_ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint64_t t0 = now_ns();
  for (int i = 0; i < 100000 && now_ns() - t0 < delay_ns; ++i) __nanosleep(100);
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}

}  // namespace

extern "C" int late_store(int32_t* dst, const int32_t* src, int n, uint64_t delay_ns, void* stream) {
  late_store_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(dst, src, n, delay_ns);
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}
