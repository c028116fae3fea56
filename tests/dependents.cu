// A kernel that lets its programmatic dependents start at once and writes only some time
// later: what calls that overlap the kernel before them have to wait for.
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace {
__device__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__global__ void late_copy_kernel(const uint8_t* from, uint8_t* to, size_t n, uint64_t ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint64_t t0 = now_ns();
  while (now_ns() - t0 < ns) __nanosleep(2000);
  for (size_t i = threadIdx.x; i < n; i += blockDim.x) to[i] = from[i];
}
}  // namespace

extern "C" int late_copy(const void* from, void* to, size_t n, uint64_t ns, void* stream) {
  late_copy_kernel<<<1, 1024, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(from), static_cast<uint8_t*>(to), n, ns);
  return int(cudaGetLastError());
}
