// A kernel that lets the next one in its stream start at once (programmatic
// dependent launch) and then takes its time before it reads and writes: what
// a caller's kernel in front of a library call may do.
#include <cuda_runtime.h>
#include <stdint.h>

__global__ void late_copy_kernel(int32_t* dst, const int32_t* src, long long n, unsigned long long wait_ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  for (int i = 0; i < (1 << 20); ++i) {  // ends by itself, whatever the timer says
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (t - t0 >= wait_ns) break;
    __nanosleep(500);
  }
  for (long long i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}

extern "C" int late_copy(void* dst, const void* src, long long ints, unsigned long long wait_ns, void* stream) {
  late_copy_kernel<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<int32_t*>(dst),
                                                                     static_cast<const int32_t*>(src), ints, wait_ns);
  return (int)cudaGetLastError();
}
