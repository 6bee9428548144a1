// late_copy.cu -- test helper: a kernel that lets the kernels after it on the stream
// start at once and writes its data late.  What follows it has to wait for its
// completion (griddepcontrol.wait) before it reads anything.
#include <cuda_runtime.h>
#include <stdint.h>

static __global__ void late_copy_kernel(uint32_t *dst, const uint32_t *src, int64_t words, unsigned delay_ns)
{
    asm volatile("griddepcontrol.launch_dependents;");
    uint64_t begin, now;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(begin));
    for (int i = 0; i < 4096; ++i) {   // ends in any case: 4096 sleeps of at most a few hundred ns
        __nanosleep(100);
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
        if (now - begin >= delay_ns) break;
    }
    for (int64_t i = threadIdx.x; i < words; i += blockDim.x) dst[i] = src[i];
}

extern "C" int late_copy(void *dst, const void *src, int64_t bytes, unsigned delay_ns, void *stream)
{
    if (bytes < 0 || bytes % 4) return -1;
    late_copy_kernel<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint32_t *>(dst),
                                                                     static_cast<const uint32_t *>(src), bytes / 4, delay_ns);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}
