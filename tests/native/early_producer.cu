// A kernel that lets the next one on its stream start at once and writes its output only later: dst = src after about
// `delay_ns` (a bounded spin on the clock).  What reads dst behind it has to wait for the kernel's end itself.
#include <cuda_runtime.h>
#include <stdint.h>

__global__ void late_copy(uint8_t* dst, const uint8_t* src, int64_t n, unsigned long long delay_ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < 1 << 20; ++i) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > delay_ns) break;
    }
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        dst[i] = src[i];
}

extern "C" int late_copy_launch(void* dst, const void* src, int64_t n, uint64_t delay_ns, void* stream) {
    late_copy<<<8, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint8_t*>(dst), static_cast<const uint8_t*>(src), n,
                                                                delay_ns);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}
