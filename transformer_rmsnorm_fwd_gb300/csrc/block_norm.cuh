// What the forward and the backward of the block norms share (formulas in
// liger_train.h).
#pragma once

#include <atomic>

#include "common.cuh"
#include "liger_train.h"
#include "mbarrier.cuh"

namespace liger {
namespace {

// sum of one value per thread over the block, returned to every thread
__device__ __forceinline__ float block_sum(float v, float* sh) {
    v = warp_sum(v);
    __syncthreads();   // the previous sum has been read
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) t += sh[i];
    return t;
}

// 1 / sqrt(x) for x > 0: the hardware approximation and one Newton step (within an ulp or so; the
// correctly rounded square root and division are a long serial chain between two barriers)
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = rsqrtf(x);
    const float e = fmaf(-x * r, r, 1.f);
    const float n = fmaf(0.5f * r, e, r);
    return isfinite(n) ? n : r;   // x = 0, infinity or NaN: what rsqrt says
}

// r^3 s for a row's scale r and a sum s over the row: s is of the size of 1 / r, so it is taken up factor by factor
// (r^3 alone leaves the range of fp32 for rows below 1e-12 or above 1e12 in size)
__device__ __forceinline__ float cube_times(float r, float s) { return r * (r * (r * s)); }

// ------------------------------------------- rows that are no whole 16-byte vectors
// Rings for rows whose width is no multiple of a vector: rows then start anywhere, so a slot
// takes the 16-byte aligned window around a row (the bytes of its neighbours in it are not looked at),
// and threads take single elements from it, EPT fixed columns each.  Memory still moves in
// bulk copies; the elements cost one shared-memory access each, which is what bounds these kernels.
// The last row's window may end past the tensor: the copy stops at the last whole 16 bytes, and the
// elements behind that come by plain loads.
struct Window {
    int64_t at;       // first byte of the window
    uint32_t bytes;   // multiple of 16
    int shift;        // elements from there to the row's first
    int tail;         // the row's elements from this one on are not in the window
};
template <typename T>
__device__ __forceinline__ Window window_of(int64_t t, int64_t rows, int cols) {
    constexpr int SZ = sizeof(T);
    Window w;
    const int64_t o = t * cols * SZ, end = o + static_cast<int64_t>(cols) * SZ;
    w.at = o & ~int64_t{15};
    w.shift = static_cast<int>((o - w.at) / SZ);
    int64_t stop = (end + 15) & ~int64_t{15};
    w.tail = cols;
    if (t == rows - 1 && stop != end) {
        stop = end & ~int64_t{15};
        w.tail = static_cast<int>((stop - o) / SZ);
    }
    w.bytes = static_cast<uint32_t>(stop - w.at);
    return w;
}
// bytes a slot needs for one stream
inline size_t window_max(int cols, size_t sz) { return (static_cast<size_t>(cols) * sz + 15 + 15) & ~static_cast<size_t>(15); }

// Lets a kernel have as much dynamic shared memory as the device gives, once per device (racing
// threads set the same value).
template <auto KERN>
int allow_smem() {
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return check_launch("block_norm device");
    if (done[dev].load(std::memory_order_acquire)) return LIGER_OK;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, KERN) != cudaSuccess ||
        cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_smem_optin() - static_cast<int>(fa.sharedSizeBytes)) != cudaSuccess)
        return check_launch("block_norm attribute");
    done[dev].store(true, std::memory_order_release);
    return LIGER_OK;
}

// Resident blocks per SM of a kernel, asked once per device.
template <typename K>
int resident(K kern, int threads, size_t smem, std::atomic<int> (&cache)[64]) {
    int dev = 0;
    const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
    int n = known ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess || n < 1) n = 1;
        if (known) cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

inline int check_common(const char* who, int64_t rows, int64_t cols, int64_t gates, const void* gate, int dtype) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (rows < 0 || cols <= 0 || cols > (1 << 24) || gates < 0 || rows > (int64_t{1} << 48) / cols)
        return fail(LIGER_ERR_SHAPE, "%s: rows=%lld cols=%lld gates=%lld", who, (long long)rows, (long long)cols,
                    (long long)gates);
    if (gates > 0 && rows % gates)
        return fail(LIGER_ERR_SHAPE, "%s: rows=%lld is no multiple of gates=%lld", who, (long long)rows, (long long)gates);
    if ((gates > 0) != (gate != nullptr))
        return fail(LIGER_ERR_NULL, "%s: gate and gates > 0 go together (gates=%lld)", who, (long long)gates);
    return LIGER_OK;
}

inline bool misaligned(std::initializer_list<const void*> ps, unsigned to) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return true;   // NULL is aligned
    return false;
}

}  // namespace
}  // namespace liger
