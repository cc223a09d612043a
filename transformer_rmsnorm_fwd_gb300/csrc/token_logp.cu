// Log-probabilities of given tokens from logits, with the entropy, the top
// alternatives and the gradient of the logits (formulas in liger_layer.h).
#include <math.h>

#include "common.cuh"
#include "liger_layer.h"

namespace liger {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kLowest = -3.402823466e38f;
constexpr int kThreads = 256;

struct LogpFwd {
    const void* z;
    int64_t ld;
    const int64_t* tokens;
    int64_t T, V, ignore;
    float inv_temp;
    float *logp, *row_max, *log_sum, *entropy, *top_logp;
    int64_t* top_ids;
    int k;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A number whose unsigned order is that of the floats: -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t order_of(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// ... and with the index behind it, the lowest first
__device__ __forceinline__ unsigned long long rank_key(float v, uint32_t index) {
    return static_cast<unsigned long long>(order_of(v)) << 32 | (0xFFFFFFFFu - index);
}

// Sums over the block, in every thread; sh holds a float per warp.
__device__ __forceinline__ float block_max_nan(float v, float* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = sh[0];
    for (int i = 1; i < static_cast<int>(blockDim.x >> 5); ++i) t = max_nan(t, sh[i]);
    return t;
}
__device__ __forceinline__ float block_add(float v, float* sh) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) t += sh[i];
    return t;
}

// With d = (z - m) / (temperature ln 2), m the largest logit, s = sum 2^d and u = sum d 2^d:
//     log_sum = ln 2 log2 s,  logp = (z_y - m) / temperature - log_sum,  entropy = ln 2 (log2 s - u / s)
// z - m is formed first: logits of the type's lowest value, or all far from 0, lose nothing.
// A logit of -inf has d below any limit: held at -200, where 2^d is 0, so that d 2^d is not NaN.
template <typename T>
__global__ void __launch_bounds__(kThreads) token_logp_rows(LogpFwd p) {
    __shared__ float sh[8];
    __shared__ unsigned long long shk[8];
    wait_for_stream();
    const int64_t t = blockIdx.x;
    const T* z = static_cast<const T*>(p.z) + t * p.ld;
    const float c = p.inv_temp * kLog2e;
    float m = -INFINITY;
    for (int64_t v = threadIdx.x; v < p.V; v += kThreads) m = max_nan(m, ldf(z + v));
    m = block_max_nan(m, sh);
    const bool none = m == -INFINITY;
    const float mf = m != m ? m : fmaxf(m, kLowest);
    float s = 0.f, u = 0.f;
    for (int64_t v = threadIdx.x; v < p.V; v += kThreads) {
        const float d = max_nan((ldf(z + v) - mf) * c, -200.f);
        const float e = ex2(d);
        s += e;
        u = fmaf(d, e, u);
    }
    s = block_add(s, sh);
    u = block_add(u, sh);
    const float ls = log2f(s);
    if (threadIdx.x == 0) {
        if (p.row_max != nullptr) p.row_max[t] = m;
        if (p.log_sum != nullptr) p.log_sum[t] = none ? -INFINITY : ls * kLn2;
        if (p.entropy != nullptr) p.entropy[t] = none ? 0.f : (ls - u / s) * kLn2;
        if (p.logp != nullptr) {
            const int64_t y = p.tokens[t];
            float r = 0.f;
            if (y != p.ignore) {
                if (y < 0 || y >= p.V) r = NAN;
                else r = none ? -INFINITY : fmaf(ldf(z + y) - mf, p.inv_temp, -ls * kLn2);
            }
            p.logp[t] = r;
        }
    }
    unsigned long long last = ~0ull;
    for (int i = 0; i < p.k; ++i) {
        unsigned long long best = 0;
        for (int64_t v = threadIdx.x; v < p.V; v += kThreads) {
            const unsigned long long key = rank_key(ldf(z + v), static_cast<uint32_t>(v));
            if (key < last && key > best) best = key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) shk[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int w = 0; w < 8; ++w) best = max(best, shk[w]);
        last = best;
        if (threadIdx.x == 0) {
            const uint32_t v = 0xFFFFFFFFu - static_cast<uint32_t>(best);
            p.top_ids[t * p.k + i] = v;
            p.top_logp[t * p.k + i] = none ? -INFINITY : fmaf(ldf(z + v) - mf, p.inv_temp, -ls * kLn2);
        }
    }
}

struct LogpBwd {
    const void* z;
    int64_t ld;
    const int64_t* tokens;
    const float *row_max, *log_sum, *entropy, *g_logp, *g_entropy;
    int64_t T, V, ignore;
    float inv_temp;
    void* dz;
    int64_t ldd;
};

// dz = (g 1[v = y] - p (g + h (a + H))) / temperature with a = log p, p = e^a
template <typename T>
__global__ void __launch_bounds__(kThreads) token_logp_bwd_rows(LogpBwd p) {
    wait_for_stream();
    const int64_t t = blockIdx.x;
    const T* z = static_cast<const T*>(p.z) + t * p.ld;
    T* dz = static_cast<T*>(p.dz) + t * p.ldd;
    const int64_t y = p.tokens != nullptr ? p.tokens[t] : p.ignore;
    const bool counts = p.g_logp != nullptr && y != p.ignore;
    float g = counts ? p.g_logp[t] : 0.f;
    if (counts && (y < 0 || y >= p.V)) g = NAN;
    const float h = p.g_entropy != nullptr ? p.g_entropy[t] : 0.f, H = p.g_entropy != nullptr ? p.entropy[t] : 0.f;
    const float m = p.row_max[t], ls = p.log_sum[t];
    const bool zero = (g == 0.f && h == 0.f) || (m == -INFINITY && g == g && h == h);
    for (int64_t v = threadIdx.x; v < p.V; v += kThreads) {
        float d = 0.f;
        if (!zero) {
            const float a = max_nan(fmaf(ldf(z + v) - m, p.inv_temp, -ls), -1e4f);
            const float pr = ex2(a * kLog2e);
            d = (v == y ? g : 0.f) - pr * fmaf(h, a + H, g);
        }
        stf(dz + v, d * p.inv_temp);
    }
}

int check_logits(const char* who, int64_t T, int64_t V, int64_t ld, float temperature, int dtype) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (T < 0 || T > 2147483647LL || V <= 0 || V > (1 << 30) || ld < V || ld > (int64_t{1} << 40))
        return fail(LIGER_ERR_SHAPE, "%s: T=%lld V=%lld ld=%lld", who, (long long)T, (long long)V, (long long)ld);
    if (!(temperature > 0.f) || !isfinite(temperature) || !isfinite(1.0f / temperature))
        return fail(LIGER_ERR_SHAPE, "%s: temperature must be > 0", who);
    return LIGER_OK;
}
bool off(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" int liger_token_logp_fwd(const void* logits, int64_t ld, const int64_t* tokens, int64_t T, int64_t V,
                                    int64_t ignore_index, float temperature, float* logp, float* row_max, float* log_sum,
                                    float* entropy, int64_t k, float* top_logp, int64_t* top_ids, int dtype, void* stream) {
    clear_error();
    const char* who = "token_logp_fwd";
    if (int rc = check_logits(who, T, V, ld, temperature, dtype)) return rc;
    if (k < 0 || k > LIGER_TOP_MAX || k > V)
        return fail(LIGER_ERR_SHAPE, "%s: k=%lld (0 to %d, at most V=%lld)", who, (long long)k, LIGER_TOP_MAX, (long long)V);
    if (T == 0) return LIGER_OK;
    if (!logits) return fail(LIGER_ERR_NULL, "%s: logits are required", who);
    if ((tokens == nullptr) != (logp == nullptr)) return fail(LIGER_ERR_NULL, "%s: tokens and logp go together", who);
    if ((k > 0) != (top_logp != nullptr) || (k > 0) != (top_ids != nullptr))
        return fail(LIGER_ERR_NULL, "%s: top_logp and top_ids go with k > 0", who);
    if (off(logits, dtype == LIGER_F32 ? 4 : 2) || off(tokens, 8) || off(top_ids, 8) || off(logp, 4) || off(row_max, 4) ||
        off(log_sum, 4) || off(entropy, 4) || off(top_logp, 4))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be aligned to their elements", who);
    const LogpFwd p{logits, ld, tokens, T, V, ignore_index, 1.0f / temperature, logp, row_max, log_sum, entropy, top_logp, top_ids,
                    static_cast<int>(k)};
    const dim3 grid(static_cast<unsigned>(T));
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32 ? launch_early(who, token_logp_rows<float>, grid, kThreads, 0, st, p)
                              : launch_early(who, token_logp_rows<__nv_bfloat16>, grid, kThreads, 0, st, p);
}

extern "C" int liger_token_logp_bwd(const void* logits, int64_t ld, const int64_t* tokens, const float* row_max,
                                    const float* log_sum, const float* entropy, const float* g_logp, const float* g_entropy,
                                    int64_t T, int64_t V, int64_t ignore_index, float temperature, void* dlogits, int64_t ldd,
                                    int dtype, void* stream) {
    clear_error();
    const char* who = "token_logp_bwd";
    if (int rc = check_logits(who, T, V, ld, temperature, dtype)) return rc;
    if (ldd < V || ldd > (int64_t{1} << 40)) return fail(LIGER_ERR_SHAPE, "%s: ldd=%lld", who, (long long)ldd);
    if (T == 0) return LIGER_OK;
    if (!logits || !row_max || !log_sum || !dlogits)
        return fail(LIGER_ERR_NULL, "%s: logits, row_max, log_sum and dlogits are required", who);
    if (!g_logp && !g_entropy) return fail(LIGER_ERR_NULL, "%s: g_logp or g_entropy is required", who);
    if (g_logp && !tokens) return fail(LIGER_ERR_NULL, "%s: g_logp needs tokens", who);
    if (g_entropy && !entropy) return fail(LIGER_ERR_NULL, "%s: g_entropy needs entropy", who);
    if (dlogits == logits && ldd != ld) return fail(LIGER_ERR_SHAPE, "%s: in place ldd must be ld", who);
    const size_t esz = dtype == LIGER_F32 ? 4 : 2;
    if (off(logits, esz) || off(dlogits, esz) || off(tokens, 8) || off(row_max, 4) || off(log_sum, 4) || off(entropy, 4) || off(g_logp, 4) ||
        off(g_entropy, 4))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be aligned to their elements", who);
    const LogpBwd p{logits, ld, g_logp ? tokens : nullptr, row_max, log_sum, entropy, g_logp, g_entropy, T, V, ignore_index,
                    1.0f / temperature, dlogits, ldd};
    const dim3 grid(static_cast<unsigned>(T));
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32 ? launch_early(who, token_logp_bwd_rows<float>, grid, kThreads, 0, st, p)
                              : launch_early(who, token_logp_bwd_rows<__nv_bfloat16>, grid, kThreads, 0, st, p);
}
