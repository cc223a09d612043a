// Layer norm, forward and backward (formulas in liger_layer.h).
#include "block_norm.cuh"
#include "liger_layer.h"

namespace liger {
namespace {

constexpr int kMaxPartRows = 1024;   // most partial rows of dw and of db

// ------------------------------------------------------------- any width
// A block per row, elements strided over its threads; the row is read again from the caches for
// the variance and for the result.
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_fwd_rows(const T* x, const T* w, const T* b, T* y, float* mean,
                                                           float* rstd, int64_t rows, int cols, float eps) {
    __shared__ float sh[8];
    const float n = static_cast<float>(cols);
    wait_for_stream();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * cols;
        float s = 0.f;
        for (int j = threadIdx.x; j < cols; j += blockDim.x) s += ldf(xr + j);
        const float m = block_sum(s, sh) / n;
        s = 0.f;
        for (int j = threadIdx.x; j < cols; j += blockDim.x) {
            const float d = ldf(xr + j) - m;
            s = fmaf(d, d, s);
        }
        const float rs = 1.0f / sqrtf(block_sum(s, sh) / n + eps);
        T* yr = y + r * cols;
        for (int j = threadIdx.x; j < cols; j += blockDim.x) {
            const float h = (ldf(xr + j) - m) * rs;
            stf(yr + j, fmaf(h, w != nullptr ? ldf(w + j) : 1.f, b != nullptr ? ldf(b + j) : 0.f));
        }
        if (threadIdx.x == 0) {
            if (mean != nullptr) mean[r] = m;
            if (rstd != nullptr) rstd[r] = rs;
        }
    }
}

struct LnBwd {
    const void *dy, *dres, *x, *w;
    const float *mean, *rstd;
    void* dx;
    float *part_w, *part_b;   // [blocks][cols] each, or NULL
    int64_t rows, rows_per_block;
    int cols;
};

// A block per run of rows; its partial rows of dw and db stand in the workspace, each element
// touched by one thread only.
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_bwd_rows(LnBwd p) {
    __shared__ float sh[8];
    const T *dy = static_cast<const T*>(p.dy), *dres = static_cast<const T*>(p.dres), *x = static_cast<const T*>(p.x),
            *w = static_cast<const T*>(p.w);
    T* dx = static_cast<T*>(p.dx);
    float* pw = p.part_w != nullptr ? p.part_w + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    float* pb = p.part_b != nullptr ? p.part_b + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    const float n = static_cast<float>(p.cols);
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_block, r1 = min(p.rows, r0 + p.rows_per_block);
    wait_for_stream();
    for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
        if (pw != nullptr) pw[j] = 0.f;
        if (pb != nullptr) pb[j] = 0.f;
    }
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t o = r * p.cols;
        const float m = p.mean[r], rs = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
            const float g = ldf(dy + o + j) * (w != nullptr ? ldf(w + j) : 1.f);
            s1 += g;
            s2 = fmaf(g, (ldf(x + o + j) - m) * rs, s2);
        }
        s1 = block_sum(s1, sh) / n;
        s2 = block_sum(s2, sh) / n;
        for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
            const float d = ldf(dy + o + j), xh = (ldf(x + o + j) - m) * rs;
            const float g = d * (w != nullptr ? ldf(w + j) : 1.f);
            stf(dx + o + j, fmaf(rs, g - s1 - xh * s2, dres != nullptr ? ldf(dres + o + j) : 0.f));
            if (pw != nullptr) pw[j] = fmaf(d, xh, pw[j]);
            if (pb != nullptr) pb[j] += d;
        }
    }
}

// Column sums of the partial rows in ascending order: dw (blockIdx.y 0) and db (1).
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_sums(const float* part_w, const float* part_b, T* dw, T* db, int parts,
                                                       int cols) {
    __shared__ float red[8][33];
    wait_for_stream();
    const float* part = blockIdx.y == 0 ? part_w : part_b;
    T* out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr) return;
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (col < cols)
#pragma unroll 4
        for (int i = sl; i < parts; i += 8) s += part[static_cast<int64_t>(i) * cols + col];
    red[sl][lane] = s;
    __syncthreads();
    if (sl == 0 && col < cols) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += red[i][lane];
        stf(out + col, t);
    }
}

int check_sizes(const char* who, int64_t rows, int64_t cols, int dtype) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (rows < 0 || cols <= 0 || cols > (1 << 24) || rows > (int64_t{1} << 48) / cols)
        return fail(LIGER_ERR_SHAPE, "%s: rows=%lld cols=%lld", who, (long long)rows, (long long)cols);
    return LIGER_OK;
}

template <typename T>
int run_fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, int64_t rows, int cols,
            float eps, cudaStream_t st) {
    const int64_t grid = std::min<int64_t>(rows, 8 * sm_count());
    return launch_early("layernorm_fwd", layer_norm_fwd_rows<T>, dim3(static_cast<unsigned>(grid)), 256, 0, st,
                        static_cast<const T*>(x), static_cast<const T*>(w), static_cast<const T*>(b), static_cast<T*>(y),
                        mean, rstd, rows, cols, eps);
}

template <typename T>
int run_bwd(LnBwd p, void* dw, void* db, cudaStream_t st) {
    const int64_t most = std::min<int64_t>({p.rows, kMaxPartRows, 4 * sm_count()});
    p.rows_per_block = ceil_div(p.rows, most);
    const int64_t grid = ceil_div(p.rows, p.rows_per_block);
    if (int rc = launch_early("layernorm_bwd", layer_norm_bwd_rows<T>, dim3(static_cast<unsigned>(grid)), 256, 0, st, p))
        return rc;
    if (dw == nullptr && db == nullptr) return LIGER_OK;
    return launch_early("layernorm_bwd sums", layer_norm_sums<T>, dim3(static_cast<unsigned>(ceil_div(p.cols, 32)), 2), 256, 0,
                        st, static_cast<const float*>(p.part_w), static_cast<const float*>(p.part_b), static_cast<T*>(dw),
                        static_cast<T*>(db), static_cast<int>(grid), p.cols);
}

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" int liger_layernorm_fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                                   int64_t rows, int64_t cols, float eps, int dtype, void* stream) {
    clear_error();
    const char* who = "layernorm_fwd";
    if (int rc = check_sizes(who, rows, cols, dtype)) return rc;
    if (!(eps >= 0.f)) return fail(LIGER_ERR_SHAPE, "%s: eps must be >= 0", who);
    if (rows == 0) return LIGER_OK;
    if (!x || !y) return fail(LIGER_ERR_NULL, "%s: x and y are required", who);
    if (misaligned({x, w, b, y}, 16)) return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    if (misaligned({mean, rstd}, 4)) return fail(LIGER_ERR_ALIGN, "%s: mean and rstd must be 4-byte aligned", who);
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32 ? run_fwd<float>(x, w, b, y, mean, rstd, rows, static_cast<int>(cols), eps, st)
                              : run_fwd<__nv_bfloat16>(x, w, b, y, mean, rstd, rows, static_cast<int>(cols), eps, st);
}

extern "C" size_t liger_layernorm_bwd_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || cols > (1 << 24)) return 0;
    return 2 * static_cast<size_t>(std::min<int64_t>(rows, kMaxPartRows)) * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" int liger_layernorm_bwd(const void* dy, const void* dres, const void* x, const void* w, const float* mean,
                                   const float* rstd, void* dx, void* dw, void* db, void* ws, size_t ws_bytes,
                                   int64_t rows, int64_t cols, int dtype, void* stream) {
    clear_error();
    const char* who = "layernorm_bwd";
    if (int rc = check_sizes(who, rows, cols, dtype)) return rc;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx))
        return fail(LIGER_ERR_NULL, "%s: dy, x, mean, rstd and dx are required", who);
    if (misaligned({dy, dres, x, w, dx, dw, db}, 16))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    if (misaligned({mean, rstd}, 4)) return fail(LIGER_ERR_ALIGN, "%s: mean and rstd must be 4-byte aligned", who);
    cudaStream_t st = as_stream(stream);
    const size_t esz = dtype == LIGER_F32 ? 4 : 2;
    if (rows == 0) {
        for (void* out : {dw, db})
            if (out != nullptr && cudaMemsetAsync(out, 0, static_cast<size_t>(cols) * esz, st) != cudaSuccess)
                return check_launch(who);
        return LIGER_OK;
    }
    const size_t need = liger_layernorm_bwd_workspace(rows, cols);
    if ((dw != nullptr || db != nullptr) && (!ws || ws_bytes < need || !aligned16(ws)))
        return fail(LIGER_ERR_WORKSPACE, "%s: workspace of %zu bytes (16-byte aligned) required, got %zu", who, need, ws_bytes);
    LnBwd p{dy, dres, x, w, mean, rstd, dx, nullptr, nullptr, rows, 0, static_cast<int>(cols)};
    if (dw != nullptr) p.part_w = static_cast<float*>(ws);
    if (db != nullptr) p.part_b = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + need / 2);
    return dtype == LIGER_F32 ? run_bwd<float>(p, dw, db, st) : run_bwd<__nv_bfloat16>(p, dw, db, st);
}
