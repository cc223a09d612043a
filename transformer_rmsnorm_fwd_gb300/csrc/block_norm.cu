// Block norms: post-norm, gate, scaled residual sum and pre-norm in one pass
// over the rows, forward and backward (formulas in liger_train.h).
//
// GB300 design: HBM-bound.  In bf16 the forward has to move 8 bytes an element
// (z, r in; h, y out), the backward 12 (dh, dy, z, h in; dr, dz out); every row
// is read once and written once.
//  * generic kernels (any width): a block per row, scalar accesses.
//  * backward sums over rows: with S[j] = sum D z rz over rows that share a
//    gate row, dgate = block_scale w_post S and dw_post = block_scale g S, so
//    one running sum serves both.  Rows are split into units that never cross a
//    gate row; per-unit partial rows go to the workspace and are added in a
//    fixed order.
#include "common.cuh"
#include "liger_train.h"

namespace liger {
namespace {

constexpr int kMaxParts = 1024;   // most partial rows of the backward's sums

struct FwdP {
    const void *z, *r, *w_post, *gate, *w_pre;
    void *h, *y;
    float *rstd_z, *rstd_h;
    int64_t rows, per_gate;   // per_gate: rows that share a gate row
    int cols;
    float a, b, eps;
};

struct BwdP {
    const void *dh, *dy, *z, *h, *w_post, *gate, *w_pre;
    const float *rstd_z, *rstd_h;
    void *dr, *dz, *dgate;
    float *part_s, *part_pre;
    int64_t rows, per_gate, gates;
    int64_t splits;       // > 0: each gate row's rows split into this many units, one block each (part_s: S)
                          // 0: each block takes gates_per_block whole gate rows (part_s: sum of block_scale g S)
    int64_t unit_rows;    // rows per unit (splits > 0)
    int64_t gates_per_block;
    int cols;
    float a, b;
};

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

// ---------------------------------------------------------------- generic
// Every element is written by the thread that read it, after the block's last
// read of the row by another pass, so h == r and y == z are safe.
template <typename T>
__global__ void __launch_bounds__(256) block_norm_fwd_generic(FwdP p) {
    __shared__ float sh[8];
    const T *z = static_cast<const T*>(p.z), *r = static_cast<const T*>(p.r);
    const T *wp = static_cast<const T*>(p.w_post), *wn = static_cast<const T*>(p.w_pre);
    T *h = static_cast<T*>(p.h), *y = static_cast<T*>(p.y);
    const float inv = 1.0f / static_cast<float>(p.cols);
    for (int64_t t = blockIdx.x; t < p.rows; t += gridDim.x) {
        const int64_t o = t * p.cols;
        const T* g = p.gate != nullptr ? static_cast<const T*>(p.gate) + t / p.per_gate * p.cols : nullptr;
        float rz = 1.f;
        if (wp != nullptr) {
            float ss = 0.f;
            for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
                const float f = ldf(z + o + j);
                ss = fmaf(f, f, ss);
            }
            rz = 1.0f / sqrtf(block_sum(ss, sh) * inv + p.eps);
            if (p.rstd_z != nullptr && threadIdx.x == 0) p.rstd_z[t] = rz;
        }
        auto hval = [&](int j) {
            float q = ldf(z + o + j);
            if (wp != nullptr) q = q * rz * ldf(wp + j);
            if (g != nullptr) q *= ldf(g + j);
            return fmaf(p.b, q, p.a * ldf(r + o + j));
        };
        float rh = 0.f;
        if (wn != nullptr) {
            float ss = 0.f;
            for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
                const float f = hval(j);
                ss = fmaf(f, f, ss);
            }
            rh = 1.0f / sqrtf(block_sum(ss, sh) * inv + p.eps);
            if (p.rstd_h != nullptr && threadIdx.x == 0) p.rstd_h[t] = rh;
        }
        for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
            const float f = hval(j);
            stf(h + o + j, f);
            if (wn != nullptr) stf(y + o + j, f * rh * ldf(wn + j));
        }
    }
}

// The block's partial rows live in the workspace; each element of them belongs to one thread.
template <typename T>
__global__ void __launch_bounds__(256) block_norm_bwd_generic(BwdP p) {
    __shared__ float sh[8];
    const T *dh = static_cast<const T*>(p.dh), *dy = static_cast<const T*>(p.dy), *z = static_cast<const T*>(p.z),
            *h = static_cast<const T*>(p.h), *wp = static_cast<const T*>(p.w_post), *wn = static_cast<const T*>(p.w_pre);
    T *dr = static_cast<T*>(p.dr), *dz = static_cast<T*>(p.dz);
    float* ps = p.part_s != nullptr ? p.part_s + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    float* pp = p.part_pre != nullptr ? p.part_pre + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    const bool need_s = wp != nullptr || p.gate != nullptr;
    const float inv = 1.0f / static_cast<float>(p.cols);
    for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
        if (ps != nullptr) ps[j] = 0.f;
        if (pp != nullptr) pp[j] = 0.f;
    }
    int64_t t0, t1;   // this block's rows
    if (p.splits > 0) {
        const int64_t gi = blockIdx.x / p.splits, s = blockIdx.x - gi * p.splits;
        t0 = gi * p.per_gate + s * p.unit_rows;
        t1 = min(t0 + p.unit_rows, (gi + 1) * p.per_gate);
    } else {
        t0 = blockIdx.x * p.gates_per_block * p.per_gate;
        t1 = min(p.rows, t0 + p.gates_per_block * p.per_gate);
    }
    for (int64_t t = t0; t < t1; ++t) {
        const int64_t o = t * p.cols, gi = t / p.per_gate;
        const T* g = p.gate != nullptr ? static_cast<const T*>(p.gate) + gi * p.cols : nullptr;
        const float rz = wp != nullptr ? p.rstd_z[t] : 1.f, rh = wn != nullptr ? p.rstd_h[t] : 0.f;
        float c1 = 0.f, c2 = 0.f;
        if (wn != nullptr) {
            float s1 = 0.f;
            for (int j = threadIdx.x; j < p.cols; j += blockDim.x)
                s1 = fmaf(ldf(dy + o + j) * ldf(wn + j), ldf(h + o + j), s1);
            c1 = rh * rh * rh * inv * block_sum(s1, sh);
        }
        auto dval = [&](int j) {
            float d = dh != nullptr ? ldf(dh + o + j) : 0.f;
            if (wn != nullptr) d += rh * (ldf(dy + o + j) * ldf(wn + j)) - c1 * ldf(h + o + j);
            return d;
        };
        auto qval = [&](int j) {
            float q = p.b;
            if (g != nullptr) q *= ldf(g + j);
            if (wp != nullptr) q *= ldf(wp + j);
            return q;
        };
        if (wp != nullptr) {
            float s2 = 0.f;
            for (int j = threadIdx.x; j < p.cols; j += blockDim.x)
                s2 = fmaf(qval(j) * dval(j), ldf(z + o + j), s2);
            c2 = rz * rz * rz * inv * block_sum(s2, sh);
        }
        const bool last_of_gate = p.splits == 0 && (t + 1) % p.per_gate == 0;
        const bool first_of_gate = p.splits == 0 && t % p.per_gate == 0;
        for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
            const float d = dval(j), q = qval(j);
            const float zj = need_s ? ldf(z + o + j) : 0.f;
            if (pp != nullptr) pp[j] = fmaf(ldf(dy + o + j) * ldf(h + o + j), rh, pp[j]);
            stf(dr + o + j, p.a * d);
            stf(dz + o + j, wp != nullptr ? rz * (q * d) - c2 * zj : q * d);
            if (need_s) {
                const float sv = d * zj * rz;
                if (p.splits > 0) {
                    ps[j] += sv;
                } else {
                    // whole gate rows: the running sum of this gate row sits in the second half
                    float* run = p.part_s + (static_cast<int64_t>(gridDim.x) + blockIdx.x) * p.cols;
                    const float acc = (first_of_gate ? 0.f : run[j]) + sv;
                    run[j] = acc;
                    if (last_of_gate) {
                        if (g != nullptr)
                            stf(static_cast<T*>(p.dgate) + gi * p.cols + j, p.b * acc * (wp != nullptr ? ldf(wp + j) : 1.f));
                        ps[j] = fmaf(p.b * (g != nullptr ? ldf(g + j) : 1.f), acc, ps[j]);
                    }
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------- sums over the partial rows
struct SumP {
    const float *part_s, *part_pre;
    const void *w_post, *gate;
    void *dw_post, *dgate, *dw_pre;
    int64_t nparts, gates, splits;
    int cols;
    float b;
};

// Block of 32 warps over 32 groups of V columns: warp w adds the partial rows w, w + 32, ... in
// ascending order, the 32 slice sums are then added in slice order (deterministic for a given
// number of partial rows).  blockIdx.y picks the sum: 0 dw_pre, 1 dw_post (with one gate row dgate
// too, from the same sum), 2 + i the gradient of gate row i.
template <typename T, int V>
__global__ void __launch_bounds__(1024) block_norm_sums(SumP p) {
    __shared__ float red[32][32][V];
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * V;
    const int task = blockIdx.y;
    if (task == 0 && p.dw_pre == nullptr) return;
    if (task == 1 && p.dw_post == nullptr && !(p.dgate != nullptr && p.gates == 1 && p.splits > 0)) return;
    const float* part = task == 0 ? p.part_pre : p.part_s;
    const bool weighted = task == 1 && p.splits > 0 && p.gates > 1;   // by the unit's gate row
    int64_t b0 = 0, b1 = p.nparts;
    if (task >= 2) {
        b0 = (task - 2) * p.splits;
        b1 = b0 + p.splits;
    }
    const T* gate = static_cast<const T*>(p.gate);
    float s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = 0.f;
    if (c < p.cols) {
#pragma unroll 4
        for (int64_t b = b0 + sl; b < b1; b += 32) {
            float v[V];
            const float* src = part + b * p.cols + c;
            if constexpr (V == 4) unpack(ldg16(src), v);
            else v[0] = *src;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (weighted) v[e] *= ldf(gate + b / p.splits * p.cols + c + e);
                s[e] += v[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[sl][lane][e] = s[e];
    __syncthreads();
    if (sl != 0 || c >= p.cols) return;
    for (int i = 1; i < 32; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] += red[i][lane][e];
    const T* wp = static_cast<const T*>(p.w_post);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (task == 0) {
            stf(static_cast<T*>(p.dw_pre) + c + e, s[e]);
        } else if (task == 1) {
            if (p.dw_post != nullptr) {
                float v = s[e];
                if (p.splits > 0) v *= p.b;
                if (p.splits > 0 && p.gates == 1 && gate != nullptr) v *= ldf(gate + c + e);
                stf(static_cast<T*>(p.dw_post) + c + e, v);
            }
            if (p.dgate != nullptr && p.gates == 1 && p.splits > 0)
                stf(static_cast<T*>(p.dgate) + c + e, p.b * s[e] * (wp != nullptr ? ldf(wp + c + e) : 1.f));
        } else {
            stf(static_cast<T*>(p.dgate) + static_cast<int64_t>(task - 2) * p.cols + c + e,
                p.b * s[e] * (wp != nullptr ? ldf(wp + c + e) : 1.f));
        }
    }
}

template <typename T>
int launch_sums(const SumP& s, cudaStream_t st) {
    if (s.dw_pre == nullptr && s.dw_post == nullptr && s.dgate == nullptr) return LIGER_OK;
    const unsigned tasks = 2u + (s.dgate != nullptr && s.gates > 1 && s.splits > 0 ? static_cast<unsigned>(s.gates) : 0u);
    if (s.cols % 4 == 0)
        block_norm_sums<T, 4><<<dim3(static_cast<unsigned>(ceil_div(s.cols, 128)), tasks), 1024, 0, st>>>(s);
    else
        block_norm_sums<T, 1><<<dim3(static_cast<unsigned>(ceil_div(s.cols, 32)), tasks), 1024, 0, st>>>(s);
    return check_launch("block_norm_sums");
}

// ------------------------------------------------------------------ launches
template <typename T>
int launch_fwd(const FwdP& p, cudaStream_t st) {
    const int64_t grid = std::min<int64_t>(p.rows, static_cast<int64_t>(sm_count()) * 8);
    block_norm_fwd_generic<T><<<static_cast<unsigned>(grid), 256, 0, st>>>(p);
    return check_launch("block_norm_fwd");
}

// Splits the rows into blocks: at most `want` of them (and kMaxParts), none across a gate row
// unless it takes whole gate rows.  Returns the grid.
int64_t split_rows(BwdP& p, int64_t want) {
    want = std::max<int64_t>(1, std::min<int64_t>({want, kMaxParts, p.rows}));
    const int64_t per_gate_blocks = std::min(want / p.gates, p.per_gate);
    if (per_gate_blocks >= 2 || p.gates == 1) {
        p.unit_rows = ceil_div(p.per_gate, std::max<int64_t>(1, per_gate_blocks));
        p.splits = ceil_div(p.per_gate, p.unit_rows);
        p.gates_per_block = 0;
        return p.gates * p.splits;
    }
    p.splits = 0;
    p.unit_rows = 0;
    p.gates_per_block = ceil_div(p.gates, want);
    return ceil_div(p.gates, p.gates_per_block);
}

template <typename T>
int launch_bwd(BwdP p, void* dw_post, void* dw_pre, float* ws, cudaStream_t st) {
    const int64_t grid = split_rows(p, static_cast<int64_t>(sm_count()) * 4);
    const int64_t room = std::min<int64_t>(p.rows, kMaxParts) * p.cols;
    const bool need_s = p.w_post != nullptr || p.gate != nullptr;
    p.part_pre = p.w_pre != nullptr ? ws : nullptr;
    p.part_s = need_s ? ws + room : nullptr;
    block_norm_bwd_generic<T><<<static_cast<unsigned>(grid), 256, 0, st>>>(p);
    if (int rc = check_launch("block_norm_bwd")) return rc;
    const SumP s{p.part_s, p.part_pre, p.w_post, p.gate, dw_post, p.gate != nullptr ? p.dgate : nullptr, dw_pre, grid,
                 p.gates, p.splits, p.cols, p.b};
    return launch_sums<T>(s, st);
}

int check_common(const char* who, int64_t rows, int64_t cols, int64_t gates, const void* gate, int dtype) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (rows < 0 || cols <= 0 || cols > (1 << 24) || gates < 0 || rows > (int64_t{1} << 40))
        return fail(LIGER_ERR_SHAPE, "%s: rows=%lld cols=%lld gates=%lld", who, (long long)rows, (long long)cols,
                    (long long)gates);
    if (gates > 0 && rows % gates)
        return fail(LIGER_ERR_SHAPE, "%s: rows=%lld is no multiple of gates=%lld", who, (long long)rows, (long long)gates);
    if ((gates > 0) != (gate != nullptr))
        return fail(LIGER_ERR_NULL, "%s: gate and gates > 0 go together (gates=%lld)", who, (long long)gates);
    return LIGER_OK;
}

bool misaligned(std::initializer_list<const void*> ps, unsigned to) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return true;   // NULL is aligned
    return false;
}

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" int liger_block_norm_fwd(const void* z, const void* r, const void* w_post, const void* gate,
                                    const void* w_pre, void* h, void* y, float* rstd_z, float* rstd_h, int64_t rows,
                                    int64_t cols, int64_t gates, float res_scale, float block_scale, float eps,
                                    int dtype, void* stream) {
    clear_error();
    const char* who = "block_norm_fwd";
    if (int rc = check_common(who, rows, cols, gates, gate, dtype)) return rc;
    if (!(eps >= 0.f)) return fail(LIGER_ERR_SHAPE, "%s: eps must be >= 0", who);
    if (rows == 0) return LIGER_OK;
    if (!z || !r || !h || (w_pre && !y)) return fail(LIGER_ERR_NULL, "%s: z, r, h (and y with w_pre) are required", who);
    if (misaligned({z, r, w_post, gate, w_pre, h, y}, 16) || misaligned({rstd_z, rstd_h}, 4))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    const FwdP p{z, r, w_post, gate, w_pre, h, y, rstd_z, rstd_h, rows, gates > 0 ? rows / gates : rows,
                 static_cast<int>(cols), res_scale, block_scale, eps};
    return dtype == LIGER_F32 ? launch_fwd<float>(p, as_stream(stream)) : launch_fwd<__nv_bfloat16>(p, as_stream(stream));
}

extern "C" size_t liger_block_norm_bwd_workspace(int64_t rows, int64_t cols, int64_t gates) {
    if (rows <= 0 || cols <= 0 || gates < 0) return 0;
    return 3 * static_cast<size_t>(std::min<int64_t>(rows, kMaxParts)) * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" int liger_block_norm_bwd(const void* dh, const void* dy, const void* z, const void* h, const void* w_post,
                                    const void* gate, const void* w_pre, const float* rstd_z, const float* rstd_h,
                                    void* dr, void* dz, void* dw_post, void* dgate, void* dw_pre, void* ws,
                                    size_t ws_bytes, int64_t rows, int64_t cols, int64_t gates, float res_scale,
                                    float block_scale, int dtype, void* stream) {
    clear_error();
    const char* who = "block_norm_bwd";
    if (int rc = check_common(who, rows, cols, gates, gate, dtype)) return rc;
    if ((w_post && !dw_post) || (gate && !dgate) || (w_pre && !dw_pre))
        return fail(LIGER_ERR_NULL, "%s: dw_post, dgate, dw_pre are required with w_post, gate, w_pre", who);
    if (rows > 0 && (!dr || !dz || (!w_pre && !dh) || (w_pre && (!dy || !h || !rstd_h)) || (w_post && !rstd_z) ||
                     ((w_post || gate) && !z)))
        return fail(LIGER_ERR_NULL,
                    "%s: required: dr, dz; dy, h, rstd_h with w_pre, else dh; z, rstd_z with w_post; z with gate", who);
    if (misaligned({dh, dy, z, h, w_post, gate, w_pre, dr, dz, dw_post, dgate, dw_pre}, 16) ||
        misaligned({rstd_z, rstd_h}, 4))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    cudaStream_t st = as_stream(stream);
    if (rows == 0) {
        const size_t row = static_cast<size_t>(cols) * (dtype == LIGER_F32 ? 4 : 2);
        bool ok = true;
        if (w_post) ok = ok && cudaMemsetAsync(dw_post, 0, row, st) == cudaSuccess;
        if (gate) ok = ok && cudaMemsetAsync(dgate, 0, row * static_cast<size_t>(gates), st) == cudaSuccess;
        if (w_pre) ok = ok && cudaMemsetAsync(dw_pre, 0, row, st) == cudaSuccess;
        return ok ? LIGER_OK : check_launch("block_norm_bwd memset");
    }
    const size_t need = liger_block_norm_bwd_workspace(rows, cols, gates);
    if (!ws || ws_bytes < need || !aligned16(ws))
        return fail(LIGER_ERR_WORKSPACE, "%s: workspace of %zu bytes (16-byte aligned) required, got %zu", who, need,
                    ws_bytes);
    const BwdP p{dh, dy, z, h, w_post, gate, w_pre, rstd_z, rstd_h, dr, dz, dgate, nullptr, nullptr, rows,
                 gates > 0 ? rows / gates : rows, std::max<int64_t>(gates, 1), 0, 0, 0, static_cast<int>(cols),
                 res_scale, block_scale};
    float* part = static_cast<float*>(ws);
    void* o_post = w_post ? dw_post : nullptr;
    void* o_pre = w_pre ? dw_pre : nullptr;
    return dtype == LIGER_F32 ? launch_bwd<float>(p, o_post, o_pre, part, st)
                              : launch_bwd<__nv_bfloat16>(p, o_post, o_pre, part, st);
}
