// SwiGLU forward that keeps gate and up in 8 bits, and the backward from them
// (formulas and format in liger_train.h).
//
// GB300 design: HBM-bound; in bf16 the forward moves 8.06 bytes an element
// (gate, up in; y, two codes, two scale bytes per 32 out), the backward 8.06
// (dy, codes, scales in; dgate, dup out).
//  * forward, rows of whole groups: a lane takes 16 elements (two lanes a checkpoint group), whose
//    largest magnitude is an integer maximum of the float bits and one shuffle, and writes its 16
//    codes at once; bf16 two such pieces in flight per thread (8192 x 11008 bf16: 108 us, 1.00 of
//    the measured copy rate; 8 elements a lane, 8-byte code stores: 122 us).
//  * backward, and the forward of other rows of whole 8-element pieces: a lane takes 8 elements,
//    two pieces in flight (backward 109 us, 0.99; 16 elements: 116 to 121).
//  * other widths: a lane per element, a warp per group, 4 groups in flight.
// Every thread runs once (no persistent grid: that was 5 to 15 % slower).
// dgate or dup may alias dy, y may alias gate or up: a thread reads its pieces
// before it writes them, and no other thread reads them.
#include "ckpt8.cuh"
#include "liger_train.h"

namespace liger {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;
constexpr int kGroupsAny = 4;   // groups per warp at a time, any width

// sigmoid as in liger_swiglu_fwd: accurate for fp32 storage, the fast exp and reciprocal for bf16
// (relative error near 2^-21, far below bf16's 2^-8)
template <typename T> __device__ __forceinline__ float sigm(float g);
template <> __device__ __forceinline__ float sigm<float>(float g) { return 1.0f / (1.0f + expf(-g)); }
template <> __device__ __forceinline__ float sigm<__nv_bfloat16>(float g) {
    return __fdividef(1.0f, 1.0f + __expf(-g));
}

// 8 consecutive elements of fp32 (two vectors) or bf16 (one)
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    uint4 a, b;
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
};
__device__ __forceinline__ void load8(const float* p, Raw8<float>& r) {
    r.a = ldg16(p);
    r.b = ldg16(p + 4);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, Raw8<__nv_bfloat16>& r) { r.a = ldg16(p); }
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&f)[8]) {
    float lo[4], hi[4];
    unpack(r.a, lo);
    unpack(r.b, hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = lo[e], f[4 + e] = hi[e];
}
__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) { unpack(r.a, f); }
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
    stg16_cs(p, pack(lo));
    stg16_cs(p + 4, pack(hi));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) { stg16_cs(p, pack(f)); }

// scale byte of the group that the four lanes of a quad hold
__device__ __forceinline__ uint32_t quad_scale(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, mag_bits(f[e]));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return ckpt_scale(m);
}
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = ckpt_code(f[e], inv);
    return make_uint2(ckpt_pack4(c[0], c[1], c[2], c[3]), ckpt_pack4(c[4], c[5], c[6], c[7]));
}

// A row is `quads` groups of 4 pieces of 8 elements (the last group's missing pieces are idle lanes).
// Piece i of the tensor: element offset, group index, and whether it exists.
struct Piece {
    int64_t at, group;
    bool live;
};
template <bool FLAT>
__device__ __forceinline__ Piece piece_of(int64_t i, int64_t n, int cols, int groups) {
    Piece p;
    if (FLAT) {   // cols a multiple of 32: pieces and groups run through the rows without gaps
        p.at = i * 8;
        p.group = i >> 2;
        p.live = i < n;
        return p;
    }
    const int64_t per = static_cast<int64_t>(groups) * 4;
    const int64_t row = n <= 0x7FFFFFFF ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(per)) : i / per;
    const int v = static_cast<int>(i - row * per);
    p.at = row * cols + static_cast<int64_t>(v) * 8;
    p.group = row * groups + (v >> 2);
    p.live = i < n && v * 8 < cols;
    return p;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) swiglu_fwd_ckpt8_vec(const T* gate, const T* up, T* y, int8_t* __restrict__ gate8,
                                                                 uint8_t* __restrict__ gs, int8_t* __restrict__ up8,
                                                                 uint8_t* __restrict__ us, int64_t n, int cols, int groups) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    wait_for_stream();
    // whole warps run the loop: base is the warp's first piece
    const int lane = threadIdx.x & 31;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x - lane; base < n; base += kUnroll * stride) {
        Raw8<T> rg[kUnroll] = {}, ru[kUnroll] = {};
        Piece pc[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            pc[k] = piece_of<false>(base + k * stride + lane, n, cols, groups);
            if (pc[k].live) {
                load8(gate + pc[k].at, rg[k]);
                load8(up + pc[k].at, ru[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            float g[8], u[8], o[8];
            widen8(rg[k], g);
            widen8(ru[k], u);
            const uint32_t sg = quad_scale(g), su = quad_scale(u);
            const uint2 cg = codes8(g, ckpt_inv(sg)), cu = codes8(u, ckpt_inv(su));
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = g[e] * sigm<T>(g[e]) * u[e];
            if (pc[k].live) {
                store8(y + pc[k].at, o);
                *reinterpret_cast<uint2*>(gate8 + pc[k].at) = cg;
                *reinterpret_cast<uint2*>(up8 + pc[k].at) = cu;
                if ((lane & 3) == 0) {
                    gs[pc[k].group] = static_cast<uint8_t>(sg);
                    us[pc[k].group] = static_cast<uint8_t>(su);
                }
            }
        }
    }
}

// rows of whole groups: n pieces of 16 elements, two lanes a group
template <typename T, int U>
__global__ void __launch_bounds__(kThreads) swiglu_fwd_ckpt8_wide(const T* gate, const T* up, T* y, int8_t* __restrict__ gate8,
                                                                  uint8_t* __restrict__ gs, int8_t* __restrict__ up8,
                                                                  uint8_t* __restrict__ us, int64_t n) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x - lane; base < n; base += U * stride) {
        Raw8<T> rg[U][2] = {}, ru[U][2] = {};
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t i = base + k * stride + lane;
            if (i < n) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    load8(gate + i * 16 + h * 8, rg[k][h]);
                    load8(up + i * 16 + h * 8, ru[k][h]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t i = base + k * stride + lane;
            float g[2][8], u[2][8];
            uint32_t mg = 0, mu = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                widen8(rg[k][h], g[h]);
                widen8(ru[k][h], u[h]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mg = max(mg, mag_bits(g[h][e]));
                    mu = max(mu, mag_bits(u[h][e]));
                }
            }
            mg = max(mg, __shfl_xor_sync(0xffffffffu, mg, 1));   // n is even: both lanes of a group or neither
            mu = max(mu, __shfl_xor_sync(0xffffffffu, mu, 1));
            if (i >= n) continue;
            const uint32_t sg = ckpt_scale(mg), su = ckpt_scale(mu);
            const float ig = ckpt_inv(sg), iu = ckpt_inv(su);
            const uint2 g0 = codes8(g[0], ig), g1 = codes8(g[1], ig), u0 = codes8(u[0], iu), u1 = codes8(u[1], iu);
            stg16_cs(gate8 + i * 16, make_uint4(g0.x, g0.y, g1.x, g1.y));
            stg16_cs(up8 + i * 16, make_uint4(u0.x, u0.y, u1.x, u1.y));
            if ((lane & 1) == 0) {
                gs[i >> 1] = static_cast<uint8_t>(sg);
                us[i >> 1] = static_cast<uint8_t>(su);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = g[h][e] * sigm<T>(g[h][e]) * u[h][e];
                store8(y + i * 16 + h * 8, o);
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void swiglu_grad(float g, float u, float d, float& dg, float& du) {
    const float s = sigm<T>(g);
    du = d * (g * s);
    dg = d * u * s * (1.0f + g * (1.0f - s));
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads) swiglu_bwd_ckpt8_vec(const T* dy, const int8_t* gate8, const uint8_t* gs,
                                                                 const int8_t* up8, const uint8_t* us, T* dgate, T* dup,
                                                                 int64_t n, int cols, int groups) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    wait_for_stream();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += kUnroll * stride) {
        Raw8<T> rd[kUnroll] = {};
        uint2 cg[kUnroll], cu[kUnroll];
        uint32_t sg[kUnroll], su[kUnroll];
        Piece pc[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            pc[k] = piece_of<FLAT>(i + k * stride, n, cols, groups);
            if (pc[k].live) {
                load8(dy + pc[k].at, rd[k]);
                cg[k] = *reinterpret_cast<const uint2*>(gate8 + pc[k].at);
                cu[k] = *reinterpret_cast<const uint2*>(up8 + pc[k].at);
                sg[k] = gs[pc[k].group];
                su[k] = us[pc[k].group];
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (!pc[k].live) continue;
            const float qg = ckpt_step(sg[k]), qu = ckpt_step(su[k]);
            float d[8], og[8], ou[8];
            widen8(rd[k], d);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float g[4], u[4];
                ckpt_unpack4(half ? cg[k].y : cg[k].x, g);
                ckpt_unpack4(half ? cu[k].y : cu[k].x, u);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    swiglu_grad<T>(g[e] * qg, u[e] * qu, d[half * 4 + e], og[half * 4 + e], ou[half * 4 + e]);
            }
            store8(dgate + pc[k].at, og);
            store8(dup + pc[k].at, ou);
        }
    }
}

// any width: warp per group of 32 columns, lane per element, kGroupsAny groups a warp at a time
struct Element {
    int64_t at;
    bool live;
};
__device__ __forceinline__ Element element_of(int64_t w, int64_t ngroups, int cols, int groups, int lane) {
    const int64_t row = ngroups <= 0x7FFFFFFF ? static_cast<int64_t>(static_cast<uint32_t>(w) / static_cast<uint32_t>(groups)) : w / groups;
    const int c = static_cast<int>(w - row * groups) * kCkptGroup + lane;
    return Element{row * cols + c, w < ngroups && c < cols};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) swiglu_fwd_ckpt8_any(const T* gate, const T* up, T* y, int8_t* __restrict__ gate8,
                                                                 uint8_t* __restrict__ gs, int8_t* __restrict__ up8,
                                                                 uint8_t* __restrict__ us, int64_t ngroups, int cols,
                                                                 int groups) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kGroupsAny;
    wait_for_stream();
    for (int64_t w = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kGroupsAny; w < ngroups; w += step) {
        Element el[kGroupsAny];
        float g[kGroupsAny], u[kGroupsAny];
#pragma unroll
        for (int k = 0; k < kGroupsAny; ++k) {
            el[k] = element_of(w + k, ngroups, cols, groups, lane);
            g[k] = el[k].live ? ldf(gate + el[k].at) : 0.f;
            u[k] = el[k].live ? ldf(up + el[k].at) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kGroupsAny; ++k) {
            const uint32_t sg = ckpt_scale(__reduce_max_sync(0xffffffffu, mag_bits(g[k])));
            const uint32_t su = ckpt_scale(__reduce_max_sync(0xffffffffu, mag_bits(u[k])));
            if (el[k].live) {
                gate8[el[k].at] = static_cast<int8_t>(ckpt_code(g[k], ckpt_inv(sg)) & 0xFFu);
                up8[el[k].at] = static_cast<int8_t>(ckpt_code(u[k], ckpt_inv(su)) & 0xFFu);
                stf(y + el[k].at, g[k] * sigm<T>(g[k]) * u[k]);
            }
            if (lane == 0 && w + k < ngroups) {
                gs[w + k] = static_cast<uint8_t>(sg);
                us[w + k] = static_cast<uint8_t>(su);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) swiglu_bwd_ckpt8_any(const T* dy, const int8_t* gate8, const uint8_t* gs,
                                                                 const int8_t* up8, const uint8_t* us, T* dgate, T* dup,
                                                                 int64_t ngroups, int cols, int groups) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kGroupsAny;
    wait_for_stream();
    for (int64_t w = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kGroupsAny; w < ngroups; w += step) {
        Element el[kGroupsAny];
        float d[kGroupsAny];
        int g[kGroupsAny], u[kGroupsAny];
        uint32_t sg[kGroupsAny], su[kGroupsAny];
#pragma unroll
        for (int k = 0; k < kGroupsAny; ++k) {
            el[k] = element_of(w + k, ngroups, cols, groups, lane);
            if (el[k].live) {
                d[k] = ldf(dy + el[k].at);
                g[k] = gate8[el[k].at];
                u[k] = up8[el[k].at];
                sg[k] = gs[w + k];
                su[k] = us[w + k];
            }
        }
#pragma unroll
        for (int k = 0; k < kGroupsAny; ++k) {
            if (!el[k].live) continue;
            float og, ou;
            swiglu_grad<T>(static_cast<float>(g[k]) * ckpt_step(sg[k]), static_cast<float>(u[k]) * ckpt_step(su[k]), d[k], og, ou);
            stf(dgate + el[k].at, og);
            stf(dup + el[k].at, ou);
        }
    }
}

// blocks so that `threads` threads run once (the kernels loop where the grid's limit is passed)
unsigned grid_for(int64_t threads) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(threads, kThreads), 0x7FFFFFFF)));
}

template <typename T>
int launch_fwd(const void* gate, const void* up, void* y, int8_t* gate8, uint8_t* gs, int8_t* up8, uint8_t* us,
               int64_t rows, int cols, cudaStream_t st) {
    const T *g = static_cast<const T*>(gate), *u = static_cast<const T*>(up);
    T* o = static_cast<T*>(y);
    const int groups = static_cast<int>(ceil_div(cols, kCkptGroup));
    const int64_t ngroups = rows * groups;
    const char* who = "swiglu_fwd_ckpt8";
    if (cols % kCkptGroup == 0) {
        constexpr int U = sizeof(T) == 2 ? 2 : 1;   // fp32: one piece is four vectors of each input already
        return launch_early(who, swiglu_fwd_ckpt8_wide<T, U>, grid_for(ceil_div(ngroups * 2, U)), kThreads, 0, st, g, u, o,
                            gate8, gs, up8, us, ngroups * 2);
    }
    if (cols % 8 == 0)
        return launch_early(who, swiglu_fwd_ckpt8_vec<T>, grid_for(ceil_div(ngroups * 4, kUnroll)), kThreads, 0, st, g, u, o,
                            gate8, gs, up8, us, ngroups * 4, cols, groups);
    return launch_early(who, swiglu_fwd_ckpt8_any<T>, grid_for(ceil_div(ngroups, kGroupsAny) * 32), kThreads, 0, st, g, u, o,
                        gate8, gs, up8, us, ngroups, cols, groups);
}

template <typename T>
int launch_bwd(const void* dy, const int8_t* gate8, const uint8_t* gs, const int8_t* up8, const uint8_t* us, void* dgate,
               void* dup, int64_t rows, int cols, cudaStream_t st) {
    const T* d = static_cast<const T*>(dy);
    T *og = static_cast<T*>(dgate), *ou = static_cast<T*>(dup);
    const int groups = static_cast<int>(ceil_div(cols, kCkptGroup));
    const int64_t ngroups = rows * groups;
    const char* who = "swiglu_bwd_ckpt8";
    if (cols % 8 == 0)
        return launch_early(who, cols % kCkptGroup == 0 ? swiglu_bwd_ckpt8_vec<T, true> : swiglu_bwd_ckpt8_vec<T, false>,
                            grid_for(ceil_div(ngroups * 4, kUnroll)), kThreads, 0, st, d, gate8, gs, up8, us, og, ou,
                            ngroups * 4, cols, groups);
    return launch_early(who, swiglu_bwd_ckpt8_any<T>, grid_for(ceil_div(ngroups, kGroupsAny) * 32), kThreads, 0, st, d, gate8,
                        gs, up8, us, og, ou, ngroups, cols, groups);
}

int check(const char* who, int64_t rows, int64_t cols, int dtype, std::initializer_list<const void*> wide,
          std::initializer_list<const void*> bytes) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (rows < 0 || cols < 0 || cols > (1 << 30) || rows > (int64_t{1} << 48) / std::max<int64_t>(cols, 1))
        return fail(LIGER_ERR_SHAPE, "%s: rows=%lld cols=%lld", who, (long long)rows, (long long)cols);
    if (rows == 0 || cols == 0) return LIGER_OK;
    for (const void* p : wide)
        if (!p) return fail(LIGER_ERR_NULL, "%s: null tensor pointer", who);
    for (const void* p : bytes)
        if (!p) return fail(LIGER_ERR_NULL, "%s: null scale pointer", who);
    for (const void* p : wide)
        if (!aligned16(p)) return fail(LIGER_ERR_ALIGN, "%s: tensors and codes must be 16-byte aligned", who);
    return LIGER_OK;
}

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" int liger_swiglu_fwd_ckpt8(const void* gate, const void* up, void* y, int8_t* gate8, uint8_t* gate_scale,
                                      int8_t* up8, uint8_t* up_scale, int64_t rows, int64_t cols, int dtype,
                                      void* stream) {
    clear_error();
    if (int rc = check("swiglu_fwd_ckpt8", rows, cols, dtype, {gate, up, y, gate8, up8}, {gate_scale, up_scale})) return rc;
    if (rows == 0 || cols == 0) return LIGER_OK;
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32
               ? launch_fwd<float>(gate, up, y, gate8, gate_scale, up8, up_scale, rows, (int)cols, st)
               : launch_fwd<__nv_bfloat16>(gate, up, y, gate8, gate_scale, up8, up_scale, rows, (int)cols, st);
}

extern "C" int liger_swiglu_bwd_ckpt8(const void* dy, const int8_t* gate8, const uint8_t* gate_scale, const int8_t* up8,
                                      const uint8_t* up_scale, void* dgate, void* dup, int64_t rows, int64_t cols,
                                      int dtype, void* stream) {
    clear_error();
    if (int rc = check("swiglu_bwd_ckpt8", rows, cols, dtype, {dy, gate8, up8, dgate, dup}, {gate_scale, up_scale}))
        return rc;
    if (rows == 0 || cols == 0) return LIGER_OK;
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32
               ? launch_bwd<float>(dy, gate8, gate_scale, up8, up_scale, dgate, dup, rows, (int)cols, st)
               : launch_bwd<__nv_bfloat16>(dy, gate8, gate_scale, up8, up_scale, dgate, dup, rows, (int)cols, st);
}
