// Activations of the biased projections and their derivatives (liger_layer.h).
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "liger_layer.h"

namespace liger {
namespace {

// FAST forms are for results that are rounded to bf16 next: the hardware's 2^x and reciprocal (relative errors near
// 2^-22), and a polynomial for the normal distribution's tail.  The others use CUDA's functions.
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Phi(p), the normal distribution function, from its tail Phi(-|p|), so that nothing cancels for p < 0; not FAST as
// erfc(-p / sqrt 2) / 2.
// FAST: Phi(-x) = e^(-x^2 / 2) t (c1 + c2 t + ... + c7 t^6), t = 1 / (1 + 0.362 x), x >= 0.  The coefficients were fitted for the least
// largest relative error over x in [0, 14]: 7.5e-7.  Evaluated in fp32 it is 1.3e-6 up to x = 3 and, as x^2 in the exponent rounds,
// 7e-6 at 13, where the tail leaves fp32's normal numbers.  The relative error counts: gelu of a far negative p is p Phi(p), rounded
// to bf16 (half a step: 2e-3 to 4e-3).  e^(-x^2 / 2) is what the density is formed from too.
struct Normal {
    float cdf, density;
};
template <bool FAST>
__device__ __forceinline__ Normal normal(float p) {
    if (!FAST) return {0.5f * erfcf(p * -0.70710678118654752f), 0.39894228040143268f * expf(-0.5f * p * p)};
    const float e = fast_exp2(p * p * -0.72134752044448170f);   // log2(e) / 2
    const float t = fast_rcp(fmaf(0.362f, fabsf(p), 1.f));
    float q = fmaf(0.0479002930f, t, -0.179877907f);
    q = fmaf(q, t, 0.176436722f);
    q = fmaf(q, t, 0.0289549623f);
    q = fmaf(q, t, 0.139385894f);
    q = fmaf(q, t, 0.142696857f);
    q = fmaf(q, t, 0.144503415f);
    q *= t * e;   // Phi(-|p|)
    return {p < 0.f ? q : 1.f - q, 0.39894228040143268f * e};
}

// 2 sqrt(2/pi) (p + 0.044715 p^3): gelu with tanh is p sigmoid of this, (1 + tanh a) / 2 = sigmoid(2 a)
__device__ __forceinline__ float tanh_arg(float p) {
    return p * fmaf(2.f * 0.79788456080286536f * 0.044715f, p * p, 2.f * 0.79788456080286536f);
}
template <bool FAST>
__device__ __forceinline__ float sigmoid(float x) {
    return FAST ? fast_rcp(1.0f + fast_exp2(x * -1.4426950408889634f)) : 1.0f / (1.0f + expf(-x));
}

template <bool FAST>
__device__ __forceinline__ float act_value(int act, float p) {
    switch (act) {
        case LIGER_ACT_RELU: return p > 0.f ? p : (p != p ? p : 0.f);
        case LIGER_ACT_GELU: return p * normal<FAST>(p).cdf;
        case LIGER_ACT_GELU_TANH: return p * sigmoid<FAST>(tanh_arg(p));
        case LIGER_ACT_SILU: return p * sigmoid<FAST>(p);
        default: return p;
    }
}

// The same for 32 values, the choice made once.
template <bool FAST>
__device__ __forceinline__ void act_values(int act, float (&v)[32]) {
    auto each = [&](auto a) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = act_value<FAST>(decltype(a)::value, v[j]);
    };
    switch (act) {
        case LIGER_ACT_RELU: each(std::integral_constant<int, LIGER_ACT_RELU>()); break;
        case LIGER_ACT_GELU: each(std::integral_constant<int, LIGER_ACT_GELU>()); break;
        case LIGER_ACT_GELU_TANH: each(std::integral_constant<int, LIGER_ACT_GELU_TANH>()); break;
        case LIGER_ACT_SILU: each(std::integral_constant<int, LIGER_ACT_SILU>()); break;
        default: break;
    }
}

// What the backward's slope is formed from (kept by the forward): half precision beside bf16 tensors, fp32 beside fp32.
// Half precision holds 2^-24 to 65504.  Larger values (where every activation's slope has its limit) are kept as that, NaN as NaN.
// Smaller ones round to 0, which only relu's slope tells from them: there a positive sum is lifted to 2^-24 (RELU).  Both limits
// for all elements by comparisons took the forward of 8192 x 4096 x 11008 with gelu from 489 us to 571; the saturating conversion of
// pairs takes what a plain one does.
constexpr float kLeastHalf = 0x1p-24f;
template <bool RELU>
__device__ __forceinline__ uint32_t kept_pair(float lo, float hi) {
    if (RELU) {
        lo = lo > 0.f ? fmaxf(lo, kLeastHalf) : lo;
        hi = hi > 0.f ? fmaxf(hi, kLeastHalf) : hi;
    }
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void keep_pre(int, float* p, float v) { *p = v; }
__device__ __forceinline__ void keep_pre(int act, __half* p, float v) {
    *p = __ushort_as_half(static_cast<unsigned short>(act == LIGER_ACT_RELU ? kept_pair<true>(v, 0.f) : kept_pair<false>(v, 0.f)));
}

// d act / dp
template <bool FAST>
__device__ __forceinline__ float act_slope(int act, float p) {
    switch (act) {
        case LIGER_ACT_RELU: return p > 0.f ? 1.f : (p != p ? p : 0.f);
        case LIGER_ACT_GELU: {
            const Normal n = normal<FAST>(p);
            return fmaf(p, n.density, n.cdf);
        }
        case LIGER_ACT_GELU_TANH: {
            // s + p s (1 - s) d(arg)/dp; past 64 s is 0 or 1, and p^2 may be infinite (not that of a half-precision p)
            const float q = FAST ? p : p > 64.f ? 64.f : p < -64.f ? -64.f : p;
            const float s = sigmoid<FAST>(tanh_arg(q));
            const float d = fmaf(6.f * 0.79788456080286536f * 0.044715f, q * q, 2.f * 0.79788456080286536f);
            return fmaf(q * s * (1.f - s), d, s);
        }
        case LIGER_ACT_SILU: {
            const float s = sigmoid<FAST>(p);
            return s * fmaf(p, 1.f - s, 1.f);
        }
        default: return 1.f;
    }
}

}  // namespace
}  // namespace liger
