// Products in fp32 FMA, for fp32 tensors and for bf16 sizes that the tensor path does not take:
// C[m, n] = sum_k A(m, k) B(k, n), any strides, then the projection's epilogue.
#pragma once

#include "activation.cuh"
#include "common.cuh"

namespace liger {
namespace {

constexpr int kFT = 64, kFK = 16;   // tile of C, k at a time

struct FmaGemm {
    int M, N, K;
    int64_t sam, sak, sbk, sbn;
};

// out = act(C + bias) + residual [M, N]; pre: C + bias
template <typename TO, typename TPRE>
struct FmaEpi {
    const TO* bias;
    const TO* residual;
    TO* out;
    TPRE* pre;
    int act;
};

template <typename TA, typename TB, typename TO, typename TPRE>
__global__ void __launch_bounds__(256) fma_gemm(const TA* A, const TB* B, FmaGemm g, FmaEpi<TO, TPRE> ep) {
    __shared__ __align__(16) float As[2][kFK][kFT + 4], Bs[2][kFK][kFT + 4];
    const unsigned tn = (static_cast<unsigned>(g.N) + kFT - 1) / kFT, tile_m = blockIdx.x / tn;
    const int64_t m0 = static_cast<int64_t>(tile_m) * kFT, n0 = static_cast<int64_t>(blockIdx.x - tile_m * tn) * kFT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    wait_for_stream();
    // consecutive threads take consecutive elements of each operand's contiguous dimension
    const bool ak = g.sak == 1, bn = g.sbn == 1;
    float ra[4], rb[4];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = threadIdx.x + i * 256;
            const int mm = ak ? e / kFK : e % kFT, ka = ak ? e % kFK : e / kFT;
            const int nn = bn ? e % kFT : e / kFK, kb = bn ? e / kFT : e % kFK;
            ra[i] = m0 + mm < g.M && k + ka < g.K ? ldf(A + (m0 + mm) * g.sam + (k + ka) * g.sak) : 0.f;
            rb[i] = n0 + nn < g.N && k + kb < g.K ? ldf(B + (k + kb) * g.sbk + (n0 + nn) * g.sbn) : 0.f;
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = threadIdx.x + i * 256;
            As[buf][ak ? e % kFK : e / kFT][ak ? e / kFK : e % kFT] = ra[i];
            Bs[buf][bn ? e / kFT : e % kFK][bn ? e % kFT : e / kFK] = rb[i];
        }
    };
    float acc[4][4] = {};
    int buf = 0;
    fetch(0);
    put(0);
    __syncthreads();
    for (int k = 0; k < g.K; k += kFK) {
        const bool more = k + kFK < g.K;
        if (more) fetch(k + kFK);
#pragma unroll
        for (int kk = 0; kk < kFK; ++kk) {
            const float4 a = *reinterpret_cast<const float4*>(&As[buf][kk][ty * 4]);
            const float4 b = *reinterpret_cast<const float4*>(&Bs[buf][kk][tx * 4]);
            const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        if (more) put(buf ^ 1);   // last read before the barrier of the step before
        __syncthreads();
        buf ^= 1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            if (n >= g.N) continue;
            const int64_t o = m * g.N + n;
            float v = acc[i][j];
            if (ep.bias != nullptr) v += ldf(ep.bias + n);
            if (ep.pre != nullptr) keep_pre(ep.pre + o, v);
            v = act_value<false>(ep.act, v);
            if (ep.residual != nullptr) v += ldf(ep.residual + o);
            stf(ep.out + o, v);
        }
    }
}

template <typename TA, typename TB, typename TO, typename TPRE>
int launch_fma_gemm(const char* who, const TA* A, const TB* B, const FmaGemm& g, const FmaEpi<TO, TPRE>& ep, cudaStream_t st) {
    const int64_t tm = ceil_div(g.M, kFT), tn = ceil_div(g.N, kFT);
    return launch_early(who, fma_gemm<TA, TB, TO, TPRE>, dim3(static_cast<unsigned>(tn * tm)), 256, 0, st, A, B, g, ep);
}

}  // namespace
}  // namespace liger
