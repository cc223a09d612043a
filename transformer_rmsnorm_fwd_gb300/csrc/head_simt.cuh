// fp32 products of the heads off the tensor cores (fp32, and bf16 shapes that
// TMA cannot take): C[m, n] = sum_k A(m, k) B(k, n), any strides, fp32 FMA.
//
// 64 x 64 tiles, 256 threads with 4 x 4 each, 16 k at a time through two
// shared-memory buffers, the next 16 loaded to registers while these are used.
// Small products have few tiles, so K is split over up to 32 blocks per tile:
// partial tiles go to the workspace and a second kernel adds them in order
// (256 x 256 outputs over K = 1024 in fp32: 15 us with the join, 58 us from 32 x 32 tiles without
// a split).  Bound by FMA issue when large, by latency when small.
#pragma once

#include "common.cuh"

namespace liger {
namespace {

constexpr int kHT = 64, kHK = 16;
constexpr int64_t kHeadRows = 65535 * kHT;           // most rows of a product (grid limit)
constexpr int64_t kSplitFloats = int64_t{1} << 22;   // workspace of the partial tiles

struct HeadGemm {
    int M, N, K;
    int64_t sam, sak, sbk, sbn, ldo;
    int splits, k_per;        // K split into `splits` runs of k_per (a multiple of kHK)
    float* part;              // [splits][M][N] when splits > 1
    const int64_t* labels;    // rows labelled `ignore` are written +0 (NULL: none)
    const int64_t* klabels;   // B's rows k labelled `ignore` count as zeros, whatever they hold (NULL: none)
    int64_t ignore;
    int add;                  // out += (fp32 outputs)
    const float* base;        // added before the store (the sum of earlier chunks), ldo apart, or NULL
};

template <typename TO>
__device__ __forceinline__ void head_store(const HeadGemm& g, TO* out, int m, int n, float v) {
    const int64_t o = static_cast<int64_t>(m) * g.ldo + n;
    if (g.labels != nullptr && g.labels[m] == g.ignore) v = 0.f;
    if (g.base != nullptr) v += g.base[o];
    if (g.add) v += ldf(out + o);
    stf(out + o, v);
}

template <typename TA, typename TB, typename TO>
__global__ void __launch_bounds__(256) head_gemm(const TA* A, const TB* B, TO* out, HeadGemm g) {
    __shared__ __align__(16) float As[2][kHK][kHT + 4], Bs[2][kHK][kHT + 4];
    const int m0 = blockIdx.y * kHT, n0 = blockIdx.x * kHT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int k0 = blockIdx.z * g.k_per, k1 = min(g.K, k0 + g.k_per);
    wait_for_stream();
    // consecutive threads take consecutive elements of each operand's contiguous dimension
    const bool ak = g.sak == 1, bn = g.sbn == 1;
    float ra[4], rb[4];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = threadIdx.x + i * 256;
            const int mm = ak ? e / kHK : e % kHT, ka = ak ? e % kHK : e / kHT;
            const int nn = bn ? e % kHT : e / kHK, kb = bn ? e / kHT : e % kHK;
            ra[i] = m0 + mm < g.M && k + ka < k1 ? ldf(A + (m0 + mm) * g.sam + (k + ka) * g.sak) : 0.f;
            const bool in = n0 + nn < g.N && k + kb < k1;
            rb[i] = in ? ldf(B + (k + kb) * g.sbk + (n0 + nn) * g.sbn) : 0.f;
            if (g.klabels != nullptr && in && g.klabels[k + kb] == g.ignore) rb[i] = 0.f;
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = threadIdx.x + i * 256;
            As[buf][ak ? e % kHK : e / kHT][ak ? e / kHK : e % kHT] = ra[i];
            Bs[buf][bn ? e / kHT : e % kHK][bn ? e % kHT : e / kHK] = rb[i];
        }
    };
    float acc[4][4] = {};
    int buf = 0;
    if (k0 < k1) {
        fetch(k0);
        put(0);
    }
    __syncthreads();
    for (int k = k0; k < k1; k += kHK) {
        const bool more = k + kHK < k1;
        if (more) fetch(k + kHK);
#pragma unroll
        for (int kk = 0; kk < kHK; ++kk) {
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
        const int m = m0 + ty * 4 + i;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= g.N) continue;
            if (g.splits > 1) g.part[(static_cast<int64_t>(blockIdx.z) * g.M + m) * g.N + n] = acc[i][j];
            else head_store(g, out, m, n, acc[i][j]);
        }
    }
}

template <typename TO>
__global__ void __launch_bounds__(256) head_join(TO* out, HeadGemm g) {
    const int64_t mn = static_cast<int64_t>(g.M) * g.N;
    wait_for_stream();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < mn; i += static_cast<int64_t>(gridDim.x) * 256) {
        float v = 0.f;
#pragma unroll 4
        for (int s = 0; s < g.splits; ++s) v += g.part[s * mn + i];
        const int m = static_cast<int>(i / g.N);
        head_store(g, out, m, static_cast<int>(i - static_cast<int64_t>(m) * g.N), v);
    }
}

// part: kSplitFloats floats
template <typename TA, typename TB, typename TO>
int launch_head_gemm(const TA* A, const TB* B, TO* out, HeadGemm g, float* part, cudaStream_t st) {
    if (g.M == 0 || g.N == 0) return LIGER_OK;
    const int64_t tm = ceil_div(g.M, kHT), tn = ceil_div(g.N, kHT);
    const int64_t fit = kSplitFloats / (static_cast<int64_t>(g.M) * g.N);
    int64_t splits = std::min<int64_t>({ceil_div(2 * sm_count(), tm * tn), ceil_div(g.K, 2 * kHK), fit, 32});
    if (splits < 2) splits = 1;
    g.k_per = static_cast<int>(ceil_div(ceil_div(g.K, splits), kHK) * kHK);
    g.splits = static_cast<int>(std::max<int64_t>(1, ceil_div(g.K, g.k_per)));
    g.part = part;
    const dim3 grid(static_cast<unsigned>(tn), static_cast<unsigned>(tm), static_cast<unsigned>(g.splits));
    if (int rc = launch_early("head_gemm", head_gemm<TA, TB, TO>, grid, 256, 0, st, A, B, out, g)) return rc;
    if (g.splits > 1) {
        const int64_t mn = static_cast<int64_t>(g.M) * g.N;
        const dim3 blocks(static_cast<unsigned>(std::min<int64_t>(ceil_div(mn, 256), 8 * sm_count())));
        return launch_early("head_join", head_join<TO>, blocks, 256, 0, st, out, g);
    }
    return LIGER_OK;
}

}  // namespace
}  // namespace liger
