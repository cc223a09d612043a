// Products in fp32 FMA, for fp32 tensors and for bf16 sizes that the tensor path does not take:
// C[m, n] = sum_k A(m, k) B(k, n), any strides, then the projection's epilogue.
#pragma once

#include "activation.cuh"
#include "cluster.cuh"

namespace liger {
namespace {


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

template <typename TO, typename TPRE>
__device__ __forceinline__ void fma_store(const FmaGemm& g, const FmaEpi<TO, TPRE>& ep, int64_t m, int64_t n, float v) {
    const int64_t o = m * g.N + n;
    if (ep.bias != nullptr) v += ldf(ep.bias + n);
    if (ep.pre != nullptr) keep_pre(ep.pre + o, v);
    v = act_value<false>(ep.act, v);
    if (ep.residual != nullptr) v += ldf(ep.residual + o);
    stf(ep.out + o, v);
}

// Tiles of FT x FT, 256 threads with FT / 16 squared outputs each, kFK k at a time (fp32: 8 KB of an operand) through two shared
// buffers, the next ones loaded to registers while these are used.  FT = 128: 64 FMA for 16 values read (bound by FMA issue).  FT = 64,
// for fewer outputs: K split over a cluster of blocks, whose tiles are joined in order over distributed shared memory.
template <typename TA, typename TB, typename TO, typename TPRE, int FT>
__global__ void __launch_bounds__(256, FT == 64 ? 3 : 2) fma_gemm(const TA* A, const TB* B, FmaGemm g, FmaEpi<TO, TPRE> ep) {
    constexpr int kFK = 2048 / FT;
    constexpr int PT = FT / 16;             // outputs of a thread in each direction
    constexpr int LD = FT * kFK / 256;      // elements of an operand that a thread loads a step
    struct Bufs {
        float A[2][kFK][FT + 4], B[2][kFK][FT + 4];
    };
    constexpr int WORDS = sizeof(Bufs) / 4 > FT * FT ? sizeof(Bufs) / 4 : FT * FT;   // (the tile of sums: FT = 64 only)
    __shared__ __align__(16) float mem[FT == 64 ? WORDS : sizeof(Bufs) / 4];
    Bufs& s = *reinterpret_cast<Bufs*>(mem);
    const uint32_t rank = block_in_cluster(), ranks = blocks_in_cluster();
    const unsigned tn = (static_cast<unsigned>(g.N) + FT - 1) / FT, tile = blockIdx.x / ranks, tile_m = tile / tn;
    const int64_t m0 = static_cast<int64_t>(tile_m) * FT, n0 = static_cast<int64_t>(tile - tile_m * tn) * FT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int steps = (g.K + kFK - 1) / kFK;
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * rank / ranks) * kFK;
    const int k1 = min(g.K, static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / ranks) * kFK);
    wait_for_stream();
    // consecutive threads take consecutive elements of each operand's contiguous dimension: element i of a thread
    // stands im, ik further along
    const bool ak = g.sak == 1, bn = g.sbn == 1;
    const int tid = threadIdx.x;
    const int am = ak ? tid / kFK : tid % FT, ka = ak ? tid % kFK : tid / FT, aim = ak ? 256 / kFK : 0, aik = ak ? 0 : 256 / FT;
    const int nb = bn ? tid % FT : tid / kFK, kb = bn ? tid / FT : tid % kFK, bin = bn ? 0 : 256 / kFK, bik = bn ? 256 / FT : 0;
    const TA* pa = A + (m0 + am) * g.sam + ka * g.sak;
    const TB* pb = B + (n0 + nb) * g.sbn + kb * g.sbk;
    const int64_t ai = aim * g.sam + aik * g.sak, bi = bin * g.sbn + bik * g.sbk;
    float ra[LD], rb[LD];
    auto fetch = [&](int k) {
        const TA* qa = pa + k * g.sak;
        const TB* qb = pb + k * g.sbk;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            ra[i] = m0 + am + i * aim < g.M && k + ka + i * aik < k1 ? ldf(qa + i * ai) : 0.f;
            rb[i] = n0 + nb + i * bin < g.N && k + kb + i * bik < k1 ? ldf(qb + i * bi) : 0.f;
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            s.A[buf][ka + i * aik][am + i * aim] = ra[i];
            s.B[buf][kb + i * bik][nb + i * bin] = rb[i];
        }
    };
    // a thread's outputs: rows ty * 4 + (0 .. 3) of each half of 64 rows, columns tx * 4 + (0 .. 3) likewise
    float acc[PT][PT] = {};
    int buf = 0;
    fetch(k0);
    put(0);
    __syncthreads();
    for (int k = k0; k < k1; k += kFK) {
        const bool more = k + kFK < k1;
        if (more) fetch(k + kFK);
#pragma unroll
        for (int kk = 0; kk < kFK; ++kk) {
            float av[PT], bv[PT];
#pragma unroll
            for (int h = 0; h < PT / 4; ++h) {
                *reinterpret_cast<float4*>(av + 4 * h) = *reinterpret_cast<const float4*>(&s.A[buf][kk][h * 64 + ty * 4]);
                *reinterpret_cast<float4*>(bv + 4 * h) = *reinterpret_cast<const float4*>(&s.B[buf][kk][h * 64 + tx * 4]);
            }
#pragma unroll
            for (int i = 0; i < PT; ++i)
#pragma unroll
                for (int j = 0; j < PT; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        if (more) put(buf ^ 1);   // last read before the barrier of the step before
        __syncthreads();
        buf ^= 1;
    }
    if (FT == 64 && ranks > 1) {
        // the tile into shared memory, and rows rank, rank + ranks, ... of the cluster's sums out of it
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(mem + (ty * 4 + i) * 64 + tx * 4) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        __syncthreads();
        cluster_barrier();
        for (int m = static_cast<int>(rank) + static_cast<int>(ranks) * ty; m < 64; m += static_cast<int>(ranks) * 16) {
            if (m0 + m >= g.M) break;
            float4 v[8];
#pragma unroll
            for (uint32_t q = 0; q < 8; ++q)
                if (q < ranks) v[q] = peer_float4(mem + m * 64 + tx * 4, q);
#pragma unroll
            for (uint32_t q = 1; q < 8; ++q)
                if (q < ranks) {
                    v[0].x += v[q].x;
                    v[0].y += v[q].y;
                    v[0].z += v[q].z;
                    v[0].w += v[q].w;
                }
            const float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n0 + tx * 4 + j < g.N) fma_store(g, ep, m0 + m, n0 + tx * 4 + j, o[j]);
        }
        __syncwarp();
        cluster_barrier();   // no block exits while another reads its sums
        return;
    }
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int64_t m = m0 + (i / 4) * 64 + ty * 4 + i % 4;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            const int64_t n = n0 + (j / 4) * 64 + tx * 4 + j % 4;
            if (n < g.N) fma_store(g, ep, m, n, acc[i][j]);
        }
    }
}

template <typename TA, typename TB, typename TO, typename TPRE>
int launch_fma_gemm(const char* who, const TA* A, const TB* B, const FmaGemm& g, const FmaEpi<TO, TPRE>& ep, cudaStream_t st) {
    auto tiles = [&](int ft) { return ceil_div(g.M, ft) * ceil_div(g.N, ft); };
    if (tiles(128) >= sm_count())
        return launch_early(who, fma_gemm<TA, TB, TO, TPRE, 128>, dim3(static_cast<unsigned>(tiles(128))), 256, 0, st, A, B, g, ep);
    // K over so many blocks that every SM has at most one, 64 k at least each
    int ranks = 1;
    while (ranks < 8 && 2 * tiles(64) * ranks <= sm_count() && g.K >= 128 * ranks) ranks *= 2;
    return launch_cluster(who, fma_gemm<TA, TB, TO, TPRE, 64>, dim3(static_cast<unsigned>(tiles(64) * ranks)),
                          dim3(static_cast<unsigned>(ranks)), 256, 0, st, A, B, g, ep);
}

}  // namespace
}  // namespace liger
