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

// one output: the sum v with its column's bias, `res` the residual there
template <typename TO, typename TPRE>
__device__ __forceinline__ void fma_store(const FmaGemm& g, const FmaEpi<TO, TPRE>& ep, int64_t m, int64_t n, float v, float bias, float res) {
    const int64_t o = m * g.N + n;
    v += bias;
    if (ep.pre != nullptr) keep_pre(ep.act, ep.pre + o, v);
    v = act_value<false>(ep.act, v);
    if (ep.residual != nullptr) v += res;
    stf(ep.out + o, v);
}

// Tiles of FM x FN by 16 x 16 threads, FK k at a time through two shared buffers, the next ones loaded to registers while
// these are used.  The arithmetic is on column pairs with the packed fp32x2 fma.  Consecutive threads load consecutive
// elements of an operand's contiguous dimension; inside the matrices without checks.  K is split over a cluster of blocks,
// whose tiles are joined in order over distributed shared memory (not for 128 x 128, whose sums do not fit).  Bound by fma issue
// beside the shared-memory reads, the less the larger the tile, and by how evenly the blocks fill the SMs (fma_us below).
// 16 x 64: up to 16 rows; 4 x 2048 x 2048 in 17.8 us, 32.9 in tiles of 64 rows.
template <int FM, int FN>
struct FmaTile {
    static constexpr int FK = 16;
    static constexpr bool SPLIT = FM * FN <= 8192;   // its sums fit the shared memory, for a join over a cluster
    static constexpr int SA = FM + 4, SB = FN + 4;   // words of a shared row of k
    static constexpr int BUFS = 2 * FK * (SA + SB), WORDS = SPLIT && BUFS < FM * FN ? FM * FN : BUFS;
};
// A launch holds one product or two that do not depend on each other (JOBS): the blocks from `first` on are the second's.
template <typename TA, typename TB, typename TO, typename TPRE>
struct FmaJob {
    const TA* A;
    const TB* B;
    FmaGemm g;
    FmaEpi<TO, TPRE> ep;
};
template <typename TA, typename TB, typename TO, typename TPRE, int FM, int FN, int JOBS>
__global__ void __launch_bounds__(256, FN == 128 ? 2 : 3)
    fma_gemm(const FmaJob<TA, TB, TO, TPRE> job0, const FmaJob<TA, TB, TO, TPRE> job1, unsigned first) {
    using Tile = FmaTile<FM, FN>;
    constexpr int FK = Tile::FK, SA = Tile::SA, SB = Tile::SB, PM = FM / 16, PN = FN / 16;
    constexpr int NA = FM * FK / 256, NB = FN * FK / 256;   // elements of an operand that a thread loads a step
    __shared__ __align__(16) float mem[Tile::WORDS];   // two buffers of A, two of B; then the tile of sums
    float* const sa = mem;
    float* const sb = mem + 2 * FK * SA;
    const uint32_t rank = block_in_cluster(), ranks = blocks_in_cluster();
    const bool second = JOBS == 2 && blockIdx.x >= first;
    const FmaGemm g = second ? job1.g : job0.g;
    const FmaEpi<TO, TPRE> ep = second ? job1.ep : job0.ep;
    const TA* const A = second ? job1.A : job0.A;
    const TB* const B = second ? job1.B : job0.B;
    const unsigned tn = (static_cast<unsigned>(g.N) + FN - 1) / FN, tile = (blockIdx.x - (second ? first : 0)) / ranks, tile_m = tile / tn;
    const int64_t m0 = static_cast<int64_t>(tile_m) * FM, n0 = static_cast<int64_t>(tile - tile_m * tn) * FN;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int steps = (g.K + FK - 1) / FK;
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * rank / ranks) * FK;
    const int k1 = min(g.K, static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / ranks) * FK);
    wait_for_stream();
    // k contiguous: FK threads along k, the elements of a thread 256 / FK rows apart; else the rows' threads side by
    // side, and 256 / F k apart
    const bool ak = g.sak == 1, bk = g.sbk == 1;
    const int am = ak ? tid / FK : tid % FM, ka = ak ? tid % FK : tid / FM, am_i = ak ? 256 / FK : 0, ka_i = ak ? 0 : 256 / FM;
    const int bn = bk ? tid / FK : tid % FN, kb = bk ? tid % FK : tid / FN, bn_i = bk ? 256 / FK : 0, kb_i = bk ? 0 : 256 / FN;
    const TA* pa = A + (m0 + am) * g.sam + (k0 + ka) * g.sak;   // this thread's first elements of the next step
    const TB* pb = B + (n0 + bn) * g.sbn + (k0 + kb) * g.sbk;
    const int64_t da = am_i * g.sam + ka_i * g.sak, db = bn_i * g.sbn + kb_i * g.sbk, step_a = FK * g.sak, step_b = FK * g.sbk;
    const bool inside = m0 + FM <= g.M && n0 + FN <= g.N;
    uint32_t va = 0, vb = 0;   // which of this thread's rows and columns are inside
#pragma unroll
    for (int i = 0; i < NA; ++i) va |= m0 + am + i * am_i < g.M ? 1u << i : 0u;
#pragma unroll
    for (int i = 0; i < NB; ++i) vb |= n0 + bn + i * bn_i < g.N ? 1u << i : 0u;
    float ra[NA], rb[NB];
    auto fetch = [&](int k) {
        const TA* qa = pa;
        const TB* qb = pb;
        if (inside && k + FK <= k1) {
#pragma unroll
            for (int i = 0; i < NA; ++i, qa += da) ra[i] = ldf(qa);
#pragma unroll
            for (int i = 0; i < NB; ++i, qb += db) rb[i] = ldf(qb);
        } else if (k + FK <= k1) {
#pragma unroll
            for (int i = 0; i < NA; ++i, qa += da) ra[i] = va >> i & 1u ? ldf(qa) : 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i, qb += db) rb[i] = vb >> i & 1u ? ldf(qb) : 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < NA; ++i, qa += da) ra[i] = (va >> i & 1u) && k + ka + i * ka_i < k1 ? ldf(qa) : 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i, qb += db) rb[i] = (vb >> i & 1u) && k + kb + i * kb_i < k1 ? ldf(qb) : 0.f;
        }
        pa += step_a;
        pb += step_b;
    };
    // in shared memory: A's element at row k, its row's place twice; B's once
    const int wa = ka * SA + am, wa_i = ka_i * SA + am_i, wb = kb * SB + bn, wb_i = kb_i * SB + bn_i;
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < NA; ++i) sa[buf * FK * SA + wa + i * wa_i] = ra[i];
#pragma unroll
        for (int i = 0; i < NB; ++i) sb[buf * FK * SB + wb + i * wb_i] = rb[i];
    };
    // a thread's outputs: rows ty * 4 + (0 .. 3) of each 64 rows (or row ty of 16), columns tx * 4 + (0 .. 3) of each 64
    float2 acc[PM][PN / 2];
#pragma unroll
    for (int i = 0; i < PM; ++i)
#pragma unroll
        for (int j = 0; j < PN / 2; ++j) acc[i][j] = make_float2(0.f, 0.f);
    int buf = 0;
    fetch(k0);
    put(0);
    __syncthreads();
    for (int k = k0; k < k1; k += FK) {
        const bool more = k + FK < k1;
        if (more) fetch(k + FK);
        const float* ca = sa + buf * FK * SA;
        const float* cb = sb + buf * FK * SB;
#pragma unroll
        for (int kk = 0; kk < FK; ++kk) {
            float2 av[PM], bv[PN / 2];
            if constexpr (PM == 1) {
                const float q = ca[kk * SA + ty];
                av[0] = make_float2(q, q);
            } else {
#pragma unroll
                for (int h = 0; h < PM / 4; ++h) {
                    const float4 q = *reinterpret_cast<const float4*>(ca + kk * SA + h * 64 + ty * 4);
                    av[4 * h] = make_float2(q.x, q.x);
                    av[4 * h + 1] = make_float2(q.y, q.y);
                    av[4 * h + 2] = make_float2(q.z, q.z);
                    av[4 * h + 3] = make_float2(q.w, q.w);
                }
            }
#pragma unroll
            for (int h = 0; h < PN / 4; ++h) {
                const float4 q = *reinterpret_cast<const float4*>(cb + kk * SB + h * 64 + tx * 4);
                bv[2 * h] = make_float2(q.x, q.y);
                bv[2 * h + 1] = make_float2(q.z, q.w);
            }
#pragma unroll
            for (int i = 0; i < PM; ++i)
#pragma unroll
                for (int j = 0; j < PN / 2; ++j) acc[i][j] = __ffma2_rn(av[i], bv[j], acc[i][j]);
        }
        if (more) put(buf ^ 1);   // last read before the barrier of the step before
        __syncthreads();
        buf ^= 1;
    }
    auto row_of = [&](int i) { return PM == 1 ? ty : (i / 4) * 64 + ty * 4 + i % 4; };
    // the bias and the residual are asked for ahead of the stores, behind which their loads would wait (the residual may be the output)
    auto col_of = [&](int j) { return n0 + (j / 4) * 64 + tx * 4 + j % 4; };
    float bias[PN];
#pragma unroll
    for (int j = 0; j < PN; ++j) bias[j] = ep.bias != nullptr && col_of(j) < g.N ? ldf(ep.bias + col_of(j)) : 0.f;
    if constexpr (Tile::SPLIT) {
        if (ranks > 1) {
            // the tile into shared memory, and rows rank, rank + ranks, ... of the cluster's sums out of it
#pragma unroll
            for (int i = 0; i < PM; ++i)
                *reinterpret_cast<float4*>(mem + row_of(i) * FN + tx * 4) = make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
            __syncthreads();
            cluster_barrier();
            for (int m = static_cast<int>(rank) + static_cast<int>(ranks) * ty; m < FM && m0 + m < g.M; m += static_cast<int>(ranks) * 16) {
                float4 v[8];
                float res[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    res[j] = ep.residual != nullptr && col_of(j) < g.N ? ldf(ep.residual + (m0 + m) * g.N + col_of(j)) : 0.f;
#pragma unroll
                for (uint32_t q = 0; q < 8; ++q)
                    if (q < ranks) v[q] = peer_float4(mem + m * FN + tx * 4, q);
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
                    if (col_of(j) < g.N) fma_store(g, ep, m0 + m, col_of(j), o[j], bias[j], res[j]);
            }
            __syncwarp();
            cluster_barrier();   // no block exits while another reads its sums
            return;
        }
    }
    constexpr int ROWS = PM < 4 ? PM : PM == 4 ? 4 : 2;
#pragma unroll
    for (int i0 = 0; i0 < PM; i0 += ROWS) {
        float res[ROWS][PN];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < PN; ++j) {
                const int64_t m = m0 + row_of(i0 + i), n = col_of(j);
                res[i][j] = ep.residual != nullptr && m < g.M && n < g.N ? ldf(ep.residual + m * g.N + n) : 0.f;
            }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < PN; ++j) {
                const int64_t m = m0 + row_of(i0 + i), n = col_of(j);
                if (m < g.M && n < g.N) fma_store(g, ep, m, n, j % 2 ? acc[i0 + i][j / 2].y : acc[i0 + i][j / 2].x, bias[j], res[i][j]);
            }
    }
}

// What the blocks of a tile shape take with K split over `ranks` of them, in us, from measurements: the SM with the most blocks
// has their k to do, at a lower rate where it has one block alone, and each block's start, join and end.  Measured (and by
// this, with 3 for the launch), in 64 x 64 over 1, 2, 4, 8 blocks: 1024^3 72, 77, 71, 80 (76, 78, 73, 83); 2000 x 700 x 300 53, 42,
// 38, 44 (54, 42, 40, 42); 100 x 1000 x 1000 49, 28, 16, 13 (50, 28, 16, 14); in 128 x 64: 1024^3 84, 71, 70, 74 (100, 68, 72, 74);
// 1600^3 299, 251, 224, 253 (293, 250, 235, 255), in 64 x 64 over 4 240 (258), in 128 x 128 347 (324); 2048^3 in 128 x 128 411 (412).
struct FmaShape {
    int m, n;
    double us_k, alone, us_block;
};
constexpr FmaShape kFmaShapes[3] = {{64, 64, 0.0342, 1.33, 1.35}, {128, 64, 0.059, 1.57, 2.2}, {128, 128, 0.098, 1.15, 3.9}};
struct FmaPlan {
    int shape = 0, ranks = 1;
    double us = 1e30;
};
inline int64_t fma_tiles(const FmaShape& s, const FmaGemm& g) { return ceil_div(g.M, s.m) * static_cast<int64_t>(ceil_div(g.N, s.n)); }
// the plan for one product, or for two in one launch (in 64 x 64: in larger tiles the second product's parameters spill)
inline FmaPlan fma_plan(const FmaGemm& g0, const FmaGemm* g1) {
    FmaPlan best;
    for (int i = 0; i < (g1 != nullptr ? 1 : 3); ++i)
        for (int r = 1; r <= (i == 2 ? 1 : 8); r *= 2) {
            const FmaShape& s = kFmaShapes[i];
            const int64_t n0 = fma_tiles(s, g0) * r, n1 = g1 != nullptr ? fma_tiles(s, *g1) * r : 0;
            const int64_t on = ceil_div(n0 + n1, static_cast<int64_t>(sm_count()));
            bool enough = true;
            auto us = [&](int K) {
                enough = enough && (r == 1 || K >= 24 * r);
                return s.us_k * (on == 1 ? s.alone * 16 * static_cast<double>(ceil_div(ceil_div(K, 16), r)) : static_cast<double>(K) / r) + s.us_block;
            };
            const double u0 = us(g0.K), u1 = g1 != nullptr ? us(g1->K) : 0.0;
            // the SM's share of the work, and no less than its longest block beside two others
            const double t = on == 1 ? std::max(u0, u1)
                                     : std::max(static_cast<double>(on) * (n0 * u0 + n1 * u1) / static_cast<double>(n0 + n1),
                                                static_cast<double>(std::min<int64_t>(on, 3)) * std::max(u0, u1) * (g1 != nullptr ? 1.0 : 0.0));
            if (enough && t < best.us) best = {i, r, t};
        }
    return best;
}

template <typename TA, typename TB, typename TO, typename TPRE>
int launch_fma_plan(const char* who, const FmaJob<TA, TB, TO, TPRE>& a, const FmaPlan& plan, cudaStream_t st) {
    const FmaShape& s = kFmaShapes[plan.shape];
    const unsigned first = static_cast<unsigned>(fma_tiles(s, a.g) * plan.ranks);
    const dim3 grid(first), cluster(static_cast<unsigned>(plan.ranks));
    if (plan.shape == 0) return launch_cluster(who, fma_gemm<TA, TB, TO, TPRE, 64, 64, 1>, grid, cluster, 256, 0, st, a, a, first);
    if (plan.shape == 1) return launch_cluster(who, fma_gemm<TA, TB, TO, TPRE, 128, 64, 1>, grid, cluster, 256, 0, st, a, a, first);
    return launch_early(who, fma_gemm<TA, TB, TO, TPRE, 128, 128, 1>, grid, 256, 0, st, a, a, first);
}

template <typename TA, typename TB, typename TO, typename TPRE>
int launch_fma_gemm(const char* who, const FmaJob<TA, TB, TO, TPRE>& a, cudaStream_t st) {
    if (a.g.M > 16) return launch_fma_plan(who, a, fma_plan(a.g, nullptr), st);
    // K over so many blocks that all of them are still resident at once (three on an SM), 64 k at least each
    const int64_t n = ceil_div(a.g.N, 64);
    int ranks = 1;
    while (ranks < 8 && 2 * n * ranks <= 3 * sm_count() && a.g.K >= 128 * ranks) ranks *= 2;
    return launch_cluster(who, fma_gemm<TA, TB, TO, TPRE, 16, 64, 1>, dim3(static_cast<unsigned>(n * ranks)), dim3(static_cast<unsigned>(ranks)),
                          256, 0, st, a, a, static_cast<unsigned>(n * ranks));
}

// Two products that do not depend on each other, in one launch where that is estimated to take less (well less, where their sums
// differ much in length: the estimate is poor there): both are bound by the latencies of their few steps, and share them.
template <typename TA, typename TB, typename TO, typename TPRE>
int launch_fma_two(const char* who, const FmaJob<TA, TB, TO, TPRE>& a, const FmaJob<TA, TB, TO, TPRE>& b, cudaStream_t st) {
    if (a.g.M > 16 && b.g.M > 16) {
        const bool longer = a.g.K >= b.g.K;   // the longer blocks start first
        const FmaJob<TA, TB, TO, TPRE>&p = longer ? a : b, &q = longer ? b : a;
        const FmaPlan both = fma_plan(p.g, &q.g);
        const double margin = 2 * static_cast<int64_t>(q.g.K) >= p.g.K ? 1.0 : 0.85;
        if (both.us < margin * (fma_plan(a.g, nullptr).us + fma_plan(b.g, nullptr).us + 3.0)) {
            const unsigned first = static_cast<unsigned>(fma_tiles(kFmaShapes[0], p.g) * both.ranks);
            return launch_cluster(who, fma_gemm<TA, TB, TO, TPRE, 64, 64, 2>,
                                  dim3(first + static_cast<unsigned>(fma_tiles(kFmaShapes[0], q.g) * both.ranks)),
                                  dim3(static_cast<unsigned>(both.ranks)), 256, 0, st, p, q, first);
        }
    }
    if (int rc = launch_fma_gemm(who, a, st)) return rc;
    return launch_fma_gemm(who, b, st);
}

}  // namespace
}  // namespace liger
