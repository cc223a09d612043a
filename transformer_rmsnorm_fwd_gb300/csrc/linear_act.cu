// The projection with bias, activation and residual sum in its epilogue, and its
// backward (formulas in liger_layer.h).
// Y = act(X W^T + b) + R is one GEMM with the rest in its epilogue; the backward is one pass dP = dY act'(P) with db, then
// dX = dP W and dW = dP^T X.  bf16 goes on the tensor cores, in 256 x 256 tiles of CTA pairs (tc_gemm.cuh) or, with few tiles, in
// 128-feature tiles (linear_small.cuh); fp32 and sizes of no whole vectors on fp32 FMA (linear_fma.cuh).  8192 x 4096 x 11008 bf16
// with gelu: forward 412 us (1790 TFLOP/s), dP and db 91, dW 390, dX 393: the tensor pipe under the power cap; 4 tokens: 19 us from
// a cold L2, the weight's 90 MB.
#include "activation.cuh"
#include "linear_fma.cuh"
#include "linear_small.cuh"

namespace liger {
namespace {

constexpr int64_t kSmallTokens = 128;
constexpr unsigned kDpShares = 8;   // most blocks of a cluster that share the rows of a column sum
constexpr int64_t kDpLong = 2048, kDpParts = 64;
constexpr int kDpRows = 3;   // 8192 x 11008 with gelu: 95 us, 210 with one row in flight and erfcf

// dP = dY act'(P) and db, in one pass: a block takes some columns and its share of the rows, the blocks of a
// cluster all rows of the same columns.  The column sums go from threads to the block over shared memory, and
// over the cluster in the order of its blocks: no partial rows in device memory, no second kernel.
// From kDpLong rows on a cluster's blocks have too many each: more blocks, no cluster, each leaves its sums as a partial row in
// the workspace, and linear_db adds those in their order.  2048 x 4096: 12.2 us so, 18.3 by clusters; 1024 x 4096 10.3 and 10.0;
// 1111 x 520 6.1 and 4.3.

// The cluster's column sums into db: `mine` holds this block's for columns [col0, col0 + n).
template <typename T>
__device__ __forceinline__ void join_db(const float* mine, T* db, float* part, int64_t col0, int n, int cols) {
    const uint32_t ranks = blocks_in_cluster();
    __syncthreads();
    if (part != nullptr) {
        for (int i = threadIdx.x; i < n; i += blockDim.x)
            if (col0 + i < cols) part[static_cast<int64_t>(blockIdx.y) * cols + col0 + i] = mine[i];
        return;
    }
    if (ranks > 1) cluster_barrier();
    if (block_in_cluster() == 0)
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            float v[kDpShares];
#pragma unroll
            for (uint32_t q = 0; q < kDpShares; ++q)
                if (q < ranks) v[q] = ranks > 1 ? peer_float(mine + i, q) : mine[i];
#pragma unroll
            for (uint32_t q = 1; q < kDpShares; ++q)
                if (q < ranks) v[0] += v[q];
            if (col0 + i < cols) stf(db + col0 + i, v[0]);
        }
    __syncwarp();
    if (ranks > 1) cluster_barrier();   // no block exits while another reads its sums
}

// Any width: 32 columns a block, 8 threads a column.  TP: type dP is kept in; dp NULL: not kept (dP is dY).
template <typename T, typename TPRE, typename TP>
__global__ void __launch_bounds__(256) linear_dp(const T* dy, const TPRE* pre, TP* dp, T* db, float* part, int64_t rows, int cols,
                                                 int act) {
    __shared__ float red[8][33], sums[32];
    wait_for_stream();
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 32, col = col0 + lane;
    const int64_t r0 = rows * blockIdx.y / gridDim.y, r1 = rows * (blockIdx.y + 1) / gridDim.y;
    float s = 0.f;
    if (col < cols)
#pragma unroll 4
        for (int64_t r = r0 + sl; r < r1; r += 8) {
            float d = ldf(dy + r * cols + col);
            if (dp != nullptr) {
                d *= act_slope<sizeof(T) == 2>(act, static_cast<float>(pre[r * cols + col]));
                stf(dp + r * cols + col, d);
            }
            s += d;
        }
    if (db == nullptr) return;
    red[sl][lane] = s;
    __syncthreads();
    if (sl == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += red[i][lane];
        sums[lane] = t;
    }
    join_db(sums, db, part, col0, 32, cols);
}

// bf16 in whole 16-byte vectors: LX threads of 8 columns a row, 256 / LX rows side by side, kDpRows of them in flight
// a thread.  dP is rounded to bf16, the type of the tensor cores' operands beside W and X: dX and dW come out 2.3e-3 off in norm, where
// fp32 products rounded once to bf16 are 1.7e-3 off.  A second word for the rest would take each product twice (8192 x 4096 x 11008:
// 780 us more), fp32 FMA some 20 times as long.  db is summed from what is not rounded.
template <int ACT, int LX>
__global__ void __launch_bounds__(256, 4) linear_dp_vec(const __nv_bfloat16* dy, const __half* pre, __nv_bfloat16* dp,
                                                        __nv_bfloat16* db, float* part, int64_t rows, int cols) {
    constexpr int SL = 256 / LX, C = LX * 8;   // row slices, columns
    __shared__ __align__(16) float red[SL][C + 4];
    __shared__ float sums[C];
    wait_for_stream();
    const int lane = threadIdx.x % LX, sl = threadIdx.x / LX;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * C, col = col0 + lane * 8;
    const int64_t r0 = rows * blockIdx.y / gridDim.y, r1 = rows * (blockIdx.y + 1) / gridDim.y;
    float s[8] = {};
    if (col < cols) {
        for (int64_t r = r0 + sl; r < r1; r += SL * kDpRows) {
            uint4 d[kDpRows], h[kDpRows];
#pragma unroll
            for (int i = 0; i < kDpRows; ++i)
                if (r + SL * i < r1) {
                    d[i] = ldg16_cs(dy + (r + SL * i) * cols + col);
                    if (ACT != LIGER_ACT_NONE) h[i] = ldg16_cs(pre + (r + SL * i) * cols + col);
                }
#pragma unroll
            for (int i = 0; i < kDpRows; ++i)
                if (r + SL * i < r1) {
                    float f[8];
                    unpack(d[i], f);
                    if (ACT != LIGER_ACT_NONE) {
                        const __half2* q = reinterpret_cast<const __half2*>(&h[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 w = __half22float2(q[e]);
                            f[2 * e] *= act_slope<true>(ACT, w.x);
                            f[2 * e + 1] *= act_slope<true>(ACT, w.y);
                        }
                        stg16(dp + (r + SL * i) * cols + col, pack(f));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] += f[e];
                }
        }
    }
    if (db == nullptr) return;
#pragma unroll
    for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(&red[sl][lane * 8 + e]) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
    __syncthreads();
    if (threadIdx.x < C) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < SL; ++i) t += red[i][threadIdx.x];
        sums[threadIdx.x] = t;
    }
    join_db(sums, db, part, col0, C, cols);
}

template <typename T>
__global__ void __launch_bounds__(128) linear_db(const float* part, T* db, int parts, int cols) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    wait_for_stream();
    if (col >= cols) return;
    float s = 0.f;
#pragma unroll 16
    for (int i = 0; i < parts; ++i) s += part[static_cast<int64_t>(i) * cols + col];
    stf(db + col, s);
}

// Blocks that share the rows of a column sum: a cluster of up to kDpShares with at least 32 rows each, or, from
// kDpLong rows on, one for each 128 rows, kDpParts at most.
struct DpShares {
    unsigned blocks;
    bool cluster;
};
DpShares dp_shares(int64_t rows) {
    if (rows >= kDpLong) return {static_cast<unsigned>(std::min<int64_t>(kDpParts, ceil_div(rows, 128))), false};
    unsigned n = kDpShares;
    while (n > 1 && rows < 32 * static_cast<int64_t>(n)) n /= 2;
    return {n, true};
}

bool on_tensor_cores(int64_t H, int64_t N, int dtype) {
    return dtype == LIGER_BF16 && H % 8 == 0 && N % 8 == 0 && H >= 64 && N >= 64;
}

int check_sizes(const char* who, int64_t T, int64_t H, int64_t N, int act, int dtype) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    const int64_t most = int64_t{1} << 30, area = int64_t{1} << 40;
    if (T < 0 || H <= 0 || N <= 0 || T > most || H > most || N > most || T * std::max(H, N) > area || H * N > area)
        return fail(LIGER_ERR_SHAPE, "%s: T=%lld H=%lld N=%lld", who, (long long)T, (long long)H, (long long)N);
    if (act < LIGER_ACT_NONE || act > LIGER_ACT_SILU) return fail(LIGER_ERR_SHAPE, "%s: act %d", who, act);
    return LIGER_OK;
}
bool off16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p)) return true;
    return false;
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
// bytes of dP in the workspace, and of db's partial rows behind it
size_t dp_bytes(int64_t T, int64_t H, int64_t N, int act, int dtype) {
    if (act == LIGER_ACT_NONE) return 0;
    return round256(static_cast<size_t>(T) * static_cast<size_t>(N) * (on_tensor_cores(H, N, dtype) ? 2 : 4));
}
size_t part_bytes(int64_t T, int64_t N) {
    const DpShares s = dp_shares(T);
    return s.cluster ? 0 : round256(static_cast<size_t>(s.blocks) * static_cast<size_t>(N) * 4);
}

template <typename T, typename TPRE>
int fwd_fma(const void* X, const void* W, FmaEpi<T, TPRE> e, int64_t Tn, int64_t H, int64_t N, cudaStream_t st) {
    FmaGemm g{static_cast<int>(Tn), static_cast<int>(N), static_cast<int>(H), H, 1, 1, H};
    return launch_fma_gemm("linear_act_fwd", FmaJob<T, T, T, TPRE>{static_cast<const T*>(X), static_cast<const T*>(W), g, e}, st);
}

// dX = dP W and dW = dP^T X from dP [T, N] in TP
template <typename T, typename TP>
int grads_fma(const TP* dP, const void* X, const void* W, void* dX, void* dW, int64_t Tn, int64_t H, int64_t N,
              cudaStream_t st) {
    FmaEpi<T, float> ex{}, ew{};
    ex.out = static_cast<T*>(dX);
    ew.out = static_cast<T*>(dW);
    const FmaJob<TP, T, T, float> x{dP, static_cast<const T*>(W), {static_cast<int>(Tn), static_cast<int>(H), static_cast<int>(N), N, 1, H, 1}, ex};
    const FmaJob<TP, T, T, float> w{dP, static_cast<const T*>(X), {static_cast<int>(N), static_cast<int>(H), static_cast<int>(Tn), 1, N, H, 1}, ew};
    if (dX != nullptr && dW != nullptr) return launch_fma_two("linear_act_bwd dX, dW", x, w, st);
    if (dX != nullptr) return launch_fma_gemm("linear_act_bwd dX", x, st);
    return dW != nullptr ? launch_fma_gemm("linear_act_bwd dW", w, st) : LIGER_OK;
}

struct LinearBwd {
    const void *dY, *X, *W, *pre;
    void *dX, *dW, *db, *dP;
    float* part;
    int64_t T, H, N;
    int act;
    cudaStream_t st;
};

// ------------------------------------------------------------- tensor cores
int64_t pair_tiles(int64_t M, int64_t N) {
    return ceil_div(M, static_cast<int64_t>(tc::TileCfg<1>::TM)) * ceil_div(N, static_cast<int64_t>(tc::BN));
}
// Whether T tokens by F features go in 128-feature tiles (linear_small.cuh) and not in 256 x 256 tiles of CTA pairs: up to
// 128 tokens, and where the pairs' tiles leave most of the SMs idle.  us in small tiles and in pairs', tokens x sum length x features:
//   128 x 4096 x 11008 20.7, 26.9 (43 tiles of pairs)   256 x 4096 x 11008 35.1, 27.6 (43)   256 x 4096 x 4096 16.0, 24.9 (16)
//   512 x 4096 x 4096  26.8, 24.9 (32)   600 x 4096 x 2048 18.7, 24.3 (24)   1024 x 1024 x 1024 9.7, 11.2 (16)
//   2394 x 1600 x 696  16.1, 13.2 (30)   160 x 2048 x 8192 13.6, 15.7 (32)   1111 x 520 x 1384  10.5, 9.5 (30)
bool goes_small(int64_t T, int64_t F) {
    const int64_t pairs = sm_count() / 2;
    return F <= 65535 * int64_t{tc::kSmallRows} && (T <= kSmallTokens || (T <= 256 ? 2 : 3) * pair_tiles(T, F) <= pairs);
}
// Tokens of a small tile: all of them up to 256 (256 x 4096 x 4096: 16.1 us, 17.4 in tiles of 128), else 128 (1024 x 2048 x 2048:
// 16.9 us, 30.7 in tiles of 192; 700 x 2048 x 2048: 14.5, 13.3 in tiles of 192, 23.1 of 256).
int small_tokens(int64_t T) { return T <= 256 ? 256 : 128; }

int fwd_tc(const void* X, const void* W, const void* bias, const void* residual, void* Y, void* pre, int64_t T, int64_t H,
           int64_t N, int act, cudaStream_t st) {
    using namespace tc;
    int* err = nullptr;
    int rc;
    if ((rc = lsw_err_word(&err))) return rc;
    if (goes_small(T, N)) {
        SmallParams p{};
        p.F = static_cast<int>(N);
        p.T = static_cast<int>(T);
        p.K = static_cast<int>(H);
        p.bias = static_cast<const __nv_bfloat16*>(bias);
        p.residual = static_cast<const __nv_bfloat16*>(residual);
        p.out = static_cast<__nv_bfloat16*>(Y);
        p.pre = static_cast<__half*>(pre);
        p.act = act;
        p.err = err;
        return launch_small<0, 0>("linear_act_fwd", W, X, p, small_tokens(T), st);
    }
    CUtensorMap mX, mW;
    if ((rc = make_map(&mX, X, H, T, H, BK, BM))) return rc;
    if ((rc = make_map(&mW, W, H, N, H, BK, B_BOX_ROWS))) return rc;
    EpiParams e{};
    e.err = err;
    e.M = static_cast<int>(T);
    e.N = static_cast<int>(N);
    e.out = static_cast<__nv_bfloat16*>(Y);
    e.ldo = N;
    e.src = static_cast<const __nv_bfloat16*>(residual);
    e.bias16 = static_cast<const __nv_bfloat16*>(bias);
    e.pre16 = static_cast<__half*>(pre);
    e.act = act;
    e.hint_a = HINT_EVICT_LAST;    // X: reused by every column tile
    e.hint_b = HINT_EVICT_FIRST;   // W: streamed once per group of rows
    e.m_group = static_cast<int>(ceil_div(rows_in_l2(H, T), static_cast<int64_t>(TileCfg<1>::TM)));
    e.early = 1;
    e.nan_unfinished = 1;
    return launch_gemm<0, 0, EPI_LINEAR, 1>(mX, mW, e.M, e.N, static_cast<int>(H), e, st);
}

// dX = dP W and dW = dP^T X from dP [T, N] bf16.  The last, partly filled round of dW's tiles is split along
// the tokens, its fp32 sums standing in dX's memory, which is formed after it.
int grads_tc(const LinearBwd& a, const void* dP) {
    using namespace tc;
    const int T = static_cast<int>(a.T), H = static_cast<int>(a.H), N = static_cast<int>(a.N);
    int* err = nullptr;
    int rc;
    if ((rc = lsw_err_word(&err))) return rc;
    if (a.dW != nullptr && goes_small(a.N, a.H)) {
        SmallParams p{};
        p.F = H;
        p.T = N;
        p.K = T;
        p.out = static_cast<__nv_bfloat16*>(a.dW);
        p.err = err;
        if ((rc = launch_small<1, 1>("linear_act_bwd dW", a.X, dP, p, 128, a.st))) return rc;
    } else if (a.dW != nullptr) {
        CUtensorMap mP, mX;
        if ((rc = make_map(&mP, dP, N, T, N, MN_BOX, BK))) return rc;
        if ((rc = make_map(&mX, a.X, H, T, H, MN_BOX, BK))) return rc;
        EpiParams w{};
        w.err = err;
        w.M = N;
        w.N = H;
        w.out = static_cast<__nv_bfloat16*>(a.dW);
        w.ldo = H;
        w.out_write = 1;
        // n fastest touches all of X in every round: fine while X stays in L2 (up to 32 MiB), above that groups
        // of 8 column blocks of it do
        w.raster = a.T * a.H * 2 > (int64_t{32} << 20) ? RASTER_N_GROUPS : RASTER_N_FASTEST;
        w.hint_a = HINT_EVICT_FIRST;
        w.hint_b = HINT_EVICT_LAST;   // X: reused by every row block
        w.early = 1;
        w.nan_unfinished = 1;
        // The last, partly filled round of tiles is split along the tokens over the idle pairs, their sums in dX, which is written after:
        // 8192 x 4096 x 11008, dW and dX: 746 us, 789 with whole tiles; 8192 x 2048 x 5504: 225, 245
        const int64_t tiles = pair_tiles(N, H), pairs = sm_count() / 2, rem = tiles % pairs;
        const int64_t tile_bytes = int64_t{TileCfg<1>::TM} * BN * 4;
        const int64_t splits = a.dX == nullptr || rem == 0 ? 0
                               : std::min<int64_t>({pairs / rem, a.T / (16 * BK), a.T * a.H * 2 / (rem * tile_bytes)});
        if (splits < 2) {
            if ((rc = launch_gemm<1, 1, EPI_ACCUM, 1>(mP, mX, N, H, T, w, a.st))) return rc;
        } else {
            w.full_tiles = static_cast<int>(tiles - rem);
            w.ksplits = static_cast<int>(splits);
            w.kpart_rows = TileCfg<1>::TM;
            w.kpart = static_cast<float*>(a.dX);
            if ((rc = launch_gemm<1, 1, EPI_ACCUM, 1, MODE_SPLIT>(mP, mX, N, H, T, w, a.st))) return rc;
            SplitJoin j{};
            j.part = w.kpart;
            j.rem = static_cast<int>(rem);
            j.splits = w.ksplits;
            j.slabs = 1;
            j.full = w.full_tiles;
            j.part_rows = w.kpart_rows;
            j.num_m = static_cast<int>(ceil_div(a.N, static_cast<int64_t>(TileCfg<1>::TM)));
            j.num_n = static_cast<int>(ceil_div(a.H, static_cast<int64_t>(BN)));
            j.out = w.out;
            j.M = N;
            j.N = H;
            j.n_fastest = w.raster == RASTER_N_FASTEST ? 1 : 0;
            if ((rc = launch_early("linear_act_bwd dW", split_join,
                                   dim3(static_cast<unsigned>(rem), static_cast<unsigned>(j.part_rows / 8)), 256, 0, a.st, j)))
                return rc;
        }
    }
    if (a.dX == nullptr) return LIGER_OK;
    if (goes_small(a.T, a.H)) {
        SmallParams p{};
        p.F = H;
        p.T = T;
        p.K = N;
        p.out = static_cast<__nv_bfloat16*>(a.dX);
        p.err = err;
        return launch_small<1, 0>("linear_act_bwd dX", a.W, dP, p, small_tokens(a.T), a.st);
    }
    CUtensorMap mP, mW;
    if ((rc = make_map(&mP, dP, N, T, N, BK, BM))) return rc;
    if ((rc = make_map(&mW, a.W, H, N, H, MN_BOX, BK))) return rc;
    EpiParams d{};
    d.err = err;
    d.M = T;
    d.N = H;
    d.out = static_cast<__nv_bfloat16*>(a.dX);
    d.ldo = H;
    d.raster = RASTER_N_GROUPS;
    d.early = 1;
    d.nan_unfinished = 1;
    return launch_gemm<0, 1, EPI_STORE, 1>(mP, mW, T, H, N, d, a.st);
}

template <typename T, typename TPRE, typename TP>
int bwd_typed(const LinearBwd& a) {
    const bool keep = a.act != LIGER_ACT_NONE;
    constexpr bool TC = sizeof(T) == 2 && sizeof(TP) == 2;   // bf16 in whole vectors, for the tensor cores
    if (keep || a.db != nullptr) {
        const DpShares sh = dp_shares(a.T);
        // 256 columns a block where there are blocks enough, else 64: dP and db of 8192 x 11008 in 92 us (103 with 64), of 4096 x 4096 in
        // 20.3 (20.7); of 2048 x 4096 in 12.4 (11.5), 1024 x 4096 in 10.0 (7.1)
        const bool wide = TC && a.N >= 2048 && a.T >= 4096;
        const dim3 grid(static_cast<unsigned>(ceil_div(a.N, !TC ? 32 : wide ? 256 : 64)), sh.blocks), cluster(1, sh.cluster ? sh.blocks : 1);
        float* part = a.db != nullptr && !sh.cluster ? a.part : nullptr;
        const T* dy = static_cast<const T*>(a.dY);
        const TPRE* pre = static_cast<const TPRE*>(a.pre);
        TP* dp = static_cast<TP*>(keep ? a.dP : nullptr);
        T* db = static_cast<T*>(a.db);
        const char* who = "linear_act_bwd dP";
        int rc = LIGER_OK;
        if constexpr (TC) {
            auto go = [&](auto k) {
                rc = launch_cluster(who, k, grid, cluster, 256, 0, a.st, dy, pre, dp, db, part, a.T, static_cast<int>(a.N));
            };
            switch (a.act) {
                case LIGER_ACT_RELU: wide ? go(linear_dp_vec<LIGER_ACT_RELU, 32>) : go(linear_dp_vec<LIGER_ACT_RELU, 8>); break;
                case LIGER_ACT_GELU: wide ? go(linear_dp_vec<LIGER_ACT_GELU, 32>) : go(linear_dp_vec<LIGER_ACT_GELU, 8>); break;
                case LIGER_ACT_GELU_TANH:
                    wide ? go(linear_dp_vec<LIGER_ACT_GELU_TANH, 32>) : go(linear_dp_vec<LIGER_ACT_GELU_TANH, 8>);
                    break;
                case LIGER_ACT_SILU: wide ? go(linear_dp_vec<LIGER_ACT_SILU, 32>) : go(linear_dp_vec<LIGER_ACT_SILU, 8>); break;
                default: wide ? go(linear_dp_vec<LIGER_ACT_NONE, 32>) : go(linear_dp_vec<LIGER_ACT_NONE, 8>); break;
            }
        } else {
            rc = launch_cluster(who, linear_dp<T, TPRE, TP>, grid, cluster, 256, 0, a.st, dy, pre, dp, db, part, a.T,
                                static_cast<int>(a.N), a.act);
        }
        if (rc) return rc;
        if (part != nullptr)
            if ((rc = launch_early(who, linear_db<T>, dim3(static_cast<unsigned>(ceil_div(a.N, 128))), 128, 0, a.st,
                                   static_cast<const float*>(part), db, static_cast<int>(sh.blocks), static_cast<int>(a.N))))
                return rc;
    }
    if constexpr (TC) return grads_tc(a, keep ? a.dP : a.dY);
    else if (keep) return grads_fma<T, TP>(static_cast<const TP*>(a.dP), a.X, a.W, a.dX, a.dW, a.T, a.H, a.N, a.st);
    else return grads_fma<T, T>(static_cast<const T*>(a.dY), a.X, a.W, a.dX, a.dW, a.T, a.H, a.N, a.st);
}

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" int liger_linear_act_fwd(const void* X, const void* W, const void* bias, const void* residual, void* Y, void* pre,
                                    int64_t T, int64_t H, int64_t N, int act, int dtype, void* stream) {
    clear_error();
    const char* who = "linear_act_fwd";
    if (int rc = check_sizes(who, T, H, N, act, dtype)) return rc;
    if (T == 0) return LIGER_OK;
    if (!X || !W || !Y) return fail(LIGER_ERR_NULL, "%s: X, W and Y are required", who);
    if (off16({X, W, bias, residual, Y, pre})) return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    cudaStream_t st = as_stream(stream);
    if (dtype == LIGER_F32) {
        FmaEpi<float, float> e{static_cast<const float*>(bias), static_cast<const float*>(residual), static_cast<float*>(Y),
                               static_cast<float*>(pre), act};
        return fwd_fma(X, W, e, T, H, N, st);
    }
    if (on_tensor_cores(H, N, dtype)) return fwd_tc(X, W, bias, residual, Y, pre, T, H, N, act, st);
    using Bf = __nv_bfloat16;
    FmaEpi<Bf, __half> e{static_cast<const Bf*>(bias), static_cast<const Bf*>(residual), static_cast<Bf*>(Y),
                         static_cast<__half*>(pre), act};
    return fwd_fma(X, W, e, T, H, N, st);
}

extern "C" size_t liger_linear_act_bwd_workspace(int64_t T, int64_t H, int64_t N, int act, int dtype) {
    const bool good = check_sizes("linear_act_bwd_workspace", T, H, N, act, dtype) == LIGER_OK;
    clear_error();
    if (!good || T == 0) return 0;
    return dp_bytes(T, H, N, act, dtype) + part_bytes(T, N);
}

extern "C" int liger_linear_act_bwd(const void* dY, const void* X, const void* W, const void* pre, void* dX, void* dW, void* db,
                                    void* ws, size_t ws_bytes, int64_t T, int64_t H, int64_t N, int act, int dtype,
                                    void* stream) {
    clear_error();
    const char* who = "linear_act_bwd";
    if (int rc = check_sizes(who, T, H, N, act, dtype)) return rc;
    if (off16({dY, X, W, pre, dX, dW, db})) return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    cudaStream_t st = as_stream(stream);
    const size_t esz = dtype == LIGER_F32 ? 4 : 2;
    if (T == 0) {
        if (dW != nullptr && cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * static_cast<size_t>(H) * esz, st) != cudaSuccess)
            return check_launch(who);
        if (db != nullptr && cudaMemsetAsync(db, 0, static_cast<size_t>(N) * esz, st) != cudaSuccess) return check_launch(who);
        return LIGER_OK;
    }
    if (!dY || (dX && !W) || (dW && !X) || (act != LIGER_ACT_NONE && !pre))
        return fail(LIGER_ERR_NULL, "%s: dY is required, W for dX, X for dW, pre for an activation", who);
    const size_t need = liger_linear_act_bwd_workspace(T, H, N, act, dtype);
    if (need > 0 && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255)))
        return fail(LIGER_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) required, got %zu", who, need, ws_bytes);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + dp_bytes(T, H, N, act, dtype));
    const LinearBwd a{dY, X, W, pre, dX, dW, db, ws, part, T, H, N, act, st};
    if (dtype == LIGER_F32) return bwd_typed<float, float, float>(a);
    if (on_tensor_cores(H, N, dtype)) return bwd_typed<__nv_bfloat16, __half, __nv_bfloat16>(a);
    return bwd_typed<__nv_bfloat16, __half, float>(a);
}
