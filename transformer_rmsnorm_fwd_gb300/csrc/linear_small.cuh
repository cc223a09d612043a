// Products with few output tiles on the tensor cores: few tokens, or narrow outputs.
//
//   D[f, t] = sum_k A(f, k) B(t, k)     bf16 x bf16 -> fp32 in TMEM, then Y[t, f] = act(D + bias[f]) + residual[t, f]
//
// The features are the MMA's rows (128 of them a block) and the tokens its columns (16 to 256), so that a
// single token wastes nothing of the weight's traffic, which bounds these products: a block's ring holds up to
// 110 KB of the weight's tiles (two blocks on an SM), and K is split over a cluster of up to 8 blocks, as many
// as fill the card once.  Each block leaves its fp32 sums in its shared memory; after a cluster barrier block r
// adds up the sums of tokens r, r + size, ... over distributed shared memory in the order of the k ranges and
// applies the epilogue: one launch, no workspace, no atomics.  4 x 4096 x 11008: 18.5 us from a cold L2 (a plain streaming read of
// those 90 MB takes 23.6 with its launch), 13.6 from a warm one; 256 x 4096 x 4096 16.0: what an SM takes in from L2 bounds it, a
// k-block of 48 KB in 0.4 us.
//   warp 0      TMA producer (one lane);  warp 1  TMEM owner and MMA issuer (one lane);
//   warps 2..5  accumulator to shared memory;  then all six the sums and the epilogue.
// Every wait is bounded; on expiry the block's sums are NaN and the error word is set.
#pragma once

#include <cuda_fp16.h>

#include "activation.cuh"
#include "cluster.cuh"
#include "tc_gemm.cuh"

namespace liger {
namespace tc {
namespace {

constexpr int kSmallThreads = 192, kSmallWarps = kSmallThreads / 32;
constexpr int kSmallRows = 128;   // features of a block
constexpr int kSmallRanks = 8;    // most blocks of a cluster

struct SmallParams {
    int F, T, K;                  // features (rows of Y's last dimension), tokens, sum length
    int nt, stages, tmem_cols;    // tokens of a tile (a multiple of 16), ring depth, TMEM columns (a power of two)
    const __nv_bfloat16* bias;    // [F] or NULL
    const __nv_bfloat16* residual;
    __nv_bfloat16* out;           // [T, F]
    __half* pre;                  // [T, F] or NULL: the sums with the bias
    int act;
    int* err;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// A_MN, B_MN: the features (tokens) of an operand are contiguous, else its k is: Y = X W^T 0, 0; dX = dP W 1, 0;
// dW = dP^T X 1, 1, with the inputs as features, the outputs as "tokens" and the tokens as k.
template <int A_MN, int B_MN>
__global__ void __launch_bounds__(kSmallThreads, 2)
    linear_small(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const SmallParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t stage_bytes = A_BYTES + static_cast<uint32_t>(p.nt) * (BK * 2);
    const uint32_t bar0 = base + p.stages * stage_bytes;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (p.stages + s); };
    const uint32_t done_bar = bar0 + 16u * p.stages;
    const uint32_t spare_bar = done_bar + 8u, slot = done_bar + 16u;
    volatile uint32_t* slot_ptr = reinterpret_cast<uint32_t*>(gbase + p.stages * stage_bytes + 16 * p.stages + 16);
    __shared__ int good;   // 0 where a wait has expired
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = block_in_cluster(), ranks = blocks_in_cluster();
    const int f0 = static_cast<int>(blockIdx.y) * kSmallRows, t0 = static_cast<int>(blockIdx.z) * p.nt;
    const int nkb = (p.K + BK - 1) / BK;   // at least one for every block of the cluster
    const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / ranks);
    const int kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / ranks);
    if (threadIdx.x == 0) {
        good = 1;
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        mbar_init(spare_bar, 1);
        mbar_init_fence();
        prefetch_map(&tmA);
        prefetch_map(&tmB);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(p.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot_ptr;
    wait_for_stream();
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = make_policy(HINT_NORMAL);
            int s = 0;
            uint32_t ph = 0;
            int kb = kb0;
            for (; kb < kb1; ++kb) {
                if (!mbar_wait(empty_bar(s), ph ^ 1u)) {
                    atomicExch(p.err, ERR_TMA_EMPTY);
                    break;
                }
                const uint32_t sa = base + s * stage_bytes;
                mbar_expect_tx(full_bar(s), stage_bytes);
                if (A_MN) {
#pragma unroll
                    for (int j = 0; j < kSmallRows / MN_BOX; ++j)
                        tma_load_2d_hint(sa + j * MN_BOX_BYTES, &tmA, full_bar(s), f0 + j * MN_BOX, kb * BK, pol);
                } else {
                    tma_load_2d_hint(sa, &tmA, full_bar(s), kb * BK, f0, pol);
                }
                if (B_MN) {
                    for (int j = 0; j < p.nt / MN_BOX; ++j)
                        tma_load_2d_hint(sa + A_BYTES + j * MN_BOX_BYTES, &tmB, full_bar(s), t0 + j * MN_BOX, kb * BK, pol);
                } else {
                    tma_load_2d_hint(sa + A_BYTES, &tmB, full_bar(s), kb * BK, t0, pol);
                }
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (kb < kb1) {
                // let the copies in flight land before the block goes on: the last of up to `stages` uses
                const int used = kb - kb0, first = used > p.stages ? used - p.stages : 0;
                for (int i = first; i < used; ++i) mbar_wait(full_bar(i % p.stages), static_cast<uint32_t>(i / p.stages) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc(kSmallRows, p.nt, A_MN, B_MN);
            const uint32_t a_lbo = A_MN ? MN_BOX_BYTES : 16u, a_kstep = A_MN ? UMMA_K * 128u : UMMA_K * 2u;
            const uint32_t b_lbo = B_MN ? MN_BOX_BYTES : 16u, b_kstep = B_MN ? UMMA_K * 128u : UMMA_K * 2u;
            int s = 0;
            uint32_t ph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(full_bar(s), ph)) {
                    atomicExch(p.err, ERR_MMA_FULL);
                    mma_commit(spare_bar);   // the MMAs issued so far end before their TMEM is freed
                    mbar_wait(spare_bar, 0);
                    break;
                }
                tc_fence_after();
                const uint32_t sa = base + s * stage_bytes, sb = sa + A_BYTES;
#pragma unroll
                for (int k = 0; k < BK / UMMA_K; ++k)
                    mma_bf16(tmem, smem_desc(sa + k * a_kstep, a_lbo, 1024u), smem_desc(sb + k * b_kstep, b_lbo, 1024u), idesc,
                             ((kb - kb0) | k) != 0 ? 1u : 0u);
                mma_commit(empty_bar(s));
                if (kb + 1 == kb1) mma_commit(done_bar);   // not reached after an expired wait: the epilogue's expires too
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        __syncwarp();
    }
    // the accumulator into the ring's memory, [token][feature] fp32: no copy or MMA uses that any more once the last
    // commit has arrived.  After an expired wait MMAs or copies may be left: the sums go nowhere then.
    float* part = reinterpret_cast<float*>(gbase);
    if (warp >= 2) {
        const int q = warp & 3;   // TMEM lane quarter this warp may access
        const bool got = __all_sync(0xffffffffu, mbar_wait(done_bar, 0));
        if (got) {
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
            for (int c = 0; c < p.nt; c += 16) {
                float v[16];
                tmem_ld16(taddr + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(c + i) * kSmallRows + q * 32 + lane] = v[i];
            }
            tc_fence_before();
        } else if (lane == 0) {
            good = 0;
            atomicExch(p.err, ERR_EPI_TMEM);
        }
    }
    __syncthreads();
    // (a wait that expired anywhere in the cluster shows in every block's word)
    if (ranks > 1) {
        if (good == 0 && threadIdx.x < ranks) peer_store(&good, threadIdx.x, 0);
        __syncwarp();
        cluster_barrier();
    }
    const bool all = good != 0;
    const int f = f0 + lane * 4;
    const int nt = min(p.nt, p.T - t0);
    if (f < p.F) {   // F is a multiple of 8: four features are in or out together
        float b[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.bias != nullptr) {
            const uint2 u = *reinterpret_cast<const uint2*>(p.bias + f);
            b[0] = bf_lo(u.x); b[1] = bf_hi(u.x);
            b[2] = bf_lo(u.y); b[3] = bf_hi(u.y);
        }
        // four tokens of a warp at a time, so that their loads are in flight together
        constexpr int U = 4;
        const int stride = static_cast<int>(ranks) * kSmallWarps;
        for (int t = static_cast<int>(rank) + static_cast<int>(ranks) * warp; t < nt; t += U * stride) {
            uint2 res[U];
            float4 v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                res[i] = make_uint2(0, 0);
                if (p.residual != nullptr && t + i * stride < nt)
                    res[i] = *reinterpret_cast<const uint2*>(p.residual + static_cast<int64_t>(t0 + t + i * stride) * p.F + f);
            }
            const float* at = part + t * kSmallRows + lane * 4;
            if (ranks > 1) {   // the blocks' sums in their order; tokens past the tile read what stands there (inside the ring)
#pragma unroll
                for (int i = 0; i < U; ++i) v[i] = peer_float4(at + (t + i * stride < nt ? i * stride * kSmallRows : 0), 0);
#pragma unroll 2
                for (uint32_t r = 1; r < ranks; ++r)
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const float4 s = peer_float4(at + (t + i * stride < nt ? i * stride * kSmallRows : 0), r);
                        v[i].x += s.x;
                        v[i].y += s.y;
                        v[i].z += s.z;
                        v[i].w += s.w;
                    }
            } else {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    v[i] = *reinterpret_cast<const float4*>(at + (t + i * stride < nt ? i * stride * kSmallRows : 0));
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (t + i * stride >= nt) break;
                const int64_t o = static_cast<int64_t>(t0 + t + i * stride) * p.F + f;
                float w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = all ? w[e] + b[e] : __int_as_float(0x7FC00000);
                if (p.pre != nullptr) {
                    const bool relu = p.act == LIGER_ACT_RELU;
                    *reinterpret_cast<uint2*>(p.pre + o) =
                        relu ? make_uint2(kept_pair<true>(w[0], w[1]), kept_pair<true>(w[2], w[3]))
                             : make_uint2(kept_pair<false>(w[0], w[1]), kept_pair<false>(w[2], w[3]));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = act_value<true>(p.act, w[e]);
                if (p.residual != nullptr) {
                    w[0] += bf_lo(res[i].x);
                    w[1] += bf_hi(res[i].x);
                    w[2] += bf_lo(res[i].y);
                    w[3] += bf_hi(res[i].y);
                }
                *reinterpret_cast<uint2*>(p.out + o) = make_uint2(pack_bf2(w[0], w[1]), pack_bf2(w[2], w[3]));
            }
        }
    }
    __syncwarp();
    if (ranks > 1) cluster_barrier();   // no block exits while another reads its sums
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
    }
}

// Tokens of a tile for T tokens: all of them up to 256 (the weight is read once), else equal tiles of at most `most`.
inline int small_tile(int64_t T, int most, int unit) {
    const int64_t tiles = ceil_div(T, most);
    return static_cast<int>(ceil_div(ceil_div(T, tiles), unit) * unit);
}

// A [F, K], or [K, F] with A_MN; B [T, K], or [K, T] with B_MN.
template <int A_MN, int B_MN>
int launch_small(const char* who, const void* A, const void* B, SmallParams p, int most_tokens, cudaStream_t st) {
    p.nt = small_tile(p.T, most_tokens, B_MN ? MN_BOX : 16);
    CUtensorMap ma, mb;
    int rc;
    if (A_MN) rc = make_map(&ma, A, p.F, p.K, p.F, MN_BOX, BK);
    else rc = make_map(&ma, A, p.K, p.F, p.K, BK, kSmallRows);
    if (rc) return rc;
    if (B_MN) rc = make_map(&mb, B, p.T, p.K, p.T, MN_BOX, BK);
    else rc = make_map(&mb, B, p.K, p.T, p.K, BK, p.nt);
    if (rc) return rc;
    const int stage = A_BYTES + p.nt * BK * 2;
    const int64_t ft = ceil_div(p.F, kSmallRows), tt = ceil_div(p.T, p.nt), nkb = ceil_div(p.K, BK), sms = sm_count();
    if (ft > 65535 || tt > 65535) return fail(LIGER_ERR_SHAPE, "%s: too many tiles", who);
    p.tmem_cols = 32;
    while (p.tmem_cols < p.nt) p.tmem_cols *= 2;
    // K over `ranks` blocks a tile, so that the SM with the most blocks has the least to do, all of them resident at
    // once where that can be: m blocks on an SM share its memory, three stages each, and its 512 TMEM columns
    const int whole = 226 * 1024, over = 1024 + 256, extra = 2048;
    int ranks = 1, m = 1;
    double least = 1e30;
    for (int r = 1; r <= kSmallRanks && nkb >= (r == 1 ? 1 : 4 * r); ++r) {
        int64_t on = ceil_div(ft * tt * r, sms);
        const int64_t fit = std::min<int64_t>({whole / (3 * stage + over + extra), 512 / p.tmem_cols, 4});
        const double rounds = static_cast<double>(ceil_div(on, fit));
        const double cost = static_cast<double>(on) / r + 0.05 * r + 0.1 * (rounds - 1);
        if (cost < least) {
            least = cost;
            ranks = r;
            m = static_cast<int>(std::min(on, fit));
        }
    }
    p.stages = std::min(12, (whole / m - over - extra) / stage);
    const size_t smem = static_cast<size_t>(p.stages) * stage + over;
    constexpr auto k = linear_small<A_MN, B_MN>;
    if ((rc = allow_smem<k>())) return rc;
    return launch_cluster(who, k, dim3(static_cast<unsigned>(ranks), static_cast<unsigned>(ft), static_cast<unsigned>(tt)),
                          dim3(static_cast<unsigned>(ranks)), kSmallThreads, smem, st, ma, mb, p);
}

}  // namespace
}  // namespace tc
}  // namespace liger
