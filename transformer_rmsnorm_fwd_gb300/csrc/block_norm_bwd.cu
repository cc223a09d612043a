// Block norms, backward (formulas in liger_train.h).
//
// GB300 design: HBM-bound.  In bf16 12 bytes an element have to move (dh, dy, z,
// h in; dr, dz out); every row is read once and written once.
// Sums over rows: with S[j] = sum D z rz over rows that share a gate row, dgate =
// block_scale w_post S and dw_post = block_scale g S, so one running sum serves
// both.  Rows are split into units that never cross a gate row; per-unit partial
// rows go to the workspace and are added in a fixed order.
#include "block_norm.cuh"

namespace liger {
namespace {

constexpr int kMaxParts = 1024;   // most partial rows of the sums

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
    int interleave;       // the ring kernel's units of a gate row take every splits-th row, not a run of rows
};

// ---------------------------------------------------------------- generic
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
    wait_for_stream();
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
            c1 = cube_times(rh, inv * block_sum(s1, sh));
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
            c2 = cube_times(rz, inv * block_sum(s2, sh));
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

// ------------------------------------------------------- backward, rows staged by bulk copies
// A block per unit of rows; a team of `tw` warps takes every teams-th row of it, the row's dh, dy,
// z, h (those that the call has) brought into the team's ring of `nst` slots by bulk copies.  Each
// thread owns VPT 16-byte column vectors: the weights and its share of the column sums S = sum D z rz
// and sum dy h rh stay in fp32 registers over the rows.
// D needs the row sum s1 and dz the row sum s2 of q D z, but with c1 = rh^3 / cols s1
//     s2 = sum (dh + rh u) q z - c1 sum h q z,
// so the three sums are formed in one pass over the row and reduced together: one team barrier a row,
// whose values stay in registers across it, and the slot is free at once for the next copies.
// Arithmetic on column pairs with the packed fp32x2 instructions.
// WHOLE 0: the block's rows share one gate row (or there is none).  WHOLE 1 (one team): the block
// takes whole gate rows; as one ends its dgate is written, and sum block_scale g S is kept.
// ONE: a single team, known at compile time (its strides and widths are then constants: 0.97 of the
// copy rate against 0.92 at 4096 bf16 columns).
// Every wait is bounded; on expiry the block records it, waits (bounded) for its copies and writes
// NaN into the rows and sums it did not finish.
template <typename T, int VPT, int WHOLE, int NT, int ONE>
__global__ void __launch_bounds__(NT, 1) block_norm_bwd_ring(BwdP p, int tw, int nst, int* err) {
    constexpr int VEC = Vec<T>::N, NP = VEC / 2;
    extern __shared__ __align__(128) uint8_t sm[];
    // per team its warps' sums, from a multiple of 4: at most 4 entries for every 2 warps
    __shared__ __align__(16) float red[2][3][NT / 32 * 2];
    __shared__ int failed;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (ONE) tw = blockDim.x >> 5;
    const int team = ONE ? 0 : warp / tw, wt = warp - team * tw, teams = ONE ? 1 : (blockDim.x >> 5) / tw;
    const int tt = wt * 32 + lane, nt = tw * 32;
    const int nvec = p.cols / VEC;
    const uint32_t rb = static_cast<uint32_t>(p.cols) * sizeof(T);
    const T *dh = static_cast<const T*>(p.dh), *dy = static_cast<const T*>(p.dy), *z = static_cast<const T*>(p.z),
            *h = static_cast<const T*>(p.h);
    const T *wp = static_cast<const T*>(p.w_post), *wn = static_cast<const T*>(p.w_pre), *gate = static_cast<const T*>(p.gate);
    const bool post = wp != nullptr, pre = wn != nullptr, need_z = post || gate != nullptr, has_dh = dh != nullptr;
    // offsets of the streams in a slot
    uint32_t off = 0;
    const uint32_t o_dh = off; off += has_dh ? rb : 0;
    const uint32_t o_dy = off; off += pre ? rb : 0;
    const uint32_t o_h = off; off += pre ? rb : 0;
    const uint32_t o_z = off; off += need_z ? rb : 0;
    const uint32_t slot_bytes = off;
    const uint8_t* ring = sm + static_cast<size_t>(team) * nst * slot_bytes;
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(teams) * nst * slot_bytes) + 8u * team * nst;
    int64_t u0, t1;   // the block's rows
    int64_t gate_row = 0;
    if (WHOLE) {
        u0 = blockIdx.x * p.gates_per_block * p.per_gate;
        t1 = min(p.rows, u0 + p.gates_per_block * p.per_gate);
        gate_row = blockIdx.x * p.gates_per_block;
    } else {
        gate_row = blockIdx.x / p.splits;
        const int64_t sp = blockIdx.x - gate_row * p.splits;
        u0 = gate_row * p.per_gate + (p.interleave ? sp : sp * p.unit_rows);
        t1 = (gate_row + 1) * p.per_gate;
        if (!p.interleave) t1 = min(t1, u0 + p.unit_rows);
    }
    const int64_t unit = !WHOLE && p.interleave ? p.splits : 1;   // the block's rows: u0, u0 + unit, ... below t1
    const int64_t t0 = u0 + team * unit, step = teams * unit;   // the team's rows: t0, t0 + step, ...
    auto issue = [&](int64_t t, int s) {
        const uint32_t bar = bars + 8u * s, dst = smem_u32(ring + static_cast<size_t>(s) * slot_bytes);
        mbar_expect_tx(bar, slot_bytes);
        if (has_dh) bulk_g2s(dst + o_dh, dh + t * p.cols, rb, bar);
        if (pre) bulk_g2s(dst + o_dy, dy + t * p.cols, rb, bar);
        if (pre) bulk_g2s(dst + o_h, h + t * p.cols, rb, bar);
        if (need_z) bulk_g2s(dst + o_z, z + t * p.cols, rb, bar);
    };
    if (tt == 0)
        for (int s = 0; s < nst; ++s) mbar_init(bars + 8u * s, 1);
    if (threadIdx.x == 0) failed = 0;
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(red) / 4); i += blockDim.x) (&red[0][0][0])[i] = 0.f;
    mbar_init_fence();
    __syncthreads();
    wait_for_stream();
    if (tt == 0)
        for (int s = 0; s < nst; ++s)
            if (t0 + s * step < t1) issue(t0 + s * step, s);
    // q = block_scale g w_post and w_pre in fp32; sums
    float2 q[VPT][NP], wf[VPT][NP], S[VPT][NP], Sn[VPT][NP], Sp[WHOLE ? VPT : 1][NP];
    bool live[VPT];
    const float2 zero2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * nt + tt;
        live[j] = v < nvec;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            wf[j][e] = S[j][e] = Sn[j][e] = zero2;
            if (WHOLE) Sp[j][e] = zero2;
        }
        if (live[j] && pre) unpack2(ldg16(wn + static_cast<int64_t>(v) * VEC), wf[j]);
    }
    auto gate_in = [&]() {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int64_t c = static_cast<int64_t>(j * nt + tt) * VEC;
            float2 f[NP];
#pragma unroll
            for (int e = 0; e < NP; ++e) q[j][e] = make_float2(p.b, p.b);
            if (!live[j]) continue;
            if (post) {
                unpack2(ldg16(wp + c), f);
#pragma unroll
                for (int e = 0; e < NP; ++e) q[j][e] = __fmul2_rn(q[j][e], f[e]);
            }
            if (gate != nullptr) {
                unpack2(ldg16(gate + gate_row * p.cols + c), f);
#pragma unroll
                for (int e = 0; e < NP; ++e) q[j][e] = __fmul2_rn(q[j][e], f[e]);
            }
        }
    };
    gate_in();
    int64_t gate_end = WHOLE ? (gate_row + 1) * p.per_gate : 0;   // first row past the current gate row
    // a gate row ends: its gradient, and its share of dw_post
    auto flush = [&]() {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (!live[j]) continue;
            const int64_t c = static_cast<int64_t>(j * nt + tt) * VEC;
            float2 g[NP], w[NP];
            unpack2(ldg16(gate + gate_row * p.cols + c), g);
#pragma unroll
            for (int e = 0; e < NP; ++e) w[e] = make_float2(1.f, 1.f);
            if (post) unpack2(ldg16(wp + c), w);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 bs = __fmul2_rn(make_float2(p.b, p.b), S[j][e]);
                Sp[WHOLE ? j : 0][e] = __ffma2_rn(g[e], bs, Sp[WHOLE ? j : 0][e]);
                w[e] = __fmul2_rn(w[e], bs);
                S[j][e] = zero2;
            }
            stg16(static_cast<T*>(p.dgate) + gate_row * p.cols + c, pack2(w));
        }
    };
    const float inv = 1.0f / static_cast<float>(p.cols);
    int s = 0, turn = 0;
    uint32_t ph = 0;
    int64_t t = t0;
    bool ok = true;
    // the next row's scales, fetched a row ahead
    float rzn = post && t < t1 ? p.rstd_z[t] : 1.f, rhn = pre && t < t1 ? p.rstd_h[t] : 0.f;
    for (; t < t1; t += step) {
        const float rz = rzn, rh = rhn;
        const bool more = t + step < t1;
        rzn = post && more ? p.rstd_z[t + step] : 1.f;
        rhn = pre && more ? p.rstd_h[t + step] : 0.f;
        if (WHOLE && t >= gate_end) {
            flush();
            ++gate_row;
            gate_end += p.per_gate;
            gate_in();
        }
        ok = mbar_wait(bars + 8u * s, ph);
        const uint8_t* slot = ring + static_cast<size_t>(s) * slot_bytes;
        uint4 cd[VPT], cy[VPT], ch[VPT], cz[VPT];
        float2 a1 = zero2, a2 = zero2, a3 = zero2;
        const float2 rh2 = make_float2(rh, rh), rz2 = make_float2(rz, rz);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const size_t at = static_cast<size_t>(j * nt + tt) * 16;
            cd[j] = cy[j] = ch[j] = cz[j] = make_uint4(0, 0, 0, 0);
            if (live[j] && ok) {
                if (has_dh) cd[j] = *reinterpret_cast<const uint4*>(slot + o_dh + at);
                if (pre) cy[j] = *reinterpret_cast<const uint4*>(slot + o_dy + at);
                if (pre) ch[j] = *reinterpret_cast<const uint4*>(slot + o_h + at);
                if (need_z) cz[j] = *reinterpret_cast<const uint4*>(slot + o_z + at);
            }
            float2 fd[NP], fy[NP], fh[NP], fz[NP];
            unpack2(cd[j], fd);
            unpack2(cy[j], fy);
            unpack2(ch[j], fh);
            unpack2(cz[j], fz);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 yh = __fmul2_rn(fy[e], fh[e]);
                a1 = __ffma2_rn(wf[j][e], yh, a1);
                Sn[j][e] = __ffma2_rn(yh, rh2, Sn[j][e]);
                const float2 v = __ffma2_rn(rh2, __fmul2_rn(fy[e], wf[j][e]), fd[e]);
                const float2 qz = __fmul2_rn(q[j][e], fz[e]);
                a2 = __ffma2_rn(v, qz, a2);
                a3 = __ffma2_rn(fh[e], qz, a3);
            }
        }
        float sums[3] = {a1.x + a1.y, a2.x + a2.y, a3.x + a3.y};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < 3; ++k) sums[k] += __shfl_xor_sync(0xffffffffu, sums[k], o);
        const int at = ONE ? 0 : team * ((tw + 3) & ~3);
        if (!ONE && tw == 1) {
            ok = __all_sync(0xffffffffu, ok);
        } else {
            if (lane == 0)
#pragma unroll
                for (int k = 0; k < 3; ++k) red[turn][k][at + wt] = sums[k];
            if (ONE) {
                ok = __syncthreads_and(ok ? 1 : 0) != 0;
            } else {
                uint32_t all;
                asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 q, %3, 0;\n\t"
                "barrier.cta.red.and.pred p, %1, %2, q;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(all)
                : "r"(team + 1), "r"(nt), "r"(ok ? 1u : 0u)
                : "memory");
                ok = all != 0;
            }
        }
        if (!ok) break;
        if (ONE || tw > 1) {
#pragma unroll
            for (int k = 0; k < 3; ++k) {   // entries past the team's warps hold 0
                const float4* r4 = reinterpret_cast<const float4*>(red[turn][k] + at);
                float a = 0.f;
#pragma unroll
                for (int w = 0; w < (NT / 32 + 3) / 4; ++w)
                    if (ONE || w * 4 < tw) {
                        const float4 f = r4[w];
                        a += (f.x + f.y) + (f.z + f.w);
                    }
                sums[k] = a;
            }
            turn ^= 1;   // this buffer is written again only after the next barrier
        }
        if (tt == 0 && t + nst * step < t1) {   // every thread of the team has the row's values
            fence_proxy_async_smem();
            issue(t + nst * step, s);
        }
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
        const float c1 = cube_times(rh, inv * sums[0]);
        const float c2 = post ? cube_times(rz, inv * (sums[1] - c1 * sums[2])) : 0.f;
        const float2 nc1 = make_float2(-c1, -c1), nc2 = make_float2(-c2, -c2), ra = make_float2(p.a, p.a);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (!live[j]) continue;
            float2 fd[NP], fy[NP], fh[NP], fz[NP], od[NP], oz[NP];
            unpack2(cd[j], fd);
            unpack2(cy[j], fy);
            unpack2(ch[j], fh);
            unpack2(cz[j], fz);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                float2 D = __ffma2_rn(rh2, __fmul2_rn(fy[e], wf[j][e]), fd[e]);
                D = __ffma2_rn(nc1, fh[e], D);
                od[e] = __fmul2_rn(ra, D);
                const float2 Dr = __fmul2_rn(D, rz2);
                oz[e] = __fmul2_rn(q[j][e], Dr);
                if (post) oz[e] = __ffma2_rn(nc2, fz[e], oz[e]);   // without it z has no part in dz: 0 z is NaN at an infinity
                S[j][e] = __ffma2_rn(Dr, fz[e], S[j][e]);
            }
            const int64_t at = t * p.cols + static_cast<int64_t>(j * nt + tt) * VEC;
            stg16_cs(static_cast<T*>(p.dr) + at, pack2(od));
            stg16_cs(static_cast<T*>(p.dz) + at, pack2(oz));
        }
    }
    float* ps = p.part_s != nullptr ? p.part_s + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    float* pp = p.part_pre != nullptr ? p.part_pre + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    if (!ok) {
        if (tt == 0) {
            failed = 1;
            atomicExch(err, 1);
            // the team's copies in flight: rows t, t + step, ..., the first in slot s
            int64_t row = t;
            for (int i = 0; i < nst && row < t1; ++i, row += step) {
                mbar_wait(bars + 8u * s, ph);
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        for (int64_t row = t; row < t1; row += step)
            for (int v = tt; v < nvec; v += nt) {
                stg16(static_cast<T*>(p.dr) + row * p.cols + static_cast<int64_t>(v) * VEC, nan16<T>());
                stg16(static_cast<T*>(p.dz) + row * p.cols + static_cast<int64_t>(v) * VEC, nan16<T>());
            }
        if (WHOLE)
            for (int64_t gi = gate_row; gi * p.per_gate < t1; ++gi)
                for (int v = tt; v < nvec; v += nt)
                    stg16(static_cast<T*>(p.dgate) + gi * p.cols + static_cast<int64_t>(v) * VEC, nan16<T>());
    } else if (WHOLE) {
        flush();
    }
    // the block's partial rows: the teams' sums in the order of the teams, through the ring's memory
    // once no copy is in flight (every team has waited for all its rows, or for its copies above)
    __syncthreads();
    const bool bad = failed != 0;
    float2* acc = reinterpret_cast<float2*>(sm);   // per column vector: NP of S, NP of Sn
    for (int k = 0; k < teams; ++k) {
        if (team == k) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (!live[j]) continue;
                const int v = j * nt + tt;
                const int64_t c = static_cast<int64_t>(v) * VEC;
                float2 s2[NP], n2[NP];
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    s2[e] = WHOLE ? Sp[WHOLE ? j : 0][e] : S[j][e];
                    n2[e] = Sn[j][e];
                    if (k > 0) {
                        s2[e] = __fadd2_rn(acc[v * 2 * NP + e], s2[e]);
                        n2[e] = __fadd2_rn(acc[v * 2 * NP + NP + e], n2[e]);
                    }
                    if (k + 1 < teams) {
                        acc[v * 2 * NP + e] = s2[e];
                        acc[v * 2 * NP + NP + e] = n2[e];
                    }
                }
                if (k + 1 == teams) {
#pragma unroll
                    for (int e = 0; e < NP; e += 2) {
                        const float2 so[2] = {s2[e], s2[e + 1]}, no[2] = {n2[e], n2[e + 1]};
                        if (ps != nullptr) stg16(ps + c + 2 * e, bad ? nan16<float>() : pack2(so));
                        if (pp != nullptr) stg16(pp + c + 2 * e, bad ? nan16<float>() : pack2(no));
                    }
                }
            }
        }
        if (k + 1 < teams) __syncthreads();
    }
}

// ------------------------------------------- rows that are no whole 16-byte vectors
template <typename T, int EPT, int WHOLE, int NT>
__global__ void __launch_bounds__(NT, 1) block_norm_bwd_odd(BwdP p, int nst, uint32_t wmax, int* err) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float red[2][3][NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const T *dh = static_cast<const T*>(p.dh), *dy = static_cast<const T*>(p.dy), *z = static_cast<const T*>(p.z),
            *h = static_cast<const T*>(p.h);
    const T *wp = static_cast<const T*>(p.w_post), *wn = static_cast<const T*>(p.w_pre), *gate = static_cast<const T*>(p.gate);
    const bool post = wp != nullptr, pre = wn != nullptr, need_z = post || gate != nullptr, has_dh = dh != nullptr;
    uint32_t off = 0;
    const uint32_t o_dh = off; off += has_dh ? wmax : 0;
    const uint32_t o_dy = off; off += pre ? wmax : 0;
    const uint32_t o_h = off; off += pre ? wmax : 0;
    const uint32_t o_z = off; off += need_z ? wmax : 0;
    const uint32_t slot_bytes = off;
    const uint32_t streams = slot_bytes / wmax;
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(nst) * slot_bytes);
    int64_t t0, t1, unit = 1, gate_row;
    if (WHOLE) {
        t0 = blockIdx.x * p.gates_per_block * p.per_gate;
        t1 = min(p.rows, t0 + p.gates_per_block * p.per_gate);
        gate_row = blockIdx.x * p.gates_per_block;
    } else {
        gate_row = blockIdx.x / p.splits;
        t0 = gate_row * p.per_gate + (blockIdx.x - gate_row * p.splits);
        t1 = (gate_row + 1) * p.per_gate;
        unit = p.splits;
    }
    auto issue = [&](int64_t t, int s) {
        const Window w = window_of<T>(t, p.rows, p.cols);
        const uint32_t bar = bars + 8u * s, dst = smem_u32(sm + static_cast<size_t>(s) * slot_bytes);
        mbar_expect_tx(bar, streams * w.bytes);
        auto copy = [&](uint32_t o, const void* src) { bulk_g2s(dst + o, static_cast<const uint8_t*>(src) + w.at, w.bytes, bar); };
        if (has_dh) copy(o_dh, p.dh);
        if (pre) copy(o_dy, p.dy);
        if (pre) copy(o_h, p.h);
        if (need_z) copy(o_z, p.z);
    };
    if (tid == 0)
        for (int s = 0; s < nst; ++s) mbar_init(bars + 8u * s, 1);
    mbar_init_fence();
    __syncthreads();
    wait_for_stream();
    if (tid == 0)
        for (int s = 0; s < nst; ++s)
            if (t0 + s * unit < t1) issue(t0 + s * unit, s);
    float q[EPT], wf[EPT], S[EPT], Sn[EPT], Sp[WHOLE ? EPT : 1];
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        S[j] = Sn[j] = 0.f;
        if (WHOLE) Sp[j] = 0.f;
        wf[j] = pre && j * NT + tid < p.cols ? ldf(wn + j * NT + tid) : 0.f;
    }
    auto gate_in = [&]() {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            q[j] = 0.f;
            if (c < p.cols) {
                q[j] = p.b;
                if (post) q[j] *= ldf(wp + c);
                if (gate != nullptr) q[j] *= ldf(gate + gate_row * p.cols + c);
            }
        }
    };
    gate_in();
    int64_t gate_end = WHOLE ? (gate_row + 1) * p.per_gate : 0;
    auto flush = [&]() {   // a gate row ends: its gradient, and its share of dw_post
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            if (c >= p.cols) continue;
            const float bs = p.b * S[j];
            Sp[WHOLE ? j : 0] = fmaf(ldf(gate + gate_row * p.cols + c), bs, Sp[WHOLE ? j : 0]);
            stf(static_cast<T*>(p.dgate) + gate_row * p.cols + c, post ? bs * ldf(wp + c) : bs);
            S[j] = 0.f;
        }
    };
    const float inv = 1.0f / static_cast<float>(p.cols);
    int s = 0, prev = 0, turn = 0;
    uint32_t ph = 0;
    bool ok = true, first = true;
    int64_t t = t0;
    float rzn = post && t < t1 ? p.rstd_z[t] : 1.f, rhn = pre && t < t1 ? p.rstd_h[t] : 0.f;
    for (; t < t1; t += unit) {
        const float rz = rzn, rh = rhn;
        const bool more = t + unit < t1;
        rzn = post && more ? p.rstd_z[t + unit] : 1.f;
        rhn = pre && more ? p.rstd_h[t + unit] : 0.f;
        if (WHOLE && t >= gate_end) {
            flush();
            ++gate_row;
            gate_end += p.per_gate;
            gate_in();
        }
        const Window win = window_of<T>(t, p.rows, p.cols);
        ok = mbar_wait(bars + 8u * s, ph);
        const uint8_t* slot = sm + static_cast<size_t>(s) * slot_bytes;
        const int64_t o = t * p.cols;
        auto get = [&](uint32_t so, const T* g, int c) {
            return c < win.tail ? ldf(reinterpret_cast<const T*>(slot + so) + win.shift + c) : ldf(g + o + c);
        };
        float a[3] = {0.f, 0.f, 0.f};
        float v[EPT];   // dh + rh u
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            v[j] = 0.f;
            if (c >= p.cols || !ok) continue;
            float fh = 0.f;
            if (has_dh) v[j] = get(o_dh, dh, c);
            if (pre) {
                const float fy = get(o_dy, dy, c);
                fh = get(o_h, h, c);
                a[0] = fmaf(wf[j], fy * fh, a[0]);
                Sn[j] = fmaf(fy * fh, rh, Sn[j]);
                v[j] = fmaf(rh, fy * wf[j], v[j]);
            }
            if (post) {
                const float qz = q[j] * get(o_z, z, c);
                a[1] = fmaf(v[j], qz, a[1]);
                a[2] = fmaf(fh, qz, a[2]);
            }
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1)
#pragma unroll
            for (int k = 0; k < 3; ++k) a[k] += __shfl_xor_sync(0xffffffffu, a[k], i);
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < 3; ++k) red[turn][k][wid] = a[k];
        ok = __syncthreads_and(ok ? 1 : 0) != 0;
        if (!ok) break;
        if (tid == 0 && !first && t + (nst - 1) * unit < t1) {   // every thread is past the row before
            fence_proxy_async_smem();
            issue(t + (nst - 1) * unit, prev);
        }
        first = false;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            a[k] = 0.f;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) a[k] += red[turn][k][w];
        }
        turn ^= 1;
        const float c1 = cube_times(rh, inv * a[0]);
        const float c2 = post ? cube_times(rz, inv * (a[1] - c1 * a[2])) : 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            if (c >= p.cols) continue;
            float D = v[j];
            if (pre) D = fmaf(-c1, get(o_h, h, c), D);
            // dr may be dh: this thread has read its dh already
            const float fz = need_z ? get(o_z, z, c) : 0.f;
            const float Dr = D * rz;
            stf(static_cast<T*>(p.dr) + o + c, p.a * D);
            stf(static_cast<T*>(p.dz) + o + c, post ? fmaf(-c2, fz, q[j] * Dr) : q[j] * Dr);
            S[j] = fmaf(Dr, fz, S[j]);
        }
        prev = s;
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
    }
    float* ps = p.part_s != nullptr ? p.part_s + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    float* pp = p.part_pre != nullptr ? p.part_pre + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    const float nan = __int_as_float(0x7FC00000);
    if (!ok) {
        if (tid == 0) {
            atomicExch(err, 1);
            int64_t row = t;
            for (int i = 0; i + (first ? 0 : 1) < nst && row < t1; ++i, row += unit) {
                mbar_wait(bars + 8u * s, ph);
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        for (int64_t row = t; row < t1; row += unit)
            for (int c = tid; c < p.cols; c += NT) {
                stf(static_cast<T*>(p.dr) + row * p.cols + c, nan);
                stf(static_cast<T*>(p.dz) + row * p.cols + c, nan);
            }
        if (WHOLE)
            for (int64_t gi = gate_row; gi * p.per_gate < t1; ++gi)
                for (int c = tid; c < p.cols; c += NT) stf(static_cast<T*>(p.dgate) + gi * p.cols + c, nan);
    } else if (WHOLE) {
        flush();
    }
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const int c = j * NT + tid;
        if (c >= p.cols) continue;
        if (ps != nullptr) ps[c] = ok ? (WHOLE ? Sp[WHOLE ? j : 0] : S[j]) : nan;
        if (pp != nullptr) pp[c] = ok ? Sn[j] : nan;
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
    wait_for_stream();
    if (task == 0 && p.dw_pre == nullptr) return;
    if (task == 1 && p.dw_post == nullptr && !(p.dgate != nullptr && p.gates == 1 && p.splits > 0)) return;
    const float* part = task == 0 ? p.part_pre : p.part_s;
    const bool weighted = task == 1 && p.splits > 0 && p.gates > 1;   // by the unit's gate row
    const int splits = static_cast<int>(p.splits);   // as the number of partial rows at most kMaxParts
    int b0 = 0, b1 = static_cast<int>(p.nparts);
    if (task >= 2) {
        b0 = (task - 2) * splits;
        b1 = b0 + splits;
    }
    const T* gate = static_cast<const T*>(p.gate);
    float s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = 0.f;
    if (c < p.cols) {
#pragma unroll 8
        for (int b = b0 + sl; b < b1; b += 32) {
            float v[V];
            const float* src = part + static_cast<int64_t>(b) * p.cols + c;
            if constexpr (V == 4) unpack(ldg16(src), v);
            else v[0] = *src;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (weighted) v[e] *= ldf(gate + static_cast<int64_t>(b / splits) * p.cols + c + e);
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
        return launch_early("block_norm_sums", block_norm_sums<T, 4>, dim3(static_cast<unsigned>(ceil_div(s.cols, 128)), tasks),
                            1024, 0, st, s);
    return launch_early("block_norm_sums", block_norm_sums<T, 1>, dim3(static_cast<unsigned>(ceil_div(s.cols, 32)), tasks),
                        1024, 0, st, s);
}

// ------------------------------------------------------------------ launches
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

// The ring kernel for rows of nvec vectors, `slot` bytes a row of all streams; grid: the partial rows written.
template <typename T, int VPT, int WHOLE, int NT, int ONE>
int launch_bwd_ring(const BwdP& p, int nvec, size_t slot, int64_t grid, int teams, int per_sm, cudaStream_t st) {
    const int tw = static_cast<int>(ceil_div(nvec, 32 * VPT));
    constexpr auto k = block_norm_bwd_ring<T, VPT, WHOLE, NT, ONE>;
    // about 128 KB of rows in flight on an SM (4096 bf16 columns, 32 KB a row, 1 vector a thread: 3 slots
    // 0.96 of the copy rate, 4 0.97, 8 0.91); one slot if no more fit (the copy of the next row then overlaps the second
    // half of a row's work only)
    size_t nst = std::max<size_t>(1, std::min<size_t>(8, (128u * 1024u) / (per_sm * teams * slot)));
    if (nst == 1 && 2 * teams * slot <= 220u * 1024u) nst = 2;
    // the sums of the teams go through the ring's memory at the end: 16 bytes a vector and element pair
    const size_t sums = teams > 1 ? static_cast<size_t>(nvec) * Vec<T>::N * 8 : 0;
    const size_t smem = std::max(teams * nst * (slot + 8), sums);
    if (int rc = allow_smem<k>()) return rc;
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    return launch_early("block_norm_bwd_ring", k, dim3(static_cast<unsigned>(grid)), teams * tw * 32, smem, st, p, tw,
                        static_cast<int>(nst), err);
}

// Splits the rows and launches: 256 threads' worth of teams where a row takes less (TEAMS: whether it can).
template <typename T, int VPT, int NT, int TEAMS>
int launch_bwd_ring(BwdP& p, int nvec, size_t slot, int64_t& grid, cudaStream_t st) {
    const int tw = static_cast<int>(ceil_div(nvec, 32 * VPT));
    const int teams = std::max(1, 8 / tw);
    int per_sm = 0;
    constexpr auto k = block_norm_bwd_ring<T, VPT, 0, NT, TEAMS ? 0 : 1>;
    if (int rc = allow_smem<k>()) return rc;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, teams * tw * 32, teams * slot);
    per_sm = std::max(1, per_sm);
    grid = split_rows(p, static_cast<int64_t>(sm_count()) * per_sm);
    // Rows up to 8 KB: the blocks walk through memory side by side (4096 bf16 columns 0.97 of the copy rate,
    // 0.90 with a run of rows each; 2048: 0.91, 0.86).  Longer rows: a run each (5120: 0.97, side by side
    // 0.77; 8192: 0.95, 0.89).
    p.interleave = static_cast<size_t>(p.cols) * sizeof(T) <= 8192 ? 1 : 0;
    if (p.splits == 0) return launch_bwd_ring<T, VPT, 1, NT, 1>(p, nvec, slot, grid, 1, per_sm, st);
    if constexpr (TEAMS != 0)
        if (teams > 1) return launch_bwd_ring<T, VPT, 0, NT, 0>(p, nvec, slot, grid, teams, per_sm, st);
    return launch_bwd_ring<T, VPT, 0, NT, 1>(p, nvec, slot, grid, 1, per_sm, st);
}

template <typename T, int EPT, int NT>
int launch_bwd_odd(BwdP& p, int streams, int64_t& grid, cudaStream_t st) {
    constexpr auto k = block_norm_bwd_odd<T, EPT, 0, NT>;
    constexpr auto kw = block_norm_bwd_odd<T, EPT, 1, NT>;
    if (int rc = allow_smem<k>()) return rc;
    if (int rc = allow_smem<kw>()) return rc;
    const size_t wmax = window_max(p.cols, sizeof(T)), slot = streams * wmax + 8;
    int nst = 4;   // one row in use, three in flight
    while (nst > 2 && nst * slot > 200u * 1024u) --nst;
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kw, NT, nst * slot);
    grid = split_rows(p, static_cast<int64_t>(sm_count()) * std::max(1, per_sm));
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    return launch_early("block_norm_bwd_odd", p.splits == 0 ? kw : k, dim3(static_cast<unsigned>(grid)), NT, nst * slot, st, p,
                        nst, static_cast<uint32_t>(wmax), err);
}

template <typename T>
int launch_bwd(BwdP p, void* dw_post, void* dw_pre, float* ws, cudaStream_t st) {
    constexpr int EPV = Vec<T>::N;
    const bool need_s = p.w_post != nullptr || p.gate != nullptr;
    const int64_t room = std::min<int64_t>(p.rows, kMaxParts) * p.cols;
    p.part_pre = p.w_pre != nullptr ? ws : nullptr;
    p.part_s = need_s ? ws + room : nullptr;
    int64_t grid = 0;
    const int streams = (p.dh != nullptr ? 1 : 0) + (p.w_pre != nullptr ? 2 : 0) + (need_s ? 1 : 0);
    const size_t slot = static_cast<size_t>(streams) * p.cols * sizeof(T);
    const int nvec = p.cols % EPV == 0 ? p.cols / EPV : 0;
    int rc;
    constexpr bool F32 = sizeof(T) == 4;
    // By the row's 16-byte vectors; fractions of the measured copy rate with many rows, bf16 unless said:
    // 1 a thread 2048 columns 0.93 (2: 0.87), 1024 0.89, 512 0.90, 256 0.86; 2 a thread 4096 0.97
    // (1, 512 threads: 0.90 to 0.93), 5120 0.95, fp32 4096 0.94, fp32 1024 0.90 (1: 0.84); 4 a thread 8192
    // 0.96, fp32 8192 0.86, 16384 0.44 (its sums spill).  Odd widths: fp32 1001 0.64, bf16 4095 0.33 (the
    // generic kernel: 0.23, 0.10).
    if (nvec == 0 && p.cols >= 64 && p.cols <= 8192 && 2 * (streams * window_max(p.cols, sizeof(T)) + 8) <= 220u * 1024u) {
        if (p.cols <= 256) rc = launch_bwd_odd<T, 4, 64>(p, streams, grid, st);
        else if (p.cols <= 512) rc = launch_bwd_odd<T, 4, 128>(p, streams, grid, st);
        else if (p.cols <= 1024) rc = launch_bwd_odd<T, 4, 256>(p, streams, grid, st);
        else if (p.cols <= 2048) rc = launch_bwd_odd<T, 8, 256>(p, streams, grid, st);
        else if (p.cols <= 4096) rc = launch_bwd_odd<T, 8, 512>(p, streams, grid, st);
        else rc = launch_bwd_odd<T, 16, 512>(p, streams, grid, st);
    } else if (nvec == 0 || nvec > 2048 || slot > 200u * 1024u) {
        grid = split_rows(p, static_cast<int64_t>(sm_count()) * 4);
        rc = launch_early("block_norm_bwd", block_norm_bwd_generic<T>, dim3(static_cast<unsigned>(grid)), 256, 0, st, p);
    } else if (!F32 && nvec <= 256) rc = launch_bwd_ring<T, 1, 256, 1>(p, nvec, slot, grid, st);
    else if (nvec <= 512) rc = launch_bwd_ring<T, 2, 256, 1>(p, nvec, slot, grid, st);
    else if (nvec <= 768) rc = launch_bwd_ring<T, 2, 384, 0>(p, nvec, slot, grid, st);
    else if (F32 && nvec <= 1024) rc = launch_bwd_ring<T, 2, 512, 0>(p, nvec, slot, grid, st);
    else if (nvec <= 1024) rc = launch_bwd_ring<T, 4, 256, 0>(p, nvec, slot, grid, st);
    else rc = launch_bwd_ring<T, 4, 512, 0>(p, nvec, slot, grid, st);
    if (rc) return rc;
    const SumP s{p.part_s, p.part_pre, p.w_post, p.gate, dw_post, p.gate != nullptr ? p.dgate : nullptr, dw_pre, grid,
                 p.gates, p.splits, p.cols, p.b};
    return launch_sums<T>(s, st);
}

}  // namespace
}  // namespace liger

using namespace liger;

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
