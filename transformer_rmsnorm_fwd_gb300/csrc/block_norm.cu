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
#include <atomic>

#include "common.cuh"
#include "liger_train.h"
#include "mbarrier.cuh"

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
    int interleave;       // the ring kernel's units of a gate row take every splits-th row, not a run of rows
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

// ------------------------------------------------------- forward, rows in registers
// VEC consecutive elements of a row as one thread holds them: a 16-byte vector, or one element
// where the rows are no whole vectors.
template <typename T, int VEC> struct Frag {
    static_assert(VEC == Vec<T>::N, "whole vectors or single elements");
    uint4 u;
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const T* p) { u = ldg16(p); }
    __device__ __forceinline__ void get(float (&f)[VEC]) const { unpack(u, f); }
    static __device__ __forceinline__ void put(T* p, const float (&f)[VEC]) { stg16(p, pack(f)); }
};
template <typename T> struct Frag<T, 1> {
    float v;
    __device__ __forceinline__ void zero() { v = 0.f; }
    __device__ __forceinline__ void load(const T* p) { v = ldf(p); }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v; }
    static __device__ __forceinline__ void put(T* p, const float (&f)[1]) { stf(p, f[0]); }
};

// A team of `tw` warps holds a row in registers (VPT fragments per thread), a block `teams` of them;
// a team keeps its columns' weights in registers over its rows and has its next row's loads in
// flight while it works on one.  The two row sums go over the team by shuffles and one named
// barrier each; the exchange buffers alternate, so that a buffer is written again only after a
// barrier that follows every read of it.
template <typename T, int VEC, int VPT>
__global__ void __launch_bounds__(512) block_norm_fwd_team(FwdP p, int tw) {
    __shared__ float red[2][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int team = warp / tw, wt = warp - team * tw, teams = (blockDim.x >> 5) / tw;
    const int tt = wt * 32 + lane, nt = tw * 32;   // thread of the team, threads of the team
    const int nfrag = p.cols / VEC;
    const T *z = static_cast<const T*>(p.z), *r = static_cast<const T*>(p.r);
    const T *wp = static_cast<const T*>(p.w_post), *wn = static_cast<const T*>(p.w_pre);
    T *h = static_cast<T*>(p.h), *y = static_cast<T*>(p.y);
    const float inv = 1.0f / static_cast<float>(p.cols);
    Frag<T, VEC> fp[VPT], fn[VPT], fg[VPT];
    bool live[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = j * nt + tt;
        live[j] = c < nfrag;
        fp[j].zero();
        fn[j].zero();
        fg[j].zero();
        if (live[j] && wp != nullptr) fp[j].load(wp + static_cast<int64_t>(c) * VEC);
        if (live[j] && wn != nullptr) fn[j].load(wn + static_cast<int64_t>(c) * VEC);
    }
    int turn = 0;
    auto team_sum = [&](float v) {
        v = warp_sum(v);
        if (tw == 1) return v;
        float* sh = red[turn & 1] + team * tw;
        ++turn;
        if (lane == 0) sh[wt] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(nt) : "memory");
        float t = 0.f;
        for (int i = 0; i < tw; ++i) t += sh[i];
        return t;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t t = static_cast<int64_t>(blockIdx.x) * teams + team;
    Frag<T, VEC> nz[VPT], nr[VPT];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            nz[j].zero();
            nr[j].zero();
            if (live[j]) {
                const int64_t o = row * p.cols + static_cast<int64_t>(j * nt + tt) * VEC;
                nz[j].load(z + o);
                nr[j].load(r + o);
            }
        }
    };
    if (t < p.rows) fetch(t);
    int64_t gate_row = -1;
    for (; t < p.rows; t += step) {
        Frag<T, VEC> cz[VPT], cr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) cz[j] = nz[j], cr[j] = nr[j];
        if (t + step < p.rows) fetch(t + step);   // rows of other teams are never written before they are read
        if (p.gate != nullptr && t / p.per_gate != gate_row) {
            gate_row = t / p.per_gate;
            const T* g = static_cast<const T*>(p.gate) + gate_row * p.cols;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (live[j]) fg[j].load(g + static_cast<int64_t>(j * nt + tt) * VEC);
        }
        float rz = 1.f;
        if (wp != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float f[VEC];
                cz[j].get(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = fmaf(f[e], f[e], ss);
            }
            rz = 1.0f / sqrtf(team_sum(ss) * inv + p.eps);
            if (p.rstd_z != nullptr && tt == 0) p.rstd_z[t] = rz;
        }
        const int64_t o = t * p.cols;
        float hv[VPT][VEC];
        float ss = 0.f;
        const float bz = p.b * rz;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float fz[VEC], fr[VEC], w[VEC];
            cz[j].get(fz);
            cr[j].get(fr);
            if (wp != nullptr) {
                fp[j].get(w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) fz[e] *= w[e];
            }
            if (p.gate != nullptr) {
                fg[j].get(w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) fz[e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                hv[j][e] = fmaf(bz, fz[e], p.a * fr[e]);
                ss = fmaf(hv[j][e], hv[j][e], ss);
            }
            if (live[j]) Frag<T, VEC>::put(h + o + static_cast<int64_t>(j * nt + tt) * VEC, hv[j]);
        }
        if (wn == nullptr) continue;
        const float rh = 1.0f / sqrtf(team_sum(ss) * inv + p.eps);
        if (p.rstd_h != nullptr && tt == 0) p.rstd_h[t] = rh;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float w[VEC];
            fn[j].get(w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) hv[j][e] = hv[j][e] * rh * w[e];
            if (live[j]) Frag<T, VEC>::put(y + o + static_cast<int64_t>(j * nt + tt) * VEC, hv[j]);
        }
    }
}

// ------------------------------------------------------- forward, rows staged by bulk copies
// 1 / sqrt(x) for x > 0: the hardware approximation and one Newton step (within an ulp or so; the
// correctly rounded square root and division are a long serial chain between two barriers)
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = rsqrtf(x);
    const float e = fmaf(-x * r, r, 1.f);
    const float n = fmaf(0.5f * r, e, r);
    return isfinite(n) ? n : r;   // x = 0, infinity or NaN: what rsqrt says
}

// The same team per row, with the rows of z and r brought into a ring of `nst` slots per team by
// bulk copies, so that several rows per team are in flight without registers.  A slot is read into
// registers at once and is free again after the next team barrier.  Every wait is bounded; on
// expiry the team records it, waits (bounded) for its copies and writes NaN into the rows it did
// not finish.  Streaming stores and issuing the next copy only after the sums measured 0.95 of the
// copy rate at 4096 bf16 columns, against 0.93 with the copy first and 0.91 with plain stores (other
// widths: within 0.01).
// GATE: 0 none, 1 one gate row (folded into the post-norm's weights once), 2 several (read anew
// where a row's gate differs from that of the team's row before).
template <typename T, int VPT, int GATE, int NT, int MB, int ONE>
__global__ void __launch_bounds__(NT, MB) block_norm_fwd_ring(FwdP p, int tw, int nst, int* err) {
    constexpr int VEC = Vec<T>::N;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ __align__(16) float red[2][NT / 32 + 4][4];   // rows of 4: a team starts on a multiple of 4 warps or is a warp alone
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (ONE) tw = blockDim.x >> 5;
    const int team = ONE ? 0 : warp / tw, wt = warp - team * tw, teams = ONE ? 1 : (blockDim.x >> 5) / tw;
    const int tt = wt * 32 + lane, nt = tw * 32;
    const int nvec = p.cols / VEC;
    const uint32_t rb = static_cast<uint32_t>(p.cols) * sizeof(T);
    const uint8_t* ring = sm + static_cast<size_t>(team) * nst * 2 * rb;
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(teams) * nst * 2 * rb) + 8u * team * nst;
    const T *z = static_cast<const T*>(p.z), *r = static_cast<const T*>(p.r);
    const T *wp = static_cast<const T*>(p.w_post), *wn = static_cast<const T*>(p.w_pre);
    T *h = static_cast<T*>(p.h), *y = static_cast<T*>(p.y);
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t t = static_cast<int64_t>(blockIdx.x) * teams + team;
    auto issue = [&](int64_t row, int s) {
        const uint32_t bar = bars + 8u * s, dst = smem_u32(ring + static_cast<size_t>(s) * 2 * rb);
        mbar_expect_tx(bar, 2 * rb);
        bulk_g2s(dst, z + row * p.cols, rb, bar);
        bulk_g2s(dst + rb, r + row * p.cols, rb, bar);
    };
    for (int i = threadIdx.x; i < 2 * (NT / 32 + 4) * 4; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
    if (tt == 0)
        for (int s = 0; s < nst; ++s) mbar_init(bars + 8u * s, 1);
    mbar_init_fence();
    __syncthreads();
    if (tt == 0)
        for (int s = 0; s < nst; ++s)
            if (t + s * step < p.rows) issue(t + s * step, s);
    // wq = block_scale w_post (and the one gate row) in fp32, wn as stored
    float wq[VPT][VEC];
    uint4 fn[VPT];
    bool live[VPT];
    auto gate_in = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int64_t c = static_cast<int64_t>(j * nt + tt) * VEC;
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) wq[j][e] = p.b;
            if (!live[j]) continue;
            if (wp != nullptr) {
                unpack(ldg16(wp + c), f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) wq[j][e] *= f[e];
            }
            if (GATE != 0) {
                unpack(ldg16(static_cast<const T*>(p.gate) + row * p.cols + c), f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) wq[j][e] *= f[e];
            }
        }
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        live[j] = j * nt + tt < nvec;
        fn[j] = make_uint4(0, 0, 0, 0);
        if (live[j] && wn != nullptr) fn[j] = ldg16(wn + static_cast<int64_t>(j * nt + tt) * VEC);
    }
    if (GATE != 2) gate_in(0);
    int turn = 0;
    // Team-wide sum in two halves: gather() brings the warps' sums together and says whether every
    // thread of the team got its row (one team barrier), total() adds them up.
    const int at0 = ONE ? 0 : team * ((tw + 3) & ~3);
    auto gather = [&](float& v, bool& ok) {
        v = warp_sum(v);
        if (!ONE && tw == 1) {
            ok = __all_sync(0xffffffffu, ok);
            return;
        }
        if (lane == 0) (&red[turn][0][0])[at0 + wt] = v;
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
    };
    auto total = [&](float v) {
        if (!ONE && tw == 1) return v;
        const float4* q = reinterpret_cast<const float4*>(&red[turn][0][0] + at0);   // slots past the team's warps hold 0
        turn ^= 1;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < (NT / 32 + 3) / 4; ++w)
            if (w * 4 < tw) {
                const float4 a = q[w];
                s += (a.x + a.y) + (a.z + a.w);
            }
        return s;
    };
    // the gate row of row t, kept without a division: t = gate * per_gate + rem
    int64_t gate_row = 0, rem = 0, step_gates = 0, step_rem = 0;
    if (GATE == 2) {
        gate_row = t / p.per_gate;
        rem = t - gate_row * p.per_gate;
        step_gates = step / p.per_gate;
        step_rem = step - step_gates * p.per_gate;
    }
    bool new_gate = true;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; t < p.rows; t += step) {
        uint4 cz[VPT], cr[VPT];
        if (GATE == 2) {   // its loads run while the row is waited for
            if (new_gate) gate_in(gate_row);
            rem += step_rem;
            const int64_t on = step_gates + (rem >= p.per_gate ? 1 : 0);
            if (rem >= p.per_gate) rem -= p.per_gate;
            gate_row += on;
            new_gate = on != 0;
        }
        ok = mbar_wait(bars + 8u * s, ph);
        const uint8_t* slot = ring + static_cast<size_t>(s) * 2 * rb;
        float sz = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            cz[j] = cr[j] = make_uint4(0, 0, 0, 0);
            if (live[j] && ok) {
                cz[j] = *reinterpret_cast<const uint4*>(slot + static_cast<size_t>(j * nt + tt) * 16);
                cr[j] = *reinterpret_cast<const uint4*>(slot + rb + static_cast<size_t>(j * nt + tt) * 16);
            }
            float f[VEC];
            unpack(cz[j], f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sz = fmaf(f[e], f[e], sz);
        }
        gather(sz, ok);
        if (!ok) break;
        const float tz = total(sz);
        if (tt == 0 && t + nst * step < p.rows) {   // every thread of the team has read the slot
            fence_proxy_async_smem();
            issue(t + nst * step, s);
        }
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
        float rz = 1.f;
        if (wp != nullptr) {
            rz = inv_sqrt(fmaf(tz, inv, p.eps));
            if (p.rstd_z != nullptr && tt == 0) p.rstd_z[t] = rz;
        }
        const int64_t o = t * p.cols;
        float hv[VPT][VEC];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float fz[VEC], fr[VEC];
            unpack(cz[j], fz);
            unpack(cr[j], fr);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                hv[j][e] = fmaf(fz[e] * wq[j][e], rz, p.a * fr[e]);
                ss = fmaf(hv[j][e], hv[j][e], ss);
            }
            if (live[j]) stg16_cs(h + o + static_cast<int64_t>(j * nt + tt) * VEC, pack(hv[j]));
        }
        if (wn == nullptr) continue;
        bool same = true;
        gather(ss, same);
        const float rh = inv_sqrt(fmaf(total(ss), inv, p.eps));
        if (p.rstd_h != nullptr && tt == 0) p.rstd_h[t] = rh;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float w[VEC];
            unpack(fn[j], w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) hv[j][e] = hv[j][e] * rh * w[e];
            if (live[j]) stg16_cs(y + o + static_cast<int64_t>(j * nt + tt) * VEC, pack(hv[j]));
        }
    }
    if (ok) return;
    if (tt == 0) {
        atomicExch(err, 1);
        int64_t row = t;
        for (int i = 0; i < nst && row < p.rows; ++i, row += step) {   // the copies in flight
            mbar_wait(bars + 8u * s, ph);
            if (++s == nst) {
                s = 0;
                ph ^= 1u;
            }
        }
    }
    const float nan = __int_as_float(0x7FC00000);
    for (; t < p.rows; t += step) {
        for (int v = tt; v < nvec; v += nt) {
            stg16(h + t * p.cols + static_cast<int64_t>(v) * VEC, nan16<T>());
            if (wn != nullptr) stg16(y + t * p.cols + static_cast<int64_t>(v) * VEC, nan16<T>());
        }
        if (tt == 0 && wp != nullptr && p.rstd_z != nullptr) p.rstd_z[t] = nan;
        if (tt == 0 && wn != nullptr && p.rstd_h != nullptr) p.rstd_h[t] = nan;
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
    __shared__ __align__(16) float red[2][3][(NT / 32 + 3) / 4 * 4 + 4];
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
        const float c1 = rh * rh * rh * inv * sums[0];
        const float c2 = post ? rz * rz * rz * inv * (sums[1] - c1 * sums[2]) : 0.f;
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
                oz[e] = __ffma2_rn(nc2, fz[e], __fmul2_rn(q[j][e], Dr));
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
// The same rings for rows whose width is no multiple of a vector: rows then start anywhere, so a slot
// takes the 16-byte aligned window around a row (the bytes of its neighbours in it are not looked at),
// and threads take single elements from it, EPT fixed columns each.  Memory still moves in
// bulk copies; the elements cost one shared-memory access each, which is what bounds these kernels.
// The last row's window may end past the tensor: the copy stops at the last whole 16 bytes, and the
// elements behind that come by plain loads.
struct Window {
    int64_t at;       // first byte of the window
    uint32_t bytes;   // multiple of 16
    int shift;        // elements from there to the row's first
    int tail;         // the row's elements from this one on are not in the window
};
template <typename T>
__device__ __forceinline__ Window window_of(int64_t t, int64_t rows, int cols) {
    constexpr int SZ = sizeof(T);
    Window w;
    const int64_t o = t * cols * SZ, end = o + static_cast<int64_t>(cols) * SZ;
    w.at = o & ~int64_t{15};
    w.shift = static_cast<int>((o - w.at) / SZ);
    int64_t stop = (end + 15) & ~int64_t{15};
    w.tail = cols;
    if (t == rows - 1 && stop != end) {
        stop = end & ~int64_t{15};
        w.tail = static_cast<int>((stop - o) / SZ);
    }
    w.bytes = static_cast<uint32_t>(stop - w.at);
    return w;
}
// bytes a slot needs for one stream
inline size_t window_max(int cols, size_t sz) { return (static_cast<size_t>(cols) * sz + 15 + 15) & ~static_cast<size_t>(15); }

template <typename T, int EPT, int NT>
__global__ void __launch_bounds__(NT, 1) block_norm_fwd_odd(FwdP p, int nst, uint32_t wmax, int* err) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float red[2][NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(nst) * 2 * wmax);
    const T *z = static_cast<const T*>(p.z), *r = static_cast<const T*>(p.r);
    const T *wp = static_cast<const T*>(p.w_post), *wn = static_cast<const T*>(p.w_pre), *gate = static_cast<const T*>(p.gate);
    T *h = static_cast<T*>(p.h), *y = static_cast<T*>(p.y);
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int64_t step = gridDim.x;
    int64_t t = blockIdx.x;
    auto issue = [&](int64_t row, int s) {
        const Window w = window_of<T>(row, p.rows, p.cols);
        const uint32_t bar = bars + 8u * s, dst = smem_u32(sm + static_cast<size_t>(s) * 2 * wmax);
        mbar_expect_tx(bar, 2 * w.bytes);
        bulk_g2s(dst, static_cast<const uint8_t*>(p.z) + w.at, w.bytes, bar);
        bulk_g2s(dst + wmax, static_cast<const uint8_t*>(p.r) + w.at, w.bytes, bar);
    };
    if (tid == 0)
        for (int s = 0; s < nst; ++s) mbar_init(bars + 8u * s, 1);
    mbar_init_fence();
    __syncthreads();
    if (tid == 0)
        for (int s = 0; s < nst; ++s)
            if (t + s * step < p.rows) issue(t + s * step, s);
    float wq[EPT], wy[EPT];
    auto gate_in = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            wq[j] = 0.f;
            if (c < p.cols) {
                wq[j] = p.b;
                if (wp != nullptr) wq[j] *= ldf(wp + c);
                if (gate != nullptr) wq[j] *= ldf(gate + row * p.cols + c);
            }
        }
    };
#pragma unroll
    for (int j = 0; j < EPT; ++j) wy[j] = wn != nullptr && j * NT + tid < p.cols ? ldf(wn + j * NT + tid) : 0.f;
    int64_t gate_row = -1;
    int turn = 0, s = 0, prev = 0;
    uint32_t ph = 0;
    bool ok = true, first = true;
    auto total = [&]() {
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) a += red[turn][w];
        turn ^= 1;   // written again only after the next barrier
        return a;
    };
    for (; t < p.rows; t += step) {
        if (gate_row < 0 || (gate != nullptr && t / p.per_gate != gate_row)) {
            gate_row = t / p.per_gate;
            gate_in(gate_row);
        }
        const Window win = window_of<T>(t, p.rows, p.cols);
        ok = mbar_wait(bars + 8u * s, ph);
        const T* zs = reinterpret_cast<const T*>(sm + static_cast<size_t>(s) * 2 * wmax) + win.shift;
        const T* rs = reinterpret_cast<const T*>(sm + static_cast<size_t>(s) * 2 * wmax + wmax) + win.shift;
        const int64_t o = t * p.cols;
        float fz[EPT];
        float sz = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            fz[j] = 0.f;
            if (c < p.cols && ok) fz[j] = c < win.tail ? ldf(zs + c) : ldf(z + o + c);
            sz = fmaf(fz[j], fz[j], sz);
        }
        sz = warp_sum(sz);
        if (lane == 0) red[turn][wid] = sz;
        ok = __syncthreads_and(ok ? 1 : 0) != 0;
        if (!ok) break;
        // every thread is past the row before: its slot's next copy
        if (tid == 0 && !first && t + (nst - 1) * step < p.rows) {
            fence_proxy_async_smem();
            issue(t + (nst - 1) * step, prev);
        }
        first = false;
        const float tz = total();
        float rz = 1.f;
        if (wp != nullptr) {
            rz = inv_sqrt(fmaf(tz, inv, p.eps));
            if (p.rstd_z != nullptr && tid == 0) p.rstd_z[t] = rz;
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            if (c < p.cols) {
                const float fr = c < win.tail ? ldf(rs + c) : ldf(r + o + c);
                fz[j] = fmaf(fz[j] * wq[j], rz, p.a * fr);
                ss = fmaf(fz[j], fz[j], ss);
                stf(h + o + c, fz[j]);
            }
        }
        prev = s;
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
        if (wn == nullptr) continue;
        ss = warp_sum(ss);
        if (lane == 0) red[turn][wid] = ss;
        __syncthreads();
        const float rh = inv_sqrt(fmaf(total(), inv, p.eps));
        if (p.rstd_h != nullptr && tid == 0) p.rstd_h[t] = rh;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = j * NT + tid;
            if (c < p.cols) stf(y + o + c, fz[j] * rh * wy[j]);
        }
    }
    if (ok) return;
    if (tid == 0) {
        atomicExch(err, 1);
        int64_t row = t;   // rows t, t + step, ... are in flight; the slot of the row before t was not filled again
        for (int i = 0; i + (first ? 0 : 1) < nst && row < p.rows; ++i, row += step) {
            mbar_wait(bars + 8u * s, ph);
            if (++s == nst) {
                s = 0;
                ph ^= 1u;
            }
        }
    }
    const float nan = __int_as_float(0x7FC00000);
    for (; t < p.rows; t += step) {
        for (int c = tid; c < p.cols; c += NT) {
            stf(h + t * p.cols + c, nan);
            if (wn != nullptr) stf(y + t * p.cols + c, nan);
        }
        if (tid == 0 && wp != nullptr && p.rstd_z != nullptr) p.rstd_z[t] = nan;
        if (tid == 0 && wn != nullptr && p.rstd_h != nullptr) p.rstd_h[t] = nan;
    }
}

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
        const float c1 = rh * rh * rh * inv * a[0];
        const float c2 = post ? rz * rz * rz * inv * (a[1] - c1 * a[2]) : 0.f;
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
            stf(static_cast<T*>(p.dz) + o + c, fmaf(-c2, fz, q[j] * Dr));
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
// Lets a kernel have as much dynamic shared memory as the device gives, once per device (racing
// threads set the same value).
template <auto KERN>
int allow_smem() {
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return check_launch("block_norm device");
    if (done[dev].load(std::memory_order_acquire)) return LIGER_OK;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, KERN) != cudaSuccess ||
        cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_smem_optin() - static_cast<int>(fa.sharedSizeBytes)) != cudaSuccess)
        return check_launch("block_norm attribute");
    done[dev].store(true, std::memory_order_release);
    return LIGER_OK;
}

// Resident blocks per SM of a kernel, asked once per device.
template <typename K>
int resident(K kern, int threads, size_t smem, std::atomic<int> (&cache)[64]) {
    int dev = 0;
    const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
    int n = known ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess || n < 1) n = 1;
        if (known) cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <typename T, int VEC, int VPT>
int launch_fwd_team(const FwdP& p, int tw, cudaStream_t st) {
    static std::atomic<int> cache[17][64];   // per team width: the block's threads follow from it
    const int teams = std::max(1, 8 / tw), threads = teams * tw * 32;
    auto k = block_norm_fwd_team<T, VEC, VPT>;
    const int64_t grid = std::min<int64_t>(ceil_div(p.rows, teams), static_cast<int64_t>(sm_count()) * resident(k, threads, 0, cache[tw]));
    k<<<static_cast<unsigned>(grid), threads, 0, st>>>(p, tw);
    return check_launch("block_norm_fwd_team");
}

template <typename T, int VPT, int GATE, int NT, int MB, int ONE>
int launch_fwd_ring(const FwdP& p, int tw, cudaStream_t st) {
    const int teams = std::max(1, NT / 32 / tw), threads = teams * tw * 32;
    const size_t slot = static_cast<size_t>(teams) * (2 * static_cast<size_t>(p.cols) * sizeof(T) + 8);
    constexpr auto k = block_norm_fwd_ring<T, VPT, GATE, NT, MB, ONE>;
    if (int rc = allow_smem<k>()) return rc;
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, 2 * slot);
    per_sm = std::max(1, per_sm);
    // Two slots where that holds about 52 KB of rows on an SM, else three: less in flight leaves the
    // memory idle, and more was slower (4096 bf16 columns: 64 KB 0.94 of the copy rate, 96 KB 0.84;
    // 3000: 48 KB 0.90, 72 KB 0.96).
    const int nst = per_sm * 2 * slot >= 52 * 1024 ? 2 : 3;
    if (nst == 3) {
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, 3 * slot);
        per_sm = std::max(1, per_sm);
    }
    const int64_t grid = std::min<int64_t>(ceil_div(p.rows, teams), static_cast<int64_t>(sm_count()) * per_sm);
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    k<<<static_cast<unsigned>(grid), threads, nst * slot, st>>>(p, tw, nst, err);
    return check_launch("block_norm_fwd_ring");
}

template <typename T, int VPT, int NT, int MB, int ONE>
int launch_fwd_ring(const FwdP& p, int tw, cudaStream_t st) {
    if (p.gate == nullptr) return launch_fwd_ring<T, VPT, 0, NT, MB, ONE>(p, tw, st);
    if (p.per_gate == p.rows) return launch_fwd_ring<T, VPT, 1, NT, MB, ONE>(p, tw, st);
    return launch_fwd_ring<T, VPT, 2, NT, MB, ONE>(p, tw, st);
}

template <typename T, int VPT, int NT, int MB>
int launch_fwd_ring(const FwdP& p, int nvec, cudaStream_t st) {
    const int tw = static_cast<int>(ceil_div(nvec, 32 * VPT));
    if (NT / 32 / tw > 1) return launch_fwd_ring<T, VPT, NT, MB, 0>(p, tw, st);
    return launch_fwd_ring<T, VPT, NT, MB, 1>(p, tw, st);
}

template <typename T, int EPT, int NT>
int launch_fwd_odd(const FwdP& p, cudaStream_t st) {
    constexpr auto k = block_norm_fwd_odd<T, EPT, NT>;
    if (int rc = allow_smem<k>()) return rc;
    const size_t wmax = window_max(p.cols, sizeof(T));
    int nst = 4;   // one row in use, three in flight
    while (nst > 2 && nst * (2 * wmax + 8) > 200u * 1024u) --nst;
    const size_t smem = nst * (2 * wmax + 8);
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, NT, smem);
    const int64_t grid = std::min<int64_t>(p.rows, static_cast<int64_t>(sm_count()) * std::max(1, per_sm));
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    k<<<static_cast<unsigned>(grid), NT, smem, st>>>(p, nst, static_cast<uint32_t>(wmax), err);
    return check_launch("block_norm_fwd_odd");
}

// Which kernel: by the row's 16-byte vectors, and whether there are rows enough that a team takes
// several.  Fractions of the measured copy rate with many rows, bf16 unless said:
//   ring, 1 vector a thread  256 columns 0.92, 512 0.94, 1024 0.94, 2048 0.91 (2 vectors: 0.87 and less)
//         2 vectors          1536 columns 0.93, 320 0.84 (1 vector, two half-empty warps a row: 0.60),
//                            4096 0.94, fp32 1024 0.94, fp32 4096 (512 threads) 0.97
//         2, 384 threads     5120 0.90, 6144 0.93
//         4 vectors          7168 1.00, 8192 0.96 (2 vectors, 512 threads: 0.96, 0.94), 16384 0.76
//   registers               0.67 to 0.87 over the same widths; first to finish when a team has one row
//   odd widths              fp32 1001 0.73, bf16 4095 0.35 (registers, element loads: 0.59, 0.22)
template <typename T>
int launch_fwd(const FwdP& p, cudaStream_t st) {
    constexpr int EPV = Vec<T>::N;
    constexpr bool F32 = sizeof(T) == 4;
    if (p.cols % EPV == 0) {
        const int nvec = p.cols / EPV;
        const int64_t few = static_cast<int64_t>(sm_count()) * std::max(1, 512 / std::max(nvec, 32));
        if (p.rows <= few && nvec <= 512) return launch_fwd_team<T, EPV, 1>(p, (nvec + 31) / 32, st);
        if (p.rows > few) {
            const bool whole = nvec % 32 == 0 && 8 % (nvec / 32) == 0;   // one vector a thread fills the block's warps
            if (nvec <= 32 || (!F32 && nvec <= 256 && whole)) return launch_fwd_ring<T, 1, 256, 2>(p, nvec, st);
            if (nvec <= 512) return launch_fwd_ring<T, 2, 256, 2>(p, nvec, st);
            if (nvec <= 768) return launch_fwd_ring<T, 2, 384, 2>(p, nvec, st);
            if (nvec <= 1024 && F32) return launch_fwd_ring<T, 2, 512, 1>(p, nvec, st);
            if (nvec <= 1024) return launch_fwd_ring<T, 4, 256, 1>(p, nvec, st);
            if (nvec <= 1536) return launch_fwd_ring<T, 4, 384, 1>(p, nvec, st);
            if (nvec <= 2048) return launch_fwd_ring<T, 4, 512, 1>(p, nvec, st);
        }
        if (nvec <= 1024) return launch_fwd_team<T, EPV, 2>(p, (nvec + 63) / 64, st);
        if (nvec <= 2048) return launch_fwd_team<T, EPV, 4>(p, (nvec + 127) / 128, st);
    } else {
        if (p.cols <= 128) return launch_fwd_team<T, 1, 4>(p, 1, st);
        if (p.rows <= sm_count() && p.cols <= 2048) return launch_fwd_team<T, 1, 4>(p, (p.cols + 127) / 128, st);
        if (p.cols <= 256) return launch_fwd_odd<T, 4, 64>(p, st);
        if (p.cols <= 512) return launch_fwd_odd<T, 4, 128>(p, st);
        if (p.cols <= 1024) return launch_fwd_odd<T, 4, 256>(p, st);
        if (p.cols <= 2048) return launch_fwd_odd<T, 8, 256>(p, st);
        if (p.cols <= 4096) return launch_fwd_odd<T, 8, 512>(p, st);
        if (p.cols <= 8192) return launch_fwd_odd<T, 16, 512>(p, st);
    }
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
    k<<<static_cast<unsigned>(grid), teams * tw * 32, smem, st>>>(p, tw, static_cast<int>(nst), err);
    return check_launch("block_norm_bwd_ring");
}

// Splits the rows and launches: 256 threads' worth of teams where a row takes less.
template <typename T, int VPT, int NT>
int launch_bwd_ring(BwdP& p, int nvec, size_t slot, int64_t& grid, cudaStream_t st) {
    const int tw = static_cast<int>(ceil_div(nvec, 32 * VPT));
    const int teams = std::max(1, 8 / tw);
    int per_sm = 0;
    if (int rc = allow_smem<block_norm_bwd_ring<T, VPT, 0, NT, 0>>()) return rc;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, block_norm_bwd_ring<T, VPT, 0, NT, 0>, teams * tw * 32, teams * slot);
    per_sm = std::max(1, per_sm);
    grid = split_rows(p, static_cast<int64_t>(sm_count()) * per_sm);
    // Rows up to 8 KB: the blocks walk through memory side by side (4096 bf16 columns 0.97 of the copy rate,
    // 0.90 with a run of rows each; 2048: 0.91, 0.86).  Longer rows: a run each (5120: 0.97, side by side
    // 0.77; 8192: 0.95, 0.89).
    p.interleave = static_cast<size_t>(p.cols) * sizeof(T) <= 8192 ? 1 : 0;
    if (p.splits == 0) return launch_bwd_ring<T, VPT, 1, NT, 1>(p, nvec, slot, grid, 1, per_sm, st);
    if (teams == 1) return launch_bwd_ring<T, VPT, 0, NT, 1>(p, nvec, slot, grid, 1, per_sm, st);
    return launch_bwd_ring<T, VPT, 0, NT, 0>(p, nvec, slot, grid, teams, per_sm, st);
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
    if (p.splits == 0) kw<<<static_cast<unsigned>(grid), NT, nst * slot, st>>>(p, nst, static_cast<uint32_t>(wmax), err);
    else k<<<static_cast<unsigned>(grid), NT, nst * slot, st>>>(p, nst, static_cast<uint32_t>(wmax), err);
    return check_launch("block_norm_bwd_odd");
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
        block_norm_bwd_generic<T><<<static_cast<unsigned>(grid), 256, 0, st>>>(p);
        rc = check_launch("block_norm_bwd");
    } else if (!F32 && nvec <= 256) rc = launch_bwd_ring<T, 1, 256>(p, nvec, slot, grid, st);
    else if (nvec <= 512) rc = launch_bwd_ring<T, 2, 256>(p, nvec, slot, grid, st);
    else if (nvec <= 768) rc = launch_bwd_ring<T, 2, 384>(p, nvec, slot, grid, st);
    else if (F32 && nvec <= 1024) rc = launch_bwd_ring<T, 2, 512>(p, nvec, slot, grid, st);
    else if (nvec <= 1024) rc = launch_bwd_ring<T, 4, 256>(p, nvec, slot, grid, st);
    else rc = launch_bwd_ring<T, 4, 512>(p, nvec, slot, grid, st);
    if (rc) return rc;
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
