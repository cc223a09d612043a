// Block norms, forward: post-norm, gate, scaled residual sum and pre-norm in one
// pass over the rows (formulas in liger_train.h).
//
// GB300 design: HBM-bound.  In bf16 8 bytes an element have to move (z, r in; h,
// y out); every row is read once and written once.  By the row's width and the
// number of rows: a team of warps per row over a ring of bulk copies, a team
// with the row in registers, single elements from aligned windows, or a
// generic kernel.
#include "block_norm.cuh"

namespace liger {
namespace {

struct FwdP {
    const void *z, *r, *w_post, *gate, *w_pre;
    void *h, *y;
    float *rstd_z, *rstd_h;
    int64_t rows, per_gate;   // per_gate: rows that share a gate row
    int cols;
    float a, b, eps;
};

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
    wait_for_stream();
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
    wait_for_stream();
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
// The same team per row, with the rows of z and r brought into a ring of `nst` slots per team by
// bulk copies, so that several rows per team are in flight without registers.  A slot is read into
// registers at once and is free again after the next team barrier.  Every wait is bounded; on
// expiry the team records it, waits (bounded) for its copies and writes NaN into the rows it did
// not finish.  Streaming stores and issuing the next copy only after the sums measured 0.95 of the
// copy rate at 4096 bf16 columns, against 0.93 with the copy first and 0.91 with plain stores (other
// widths: within 0.01).
// GATES 0: no gate or one gate row (folded into the post-norm's weights once); 1: several (read anew
// where a row's gate differs from that of the team's row before).
template <typename T, int VPT, int GATES, int NT, int MB, int ONE>
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
    wait_for_stream();
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
            if (p.gate != nullptr) {
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
    if (!GATES) gate_in(0);
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
    if (GATES) {
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
        if (GATES) {   // its loads run while the row is waited for
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

// ------------------------------------------- rows that are no whole 16-byte vectors
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
    wait_for_stream();
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

// ------------------------------------------------------------------ launches
template <typename T, int VEC, int VPT>
int launch_fwd_team(const FwdP& p, int tw, cudaStream_t st) {
    static std::atomic<int> cache[17][64];   // per team width: the block's threads follow from it
    const int teams = std::max(1, 8 / tw), threads = teams * tw * 32;
    auto k = block_norm_fwd_team<T, VEC, VPT>;
    const int64_t grid = std::min<int64_t>(ceil_div(p.rows, teams), static_cast<int64_t>(sm_count()) * resident(k, threads, 0, cache[tw]));
    return launch_early("block_norm_fwd_team", k, dim3(static_cast<unsigned>(grid)), threads, 0, st, p, tw);
}

template <typename T, int VPT, int GATES, int NT, int MB, int ONE>
int launch_fwd_ring(const FwdP& p, int tw, cudaStream_t st) {
    const int teams = std::max(1, NT / 32 / tw), threads = teams * tw * 32;
    const size_t slot = static_cast<size_t>(teams) * (2 * static_cast<size_t>(p.cols) * sizeof(T) + 8);
    constexpr auto k = block_norm_fwd_ring<T, VPT, GATES, NT, MB, ONE>;
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
    return launch_early("block_norm_fwd_ring", k, dim3(static_cast<unsigned>(grid)), threads, nst * slot, st, p, tw, nst, err);
}

template <typename T, int VPT, int NT, int MB, int ONE>
int launch_fwd_ring(const FwdP& p, int tw, cudaStream_t st) {
    if (p.per_gate == p.rows) return launch_fwd_ring<T, VPT, 0, NT, MB, ONE>(p, tw, st);
    return launch_fwd_ring<T, VPT, 1, NT, MB, ONE>(p, tw, st);
}

// TEAMS: whether rows can be short enough that a block holds several teams
template <typename T, int VPT, int NT, int MB, int TEAMS>
int launch_fwd_ring(const FwdP& p, int64_t nvec, cudaStream_t st) {
    const int tw = static_cast<int>(ceil_div(nvec, 32 * VPT));
    if constexpr (TEAMS != 0)
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
    return launch_early("block_norm_fwd_odd", k, dim3(static_cast<unsigned>(grid)), NT, smem, st, p, nst,
                        static_cast<uint32_t>(wmax), err);
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
            const int64_t nvec64 = nvec;
            const bool whole = nvec % 32 == 0 && 8 % (nvec / 32) == 0;   // one vector a thread fills the block's warps
            if (nvec <= 32 || (!F32 && nvec <= 256 && whole)) return launch_fwd_ring<T, 1, 256, 2, 1>(p, nvec64, st);
            if (nvec <= 512) return launch_fwd_ring<T, 2, 256, 2, 1>(p, nvec64, st);
            if (nvec <= 768) return launch_fwd_ring<T, 2, 384, 2, 0>(p, nvec64, st);
            if (nvec <= 1024 && F32) return launch_fwd_ring<T, 2, 512, 1, 0>(p, nvec64, st);
            if (nvec <= 1024) return launch_fwd_ring<T, 4, 256, 1, 0>(p, nvec64, st);
            if (nvec <= 1536) return launch_fwd_ring<T, 4, 384, 1, 0>(p, nvec64, st);
            if (nvec <= 2048) return launch_fwd_ring<T, 4, 512, 1, 0>(p, nvec64, st);
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
    return launch_early("block_norm_fwd", block_norm_fwd_generic<T>, dim3(static_cast<unsigned>(grid)), 256, 0, st, p);
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
