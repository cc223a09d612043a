// Layer norm, forward and backward (formulas in liger_layer.h).
// A row's mean comes first and its variance from the differences to it, both in fp32 over values that stay in registers, so
// that a row is read once.  The mean m is rounded, and so is the sum it comes from, by what may be many steps of the differences
// x - m where the mean is large.  fp32 rows with a mean above twice their deviation: the differences' own mean `off` is what is
// missing, the mean is m + off, the variance mean((x - m)^2) - off^2, and y is formed from x - m - off, so that a large mean costs
// the forward no digits (of 1000 deviations: y off by 1e-4 without, 1e-6 with).  Formed in every row it would cost a seventh of the
// time of wide ones; so only rows that need it pay (16384 x 8192 165 us, 205 where all do; 32768 x 4096 177 and 184).  bf16 rows:
// m is off by some 2^-14 of the inputs' own rounding, and nothing is formed.  The backward has the mean as it is stored, in fp32.
// The backward's two row sums, of dy w and of dy w xhat, are formed
// in one pass, and dw and db as fp32 column sums in registers over all rows of a block; each block leaves them as a partial row,
// added up in a fixed order.  What bounds all of it is HBM: two streams forward, three (four with dres) backward.  32768 x 4096
// bf16: forward 85 us (0.93 of the copy rate), backward with dres 155 us (1.02); a few rows: the launch (4 rows: 2.3 us of kernel).
#include "block_norm.cuh"
#include "liger_layer.h"

namespace liger {
namespace {

constexpr int kMaxPartRows = 1024;   // most partial rows of dw and of db
// Bytes of rows in flight on an SM that the rings aim at.  Forward of 32768 x 4096 bf16: 88 us with 32 KB, 85 with 64 to 192;
// of 16384 x 8192 83, 83 and 88.  Backward: 192 KB where a row is 8 KB or more (16384 x 8192 bf16: 156 us, 167 with 64 or 128 KB;
// 32768 x 4096: 155 and 158), 128 KB below (131072 x 512 bf16: 102 us, 104 with 192 KB).
constexpr size_t kFwdFlight = 64u * 1024u, kBwdFlight = 128u * 1024u, kBwdFlightLong = 192u * 1024u;

// Whether the differences' own mean is formed (above) for a row of mean m and mean square `square` of its differences to it
template <typename T> constexpr bool kOffset = sizeof(T) == 4;
template <typename T>
__device__ __forceinline__ bool far_off(float m, float square) {
    return kOffset<T> && m * m > 4.f * square;
}
// The variance from the mean square of x - m and the mean `off` of x - m (at least 0; NaN stays)
__device__ __forceinline__ float variance(float square, float off) {
    const float v = fmaf(-off, off, square);
    return v < 0.f ? 0.f : v;
}

// ------------------------------------------------------------- any width
// A block per row, elements strided over its threads; the row is read again from the caches for
// the variance and for the result.
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_fwd_rows(const T* x, const T* w, const T* b, T* y, float* mean,
                                                           float* rstd, int64_t rows, int cols, float eps) {
    __shared__ float sh[8];
    const float n = static_cast<float>(cols);
    wait_for_stream();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * cols;
        float s = 0.f;
        for (int j = threadIdx.x; j < cols; j += blockDim.x) s += ldf(xr + j);
        const float m = block_sum(s, sh) / n;
        s = 0.f;
        for (int j = threadIdx.x; j < cols; j += blockDim.x) {
            const float d = ldf(xr + j) - m;
            s = fmaf(d, d, s);
        }
        float square = block_sum(s, sh) / n, off = 0.f;
        if (far_off<T>(m, square)) {
            s = 0.f;
            for (int j = threadIdx.x; j < cols; j += blockDim.x) s += ldf(xr + j) - m;
            off = block_sum(s, sh) / n;
            square = variance(square, off);
        }
        const float rs = 1.0f / sqrtf(square + eps);
        T* yr = y + r * cols;
        for (int j = threadIdx.x; j < cols; j += blockDim.x) {
            const float h = (kOffset<T> ? ldf(xr + j) - m - off : ldf(xr + j) - m) * rs;
            stf(yr + j, fmaf(h, w != nullptr ? ldf(w + j) : 1.f, b != nullptr ? ldf(b + j) : 0.f));
        }
        if (threadIdx.x == 0) {
            if (mean != nullptr) mean[r] = kOffset<T> ? m + off : m;
            if (rstd != nullptr) rstd[r] = rs;
        }
    }
}

// ------------------------------------------------------------- rows in registers
// VEC consecutive elements as one thread holds them: a 16-byte vector, or one element where the rows
// are no whole vectors.
template <typename T, int VEC> struct Piece {
    static_assert(VEC == Vec<T>::N, "whole vectors or single elements");
    uint4 u;
    __device__ __forceinline__ void load(const T* p) { u = ldg16(p); }
    __device__ __forceinline__ void get(float (&f)[VEC]) const { unpack(u, f); }
    static __device__ __forceinline__ void put(T* p, const float (&f)[VEC]) { stg16(p, pack(f)); }
};
template <typename T> struct Piece<T, 1> {
    float v;
    __device__ __forceinline__ void load(const T* p) { v = ldf(p); }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v; }
    static __device__ __forceinline__ void put(T* p, const float (&f)[1]) { stf(p, f[0]); }
};

struct LnFwd {
    const void *x, *w, *b;
    void* y;
    float *mean, *rstd;
    int64_t rows;
    int cols;
    float eps;
};

// Few rows: a team of `tw` warps holds a row in registers, VPT pieces a thread; its mean and the
// mean of the squared differences go over the team by shuffles and one named barrier each.
template <typename T, int VEC, int VPT>
__global__ void __launch_bounds__(512) layer_norm_fwd_team(LnFwd p, int tw) {
    __shared__ float red[3][16];   // sums of the values, of the differences' squares, of the differences
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int team = warp / tw, wt = warp - team * tw, teams = (blockDim.x >> 5) / tw;
    const int tt = wt * 32 + lane, nt = tw * 32;   // thread of the team, threads of the team
    const int npiece = p.cols / VEC;
    const T *x = static_cast<const T*>(p.x), *w = static_cast<const T*>(p.w), *b = static_cast<const T*>(p.b);
    T* y = static_cast<T*>(p.y);
    const float inv = 1.0f / static_cast<float>(p.cols);
    auto team_sum = [&](int k, float v) {
        v = warp_sum(v);
        if (tw == 1) return v;
        float* sh = red[k] + team * tw;   // written again only after another barrier, which follows every read of it
        if (lane == 0) sh[wt] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(nt) : "memory");
        float s = 0.f;
        for (int i = 0; i < tw; ++i) s += sh[i];
        return s;
    };
    wait_for_stream();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * teams + team; t < p.rows; t += static_cast<int64_t>(gridDim.x) * teams) {
        const int64_t o = t * p.cols;
        Piece<T, VEC> cx[VPT], cw[VPT], cb[VPT];
        bool live[VPT];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = j * nt + tt;
            live[j] = c < npiece;
            if (live[j]) {
                cx[j].load(x + o + static_cast<int64_t>(c) * VEC);
                if (w != nullptr) cw[j].load(w + static_cast<int64_t>(c) * VEC);
                if (b != nullptr) cb[j].load(b + static_cast<int64_t>(c) * VEC);
            }
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (live[j]) {
                float f[VEC];
                cx[j].get(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += f[e];
            }
        const float m = team_sum(0, s) * inv;
        s = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (live[j]) {
                float f[VEC];
                cx[j].get(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s = fmaf(f[e] - m, f[e] - m, s);
            }
        float square = team_sum(1, s) * inv, off = 0.f;
        if (far_off<T>(m, square)) {
            s = 0.f;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (live[j]) {
                    float f[VEC];
                    cx[j].get(f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) s += f[e] - m;
                }
            off = team_sum(2, s) * inv;
            square = variance(square, off);
        }
        const float rs = inv_sqrt(square + p.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (live[j]) {
                float f[VEC], g[VEC];
                cx[j].get(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = (kOffset<T> ? f[e] - m - off : f[e] - m) * rs;
                if (w != nullptr) {
                    cw[j].get(g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[e] *= g[e];
                }
                if (b != nullptr) {
                    cb[j].get(g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[e] += g[e];
                }
                Piece<T, VEC>::put(y + o + static_cast<int64_t>(j * nt + tt) * VEC, f);
            }
        if (tt == 0) {
            if (p.mean != nullptr) p.mean[t] = kOffset<T> ? m + off : m;
            if (p.rstd != nullptr) p.rstd[t] = rs;
        }
    }
}

// ------------------------------------------------------------- rows staged by bulk copies
// Whether every thread of the team says so, with one team barrier.
__device__ __forceinline__ bool team_all(int team, int threads, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %3, 0;\n\t"
        "barrier.cta.red.and.pred p, %1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(all)
        : "r"(team + 1), "r"(threads), "r"(ok ? 1u : 0u)
        : "memory");
    return all != 0;
}

// Many rows: the same team per row, its rows brought into a ring of `nst` slots by bulk copies, so that
// several rows per team are in flight without registers; a slot is read into registers at once and is
// free again after the next team barrier.  The weights stay in registers over the rows.  Every wait is
// bounded; on expiry the team records it, waits (bounded) for its copies and writes NaN into the rows it
// did not finish.  ONE: a single team, known at compile time.
template <typename T, int VPT, int NT, int MB, int ONE>
__global__ void __launch_bounds__(NT, MB) layer_norm_fwd_ring(LnFwd p, int tw, int nst, int* err) {
    constexpr int VEC = Vec<T>::N, NP = VEC / 2;
    extern __shared__ __align__(128) uint8_t sm[];
    // sums of the values, of the differences' squares, of the differences; rows of 4: a team starts on a multiple of 4 warps or is a warp alone
    __shared__ __align__(16) float red[3][NT / 32 + 4][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (ONE) tw = blockDim.x >> 5;
    const int team = ONE ? 0 : warp / tw, wt = warp - team * tw, teams = ONE ? 1 : (blockDim.x >> 5) / tw;
    const int tt = wt * 32 + lane, nt = tw * 32;
    const int nvec = p.cols / VEC;
    const uint32_t rb = static_cast<uint32_t>(p.cols) * sizeof(T);
    const uint8_t* ring = sm + static_cast<size_t>(team) * nst * rb;
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(teams) * nst * rb) + 8u * team * nst;
    const T *x = static_cast<const T*>(p.x), *w = static_cast<const T*>(p.w), *b = static_cast<const T*>(p.b);
    T* y = static_cast<T*>(p.y);
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t t = static_cast<int64_t>(blockIdx.x) * teams + team;
    auto issue = [&](int64_t row, int s) {
        mbar_expect_tx(bars + 8u * s, rb);
        bulk_g2s(smem_u32(ring + static_cast<size_t>(s) * rb), x + row * p.cols, rb, bars + 8u * s);
    };
    for (int i = threadIdx.x; i < 3 * (NT / 32 + 4) * 4; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
    if (tt == 0)
        for (int s = 0; s < nst; ++s) mbar_init(bars + 8u * s, 1);
    mbar_init_fence();
    __syncthreads();
    wait_for_stream();
    if (tt == 0)
        for (int s = 0; s < nst; ++s)
            if (t + s * step < p.rows) issue(t + s * step, s);
    uint4 cw[VPT], cb[VPT];
    bool live[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int64_t c = static_cast<int64_t>(j * nt + tt) * VEC;
        live[j] = j * nt + tt < nvec;
        cw[j] = cb[j] = make_uint4(0, 0, 0, 0);
        if (live[j] && w != nullptr) cw[j] = ldg16(w + c);
        if (live[j] && b != nullptr) cb[j] = ldg16(b + c);
    }
    const int at0 = ONE ? 0 : team * ((tw + 3) & ~3);
    // Team-wide sum in two halves: gather() brings the warps' sums together in place k and says whether every thread
    // of the team got its row (one team barrier), total() adds them up.  A place is written again only after another barrier.
    auto gather = [&](int k, float& v, bool& ok) {
        v = warp_sum(v);
        if (!ONE && tw == 1) {
            ok = __all_sync(0xffffffffu, ok);
            return;
        }
        if (lane == 0) (&red[k][0][0])[at0 + wt] = v;
        ok = ONE ? __syncthreads_and(ok ? 1 : 0) != 0 : team_all(team, nt, ok);
    };
    auto total = [&](int k, float v) {
        if (!ONE && tw == 1) return v;
        const float4* q = reinterpret_cast<const float4*>(&red[k][0][0] + at0);   // slots past the team's warps hold 0
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < (NT / 32 + 3) / 4; ++i)
            if (i * 4 < tw) {
                const float4 a = q[i];
                s += (a.x + a.y) + (a.z + a.w);
            }
        return s;
    };
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; t < p.rows; t += step) {
        ok = mbar_wait(bars + 8u * s, ph);
        const uint8_t* slot = ring + static_cast<size_t>(s) * rb;
        uint4 cx[VPT];
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            cx[j] = make_uint4(0, 0, 0, 0);
            if (live[j] && ok) cx[j] = *reinterpret_cast<const uint4*>(slot + static_cast<size_t>(j * nt + tt) * 16);
            float2 f[NP];
            unpack2(cx[j], f);
#pragma unroll
            for (int e = 0; e < NP; ++e) a = __fadd2_rn(a, f[e]);
        }
        float sum = a.x + a.y;
        gather(0, sum, ok);
        if (!ok) break;
        const float m = total(0, sum) * inv;
        if (tt == 0 && t + nst * step < p.rows) {   // every thread of the team has read the slot
            fence_proxy_async_smem();
            issue(t + nst * step, s);
        }
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
        const float2 nm = make_float2(-m, -m);
        a = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (live[j]) {
                float2 f[NP];
                unpack2(cx[j], f);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    f[e] = __fadd2_rn(f[e], nm);
                    a = __ffma2_rn(f[e], f[e], a);
                }
            }
        sum = a.x + a.y;
        bool same = true;
        gather(1, sum, same);
        float square = total(1, sum) * inv, off = 0.f;
        if (far_off<T>(m, square)) {
            a = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (live[j]) {
                    float2 f[NP];
                    unpack2(cx[j], f);
#pragma unroll
                    for (int e = 0; e < NP; ++e) a = __fadd2_rn(a, __fadd2_rn(f[e], nm));
                }
            sum = a.x + a.y;
            gather(2, sum, same);
            off = total(2, sum) * inv;
            square = variance(square, off);
        }
        const float rs = inv_sqrt(square + p.eps);
        const float2 rs2 = make_float2(rs, rs), no2 = make_float2(-off * rs, -off * rs);   // (x - m) rstd - off rstd
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (live[j]) {
                float2 f[NP], g[NP], h[NP];
                unpack2(cx[j], f);
                unpack2(cw[j], g);
                unpack2(cb[j], h);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    f[e] = __fadd2_rn(f[e], nm);
                    f[e] = kOffset<T> ? __ffma2_rn(f[e], rs2, no2) : __fmul2_rn(f[e], rs2);
                    f[e] = w != nullptr ? __ffma2_rn(f[e], g[e], h[e]) : __fadd2_rn(f[e], h[e]);
                }
                stg16_cs(y + t * p.cols + static_cast<int64_t>(j * nt + tt) * VEC, pack2(f));
            }
        if (tt == 0) {
            if (p.mean != nullptr) p.mean[t] = kOffset<T> ? m + off : m;
            if (p.rstd != nullptr) p.rstd[t] = rs;
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
        for (int v = tt; v < nvec; v += nt) stg16(y + t * p.cols + static_cast<int64_t>(v) * VEC, nan16<T>());
        if (tt == 0 && p.mean != nullptr) p.mean[t] = nan;
        if (tt == 0 && p.rstd != nullptr) p.rstd[t] = nan;
    }
}

// Rows that are no whole vectors: aligned windows around them (block_norm.cuh).  A row starts `shift` elements into its
// window; rows that lie a multiple of VEC apart have the same shift, and a block only takes such rows.  So the columns of
// a thread's vectors stay the same from row to row, as do its weights, and only the first and the last vector of a
// window, which the neighbouring rows share, go by elements.
template <typename T> struct Span {
    static constexpr int VEC = Vec<T>::N, NP = VEC / 2;
    static constexpr uint32_t kAll = (1u << VEC) - 1u;
    int shift, end, nv;   // the row is elements [shift, end) of its window of nv vectors
    __device__ __forceinline__ Span(int64_t row, int64_t rows, int cols) {
        shift = window_of<T>(row, rows, cols).shift;
        end = shift + cols;
        nv = (end + VEC - 1) / VEC;
    }
    // a bit for each element of vector v that is the row's
    __device__ __forceinline__ uint32_t inside(int v) const {
        const int lo = min(max(shift - v * VEC, 0), VEC), hi = min(max(end - v * VEC, 0), VEC);
        return ((1u << hi) - 1u) & ~((1u << lo) - 1u);
    }
    __device__ __forceinline__ void mask(uint32_t in, float2 (&f)[NP]) const {
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            f[e].x = in >> (2 * e) & 1u ? f[e].x : 0.f;
            f[e].y = in >> (2 * e + 1) & 1u ? f[e].y : 0.f;
        }
    }
    // vector v of a row in global memory, by elements, 0 outside the row
    __device__ __forceinline__ uint4 gather(const T* row, int v) const {
        const uint32_t in = inside(v);
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = in >> e & 1u ? ldf(row + v * VEC + e - shift) : 0.f;
        return pack(f);
    }
    // the same from the row's window in shared memory
    __device__ __forceinline__ uint4 take(const uint8_t* window, int v, uint32_t in) const {
        uint4 u = *reinterpret_cast<const uint4*>(window + v * 16);
        if (in == kAll) return u;
        auto keep = [&](int i) {
            if constexpr (VEC == 4) return in >> i & 1u ? 0xffffffffu : 0u;
            else return (in >> (2 * i) & 1u ? 0xffffu : 0u) | (in >> (2 * i + 1) & 1u ? 0xffff0000u : 0u);
        };
        u.x &= keep(0);
        u.y &= keep(1);
        u.z &= keep(2);
        u.w &= keep(3);
        return u;
    }
    __device__ __forceinline__ void put(T* row, int v, uint32_t in, const float2 (&f)[NP]) const {
        T* at = row - shift + v * VEC;
        if (in == kAll) {
            stg16_cs(at, pack2(f));
            return;
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            if (in >> (2 * e) & 1u) stf(at + 2 * e, f[e].x);
            if (in >> (2 * e + 1) & 1u) stf(at + 2 * e + 1, f[e].y);
        }
    }
    // The copy of the last row's window may stop short of its end: the elements behind go by plain stores, before the thread that
    // asks for the copy arrives at its barrier.
    static __device__ __forceinline__ void rest(uint8_t* window, const Window& win, const T* row, int cols) {
        for (int c = win.tail; c < cols; ++c) reinterpret_cast<T*>(window)[win.shift + c] = row[c];
    }
};

template <typename T, int VPT, int NT, int MB>
__global__ void __launch_bounds__(NT, MB) layer_norm_fwd_odd(LnFwd p, int nst, uint32_t wmax, int* err) {
    constexpr int VEC = Vec<T>::N, NP = VEC / 2;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ __align__(16) float red[2][NT / 32];   // (slots of warps that the block has not hold 0)
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nt = blockDim.x;
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(nst) * wmax);
    const T *x = static_cast<const T*>(p.x), *w = static_cast<const T*>(p.w), *b = static_cast<const T*>(p.b);
    T* y = static_cast<T*>(p.y);
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int64_t step = gridDim.x;
    int64_t t = blockIdx.x;
    const Span<T> span(t, p.rows, p.cols);
    auto issue = [&](int64_t row, int s) {
        const Window win = window_of<T>(row, p.rows, p.cols);
        Span<T>::rest(sm + static_cast<size_t>(s) * wmax, win, x + row * p.cols, p.cols);
        mbar_expect_tx(bars + 8u * s, win.bytes);
        if (win.bytes > 0)
            bulk_g2s(smem_u32(sm + static_cast<size_t>(s) * wmax), static_cast<const uint8_t*>(p.x) + win.at, win.bytes, bars + 8u * s);
    };
    if (tid < 2 * (NT / 32)) (&red[0][0])[tid] = 0.f;
    if (tid == 0)
        for (int s = 0; s < nst; ++s) mbar_init(bars + 8u * s, 1);
    mbar_init_fence();
    __syncthreads();
    wait_for_stream();
    if (tid == 0)
        for (int s = 0; s < nst; ++s)
            if (t + s * step < p.rows) issue(t + s * step, s);
    uint4 cw[VPT], cb[VPT];
    uint32_t in[VPT];   // 0: no vector of the row
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        in[j] = span.inside(j * nt + tid);
        cw[j] = cb[j] = make_uint4(0, 0, 0, 0);
        if (w != nullptr) cw[j] = span.gather(w, j * nt + tid);
        if (b != nullptr) cb[j] = span.gather(b, j * nt + tid);
    }
    int turn = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    auto put = [&](float v) {
        v = warp_sum(v);
        if (lane == 0) red[turn][wid] = v;
    };
    auto total = [&]() {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) a += red[turn][i];
        turn ^= 1;   // written again only after the next barrier
        return a;
    };
    for (; t < p.rows; t += step) {
        ok = mbar_wait(bars + 8u * s, ph);
        const uint8_t* slot = sm + static_cast<size_t>(s) * wmax;
        const int64_t o = t * p.cols;
        uint4 cx[VPT];
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            cx[j] = make_uint4(0, 0, 0, 0);
            if (in[j] != 0 && ok) cx[j] = span.take(slot, j * nt + tid, in[j]);
            float2 f[NP];
            unpack2(cx[j], f);
#pragma unroll
            for (int e = 0; e < NP; ++e) a = __fadd2_rn(a, f[e]);
        }
        put(a.x + a.y);
        ok = __syncthreads_and(ok ? 1 : 0) != 0;
        if (!ok) break;
        if (tid == 0 && t + nst * step < p.rows) {   // every thread has its vectors of the row
            fence_proxy_async_smem();
            issue(t + nst * step, s);
        }
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
        const float m = total() * inv;
        const float2 nm = make_float2(-m, -m);
        auto differences = [&](int j, float2 (&f)[NP]) {   // 0 outside the row
            unpack2(cx[j], f);
#pragma unroll
            for (int e = 0; e < NP; ++e) f[e] = __fadd2_rn(f[e], nm);
            if (in[j] != Span<T>::kAll) span.mask(in[j], f);
        };
        a = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (in[j] != 0) {
                float2 f[NP];
                differences(j, f);
#pragma unroll
                for (int e = 0; e < NP; ++e) a = __ffma2_rn(f[e], f[e], a);
            }
        put(a.x + a.y);
        __syncthreads();
        float square = total() * inv, off = 0.f;
        if (far_off<T>(m, square)) {
            a = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (in[j] != 0) {
                    float2 f[NP];
                    differences(j, f);
#pragma unroll
                    for (int e = 0; e < NP; ++e) a = __fadd2_rn(a, f[e]);
                }
            put(a.x + a.y);
            __syncthreads();
            off = total() * inv;
            square = variance(square, off);
        }
        const float rs = inv_sqrt(square + p.eps);
        const float2 rs2 = make_float2(rs, rs), no2 = make_float2(-off * rs, -off * rs);   // (x - m) rstd - off rstd
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (in[j] != 0) {
                float2 f[NP], g[NP], h[NP];
                unpack2(cx[j], f);
                unpack2(cw[j], g);
                unpack2(cb[j], h);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    f[e] = __fadd2_rn(f[e], nm);
                    f[e] = kOffset<T> ? __ffma2_rn(f[e], rs2, no2) : __fmul2_rn(f[e], rs2);
                    f[e] = w != nullptr ? __ffma2_rn(f[e], g[e], h[e]) : __fadd2_rn(f[e], h[e]);
                }
                span.put(y + o, j * nt + tid, in[j], f);
            }
        if (tid == 0) {
            if (p.mean != nullptr) p.mean[t] = kOffset<T> ? m + off : m;
            if (p.rstd != nullptr) p.rstd[t] = rs;
        }
    }
    if (ok) return;
    if (tid == 0) {
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
        for (int c = tid; c < p.cols; c += nt) stf(y + t * p.cols + c, nan);
        if (tid == 0 && p.mean != nullptr) p.mean[t] = nan;
        if (tid == 0 && p.rstd != nullptr) p.rstd[t] = nan;
    }
}

struct LnBwd {
    const void *dy, *dres, *x, *w;
    const float *mean, *rstd;
    void* dx;
    float *part_w, *part_b;   // [blocks][cols] each, or NULL
    int64_t rows, rows_per_block;
    int cols;
};

// A block per run of rows; its partial rows of dw and db stand in the workspace, each element
// touched by one thread only.
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_bwd_rows(LnBwd p) {
    __shared__ float sh[8];
    const T *dy = static_cast<const T*>(p.dy), *dres = static_cast<const T*>(p.dres), *x = static_cast<const T*>(p.x),
            *w = static_cast<const T*>(p.w);
    T* dx = static_cast<T*>(p.dx);
    float* pw = p.part_w != nullptr ? p.part_w + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    float* pb = p.part_b != nullptr ? p.part_b + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    const float n = static_cast<float>(p.cols);
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_block, r1 = min(p.rows, r0 + p.rows_per_block);
    wait_for_stream();
    for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
        if (pw != nullptr) pw[j] = 0.f;
        if (pb != nullptr) pb[j] = 0.f;
    }
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t o = r * p.cols;
        const float m = p.mean[r], rs = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
            const float g = ldf(dy + o + j) * (w != nullptr ? ldf(w + j) : 1.f);
            s1 += g;
            s2 = fmaf(g, (ldf(x + o + j) - m) * rs, s2);
        }
        s1 = block_sum(s1, sh) / n;
        s2 = block_sum(s2, sh) / n;
        for (int j = threadIdx.x; j < p.cols; j += blockDim.x) {
            const float d = ldf(dy + o + j), xh = (ldf(x + o + j) - m) * rs;
            const float g = d * (w != nullptr ? ldf(w + j) : 1.f);
            stf(dx + o + j, fmaf(rs, g - s1 - xh * s2, dres != nullptr ? ldf(dres + o + j) : 0.f));
            if (pw != nullptr) pw[j] = fmaf(d, xh, pw[j]);
            if (pb != nullptr) pb[j] += d;
        }
    }
}

// ------------------------------------------------------------- backward, rows staged by bulk copies
// A block takes every gridDim.x-th row; in it a team of `tw` warps takes every teams-th of those, the row's
// dy, x (and dres) brought into the team's ring of `nst` slots.  Each thread owns VPT 16-byte column
// vectors: the weight and its shares of dw and db stay in fp32 registers over the rows.  The two sums of a
// row are reduced together (one team barrier a row), across which its values stay in registers, and the
// slot is free at once for the next copies.  Arithmetic on column pairs with the packed fp32x2
// instructions.  Every wait is bounded; on expiry the block records it, waits (bounded) for its copies and
// writes NaN into the rows and sums it did not finish.
template <typename T, int VPT, int NT, int ONE>
__global__ void __launch_bounds__(NT, 1) layer_norm_bwd_ring(LnBwd p, int tw, int nst, int* err) {
    constexpr int VEC = Vec<T>::N, NP = VEC / 2;
    extern __shared__ __align__(128) uint8_t sm[];
    // per team its warps' sums, from a multiple of 4: at most 4 entries for every warp
    __shared__ __align__(16) float red[2][2][NT / 32 * 4];
    __shared__ int failed;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (ONE) tw = blockDim.x >> 5;
    const int team = ONE ? 0 : warp / tw, wt = warp - team * tw, teams = ONE ? 1 : (blockDim.x >> 5) / tw;
    const int tt = wt * 32 + lane, nt = tw * 32;
    const int nvec = p.cols / VEC;
    const uint32_t rb = static_cast<uint32_t>(p.cols) * sizeof(T);
    const T *dy = static_cast<const T*>(p.dy), *x = static_cast<const T*>(p.x), *dres = static_cast<const T*>(p.dres),
            *w = static_cast<const T*>(p.w);
    T* dx = static_cast<T*>(p.dx);
    const bool res = dres != nullptr;
    const uint32_t slot_bytes = rb * (res ? 3 : 2);
    const uint8_t* ring = sm + static_cast<size_t>(team) * nst * slot_bytes;
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(teams) * nst * slot_bytes) + 8u * team * nst;
    int64_t t = blockIdx.x + static_cast<int64_t>(team) * gridDim.x;
    const int64_t step = static_cast<int64_t>(teams) * gridDim.x;
    auto issue = [&](int64_t row, int s) {
        const uint32_t bar = bars + 8u * s, dst = smem_u32(ring + static_cast<size_t>(s) * slot_bytes);
        mbar_expect_tx(bar, slot_bytes);
        bulk_g2s(dst, dy + row * p.cols, rb, bar);
        bulk_g2s(dst + rb, x + row * p.cols, rb, bar);
        if (res) bulk_g2s(dst + 2 * rb, dres + row * p.cols, rb, bar);
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
            if (t + s * step < p.rows) issue(t + s * step, s);
    float2 wf[VPT][NP], Sw[VPT][NP], Sb[VPT][NP];
    bool live[VPT];
    const float2 zero2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        live[j] = j * nt + tt < nvec;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            wf[j][e] = make_float2(1.f, 1.f);
            Sw[j][e] = Sb[j][e] = zero2;
        }
        if (live[j] && w != nullptr) unpack2(ldg16(w + static_cast<int64_t>(j * nt + tt) * VEC), wf[j]);
    }
    const float inv = 1.0f / static_cast<float>(p.cols);
    const int at = ONE ? 0 : team * ((tw + 3) & ~3);
    int s = 0, turn = 0;
    uint32_t ph = 0;
    bool ok = true;
    // the next row's mean and rstd, fetched a row ahead
    float mn = t < p.rows ? p.mean[t] : 0.f, rn = t < p.rows ? p.rstd[t] : 0.f;
    for (; t < p.rows; t += step) {
        const float m = mn, rs = rn;
        if (t + step < p.rows) {
            mn = p.mean[t + step];
            rn = p.rstd[t + step];
        }
        ok = mbar_wait(bars + 8u * s, ph);
        const uint8_t* slot = ring + static_cast<size_t>(s) * slot_bytes;
        uint4 cy[VPT], cx[VPT], cr[VPT];
        float2 a1 = zero2, a2 = zero2;
        const float2 nm = make_float2(-m, -m), rs2 = make_float2(rs, rs);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const size_t o = static_cast<size_t>(j * nt + tt) * 16;
            cy[j] = cx[j] = cr[j] = make_uint4(0, 0, 0, 0);
            if (!(live[j] && ok)) continue;
            cy[j] = *reinterpret_cast<const uint4*>(slot + o);
            cx[j] = *reinterpret_cast<const uint4*>(slot + rb + o);
            if (res) cr[j] = *reinterpret_cast<const uint4*>(slot + 2 * rb + o);
            float2 fy[NP], fx[NP];
            unpack2(cy[j], fy);
            unpack2(cx[j], fx);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 xh = __fmul2_rn(__fadd2_rn(fx[e], nm), rs2);
                const float2 g = __fmul2_rn(fy[e], wf[j][e]);
                a1 = __fadd2_rn(a1, g);
                a2 = __ffma2_rn(g, xh, a2);
                Sw[j][e] = __ffma2_rn(fy[e], xh, Sw[j][e]);
                Sb[j][e] = __fadd2_rn(Sb[j][e], fy[e]);
            }
        }
        float s1 = a1.x + a1.y, s2 = a2.x + a2.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
        if (!ONE && tw == 1) {
            ok = __all_sync(0xffffffffu, ok);
        } else {
            if (lane == 0) {
                red[turn][0][at + wt] = s1;
                red[turn][1][at + wt] = s2;
            }
            ok = ONE ? __syncthreads_and(ok ? 1 : 0) != 0 : team_all(team, nt, ok);
        }
        if (!ok) break;
        if (ONE || tw > 1) {
            s1 = s2 = 0.f;
#pragma unroll
            for (int i = 0; i < (NT / 32 + 3) / 4; ++i)   // entries past the team's warps hold 0
                if (ONE || i * 4 < tw) {
                    const float4 f = reinterpret_cast<const float4*>(red[turn][0] + at)[i];
                    const float4 g = reinterpret_cast<const float4*>(red[turn][1] + at)[i];
                    s1 += (f.x + f.y) + (f.z + f.w);
                    s2 += (g.x + g.y) + (g.z + g.w);
                }
            turn ^= 1;   // this buffer is written again only after the next barrier
        }
        if (tt == 0 && t + nst * step < p.rows) {   // every thread of the team has the row's values
            fence_proxy_async_smem();
            issue(t + nst * step, s);
        }
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
        const float2 nc1 = make_float2(-s1 * inv, -s1 * inv), nc2 = make_float2(-s2 * inv, -s2 * inv);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (!live[j]) continue;
            float2 fy[NP], fx[NP], o[NP];
            unpack2(cy[j], fy);
            unpack2(cx[j], fx);
            unpack2(cr[j], o);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 xh = __fmul2_rn(__fadd2_rn(fx[e], nm), rs2);
                float2 g = __ffma2_rn(fy[e], wf[j][e], nc1);
                g = __ffma2_rn(nc2, xh, g);
                o[e] = __ffma2_rn(rs2, g, o[e]);
            }
            stg16_cs(dx + t * p.cols + static_cast<int64_t>(j * nt + tt) * VEC, pack2(o));
        }
    }
    if (!ok) {
        if (tt == 0) {
            failed = 1;
            atomicExch(err, 1);
            int64_t row = t;   // the team's copies in flight: rows t, t + step, ..., the first in slot s
            for (int i = 0; i < nst && row < p.rows; ++i, row += step) {
                mbar_wait(bars + 8u * s, ph);
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        for (int64_t row = t; row < p.rows; row += step)
            for (int v = tt; v < nvec; v += nt) stg16(dx + row * p.cols + static_cast<int64_t>(v) * VEC, nan16<T>());
    }
    // the block's partial rows: the teams' sums in the order of the teams, through the ring's memory once no
    // copy is in flight (every team has waited for all its rows, or for its copies above)
    __syncthreads();
    const bool bad = failed != 0;
    float2* acc = reinterpret_cast<float2*>(sm);   // per column vector: NP of dw, NP of db
    float* pw = p.part_w != nullptr ? p.part_w + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    float* pb = p.part_b != nullptr ? p.part_b + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    for (int k = 0; k < teams; ++k) {
        if (team == k) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (!live[j]) continue;
                const int v = j * nt + tt;
                float2 sw[NP], sb[NP];
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    sw[e] = Sw[j][e];
                    sb[e] = Sb[j][e];
                    if (k > 0) {
                        sw[e] = __fadd2_rn(acc[v * 2 * NP + e], sw[e]);
                        sb[e] = __fadd2_rn(acc[v * 2 * NP + NP + e], sb[e]);
                    }
                    if (k + 1 < teams) {
                        acc[v * 2 * NP + e] = sw[e];
                        acc[v * 2 * NP + NP + e] = sb[e];
                    }
                }
                if (k + 1 == teams) {
#pragma unroll
                    for (int e = 0; e < NP; e += 2) {
                        const int64_t c = static_cast<int64_t>(v) * VEC + 2 * e;
                        const float2 ow[2] = {sw[e], sw[e + 1]}, ob[2] = {sb[e], sb[e + 1]};
                        if (pw != nullptr) stg16(pw + c, bad ? nan16<float>() : pack2(ow));
                        if (pb != nullptr) stg16(pb + c, bad ? nan16<float>() : pack2(ob));
                    }
                }
            }
        }
        if (k + 1 < teams) __syncthreads();
    }
}

// Rows that are no whole vectors: windows of one shift a block, as in the forward.
template <typename T, int VPT, int NT, int MB>
__global__ void __launch_bounds__(NT, MB) layer_norm_bwd_odd(LnBwd p, int nst, uint32_t wmax, int* err) {
    constexpr int VEC = Vec<T>::N, NP = VEC / 2;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float red[2][2][NT / 32];   // (slots of warps that the block has not hold 0)
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nt = blockDim.x;
    const T *dy = static_cast<const T*>(p.dy), *x = static_cast<const T*>(p.x), *dres = static_cast<const T*>(p.dres),
            *w = static_cast<const T*>(p.w);
    T* dx = static_cast<T*>(p.dx);
    const bool res = dres != nullptr;
    const uint32_t slot_bytes = wmax * (res ? 3 : 2);
    const uint32_t bars = smem_u32(sm + static_cast<size_t>(nst) * slot_bytes);
    int64_t t = blockIdx.x;
    const int64_t step = gridDim.x;
    const Span<T> span(t, p.rows, p.cols);
    auto issue = [&](int64_t row, int s) {
        const Window win = window_of<T>(row, p.rows, p.cols);
        const uint32_t bar = bars + 8u * s, dst = smem_u32(sm + static_cast<size_t>(s) * slot_bytes);
        uint8_t* at = sm + static_cast<size_t>(s) * slot_bytes;
        Span<T>::rest(at, win, dy + row * p.cols, p.cols);
        Span<T>::rest(at + wmax, win, x + row * p.cols, p.cols);
        if (res) Span<T>::rest(at + 2 * wmax, win, dres + row * p.cols, p.cols);
        mbar_expect_tx(bar, (res ? 3 : 2) * win.bytes);
        if (win.bytes == 0) return;
        bulk_g2s(dst, static_cast<const uint8_t*>(p.dy) + win.at, win.bytes, bar);
        bulk_g2s(dst + wmax, static_cast<const uint8_t*>(p.x) + win.at, win.bytes, bar);
        if (res) bulk_g2s(dst + 2 * wmax, static_cast<const uint8_t*>(p.dres) + win.at, win.bytes, bar);
    };
    for (int i = tid; i < 4 * (NT / 32); i += nt) (&red[0][0][0])[i] = 0.f;
    if (tid == 0)
        for (int s = 0; s < nst; ++s) mbar_init(bars + 8u * s, 1);
    mbar_init_fence();
    __syncthreads();
    wait_for_stream();
    if (tid == 0)
        for (int s = 0; s < nst; ++s)
            if (t + s * step < p.rows) issue(t + s * step, s);
    uint4 cw[VPT];
    uint32_t in[VPT];   // 0: no vector of the row
    float2 Sw[VPT][NP], Sb[VPT][NP];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        in[j] = span.inside(j * nt + tid);
        if (w != nullptr) {
            cw[j] = span.gather(w, j * nt + tid);
        } else {
            float one[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) one[e] = 1.f;
            cw[j] = pack(one);
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) Sw[j][e] = Sb[j][e] = make_float2(0.f, 0.f);
    }
    const float inv = 1.0f / static_cast<float>(p.cols);
    int s = 0, turn = 0;
    uint32_t ph = 0;
    bool ok = true;
    float mn = t < p.rows ? p.mean[t] : 0.f, rn = t < p.rows ? p.rstd[t] : 0.f;
    for (; t < p.rows; t += step) {
        const float m = mn, rs = rn;
        if (t + step < p.rows) {
            mn = p.mean[t + step];
            rn = p.rstd[t + step];
        }
        ok = mbar_wait(bars + 8u * s, ph);
        const uint8_t* slot = sm + static_cast<size_t>(s) * slot_bytes;
        const int64_t o = t * p.cols;
        const float2 nm = make_float2(-m, -m), rs2 = make_float2(rs, rs);
        uint4 cd[VPT], cx[VPT], cr[VPT];
        float2 a1 = make_float2(0.f, 0.f), a2 = a1;
        // a vector of the normalised row, 0 outside the row
        auto normed = [&](const uint4& u, uint32_t in, float2 (&f)[NP]) {
            unpack2(u, f);
#pragma unroll
            for (int e = 0; e < NP; ++e) f[e] = __fmul2_rn(__fadd2_rn(f[e], nm), rs2);
            if (in != Span<T>::kAll) span.mask(in, f);
        };
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * nt + tid;
            if (in[j] == 0 || !ok) continue;
            cd[j] = span.take(slot, v, in[j]);
            cx[j] = span.take(slot + wmax, v, in[j]);
            if (res) cr[j] = span.take(slot + 2 * wmax, v, in[j]);
            float2 d[NP], h[NP], g[NP];
            unpack2(cd[j], d);
            unpack2(cw[j], g);
            normed(cx[j], in[j], h);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                g[e] = __fmul2_rn(d[e], g[e]);
                a1 = __fadd2_rn(a1, g[e]);
                a2 = __ffma2_rn(g[e], h[e], a2);
                Sw[j][e] = __ffma2_rn(d[e], h[e], Sw[j][e]);
                Sb[j][e] = __fadd2_rn(Sb[j][e], d[e]);
            }
        }
        float s1 = a1.x + a1.y, s2 = a2.x + a2.y;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) {
            s1 += __shfl_xor_sync(0xffffffffu, s1, i);
            s2 += __shfl_xor_sync(0xffffffffu, s2, i);
        }
        if (lane == 0) {
            red[turn][0][wid] = s1;
            red[turn][1][wid] = s2;
        }
        ok = __syncthreads_and(ok ? 1 : 0) != 0;
        if (!ok) break;
        if (tid == 0 && t + nst * step < p.rows) {   // every thread has its vectors of the row
            fence_proxy_async_smem();
            issue(t + nst * step, s);
        }
        if (++s == nst) {
            s = 0;
            ph ^= 1u;
        }
        s1 = s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            s1 += red[turn][0][i];
            s2 += red[turn][1][i];
        }
        turn ^= 1;
        const float2 n1 = make_float2(-s1 * inv, -s1 * inv), n2 = make_float2(-s2 * inv, -s2 * inv);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (in[j] == 0) continue;
            float2 d[NP], h[NP], g[NP], r[NP];
            unpack2(cd[j], d);
            unpack2(cw[j], g);
            normed(cx[j], in[j], h);
            if (res) unpack2(cr[j], r);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                d[e] = __ffma2_rn(h[e], n2, __ffma2_rn(d[e], g[e], n1));
                d[e] = res ? __ffma2_rn(rs2, d[e], r[e]) : __fmul2_rn(rs2, d[e]);
            }
            span.put(dx + o, j * nt + tid, in[j], d);
        }
    }
    float* pw = p.part_w != nullptr ? p.part_w + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    float* pb = p.part_b != nullptr ? p.part_b + static_cast<int64_t>(blockIdx.x) * p.cols : nullptr;
    const float nan = __int_as_float(0x7FC00000);
    if (!ok) {
        if (tid == 0) {
            atomicExch(err, 1);
            int64_t row = t;
            for (int i = 0; i < nst && row < p.rows; ++i, row += step) {
                mbar_wait(bars + 8u * s, ph);
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        for (int64_t row = t; row < p.rows; row += step)
            for (int c = tid; c < p.cols; c += nt) stf(dx + row * p.cols + c, nan);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int col = (j * nt + tid) * VEC + e - span.shift;
            if ((in[j] >> e & 1u) == 0) continue;
            if (pw != nullptr) pw[col] = !ok ? nan : e % 2 ? Sw[j][e / 2].y : Sw[j][e / 2].x;
            if (pb != nullptr) pb[col] = !ok ? nan : e % 2 ? Sb[j][e / 2].y : Sb[j][e / 2].x;
        }
}

// dw (blockIdx.y 0) and db (1) from the partial rows: a block of 32 warps over 32 groups of V columns, warp w
// adding the partial rows w, w + 32, ... in ascending order, the slices then added in their order.
template <typename T, int V>
__global__ void __launch_bounds__(1024) layer_norm_sums(const float* part_w, const float* part_b, T* dw, T* db, int parts,
                                                        int cols) {
    __shared__ float red[32][32][V];
    wait_for_stream();
    const float* part = blockIdx.y == 0 ? part_w : part_b;
    T* out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr) return;
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * V;
    float s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int i = sl; i < parts; i += 32) {
            float v[V];
            const float* src = part + static_cast<int64_t>(i) * cols + c;
            if constexpr (V == 4) unpack(ldg16(src), v);
            else v[0] = *src;
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] += v[e];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[sl][lane][e] = s[e];
    __syncthreads();
    if (sl != 0 || c >= cols) return;
    for (int i = 1; i < 32; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] += red[i][lane][e];
#pragma unroll
    for (int e = 0; e < V; ++e) stf(out + c + e, s[e]);
}

int check_sizes(const char* who, int64_t rows, int64_t cols, int dtype) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (rows < 0 || cols <= 0 || cols > (1 << 24) || rows > (int64_t{1} << 48) / cols)
        return fail(LIGER_ERR_SHAPE, "%s: rows=%lld cols=%lld", who, (long long)rows, (long long)cols);
    return LIGER_OK;
}

// ------------------------------------------------------------------ launches
template <typename T, int VEC, int VPT>
int fwd_team(const LnFwd& p, int tw, cudaStream_t st) {
    const int teams = std::max(1, 8 / tw), threads = teams * tw * 32;
    const int64_t grid = std::min<int64_t>(ceil_div(p.rows, teams), 8 * sm_count());
    return launch_early("layernorm_fwd", layer_norm_fwd_team<T, VEC, VPT>, dim3(static_cast<unsigned>(grid)), threads, 0, st, p, tw);
}

template <typename T, int VPT, int NT, int MB, int ONE>
int fwd_ring_teams(const LnFwd& p, int tw, cudaStream_t st) {
    const int teams = std::max(1, NT / 32 / tw), threads = teams * tw * 32;
    const size_t slot = static_cast<size_t>(teams) * (static_cast<size_t>(p.cols) * sizeof(T) + 8);
    constexpr auto k = layer_norm_fwd_ring<T, VPT, NT, MB, ONE>;
    if (int rc = allow_smem<k>()) return rc;
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, 2 * slot);
    per_sm = std::max(1, per_sm);
    const int nst = static_cast<int>(std::max<size_t>(2, std::min<size_t>(4, (kFwdFlight + per_sm * slot - 1) / (per_sm * slot))));
    if (nst > 2) {
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, nst * slot);
        per_sm = std::max(1, per_sm);
    }
    const int64_t grid = std::min<int64_t>(ceil_div(p.rows, teams), static_cast<int64_t>(sm_count()) * per_sm);
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    return launch_early("layernorm_fwd", k, dim3(static_cast<unsigned>(grid)), threads, nst * slot, st, p, tw, nst, err);
}
// TEAMS: whether rows can be short enough that a block holds several teams
template <typename T, int VPT, int NT, int MB, int TEAMS>
int fwd_ring(const LnFwd& p, int nvec, cudaStream_t st) {
    const int tw = static_cast<int>(ceil_div(nvec, 32 * VPT));
    if constexpr (TEAMS != 0)
        if (NT / 32 / tw > 1) return fwd_ring_teams<T, VPT, NT, MB, 0>(p, tw, st);
    return fwd_ring_teams<T, VPT, NT, MB, 1>(p, tw, st);
}

// blocks of the odd kernels, whose rows must have one shift: the grid divides into whole vectors where a block takes
// more than one row
template <typename T> int64_t odd_grid(int64_t rows, int64_t most) {
    return rows <= most ? rows : most / Vec<T>::N * Vec<T>::N;
}

template <typename T, int VPT, int NT, int MB>
int fwd_odd(const LnFwd& p, int nvec, cudaStream_t st) {
    const int threads = static_cast<int>(ceil_div(nvec, 32 * VPT)) * 32;
    constexpr auto k = layer_norm_fwd_odd<T, VPT, NT, MB>;
    if (int rc = allow_smem<k>()) return rc;
    const size_t wmax = window_max(p.cols, sizeof(T)), smem = 3 * (wmax + 8);
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, smem);
    const int64_t grid = odd_grid<T>(p.rows, static_cast<int64_t>(sm_count()) * std::max(1, per_sm));
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    return launch_early("layernorm_fwd", k, dim3(static_cast<unsigned>(grid)), threads, smem, st, p, 3, static_cast<uint32_t>(wmax), err);
}

template <typename T>
int run_fwd(const LnFwd& p, cudaStream_t st) {
    constexpr int EPV = Vec<T>::N;
    if (p.cols % EPV == 0) {
        const int nvec = p.cols / EPV;
        // A team to a row that it loads itself, up to one round of blocks; then the rings.  bf16, us by team and by ring: 152 x 4096 2.7,
        // 2.9; 304 x 4096 3.6, 3.0; 608 x 1024 2.5, 2.9; 1216 x 1024 3.4, 3.1; 152 x 8192 3.1, 3.3; 608 x 8192 6.2, 5.1
        const int64_t few = static_cast<int64_t>(sm_count()) * std::max(1, 512 / std::max(nvec, 32));
        if (p.rows <= few && nvec <= 512) return fwd_team<T, EPV, 1>(p, (nvec + 31) / 32, st);
        if (p.rows <= few && nvec <= 2048) return fwd_team<T, EPV, 4>(p, (nvec + 127) / 128, st);
        if (nvec <= 32) return fwd_ring<T, 1, 256, 2, 1>(p, nvec, st);
        if (nvec <= 512) return fwd_ring<T, 2, 256, 2, 1>(p, nvec, st);
        if (nvec <= 1024) return fwd_ring<T, 4, 256, 2, 0>(p, nvec, st);
        if (nvec <= 2048) return fwd_ring<T, 4, 512, 1, 0>(p, nvec, st);
    } else {
        if (p.cols <= 128) return fwd_team<T, 1, 4>(p, 1, st);
        const int nvec = (p.cols + 2 * EPV - 2) / EPV;   // of the longest window
        // few threads a row and several rows on an SM hide a row's two barriers; what does not fit their registers takes more threads
        if (nvec <= 64) return fwd_odd<T, 2, 32, 16>(p, nvec, st);     // 131072 x 333 bf16: 82 us, 101 with 4 vectors a thread
        if (nvec <= 512) return fwd_odd<T, 4, 128, 4>(p, nvec, st);    // 65536 x 1001 bf16: 63 us, 70 with 2
        if (nvec <= 576) return fwd_odd<T, 3, 192, 3>(p, nvec, st);    // 32768 x 4097 bf16: 124 us, 143 with 2
        if (nvec <= 768) return fwd_odd<T, 2, 384, 2>(p, nvec, st);    // 16384 x 6001 bf16: 85 us, 102 with 3
        if (nvec <= 1056) return fwd_odd<T, 3, 352, 2>(p, nvec, st);   // 16384 x 4097 fp32: 89 us, 120 with 2
        if (nvec <= 2048) return fwd_odd<T, 4, 512, 1>(p, nvec, st);
    }
    const int64_t grid = std::min<int64_t>(p.rows, 8 * sm_count());
    return launch_early("layernorm_fwd", layer_norm_fwd_rows<T>, dim3(static_cast<unsigned>(grid)), 256, 0, st,
                        static_cast<const T*>(p.x), static_cast<const T*>(p.w), static_cast<const T*>(p.b), static_cast<T*>(p.y),
                        p.mean, p.rstd, p.rows, p.cols, p.eps);
}

template <typename T, int VPT, int NT, int ONE>
int bwd_ring_teams(const LnBwd& p, int nvec, int teams, int64_t& grid, cudaStream_t st) {
    const int tw = static_cast<int>(ceil_div(nvec, 32 * VPT)), threads = teams * tw * 32;
    const size_t slot = static_cast<size_t>(p.dres != nullptr ? 3 : 2) * p.cols * sizeof(T);
    constexpr auto k = layer_norm_bwd_ring<T, VPT, NT, ONE>;
    if (int rc = allow_smem<k>()) return rc;
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, teams * (slot + 8));
    per_sm = std::max(1, per_sm);
    size_t nst = std::max<size_t>(1, std::min<size_t>(8, (nvec >= 512 ? kBwdFlightLong : kBwdFlight) / (per_sm * teams * slot)));
    if (nst == 1 && 2 * teams * (slot + 8) <= 220u * 1024u) nst = 2;
    // the sums of the teams go through the ring's memory at the end: 16 bytes a vector and element pair
    const size_t sums = teams > 1 ? static_cast<size_t>(nvec) * Vec<T>::N * 8 : 0;
    const size_t smem = std::max(teams * nst * (slot + 8), sums);
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, smem);
    grid = std::min<int64_t>({ceil_div(p.rows, teams), kMaxPartRows, static_cast<int64_t>(sm_count()) * std::max(1, per_sm)});
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    return launch_early("layernorm_bwd", k, dim3(static_cast<unsigned>(grid)), threads, smem, st, p, tw, static_cast<int>(nst), err);
}
template <typename T, int VPT, int NT, int TEAMS>
int bwd_ring(const LnBwd& p, int nvec, int64_t& grid, cudaStream_t st) {
    const int teams = std::max<int>(1, 8 / static_cast<int>(ceil_div(nvec, 32 * VPT)));
    if constexpr (TEAMS != 0)
        if (teams > 1) return bwd_ring_teams<T, VPT, NT, 0>(p, nvec, teams, grid, st);
    return bwd_ring_teams<T, VPT, NT, 1>(p, nvec, 1, grid, st);
}

template <typename T, int VPT, int NT, int MB>
int bwd_odd(const LnBwd& p, int nvec, int64_t& grid, cudaStream_t st) {
    const int threads = static_cast<int>(ceil_div(nvec, 32 * VPT)) * 32;
    constexpr auto k = layer_norm_bwd_odd<T, VPT, NT, MB>;
    if (int rc = allow_smem<k>()) return rc;
    const size_t wmax = window_max(p.cols, sizeof(T)), slot = (p.dres != nullptr ? 3 : 2) * wmax + 8;
    int nst = 4;   // one row in use, three in flight
    while (nst > 2 && nst * slot > 200u * 1024u) --nst;
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, nst * slot);
    grid = odd_grid<T>(p.rows, std::min<int64_t>(kMaxPartRows, static_cast<int64_t>(sm_count()) * std::max(1, per_sm)));
    int* err = nullptr;
    if (int rc = rmsnorm_err_word(&err)) return rc;
    return launch_early("layernorm_bwd", k, dim3(static_cast<unsigned>(grid)), threads, nst * slot, st, p, nst,
                        static_cast<uint32_t>(wmax), err);
}

template <typename T>
int run_bwd(LnBwd p, void* dw, void* db, cudaStream_t st) {
    constexpr int EPV = Vec<T>::N;
    constexpr bool F32 = sizeof(T) == 4;
    const int streams = p.dres != nullptr ? 3 : 2;
    const int nvec = p.cols % EPV == 0 ? p.cols / EPV : 0;
    int64_t grid = 0;
    int rc;
    const int longest = (p.cols + 2 * EPV - 2) / EPV;   // vectors of the longest window of an odd row
    if (nvec == 0 && p.cols >= 64 && longest <= 2048 && 2 * (streams * window_max(p.cols, sizeof(T)) + 8) <= 220u * 1024u) {
        if (longest <= 128) rc = bwd_odd<T, 1, 128, 5>(p, longest, grid, st);         // 131072 x 333 bf16: 156 us, 179 with 2 vectors a thread
        else if (longest <= 256) rc = bwd_odd<T, 2, 128, 4>(p, longest, grid, st);    // 65536 x 2001 bf16: 188 us, 232 with 1
        else if (longest <= 576) rc = bwd_odd<T, 3, 192, 2>(p, longest, grid, st);    // 32768 x 4097 bf16: 234 us, 326 with 2
        else if (longest <= 1024) rc = bwd_odd<T, 2, 512, 1>(p, longest, grid, st);   // 16384 x 6001 bf16: 175 us, 292 with 3
        else if (longest <= 1088) rc = bwd_odd<T, 2, 544, 1>(p, longest, grid, st);   // 16384 x 8191 bf16: 332 us, 344 with 3, 534 with 4
        else rc = bwd_odd<T, 4, 512, 1>(p, longest, grid, st);
    } else if (nvec == 0 || nvec > 2048 || static_cast<size_t>(streams) * p.cols * sizeof(T) > 200u * 1024u) {
        const int64_t most = std::min<int64_t>({p.rows, kMaxPartRows, 4 * sm_count()});
        p.rows_per_block = ceil_div(p.rows, most);
        grid = ceil_div(p.rows, p.rows_per_block);
        rc = launch_early("layernorm_bwd", layer_norm_bwd_rows<T>, dim3(static_cast<unsigned>(grid)), 256, 0, st, p);
    } else if (!F32 && nvec <= 256) rc = bwd_ring<T, 1, 256, 1>(p, nvec, grid, st);
    else if (nvec <= 512) rc = bwd_ring<T, 2, 256, 1>(p, nvec, grid, st);
    else if (nvec <= 1024) rc = bwd_ring<T, 2, 512, 0>(p, nvec, grid, st);
    else rc = bwd_ring<T, 4, 512, 0>(p, nvec, grid, st);
    if (rc) return rc;
    if (dw == nullptr && db == nullptr) return LIGER_OK;
    const float *pw = p.part_w, *pb = p.part_b;
    if (p.cols % 4 == 0)
        return launch_early("layernorm_bwd sums", layer_norm_sums<T, 4>, dim3(static_cast<unsigned>(ceil_div(p.cols, 128)), 2), 1024,
                            0, st, pw, pb, static_cast<T*>(dw), static_cast<T*>(db), static_cast<int>(grid), p.cols);
    return launch_early("layernorm_bwd sums", layer_norm_sums<T, 1>, dim3(static_cast<unsigned>(ceil_div(p.cols, 32)), 2), 1024, 0,
                        st, pw, pb, static_cast<T*>(dw), static_cast<T*>(db), static_cast<int>(grid), p.cols);
}

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" int liger_layernorm_fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                                   int64_t rows, int64_t cols, float eps, int dtype, void* stream) {
    clear_error();
    const char* who = "layernorm_fwd";
    if (int rc = check_sizes(who, rows, cols, dtype)) return rc;
    if (!(eps >= 0.f)) return fail(LIGER_ERR_SHAPE, "%s: eps must be >= 0", who);
    if (rows == 0) return LIGER_OK;
    if (!x || !y) return fail(LIGER_ERR_NULL, "%s: x and y are required", who);
    if (misaligned({x, w, b, y}, 16)) return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    if (misaligned({mean, rstd}, 4)) return fail(LIGER_ERR_ALIGN, "%s: mean and rstd must be 4-byte aligned", who);
    cudaStream_t st = as_stream(stream);
    const LnFwd p{x, w, b, y, mean, rstd, rows, static_cast<int>(cols), eps};
    return dtype == LIGER_F32 ? run_fwd<float>(p, st) : run_fwd<__nv_bfloat16>(p, st);
}

extern "C" size_t liger_layernorm_bwd_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || cols > (1 << 24)) return 0;
    return 2 * static_cast<size_t>(std::min<int64_t>(rows, kMaxPartRows)) * static_cast<size_t>(cols) * sizeof(float);
}

extern "C" int liger_layernorm_bwd(const void* dy, const void* dres, const void* x, const void* w, const float* mean,
                                   const float* rstd, void* dx, void* dw, void* db, void* ws, size_t ws_bytes,
                                   int64_t rows, int64_t cols, int dtype, void* stream) {
    clear_error();
    const char* who = "layernorm_bwd";
    if (int rc = check_sizes(who, rows, cols, dtype)) return rc;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx))
        return fail(LIGER_ERR_NULL, "%s: dy, x, mean, rstd and dx are required", who);
    if (misaligned({dy, dres, x, w, dx, dw, db}, 16))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
    if (misaligned({mean, rstd}, 4)) return fail(LIGER_ERR_ALIGN, "%s: mean and rstd must be 4-byte aligned", who);
    cudaStream_t st = as_stream(stream);
    const size_t esz = dtype == LIGER_F32 ? 4 : 2;
    if (rows == 0) {
        for (void* out : {dw, db})
            if (out != nullptr && cudaMemsetAsync(out, 0, static_cast<size_t>(cols) * esz, st) != cudaSuccess)
                return check_launch(who);
        return LIGER_OK;
    }
    const size_t need = liger_layernorm_bwd_workspace(rows, cols);
    if ((dw != nullptr || db != nullptr) && (!ws || ws_bytes < need || !aligned16(ws)))
        return fail(LIGER_ERR_WORKSPACE, "%s: workspace of %zu bytes (16-byte aligned) required, got %zu", who, need, ws_bytes);
    LnBwd p{dy, dres, x, w, mean, rstd, dx, nullptr, nullptr, rows, 0, static_cast<int>(cols)};
    if (dw != nullptr) p.part_w = static_cast<float*>(ws);
    if (db != nullptr) p.part_b = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + need / 2);
    return dtype == LIGER_F32 ? run_bwd<float>(p, dw, db, st) : run_bwd<__nv_bfloat16>(p, dw, db, st);
}
