// Rotary positions on the first part of each head, with scaled frequencies
// (formulas in liger_layer.h).
// The angles are formed in the kernel, in double before the range reduction (rope_angle.cuh), once a token for all its heads.  HBM
// bounds long sequences: [4, 8192] tokens of 32 + 8 heads of 128 bf16, out of place and back, 195 us (1.01 of the copy rate); the
// host a few tokens' call (the kernel takes 3 us of it).
#include <math.h>

#include "common.cuh"
#include "liger_layer.h"
#include "mbarrier.cuh"
#include "rope_angle.cuh"

namespace liger {
namespace {

constexpr int kMaxPairs = 256;   // rotary_dim <= 512
constexpr int kThreads = 256;
// Fewer tokens go straight through registers.  32 + 8 heads of 128 bf16, half of each rotated, pairs across halves (neighbours), us:
// 32 tokens 3.0 (3.2) staged, 3.3 (2.8) straight; 128: 3.1 (3.1), 3.3 (3.1); 512: 3.9 (3.6), 4.8 (5.4); 8192: 27 (26), 41 (46).
constexpr int64_t kStagedTokens = 128;

// inverse frequencies, by value in the kernel's parameters
struct Freqs {
    double v[kMaxPairs];
};

struct RopeScaled {
    const void *q, *k;
    void *q_out, *k_out;
    const int32_t* pos;
    int64_t q_ts, k_ts, qo_ts, ko_ts;   // elements between tokens
    int64_t tokens, S;
    int Hq, Hk, D, R;
    int inter;                          // pairs (2i, 2i + 1)
    int copy_q, copy_k;                 // out of place: the rest of each head is copied
    int npos;                           // tokens per block
    int heads_per_block;                // rope_scaled_chunks
    float m, sign;
};

// A pair by its (cos, sin), with the roundings written out: every path below gives the same bits.
__device__ __forceinline__ float2 turned(float a, float b, float2 r) {
    return make_float2(fmaf(a, r.x, -__fmul_rn(b, r.y)), fmaf(b, r.x, __fmul_rn(a, r.y)));
}

// A block takes npos tokens: their angles into shared memory, then a thread per pair or copied element.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_scaled_elems(const RopeScaled a, const __grid_constant__ Freqs f) {
    extern __shared__ float2 cs[];   // [npos][R / 2]
    const int half = a.R >> 1;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.npos;
    const int np = static_cast<int>(min(static_cast<int64_t>(a.npos), a.tokens - t0));
    wait_for_stream();
    for (int i = threadIdx.x; i < np * half; i += kThreads) {
        const int pp = i / half;
        const int64_t t = t0 + pp, p = a.pos != nullptr ? static_cast<int64_t>(a.pos[t]) : t % a.S;
        const float2 r = angle_cs(static_cast<double>(p), f.v[i - pp * half], a.sign);
        cs[i] = make_float2(a.m * r.x, a.m * r.y);
    }
    __syncthreads();
    const int H = a.Hq + a.Hk, rest = a.D - a.R, per_head = half + rest;
    const int64_t n = static_cast<int64_t>(np) * H * per_head;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int j = static_cast<int>(i % per_head);
        const int64_t hh = i / per_head;
        const int h = static_cast<int>(hh % H), pp = static_cast<int>(hh / H);
        const bool isq = h < a.Hq;
        const int64_t t = t0 + pp;
        const T* src = isq ? static_cast<const T*>(a.q) + t * a.q_ts + static_cast<int64_t>(h) * a.D
                           : static_cast<const T*>(a.k) + t * a.k_ts + static_cast<int64_t>(h - a.Hq) * a.D;
        T* dst = isq ? static_cast<T*>(a.q_out) + t * a.qo_ts + static_cast<int64_t>(h) * a.D
                     : static_cast<T*>(a.k_out) + t * a.ko_ts + static_cast<int64_t>(h - a.Hq) * a.D;
        if (j < half) {
            const int ia = a.inter ? 2 * j : j, ib = a.inter ? 2 * j + 1 : j + half;
            const float2 y = turned(ldf(src + ia), ldf(src + ib), cs[pp * half + j]);
            stf(dst + ia, y.x);
            stf(dst + ib, y.y);
        } else if (isq ? a.copy_q : a.copy_k) {
            dst[a.R + j - half] = src[a.R + j - half];
        }
    }
}

// ------------------------------------------------------------- pieces of 16 bytes
// Where heads, their rotated part and its halves are whole pieces of P elements: P consecutive elements of
// one type move as one access: 16 bytes, or two elements.
template <typename T, int P> struct Chunk {
    static_assert(P == Vec<T>::N, "16 bytes");
    float f[P];
    __device__ __forceinline__ void get(const T* p) { unpack(*reinterpret_cast<const uint4*>(p), f); }
    __device__ __forceinline__ void put(T* p) const { *reinterpret_cast<uint4*>(p) = pack(f); }
};
template <> struct Chunk<float, 2> {
    float f[2];
    __device__ __forceinline__ void get(const float* p) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        f[0] = v.x;
        f[1] = v.y;
    }
    __device__ __forceinline__ void put(float* p) const { *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]); }
};
template <> struct Chunk<__nv_bfloat16, 2> {
    float f[2];
    __device__ __forceinline__ void get(const __nv_bfloat16* p) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
        f[0] = bf_lo(v);
        f[1] = bf_hi(v);
    }
    __device__ __forceinline__ void put(__nv_bfloat16* p) const { *reinterpret_cast<uint32_t*>(p) = pack_bf2(f[0], f[1]); }
};

// A unit of rotation: interleaved, P / 2 pairs in one chunk at a; else P pairs in the chunks at a and b.
// cs: the unit's angles, `apart` float2 between consecutive ones.
template <typename T, bool INTER, int P>
__device__ __forceinline__ void turn(Chunk<T, P>& a, Chunk<T, P>& b, const float2* cs, int apart) {
    if (INTER) {
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
            const float2 y = turned(a.f[2 * i], a.f[2 * i + 1], cs[i * apart]);
            a.f[2 * i] = y.x;
            a.f[2 * i + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 y = turned(a.f[i], b.f[i], cs[i * apart]);
            a.f[i] = y.x;
            b.f[i] = y.y;
        }
    }
}

// The block's angles, laid out [token][angle within a unit][unit] so that threads of neighbouring units
// read neighbouring words.
template <int APU>
__device__ __forceinline__ void form_angles(const RopeScaled& a, const Freqs& f, int64_t t0, int np, float2* cs) {
    const int half = a.R >> 1, units = half / APU;
    for (int i = threadIdx.x; i < np * half; i += kThreads) {
        const int pp = i / half, k = i - pp * half, u = k / APU;
        const int64_t t = t0 + pp, p = a.pos != nullptr ? static_cast<int64_t>(a.pos[t]) : t % a.S;
        const float2 r = angle_cs(static_cast<double>(p), f.v[k], a.sign);
        cs[pp * half + (k - u * APU) * units + u] = make_float2(a.m * r.x, a.m * r.y);
    }
}

// ------------------------------------------------------------- rows staged by bulk copies
// Error word: the RoPE family's (an expired wait), read and cleared by liger_device_status.
// A block takes npos consecutive tokens: their Q and K rows come into shared memory by 1-D bulk copies while
// the threads form the angles, the rotated parts are turned there, and the rows leave by bulk copies, so
// that what is only copied costs no instruction.  On an expired wait the block records it, waits (bounded)
// again for its copies and writes NaN rows.
template <typename T, bool INTER, int P>
__global__ void __launch_bounds__(kThreads) rope_scaled_staged(const RopeScaled a, const __grid_constant__ Freqs f, int* err) {
    constexpr int APU = INTER ? P / 2 : P;   // angles of a unit
    extern __shared__ __align__(128) uint8_t sm[];
    const int half = a.R >> 1, units = half / APU, H = a.Hq + a.Hk;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.npos;
    const int np = static_cast<int>(min(static_cast<int64_t>(a.npos), a.tokens - t0));
    const uint32_t qrow = static_cast<uint32_t>(a.Hq * a.D) * sizeof(T), krow = static_cast<uint32_t>(a.Hk * a.D) * sizeof(T);
    const uint32_t rowb = qrow + krow;   // a multiple of 16
    uint8_t* tile = sm;                  // [npos][rowb]
    float2* cs = reinterpret_cast<float2*>(sm + static_cast<size_t>(a.npos) * rowb);
    const uint32_t bar = smem_u32(cs + a.npos * half);
    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        mbar_init_fence();
    }
    __syncthreads();
    wait_for_stream();
    if (threadIdx.x == 0) {
        mbar_expect_tx(bar, static_cast<uint32_t>(np) * rowb);
        for (int pp = 0; pp < np; ++pp) {
            const uint32_t dst = smem_u32(tile + static_cast<size_t>(pp) * rowb);
            if (qrow) bulk_g2s(dst, static_cast<const T*>(a.q) + (t0 + pp) * a.q_ts, qrow, bar);
            if (krow) bulk_g2s(dst + qrow, static_cast<const T*>(a.k) + (t0 + pp) * a.k_ts, krow, bar);
        }
    }
    form_angles<APU>(a, f, t0, np, cs);
    const bool got = mbar_wait(bar, 0);
    if (!__syncthreads_and(got ? 1 : 0)) {
        if (threadIdx.x == 0) {
            atomicExch(err, 1);
            mbar_wait(bar, 0);   // the copies still in flight into this block's shared memory
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < np * rowb / 16; i += kThreads) reinterpret_cast<uint4*>(tile)[i] = nan16<T>();
    } else {
        // task (token, head, unit), the unit fastest: advanced with the thread's stride instead of divided out
        const int per = H * units;
        int pp = static_cast<int>(threadIdx.x) / per, r = static_cast<int>(threadIdx.x) - pp * per;
        int h = r / units, u = r - h * units;
        const int dh = kThreads / units, du = kThreads - dh * units;
        while (pp < np) {
            T* head = reinterpret_cast<T*>(tile + static_cast<size_t>(pp) * rowb) + h * a.D;
            T* pa = head + u * P;
            T* pb = head + half + u * P;
            Chunk<T, P> x0, x1;
            x0.get(pa);
            if (!INTER) x1.get(pb);
            turn<T, INTER, P>(x0, x1, cs + pp * half + u, units);
            x0.put(pa);
            if (!INTER) x1.put(pb);
            u += du;
            h += dh;
            if (u >= units) {
                u -= units;
                ++h;
            }
            while (h >= H) {
                h -= H;
                ++pp;
            }
        }
    }
    fence_proxy_async_smem();   // the turned values, before the copies out read them
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int pp = 0; pp < np; ++pp) {
            const uint32_t src = smem_u32(tile + static_cast<size_t>(pp) * rowb);
            if (qrow) bulk_s2g(static_cast<T*>(a.q_out) + (t0 + pp) * a.qo_ts, src, qrow);
            if (krow) bulk_s2g(static_cast<T*>(a.k_out) + (t0 + pp) * a.ko_ts, src + qrow, krow);
        }
        bulk_s2g_done();   // the shared memory has been read
    }
}

// ------------------------------------------------------------- straight from global memory
// Few tokens, or in place with a part of the heads that stays: a thread moves whole chunks itself.
template <typename T, bool INTER, int P>
__global__ void __launch_bounds__(kThreads) rope_scaled_chunks(const RopeScaled a, const __grid_constant__ Freqs f) {
    constexpr int APU = INTER ? P / 2 : P;
    extern __shared__ __align__(128) uint8_t sm[];
    float2* cs = reinterpret_cast<float2*>(sm);
    const int half = a.R >> 1, units = half / APU, H = a.Hq + a.Hk;
    const int rest = (a.D - a.R) / P, per_head = units + (a.copy_q || a.copy_k ? rest : 0);
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.npos;
    const int np = static_cast<int>(min(static_cast<int64_t>(a.npos), a.tokens - t0));
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(H, h0 + a.heads_per_block);
    wait_for_stream();
    form_angles<APU>(a, f, t0, np, cs);
    __syncthreads();
    const int n = np * (h1 - h0) * per_head;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int hh = i / per_head, j = i - hh * per_head;
        const int pp = hh / (h1 - h0), h = h0 + hh - pp * (h1 - h0);
        const bool isq = h < a.Hq;
        const int64_t t = t0 + pp;
        const T* src = isq ? static_cast<const T*>(a.q) + t * a.q_ts + h * a.D
                           : static_cast<const T*>(a.k) + t * a.k_ts + (h - a.Hq) * a.D;
        T* dst = isq ? static_cast<T*>(a.q_out) + t * a.qo_ts + h * a.D : static_cast<T*>(a.k_out) + t * a.ko_ts + (h - a.Hq) * a.D;
        Chunk<T, P> x0, x1;
        if (j < units) {
            x0.get(src + j * P);
            if (!INTER) x1.get(src + half + j * P);
            turn<T, INTER, P>(x0, x1, cs + pp * half + j, units);
            x0.put(dst + j * P);
            if (!INTER) x1.put(dst + half + j * P);
        } else if (isq ? a.copy_q : a.copy_k) {
            const int o = a.R + (j - units) * P;
            x0.get(src + o);
            x0.put(dst + o);
        }
    }
}

// f_i of every pair in double precision; false if the scaling gives a frequency that is no finite number
bool frequencies(Freqs& f, int R, double theta, int scaling, double factor, double low, double high, double orig_len) {
    const int half = R / 2;
    const double two_pi = 6.283185307179586;
    double base = theta;
    if (scaling == LIGER_ROPE_NTK && R > 2) base = theta * pow(factor, static_cast<double>(R) / (R - 2));
    const double step = log2(base) * -2.0 / R;
    double lo = 0, hi = 0;
    if (scaling == LIGER_ROPE_YARN) {
        auto dim = [&](double turns) { return R * log(orig_len / (turns * two_pi)) / (2.0 * log(theta)); };
        lo = std::max(floor(dim(high)), 0.0);
        hi = std::min(ceil(dim(low)), R - 1.0);
    }
    for (int i = 0; i < half; ++i) {
        double v = exp2(step * i);
        if (scaling == LIGER_ROPE_LINEAR) v /= factor;
        if (scaling == LIGER_ROPE_BANDS) {
            const double c = std::min(std::max((orig_len * v / two_pi - low) / (high - low), 0.0), 1.0);
            v *= c + (1.0 - c) / factor;
        }
        if (scaling == LIGER_ROPE_YARN) {
            const double c = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            v *= 1.0 - c + c / factor;
        }
        if (!(v >= 0.0) || !isfinite(v)) return false;
        f.v[i] = v;
    }
    return true;
}

template <typename T, bool INTER, int P>
int launch_staged(const char* who, RopeScaled a, const Freqs& f, cudaStream_t st) {
    const size_t row = static_cast<size_t>(a.Hq + a.Hk) * a.D * sizeof(T), angles = static_cast<size_t>(a.R / 2) * sizeof(float2);
    // a tile of about 32 KB, fewer tokens where that leaves SMs without a block
    const int64_t fit = std::max<int64_t>(1, static_cast<int64_t>((32u << 10) / row));
    a.npos = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({fit, 64, ceil_div(a.tokens, 2 * sm_count())})));
    while (ceil_div(a.tokens, a.npos) > 2147483647LL) a.npos *= 2;
    const size_t smem = a.npos * (row + angles) + 8;
    constexpr auto k = rope_scaled_staged<T, INTER, P>;
    if (int rc = allow_smem<k>()) return rc;
    int* err = nullptr;
    if (int rc = rope_err_word(&err)) return rc;
    return launch_early(who, k, dim3(static_cast<unsigned>(ceil_div(a.tokens, a.npos))), kThreads, smem, st, a, f, err);
}

template <typename T, bool INTER, int P>
int launch_chunks(const char* who, RopeScaled a, const Freqs& f, cudaStream_t st) {
    constexpr int APU = INTER ? P / 2 : P;
    const int H = a.Hq + a.Hk, units = a.R / 2 / APU, per_head = units + (a.copy_q || a.copy_k ? (a.D - a.R) / P : 0);
    // a block's worth of chunks is 1024, or 256 where there are few tokens; tokens together while that is less than a token has
    const int64_t want = a.tokens * H * per_head >= static_cast<int64_t>(4096) * sm_count() ? 1024 : kThreads;
    a.npos = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4096 / a.R, want / (static_cast<int64_t>(H) * per_head))));
    while (ceil_div(a.tokens, a.npos) > 2147483647LL) a.npos *= 2;
    a.heads_per_block = a.npos > 1 ? H : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(H, ceil_div(want, per_head))));
    const int64_t splits = ceil_div(H, a.heads_per_block);
    if (splits > 65535) a.heads_per_block = static_cast<int>(ceil_div(H, 65535));
    const dim3 grid(static_cast<unsigned>(ceil_div(a.tokens, a.npos)), static_cast<unsigned>(ceil_div(H, a.heads_per_block)));
    const size_t smem = static_cast<size_t>(a.npos) * (a.R / 2) * sizeof(float2);
    if (smem > 48u * 1024u) return fail(LIGER_ERR_SHAPE, "%s: too many tokens", who);
    return launch_early(who, rope_scaled_chunks<T, INTER, P>, grid, kThreads, smem, st, a, f);
}

template <typename T, bool INTER, int P>
int launch_sized(const char* who, const RopeScaled& a, const Freqs& f, bool rows16, cudaStream_t st) {
    const size_t row = static_cast<size_t>(a.Hq + a.Hk) * a.D * sizeof(T), need = row + a.R / 2 * sizeof(float2) + 8;
    const bool some_stay = a.R < a.D && !((a.Hq == 0 || a.copy_q) && (a.Hk == 0 || a.copy_k));
    if (rows16 && a.tokens >= kStagedTokens && !some_stay && need <= static_cast<size_t>(max_smem_optin()))
        return launch_staged<T, INTER, P>(who, a, f, st);
    return launch_chunks<T, INTER, P>(who, a, f, st);
}

template <typename T>
int launch_rope(const char* who, const RopeScaled& a, const Freqs& f, bool aligned, cudaStream_t st) {
    constexpr int V = Vec<T>::N;
    // 16-byte rows of Q and of K (their strides and starts are, by `aligned`); chunks by what divides a head
    const bool rows16 = aligned && a.Hq * a.D % V == 0 && a.Hk * a.D % V == 0;
    const bool whole = aligned && a.D % V == 0;
    if (a.inter) {
        if (whole && a.R % V == 0) return launch_sized<T, true, V>(who, a, f, rows16, st);
        if (aligned && a.D % 2 == 0) return launch_sized<T, true, 2>(who, a, f, rows16, st);
    } else {
        if (whole && a.R % (2 * V) == 0) return launch_sized<T, false, V>(who, a, f, rows16, st);
        if (aligned && a.D % 2 == 0 && a.R % 4 == 0) return launch_sized<T, false, 2>(who, a, f, rows16, st);
    }
    RopeScaled e = a;
    e.npos = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, 2 * kThreads / a.R)));
    while (ceil_div(e.tokens, e.npos) > 2147483647LL) e.npos *= 2;
    const size_t smem = static_cast<size_t>(e.npos) * (e.R / 2) * sizeof(float2);
    if (smem > 48u * 1024u) return fail(LIGER_ERR_SHAPE, "%s: too many tokens", who);
    return launch_early(who, rope_scaled_elems<T>, dim3(static_cast<unsigned>(ceil_div(e.tokens, e.npos))), kThreads, smem, st, e, f);
}

int rope_scaled_run(const char* who, const void* q, const void* k, void* q_out, void* k_out, const int32_t* pos, int64_t B,
                    int64_t S, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t q_ts, int64_t k_ts, int64_t qo_ts,
                    int64_t ko_ts, int pairing, double theta, int scaling, double factor, double low, double high,
                    double orig_len, double attn_factor, int dtype, void* stream, float sign) {
    clear_error();
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (B < 0 || S < 0 || Hq < 0 || Hk < 0 || B > 2147483647LL || S > 2147483647LL || Hq > (1 << 20) || Hk > (1 << 20) ||
        D <= 0 || D > 512)
        return fail(LIGER_ERR_SHAPE, "%s: batch=%lld seq=%lld heads=%lld/%lld head_dim=%lld (1 to 512)", who, (long long)B,
                    (long long)S, (long long)Hq, (long long)Hk, (long long)D);
    if (R < 2 || R > D || (R & 1))
        return fail(LIGER_ERR_SHAPE, "%s: rotary_dim=%lld (even, 2 to head_dim=%lld)", who, (long long)R, (long long)D);
    if (pairing != 0 && pairing != 1) return fail(LIGER_ERR_SHAPE, "%s: pairing must be 0 or 1", who);
    const bool has_q = Hq > 0, has_k = Hk > 0;
    if ((has_q && (q_ts < Hq * D || qo_ts < Hq * D)) || (has_k && (k_ts < Hk * D || ko_ts < Hk * D)))
        return fail(LIGER_ERR_SHAPE, "%s: a token stride is smaller than heads*head_dim", who);
    const int64_t most = int64_t{1} << 61;
    if (B > 0 && S > 0 && (B * S > (int64_t{1} << 40) || std::max({q_ts, k_ts, qo_ts, ko_ts}) > most / (B * S)))
        return fail(LIGER_ERR_SHAPE, "%s: too many tokens, or token strides too large", who);
    if (scaling < LIGER_ROPE_NONE || scaling > LIGER_ROPE_YARN) return fail(LIGER_ERR_SHAPE, "%s: scaling %d", who, scaling);
    if (!(theta > 0.0) || !isfinite(theta)) return fail(LIGER_ERR_SHAPE, "%s: theta must be > 0", who);
    if (scaling != LIGER_ROPE_NONE && (!(factor > 0.0) || !isfinite(factor)))
        return fail(LIGER_ERR_SHAPE, "%s: factor must be > 0", who);
    if (scaling >= LIGER_ROPE_BANDS && (!(orig_len > 0.0) || !isfinite(orig_len) || !isfinite(low) || !isfinite(high)))
        return fail(LIGER_ERR_SHAPE, "%s: orig_len must be > 0, low and high finite", who);
    if (scaling == LIGER_ROPE_BANDS && !(low < high)) return fail(LIGER_ERR_SHAPE, "%s: low must be below high", who);
    if (scaling == LIGER_ROPE_YARN && (!(low > 0.0) || !(high > 0.0) || !(theta > 1.0)))
        return fail(LIGER_ERR_SHAPE, "%s: yarn needs low, high > 0 and theta > 1", who);
    if (!isfinite(attn_factor)) return fail(LIGER_ERR_SHAPE, "%s: attn_factor must be finite", who);
    if (B == 0 || S == 0 || (!has_q && !has_k)) return LIGER_OK;
    if ((has_q && (!q || !q_out)) || (has_k && (!k || !k_out)))
        return fail(LIGER_ERR_NULL, "%s: inputs and outputs are required for nonzero head counts", who);
    if ((has_q && q_out == q && qo_ts != q_ts) || (has_k && k_out == k && ko_ts != k_ts))
        return fail(LIGER_ERR_SHAPE, "%s: in place the strides must be equal", who);
    const size_t esz = dtype == LIGER_F32 ? 4 : 2;
    for (const void* p : {has_q ? q : nullptr, has_q ? static_cast<const void*>(q_out) : nullptr, has_k ? k : nullptr,
                          has_k ? static_cast<const void*>(k_out) : nullptr})
        if (reinterpret_cast<uintptr_t>(p) % esz) return fail(LIGER_ERR_ALIGN, "%s: tensors must be aligned to their elements", who);
    if (reinterpret_cast<uintptr_t>(pos) & 3) return fail(LIGER_ERR_ALIGN, "%s: pos must be 4-byte aligned", who);
    Freqs f;
    if (!frequencies(f, static_cast<int>(R), theta, scaling, factor, low, high, orig_len))
        return fail(LIGER_ERR_SHAPE, "%s: the scaling gives a frequency that is no finite number", who);
    double m = attn_factor;
    if (m == 0.0) m = scaling == LIGER_ROPE_YARN && factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
    RopeScaled a{};
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.pos = pos;
    a.q_ts = q_ts;
    a.k_ts = k_ts;
    a.qo_ts = qo_ts;
    a.ko_ts = ko_ts;
    a.tokens = B * S;
    a.S = S;
    a.Hq = static_cast<int>(Hq);
    a.Hk = static_cast<int>(Hk);
    a.D = static_cast<int>(D);
    a.R = static_cast<int>(R);
    a.inter = pairing;
    a.copy_q = q_out != q;
    a.copy_k = k_out != k;
    a.m = static_cast<float>(m);
    a.sign = sign;
    const bool aligned = (!has_q || (aligned16(q) && aligned16(q_out) && q_ts * esz % 16 == 0 && qo_ts * esz % 16 == 0)) &&
                         (!has_k || (aligned16(k) && aligned16(k_out) && k_ts * esz % 16 == 0 && ko_ts * esz % 16 == 0));
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32 ? launch_rope<float>(who, a, f, aligned, st) : launch_rope<__nv_bfloat16>(who, a, f, aligned, st);
}

}  // namespace
}  // namespace liger

extern "C" int liger_rope_scaled_fwd(const void* q, const void* k, void* q_out, void* k_out, const int32_t* pos, int64_t batch,
                                     int64_t seq, int64_t n_q_heads, int64_t n_k_heads, int64_t head_dim, int64_t rotary_dim,
                                     int64_t q_token_stride, int64_t k_token_stride, int64_t q_out_token_stride,
                                     int64_t k_out_token_stride, int pairing, double theta, int scaling, double factor,
                                     double low, double high, double orig_len, double attn_factor, int dtype, void* stream) {
    return liger::rope_scaled_run("rope_scaled_fwd", q, k, q_out, k_out, pos, batch, seq, n_q_heads, n_k_heads, head_dim,
                                  rotary_dim, q_token_stride, k_token_stride, q_out_token_stride, k_out_token_stride, pairing,
                                  theta, scaling, factor, low, high, orig_len, attn_factor, dtype, stream, 1.0f);
}

extern "C" int liger_rope_scaled_bwd(const void* dq, const void* dk, void* dq_out, void* dk_out, const int32_t* pos,
                                     int64_t batch, int64_t seq, int64_t n_q_heads, int64_t n_k_heads, int64_t head_dim,
                                     int64_t rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                                     int64_t q_out_token_stride, int64_t k_out_token_stride, int pairing, double theta,
                                     int scaling, double factor, double low, double high, double orig_len, double attn_factor,
                                     int dtype, void* stream) {
    return liger::rope_scaled_run("rope_scaled_bwd", dq, dk, dq_out, dk_out, pos, batch, seq, n_q_heads, n_k_heads, head_dim,
                                  rotary_dim, q_token_stride, k_token_stride, q_out_token_stride, k_out_token_stride, pairing,
                                  theta, scaling, factor, low, high, orig_len, attn_factor, dtype, stream, -1.0f);
}
