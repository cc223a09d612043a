// Rotary positions on the first part of each head, with scaled frequencies
// (formulas in liger_layer.h).
#include <math.h>

#include "common.cuh"
#include "liger_layer.h"
#include "rope_angle.cuh"

namespace liger {
namespace {

constexpr int kMaxPairs = 256;   // rotary_dim <= 512
constexpr int kThreads = 256;

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
    float m, sign;
};

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
            const float2 r = cs[pp * half + j];
            const int ia = a.inter ? 2 * j : j, ib = a.inter ? 2 * j + 1 : j + half;
            const float x0 = ldf(src + ia), x1 = ldf(src + ib);
            stf(dst + ia, x0 * r.x - x1 * r.y);
            stf(dst + ib, x1 * r.x + x0 * r.y);
        } else if (isq ? a.copy_q : a.copy_k) {
            dst[a.R + j - half] = src[a.R + j - half];
        }
    }
}

// f_i of every pair in double precision; false if the scaling gives a frequency that is no positive number
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
    a.npos = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, 2 * kThreads / R)));
    while (ceil_div(a.tokens, a.npos) > 2147483647LL) a.npos *= 2;
    const size_t smem = static_cast<size_t>(a.npos) * (R / 2) * sizeof(float2);
    if (smem > 48u * 1024u) return fail(LIGER_ERR_SHAPE, "%s: too many tokens", who);
    const dim3 grid(static_cast<unsigned>(ceil_div(a.tokens, a.npos)));
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32 ? launch_early(who, rope_scaled_elems<float>, grid, kThreads, smem, st, a, f)
                              : launch_early(who, rope_scaled_elems<__nv_bfloat16>, grid, kThreads, smem, st, a, f);
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
