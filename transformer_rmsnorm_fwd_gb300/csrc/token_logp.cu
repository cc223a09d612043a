// Log-probabilities of given tokens from logits, with the entropy, the top
// alternatives and the gradient of the logits (formulas in liger_layer.h).
// The forward reads a row once: a running maximum with the sums of e^(z - m) and of (z - m) e^(z - m) relative to it, raised where the
// maximum rises, and the largest logit of each thread's vectors, from which the k-th largest of 64 groups bounds the alternatives:
// only vectors that reach the bound are looked at again.  4096 rows of 128256 bf16 with 8 alternatives: 189 to 192 us, 0.81 of the
// copy rate, without alternatives 159 (0.97): bound by HBM and, for the rest, by the ends of the rows (their barriers and ranking).
// The gradient, 4096 x 128256 bf16: 313 us (0.99); 1500 x 32771 fp32: 61 (0.95).  One row of 151936: 9.5 us, the latencies of one pass.
#include <math.h>

#include <type_traits>

#include "cluster.cuh"
#include "liger_layer.h"

namespace liger {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kLowest = -3.402823466e38f;
constexpr int kRowThreads = 256;

struct LogpFwd {
    const void* z;
    int64_t ld;
    const int64_t* tokens;
    int64_t T, V, ignore;
    float inv_temp;
    float *logp, *row_max, *log_sum, *entropy, *top_logp;
    int64_t* top_ids;
    int k;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A number whose unsigned order is that of the floats: -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t order_of(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// The float of an order (+0 for either zero, a NaN for all of them)
__device__ __forceinline__ float value_of(uint32_t o) {
    if (o == 0xFFFFFFFFu) return NAN;
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
// ... and with the index behind it, the lowest first
__device__ __forceinline__ unsigned long long rank_key(float v, uint32_t index) {
    return static_cast<unsigned long long>(order_of(v)) << 32 | (0xFFFFFFFFu - index);
}

// ------------------------------------------------------------------ forward
// With d = (z - m) / (temperature ln 2), m the largest logit, s = sum 2^d and u = sum d 2^d:
//     log_sum = ln 2 log2 s,  logp = (z_y - m) / temperature - log_sum,  entropy = ln 2 (log2 s - u / s)
// z - m is formed first: logits of the type's lowest value, or all far from 0, lose nothing.
//
// One pass over the row's 16-byte vectors: a thread keeps a running maximum with s and u relative to it (they
// are rescaled when it grows, which is rare after the first vectors), and the largest logit it has seen with that
// vector's index.  The block (a cluster of blocks where there are few rows, each with its share of the row)
// joins the sums.
// Alternatives: threads are taken together in kGroups groups; the k-th largest of the groups' best logits is a
// lower bound on the row's k-th largest, since k groups have one that large, and with random logits hardly more than k
// logits reach it.  So only threads whose best reaches the bound look at their vectors again (from L2), 32
// vectors at a time by their whole warp, and put what reaches it on a list, which is then ranked.  Equal logits
// go by index throughout, so a constant row leaves a short list too.  A list that overflows (largest logits
// crowded in one group's vectors) is given up, and the k largest are found one after the other.

// Largest 64-bit key or float (NaN above all) over the block, in every thread.
template <int NT>
__device__ __forceinline__ unsigned long long block_max_key(unsigned long long v, unsigned long long* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();   // the previous one has been read
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) v = max(v, sh[w]);
    return v;
}

// Running maximum with the sums relative to it (c: log2 e / temperature).
struct Sums {
    float m, s, u;
};
// The sums of `a` relative to a larger maximum m.  The difference is held at -1e4, where the factor is 0, so that 0 times it
// is not NaN.
__device__ __forceinline__ void raise(Sums& a, float m, float c) {
    const float d = max_nan((a.m - m) * c, -1e4f), f = ex2(d);
    a.u = fmaf(a.s, d, a.u) * f;
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void join(Sums& a, Sums b, float c) {
    const float m = fmaxf(a.m, b.m);
    raise(a, m, c);
    raise(b, m, c);
    a.s += b.s;
    a.u += b.u;
}
// The thread's sums while it runs: d is formed as f c - k by one fma, k = fl(m c), and so is off by e = m c - k (below
// 2^-24 of m c) in every term alike, which is put right when the sums are read: with the sums s' and u' of those,
// s = 2^-e s', u = 2^-e (u' - e s').  From kFarOut on (e would be no small number, or out of fp32's range as in a row
// of nothing but the type's lowest values) d is (f - m) c, and e is 0.
constexpr float kFarOut = 1e6f;
struct Running {
    float m, k;        // maximum, fl(m c)
    float2 s, u;
    __device__ __forceinline__ bool far() const { return !(fabsf(k) < kFarOut); }
    __device__ __forceinline__ Sums read(float c) const {
        const float e = far() ? 0.f : fmaf(m, c, -k), f = ex2(-e), sum = s.x + s.y;
        return {m, sum * f, fmaf(-e, sum, u.x + u.y) * f};
    }
    __device__ __forceinline__ void set(const Sums& a, float c) {
        m = a.m;
        k = a.m * c;
        const float e = far() ? 0.f : fmaf(m, c, -k), f = ex2(e);
        s = make_float2(a.s * f, 0.f);
        u = make_float2(fmaf(e, a.s, a.u) * f, 0.f);
    }
};

// Largest element of a 16-byte vector, NaN above all; bf16 by packed comparisons.
__device__ __forceinline__ float vec_max(const uint4& u, float) {
    return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)), max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
}
__device__ __forceinline__ float vec_max(const uint4& u, __nv_bfloat16) {
    auto larger = [](uint32_t a, uint32_t b) {
        const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    };
    const uint32_t m = larger(larger(u.x, u.y), larger(u.z, u.w));
    return max_nan(bf_lo(m), bf_hi(m));
}

constexpr int kGroups = 64;         // groups of threads
constexpr int kList = 2048;         // candidates of a block
constexpr int kSecond = LIGER_TOP_MAX * kList / kGroups;   // ... that reach the second bound: k groups' shares at most
constexpr int kUnroll = 4;          // vectors of a thread in flight
// Many rows (kManyRows an SM) of at most kShortRow vectors: 128 threads a row, whose ends overlap better; 64 for rows of few vectors,
// of which 128 threads would hold too few groups for the bound.  us with 64, 128 and 256 threads, bf16, 8 alternatives: 8192 x 2048
// 60, 58, 80; 8192 x 16384 101, 92, 115; 8192 x 32768 154, 128, 145; 4096 x 65536 173, 136, 111; 1024 x 8192 13.8, 13.0, 15.4;
// 304 x 8192 10.5, 9.7, 7.7.
constexpr int kShortRow = 5120, kManyRows = 6;

// a row's vectors: vector v holds elements v EPV - shift + (0 .. EPV - 1); those in [first, last) are whole
template <typename T>
struct RowVecs {
    const T* base;       // element 0 of vector 0 (aligned; up to EPV - 1 elements before the row)
    int shift, n, first, last, V;
    __device__ RowVecs(const T* z, int64_t vocab) {
        constexpr int EPV = Vec<T>::N;
        const uintptr_t at = reinterpret_cast<uintptr_t>(z);
        shift = static_cast<int>((at & 15) / sizeof(T));
        base = z - shift;
        V = static_cast<int>(vocab);   // at most 2^30
        n = (V + shift + EPV - 1) / EPV;
        first = shift > 0 ? 1 : 0;
        last = (V + shift) / EPV;
    }
    // vector v, -inf where it reaches past the row (nothing outside the row is read)
    __device__ __forceinline__ uint4 get(int v) const {
        constexpr int EPV = Vec<T>::N;
        if (v >= first && v < last) return ldg16(base + static_cast<int64_t>(v) * EPV);
        float f[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const int i = v * EPV + e - shift;
            f[e] = i >= 0 && i < V ? ldf(base + i + shift) : -INFINITY;
        }
        return pack(f);
    }
    __device__ __forceinline__ void get(int v, float (&f)[Vec<T>::N]) const { unpack(get(v), f); }
};

// Finds the `k` largest of n keys (all different, none 0) by counting and leaves them in order in out[0 .. k).
template <int NT>
__device__ __forceinline__ void rank_keys(const unsigned long long* keys, int n, int k, unsigned long long* out) {
    for (int i = threadIdx.x; i < n; i += NT) {
        const unsigned long long x = keys[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += keys[j] > x ? 1 : 0;
        if (above < k) out[above] = x;
    }
}

struct alignas(16) RowShared {   // (the keys by pairs too, should a loop over them be read so)
    alignas(16) unsigned long long best[LIGER_TOP_MAX];   // this block's k largest keys in order (0: no more)
    alignas(16) unsigned long long groups[kGroups];
    alignas(16) unsigned long long red[kRowThreads / 32];
    unsigned long long bound;
    Sums sums[kRowThreads / 32];
    Sums total;
    float row_max;
    int count, count2;
};

// 1024 threads on an SM with 63 registers each: 4096 x 128256 bf16 with 8 alternatives in 189 us; 1280 with 48 (which spill) 218.
template <typename T, int NT, bool ENT>
__global__ void __launch_bounds__(NT, 1024 / NT) token_logp_row(const LogpFwd p) {
    constexpr int EPV = Vec<T>::N, NP = EPV / 2;
    __shared__ RowShared sh;
    extern __shared__ __align__(16) unsigned long long list[];   // [kList + kSecond] with k > 0
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(block_in_cluster()), ranks = static_cast<int>(blocks_in_cluster());
    wait_for_stream();
    const int64_t t = blockIdx.x / static_cast<unsigned>(ranks);
    const T* z = static_cast<const T*>(p.z) + t * p.ld;
    const RowVecs<T> row(z, p.V);
    const int v0 = static_cast<int>(static_cast<int64_t>(row.n) * rank / ranks);   // this block's vectors
    const int v1 = static_cast<int>(static_cast<int64_t>(row.n) * (rank + 1) / ranks);
    const float c = p.inv_temp * kLog2e;
    // the token's logit, asked for early
    int64_t y = p.ignore;
    float zy = 0.f;
    if (rank == 0 && tid == 0 && p.tokens != nullptr) {
        y = p.tokens[t];
        if (y != p.ignore && y >= 0 && y < p.V) zy = ldf(z + y);
    }
    const float2 c2 = make_float2(c, c);
    Running run;
    run.set(Sums{kLowest, 0.f, 0.f}, c);
    // the thread's largest logit (NaN above all), and its vector
    float best = -INFINITY;
    int best_v = v0 + tid < v1 ? v0 + tid : -1;
    auto take = [&](const uint4 (&x)[kUnroll], int v, int count) {
        float m[kUnroll];
        m[0] = vec_max(x[0], T());
        float gm = m[0];
#pragma unroll
        for (int q = 1; q < kUnroll; ++q)
            if (q < count) {
                m[q] = vec_max(x[q], T());
                gm = max_nan(gm, m[q]);
            }
        if (!(gm <= best)) {   // larger, or NaN; rare after the first vectors
            if (best == best) {
                best = gm;
#pragma unroll
                for (int q = kUnroll - 1; q >= 0; --q)   // the first of equal ones
                    if (q < count && (m[q] == gm || m[q] != m[q])) best_v = v + q * NT;
            }
            if (gm > run.m) {
                Sums a = run.read(c);
                raise(a, gm, c);
                run.set(a, c);
            }
        }
        auto add = [&](auto far) {
            const float2 nk = make_float2(-run.k, -run.k), nm = make_float2(-run.m, -run.m);
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                if (q >= count) break;
                float2 f[NP];
                unpack2(x[q], f);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    float2 d = decltype(far)::value ? __fmul2_rn(__fadd2_rn(f[e], nm), c2) : __ffma2_rn(f[e], c2, nk);
                    if (ENT) {   // a logit of -inf has d below any limit: held where 2^d is 0, so that d 2^d is not NaN
                        d.x = max_nan(d.x, -200.f);
                        d.y = max_nan(d.y, -200.f);
                    }
                    const float2 w = make_float2(ex2(d.x), ex2(d.y));
                    run.s = __fadd2_rn(run.s, w);
                    if (ENT) run.u = __ffma2_rn(d, w, run.u);
                }
            }
        };
        if (run.far()) add(std::true_type());
        else add(std::false_type());
    };
    // groups of kUnroll vectors a thread, NT apart; the next group is asked for before this one is used
    constexpr int STEP = kUnroll * NT;
    auto fetch = [&](uint4 (&x)[kUnroll], int g0) {   // the block's group from vector g0 on
        const int v = g0 + tid;
        if (g0 >= row.first && g0 + STEP <= min(row.last, v1)) {
            const uint4* at = reinterpret_cast<const uint4*>(row.base) + v;
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) x[q] = ldg16(at + q * NT);
        } else {
#pragma unroll
            for (int q = 0; q < kUnroll; ++q)
                if (v + q * NT < v1) x[q] = row.get(v + q * NT);
        }
    };
    uint4 next[kUnroll];
    fetch(next, v0);
    int g0 = v0;
    for (; g0 + STEP <= v1; g0 += STEP) {
        uint4 x[kUnroll];
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) x[q] = next[q];
        if (g0 + STEP < v1) fetch(next, g0 + STEP);
        take(x, g0 + tid, kUnroll);
    }
    if (g0 + tid < v1) take(next, g0 + tid, (v1 - g0 - tid + NT - 1) / NT);
    Sums a = run.read(c);
    // the warp's sums, and the groups' best logits as keys: the order of the value, then the vector's index
    const unsigned long long mine =
        best_v < 0 ? 0 : static_cast<unsigned long long>(order_of(best)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(best_v));
    constexpr int PER = NT / kGroups;   // neighbouring threads of a group
    unsigned long long key = mine;
    float wm = a.m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o == PER && lane % PER == 0) sh.groups[tid / PER] = key;
        key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
        wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    }
    raise(a, wm, c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        if (ENT) a.u += __shfl_xor_sync(0xffffffffu, a.u, o);
    }
    if (lane == 0) {
        sh.sums[warp] = a;
        sh.red[warp] = key;
    }
    if (tid < LIGER_TOP_MAX) sh.best[tid] = 0;
    if (tid == 0) {
        sh.bound = 0;
        sh.count = sh.count2 = 0;
    }
    __syncthreads();
    if (warp == NT / 32 - 1) {   // the last warp joins the warps' sums, in pairs that do not depend on anything but their number
        Sums w = lane < NT / 32 ? sh.sums[lane] : Sums{kLowest, 0.f, 0.f};
        unsigned long long top = lane < NT / 32 ? sh.red[lane] : 0;
        float m = w.m;
#pragma unroll
        for (int o = NT / 64; o > 0; o >>= 1) {
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        raise(w, m, c);
#pragma unroll
        for (int o = NT / 64; o > 0; o >>= 1) {
            w.s += __shfl_xor_sync(0xffffffffu, w.s, o);
            w.u += __shfl_xor_sync(0xffffffffu, w.u, o);
        }
        if (lane == 0) {
            sh.total = w;
            sh.row_max = value_of(static_cast<uint32_t>(top >> 32));
        }
    }
    if (p.k > 0) {
        if (tid < kGroups) {   // the k-th largest of the groups' (those without an element: 0, and not distinct)
            const unsigned long long x = sh.groups[tid];
            int above = 0;
#pragma unroll 8
            for (int i = 0; i < kGroups; ++i) above += sh.groups[i] > x ? 1 : 0;
            if (x != 0 && above == p.k - 1) sh.bound = x;
        }
        __syncthreads();
        const unsigned long long bound = sh.bound;
        const uint32_t bound_o = static_cast<uint32_t>(bound >> 32), bound_v = 0xFFFFFFFFu - static_cast<uint32_t>(bound);
        uint32_t hot = __ballot_sync(0xffffffffu, mine != 0 && mine >= bound);
        while (hot != 0) {   // the vectors of one thread at a time, over the warp
            const int vt = v0 + warp * 32 + (__ffs(hot) - 1);
            hot &= hot - 1;
            for (int x0 = vt + lane * NT; x0 < v1; x0 += 64 * NT) {
                uint4 w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (x0 + h * 32 * NT < v1) w[h] = row.get(x0 + h * 32 * NT);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = x0 + h * 32 * NT;
                    if (x >= v1 || order_of(vec_max(w[h], T())) < bound_o) continue;
                    const bool level = bound == 0 || static_cast<uint32_t>(x) <= bound_v;
                    float f[EPV];
                    unpack(w[h], f);
#pragma unroll
                    for (int e = 0; e < EPV; ++e) {
                        const int i = x * EPV + e - row.shift;
                        const uint32_t o = order_of(f[e]);
                        if (i >= 0 && i < row.V && (o > bound_o || (o == bound_o && level))) {
                            const int at = atomicAdd(&sh.count, 1);   // in any order: the keys are ranked
                            if (at < kList) list[at] = rank_key(f[e], static_cast<uint32_t>(i));
                        }
                    }
                }
            }
        }
        __syncthreads();
        const int n = sh.count;
        if (n > kList) {
            // given up: the largest below the last one found, k times
            unsigned long long last = ~0ull;
            for (int i = 0; i < p.k; ++i) {
                unsigned long long b = 0;
                for (int x = v0 + tid; x < v1; x += NT) {
                    float f[EPV];
                    row.get(x, f);
#pragma unroll
                    for (int e = 0; e < EPV; ++e) {
                        const int j = x * EPV + e - row.shift;
                        const unsigned long long key = rank_key(f[e], static_cast<uint32_t>(j));
                        if (j >= 0 && j < row.V && key < last && key > b) b = key;
                    }
                }
                last = block_max_key<NT>(b, sh.red);
                if (tid == 0) sh.best[i] = last;
                if (last == 0) break;   // a share of fewer than k elements
            }
        } else if (n <= 2 * kGroups) {
            rank_keys<NT>(list, n, p.k, sh.best);
        } else {
            // the same bound again, over the list: the k-th largest of kGroups groups' best
            if (tid < kGroups) {
                unsigned long long g2 = 0;
                for (int i = tid; i < n; i += kGroups) g2 = max(g2, list[i]);
                sh.groups[tid] = g2;
            }
            __syncthreads();
            if (tid < kGroups) {
                const unsigned long long x = sh.groups[tid];
                int above = 0;
#pragma unroll 8
                for (int i = 0; i < kGroups; ++i) above += sh.groups[i] > x ? 1 : 0;
                if (above == p.k - 1) sh.bound = x;
            }
            __syncthreads();
            const unsigned long long b2 = sh.bound;
            for (int i = tid; i < n; i += NT)
                if (list[i] >= b2) list[kList + atomicAdd(&sh.count2, 1)] = list[i];
            __syncthreads();
            rank_keys<NT>(list + kList, sh.count2, p.k, sh.best);
        }
    }
    __syncthreads();
    if (ranks > 1) cluster_barrier();
    if (rank == 0) {
        // the blocks' sums in their order, and their alternatives ranked again
        Sums all = sh.total;
        float m = sh.row_max;
        for (int r = 1; r < ranks; ++r) {
            const Sums b{peer_float(&sh.total.m, r), peer_float(&sh.total.s, r), peer_float(&sh.total.u, r)};
            join(all, b, c);
            m = max_nan(m, peer_float(&sh.row_max, r));
        }
        const bool none = m == -INFINITY;
        const float l2 = log2f(all.s), ls = l2 * kLn2;   // relative to all.m, which is m but for NaN (all.s is NaN then)
        if (tid == 0) {
            if (p.row_max != nullptr) p.row_max[t] = m;
            if (p.log_sum != nullptr) p.log_sum[t] = none ? -INFINITY : ls;
            if (p.entropy != nullptr) p.entropy[t] = none ? 0.f : (l2 - all.u / all.s) * kLn2;
            if (p.logp != nullptr) {
                float r = 0.f;
                if (y != p.ignore) {
                    if (y < 0 || y >= p.V) r = NAN;
                    else r = none ? -INFINITY : fmaf(zy - all.m, p.inv_temp, -ls);
                }
                p.logp[t] = r;
            }
        }
        if (p.k > 0) {
            const unsigned long long* keys = sh.best;
            if (ranks > 1) {
                for (int i = tid; i < ranks * p.k; i += NT) list[i] = peer_key(&sh.best[i % p.k], i / p.k);
                __syncthreads();
                unsigned long long* out = list + ranks * p.k;   // (0 marks a missing one: below all keys, of which there are k)
                for (int i = tid; i < ranks * p.k; i += NT) {
                    const unsigned long long x = list[i];
                    int above = 0;
                    for (int j = 0; j < ranks * p.k; ++j) above += list[j] > x ? 1 : 0;
                    if (x != 0 && above < p.k) out[above] = x;
                }
                __syncthreads();
                keys = out;
            }
            for (int i = tid; i < p.k; i += NT) {
                const unsigned long long key = keys[i];
                p.top_ids[t * p.k + i] = 0xFFFFFFFFu - static_cast<uint32_t>(key);
                p.top_logp[t * p.k + i] = none ? -INFINITY : fmaf(value_of(static_cast<uint32_t>(key >> 32)) - all.m, p.inv_temp, -ls);
            }
        }
    }
    if (ranks > 1) {
        __syncwarp();
        cluster_barrier();   // no block exits while another reads from it
    }
}

struct LogpBwd {
    const void* z;
    int64_t ld;
    const int64_t* tokens;
    const float *row_max, *log_sum, *entropy, *g_logp, *g_entropy;
    int64_t T, V, ignore;
    float inv_temp;
    void* dz;
    int64_t ldd;
};

// dz = (g 1[v = y] - p (g + h (a + H))) / temperature with a = log p, p = e^a: every element read and written once.
// A block takes a run of a row's vectors; VECS: logits and gradients have the same place within 16 bytes.
template <typename T, bool VECS>
__global__ void __launch_bounds__(kRowThreads) token_logp_grad(const LogpBwd p) {
    constexpr int EPV = Vec<T>::N;
    wait_for_stream();
    const int64_t t = blockIdx.x;
    const T* z = static_cast<const T*>(p.z) + t * p.ld;
    T* dz = static_cast<T*>(p.dz) + t * p.ldd;
    // the first vectors are asked for before the row's scalars are known
    const RowVecs<T> row(z, p.V);
    const int64_t v0 = static_cast<int64_t>(row.n) * blockIdx.y / gridDim.y, v1 = static_cast<int64_t>(row.n) * (blockIdx.y + 1) / gridDim.y;
    uint4 x[kUnroll];
    auto load = [&](int64_t v) {
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int64_t w = v + q * kRowThreads;
            if (w < v1 && w >= row.first && w < row.last) x[q] = ldg16(row.base + w * EPV);
        }
    };
    if (VECS) load(v0 + threadIdx.x);
    const int64_t y = p.tokens != nullptr ? p.tokens[t] : p.ignore;
    const bool counts = p.g_logp != nullptr && y != p.ignore;
    float g = counts ? p.g_logp[t] : 0.f;
    if (counts && (y < 0 || y >= p.V)) g = NAN;
    const float h = p.g_entropy != nullptr ? p.g_entropy[t] : 0.f, H = p.g_entropy != nullptr ? p.entropy[t] : 0.f;
    const float m = p.row_max[t], ls = p.log_sum[t];
    const bool zero = (g == 0.f && h == 0.f) || (m == -INFINITY && g == g && h == h);
    // temperature dz = -e^a (h a + c), and g more at the token (scaled last: the sums of a row stay in range at any temperature)
    const float c = fmaf(h, H, g);
    auto one = [&](float zv, int64_t i) {
        const float a = max_nan(fmaf(zv - m, p.inv_temp, -ls), -1e4f);   // of -inf: held where e^a is 0
        const float d = ex2(a * kLog2e) * fmaf(-h, a, -c);
        return (i == y ? d + g : d) * p.inv_temp;
    };
    if constexpr (!VECS) {
        for (int64_t i = static_cast<int64_t>(blockIdx.y) * kRowThreads + threadIdx.x; i < p.V; i += static_cast<int64_t>(gridDim.y) * kRowThreads)
            stf(dz + i, zero ? 0.f : one(ldf(z + i), i));
        return;
    } else {
        T* out = dz - row.shift;
        const float2 nm = make_float2(-m, -m), it = make_float2(p.inv_temp, p.inv_temp), nls = make_float2(-ls, -ls),
                     l2e = make_float2(kLog2e, kLog2e), nh = make_float2(-h, -h), nc = make_float2(-c, -c);
        for (int64_t v = v0 + threadIdx.x; v < v1; v += kUnroll * kRowThreads) {
            if (!zero && v >= v0 + kUnroll * kRowThreads) load(v);
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                const int64_t w = v + q * kRowThreads, i0 = w * EPV - row.shift;
                if (w >= v1) break;
                if (w >= row.first && w < row.last) {
                    float2 f[EPV / 2] = {};
                    if (!zero) {
                        unpack2(x[q], f);
#pragma unroll
                        for (int e = 0; e < EPV / 2; ++e) {
                            float2 a = __ffma2_rn(__fadd2_rn(f[e], nm), it, nls);
                            a = make_float2(max_nan(a.x, -1e4f), max_nan(a.y, -1e4f));
                            const float2 b = __fmul2_rn(a, l2e);
                            f[e] = __fmul2_rn(make_float2(ex2(b.x), ex2(b.y)), __ffma2_rn(nh, a, nc));
                        }
                        const int64_t at = y - i0;
                        if (at >= 0 && at < EPV)
#pragma unroll
                            for (int e = 0; e < EPV / 2; ++e) {
                                if (at == 2 * e) f[e].x += g;
                                if (at == 2 * e + 1) f[e].y += g;
                            }
#pragma unroll
                        for (int e = 0; e < EPV / 2; ++e) f[e] = __fmul2_rn(f[e], it);
                    }
                    stg16_cs(out + w * EPV, pack2(f));
                } else {
                    for (int e = 0; e < EPV; ++e)
                        if (i0 + e >= 0 && i0 + e < p.V) stf(dz + i0 + e, zero ? 0.f : one(ldf(z + i0 + e), i0 + e));
                }
            }
        }
    }
}

// ------------------------------------------------------------------ launches
template <typename T, int NT, bool ENT>
int launch_row(const char* who, const LogpFwd& p, int ranks, cudaStream_t st) {
    const size_t smem = p.k > 0 ? (kList + kSecond) * sizeof(unsigned long long) : 0;
    return launch_cluster(who, token_logp_row<T, NT, ENT>, dim3(static_cast<unsigned>(p.T * ranks)), dim3(static_cast<unsigned>(ranks)),
                          NT, smem, st, p);
}

template <typename T>
int launch_fwd(const char* who, const LogpFwd& p, cudaStream_t st) {
    const int64_t vecs = ceil_div(p.V, Vec<T>::N);
    const bool ent = p.entropy != nullptr;
    // Few rows: each over a cluster of blocks, while an SM has one of them and a thread more than 8 vectors.  128256 bf16 logits with 8
    // alternatives, over 1, 2, 4, 8 blocks: one row 13.4, 10.3, 9.6, 9.5 us; 38 rows 14.1, 12.8, 10.7, 11.1; 76 rows 15.1, 12.7, 13.3,
    // 20.0; 152 rows 15.6, 15.4, 21.7, 31.2.  32768 logits: one row 6.6, 7.9, 7.7, 8.5.
    int ranks = 1;
    while (ranks < 8 && p.T * ranks * 2 <= sm_count() && vecs > 16 * ranks * kRowThreads) ranks *= 2;
    if (vecs < kRowThreads) return ent ? launch_row<T, 64, true>(who, p, 1, st) : launch_row<T, 64, false>(who, p, 1, st);
    if (vecs <= kShortRow && p.T >= kManyRows * sm_count())
        return ent ? launch_row<T, 128, true>(who, p, 1, st) : launch_row<T, 128, false>(who, p, 1, st);
    return ent ? launch_row<T, kRowThreads, true>(who, p, ranks, st) : launch_row<T, kRowThreads, false>(who, p, ranks, st);
}

template <typename T>
int launch_bwd(const char* who, const LogpBwd& p, cudaStream_t st) {
    const int64_t vecs = ceil_div(p.V, Vec<T>::N);
    const uintptr_t az = reinterpret_cast<uintptr_t>(p.z), ad = reinterpret_cast<uintptr_t>(p.dz);
    const bool same = (az - ad) % 16 == 0 && (p.T == 1 || (p.ld - p.ldd) * static_cast<int64_t>(sizeof(T)) % 16 == 0);
    // 4 rounds of vectors a thread: 4096 x 128256 bf16 in 313 us, 334 with 2, 388 with 1, 314 with 8; few rows over more blocks
    const int64_t fill = std::min<int64_t>(vecs / kRowThreads, ceil_div(2 * sm_count(), p.T));
    const int64_t y = std::min<int64_t>(65535, std::max<int64_t>({1, fill, vecs / (4 * kUnroll * kRowThreads)}));
    const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>(y));
    return same ? launch_early(who, token_logp_grad<T, true>, grid, kRowThreads, 0, st, p)
                : launch_early(who, token_logp_grad<T, false>, grid, kRowThreads, 0, st, p);
}

int check_logits(const char* who, int64_t T, int64_t V, int64_t ld, float temperature, int dtype) {
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (T < 0 || T > 2147483647LL || V <= 0 || V > (1 << 30) || ld < V || ld > (int64_t{1} << 40))
        return fail(LIGER_ERR_SHAPE, "%s: T=%lld V=%lld ld=%lld", who, (long long)T, (long long)V, (long long)ld);
    if (!(temperature >= 1e-30f) || !isfinite(temperature))   // (so that logits over it stay in range of the arithmetic)
        return fail(LIGER_ERR_SHAPE, "%s: temperature must be at least 1e-30", who);
    return LIGER_OK;
}
bool off(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" int liger_token_logp_fwd(const void* logits, int64_t ld, const int64_t* tokens, int64_t T, int64_t V,
                                    int64_t ignore_index, float temperature, float* logp, float* row_max, float* log_sum,
                                    float* entropy, int64_t k, float* top_logp, int64_t* top_ids, int dtype, void* stream) {
    clear_error();
    const char* who = "token_logp_fwd";
    if (int rc = check_logits(who, T, V, ld, temperature, dtype)) return rc;
    if (k < 0 || k > LIGER_TOP_MAX || k > V)
        return fail(LIGER_ERR_SHAPE, "%s: k=%lld (0 to %d, at most V=%lld)", who, (long long)k, LIGER_TOP_MAX, (long long)V);
    if (T == 0) return LIGER_OK;
    if (!logits) return fail(LIGER_ERR_NULL, "%s: logits are required", who);
    if ((tokens == nullptr) != (logp == nullptr)) return fail(LIGER_ERR_NULL, "%s: tokens and logp go together", who);
    if ((k > 0) != (top_logp != nullptr) || (k > 0) != (top_ids != nullptr))
        return fail(LIGER_ERR_NULL, "%s: top_logp and top_ids go with k > 0", who);
    if (off(logits, dtype == LIGER_F32 ? 4 : 2) || off(tokens, 8) || off(top_ids, 8) || off(logp, 4) || off(row_max, 4) ||
        off(log_sum, 4) || off(entropy, 4) || off(top_logp, 4))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be aligned to their elements", who);
    const LogpFwd p{logits, ld, tokens, T, V, ignore_index, 1.0f / temperature, logp, row_max, log_sum, entropy, top_logp, top_ids,
                    static_cast<int>(k)};
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32 ? launch_fwd<float>(who, p, st) : launch_fwd<__nv_bfloat16>(who, p, st);
}

extern "C" int liger_token_logp_bwd(const void* logits, int64_t ld, const int64_t* tokens, const float* row_max,
                                    const float* log_sum, const float* entropy, const float* g_logp, const float* g_entropy,
                                    int64_t T, int64_t V, int64_t ignore_index, float temperature, void* dlogits, int64_t ldd,
                                    int dtype, void* stream) {
    clear_error();
    const char* who = "token_logp_bwd";
    if (int rc = check_logits(who, T, V, ld, temperature, dtype)) return rc;
    if (ldd < V || ldd > (int64_t{1} << 40)) return fail(LIGER_ERR_SHAPE, "%s: ldd=%lld", who, (long long)ldd);
    if (T == 0) return LIGER_OK;
    if (!logits || !row_max || !log_sum || !dlogits)
        return fail(LIGER_ERR_NULL, "%s: logits, row_max, log_sum and dlogits are required", who);
    if (!g_logp && !g_entropy) return fail(LIGER_ERR_NULL, "%s: g_logp or g_entropy is required", who);
    if (g_logp && !tokens) return fail(LIGER_ERR_NULL, "%s: g_logp needs tokens", who);
    if (g_entropy && !entropy) return fail(LIGER_ERR_NULL, "%s: g_entropy needs entropy", who);
    if (dlogits == logits && ldd != ld) return fail(LIGER_ERR_SHAPE, "%s: in place ldd must be ld", who);
    const size_t esz = dtype == LIGER_F32 ? 4 : 2;
    if (off(logits, esz) || off(dlogits, esz) || off(tokens, 8) || off(row_max, 4) || off(log_sum, 4) || off(entropy, 4) || off(g_logp, 4) ||
        off(g_entropy, 4))
        return fail(LIGER_ERR_ALIGN, "%s: tensors must be aligned to their elements", who);
    const LogpBwd p{logits, ld, g_logp ? tokens : nullptr, row_max, log_sum, entropy, g_logp, g_entropy, T, V, ignore_index,
                    1.0f / temperature, dlogits, ldd};
    cudaStream_t st = as_stream(stream);
    return dtype == LIGER_F32 ? launch_bwd<float>(who, p, st) : launch_bwd<__nv_bfloat16>(who, p, st);
}
