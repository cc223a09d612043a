// Fused linear cross-entropy, forward and backward, token-chunked.
//
// Operator: the FusedCrossEntropyLoss paragraph of the page "Liger-Kernel核心
// 技术：RollingBuffer与融合算子详解", section "算子融合" -- softmax and NLL in one
// step on the classifier-head output, the softmax never stored -- with the
// online softmax merge (running maximum and rescaled normaliser per tile) of
// the page "Liger-Kernel内核级优化：FlashAttention与RollingBuffer详解".
//
// bf16 path (tensor cores), per chunk of C tokens (rows t0 .. t0+C):
//   1. Z_c = X_c W^T on tcgen05; the epilogue never stores z: per 256-wide
//      vocab tile it keeps the row max m and sum s of exp(z - m), writes
//      P = exp(z - m) in bf16 to the [C x V] chunk buffer, and the logit at
//      the label in fp32;
//   2. one block per row merges the (m, s) of all vocab tiles into lse, the
//      row's loss term, and rewrites P in place into the softmax part of D,
//      S = scale * P * exp(m_tile - lse) (bf16);
//   3. dX_c = S W on tcgen05 (W read MN-major); the epilogue subtracts the
//      one-hot part, scale * W[label], in fp32; ignored rows written +0;
//   4. dW (+)= S^T X_c on tcgen05 (both operands MN-major); the epilogue
//      subtracts scale * X_t for the tokens labelled with the row (the chunk's
//      labels sorted once, indexed by a [V+1] start table) in fp32, and
//      prefetches and accumulates across chunks in
//      an fp32 [V x H] workspace, the last chunk writing W's dtype.
// Keeping the one-hot term out of the bf16 operand matters: rounding
// -scale to bf16 at every label would cost up to 2^-9 relative on the rows of
// dW and dX that dominate their magnitude.
// The full [T x V] logits never exist; per chunk only [C x V] bf16 does.
//
// fp32 path (and bf16 with H not a multiple of 8): the same steps with an
// fp32 SIMT GEMM and an fp32 [C x V] chunk buffer holding z, then D.  TF32
// tensor cores would miss the 1e-5 fp32 tolerance, so fp32 stays on FMA.
#include <math.h>

#include <atomic>

#include "head_simt.cuh"
#include "liger_train.h"
#include "tc_gemm.cuh"

namespace liger {

namespace {

constexpr int kVT = tc::BN;   // vocab tile of the (m, s) partials
constexpr int kMaxSortKeys = 8192;      // label keys sorted together (shared memory)
constexpr int64_t kAutoChunkTC = 8192;   // tensor-core path: most rows per chunk chosen automatically
constexpr int64_t kMaxChunkTC = 65536;   // tensor-core path: most rows per chunk a caller may ask for
// The dX GEMM's K is the whole vocabulary: over 150 k vocabulary rows the tiles of a
// wave drift apart along K and stop sharing their D and W slices through L2 (it read
// 4-6x its operand bytes from DRAM).  Above this many vocabulary rows it runs in
// launches over equal slabs of at most this many rows (0: one launch), the partial sums
// kept in an fp32 [chunk x H] buffer; each launch starts the wave's tiles together.
constexpr int64_t kDxSlabRows = 65536;

// vocabulary rows per dX launch: V itself, or equal slabs (multiples of 256) of at most kDxSlabRows
int64_t dx_slab(int64_t V) {
    if (kDxSlabRows <= 0 || V <= kDxSlabRows) return V;
    const int64_t n = (V + kDxSlabRows - 1) / kDxSlabRows;
    return ((V + n - 1) / n + 255) / 256 * 256;
}

struct Hdr {
    unsigned long long n_valid;
    int bad;
    int err;
    float scale;   // the gradient scale, when it is formed on the device (no host wait)
};

struct Layout {
    bool tc;
    int64_t C, ldp, nvt, nchunks;
    int seg;   // label-sort segment: the chunk (C <= 8192, indices relative to it) or 8192 tokens (absolute)
    size_t lse, lossrow, zlab, hdr, labs, keys, lstart, part, scr, acc, dxacc, total;
};

inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool use_tc(int64_t H, int64_t V, int dtype) { return dtype == LIGER_BF16 && H % 8 == 0 && H >= 64 && V >= 256; }

Layout layout(int64_t T, int64_t H, int64_t V, int64_t chunk, int dtype) {
    Layout L{};
    L.tc = use_tc(H, V, dtype);
    int64_t C;
    if (chunk > 0) C = chunk;
    // automatic: at most half the tokens (never all T rows at once, for T > 128), at most kAutoChunkTC rows
    else if (L.tc) {
        C = std::min<int64_t>(kAutoChunkTC, std::max<int64_t>(128, (T + 1) / 2));
        // large chunks in whole 256-row tiles of the CTA-pair GEMMs (7373 tokens: 3840 + 3533
        // rows, 15 + 14 row tiles, rather than 2 x 3687 rows in 15 + 15)
        if (C >= 1024) C = std::min<int64_t>(kAutoChunkTC, (C + 255) / 256 * 256);
    }
    else C = std::max<int64_t>(128, (int64_t{1} << 26) / std::max<int64_t>(V, 1));
    if (L.tc) {
        C = std::min<int64_t>(C, kMaxChunkTC);
        // above one label-sort block, whole blocks (the chunk's labels are sorted block by block)
        if (C > kMaxSortKeys && C < T) C = (C / kMaxSortKeys) * kMaxSortKeys;
    }
    C = std::max<int64_t>(1, std::min(C, std::max<int64_t>(T, 1)));
    L.C = C;
    L.seg = static_cast<int>(std::min<int64_t>(C, kMaxSortKeys));
    L.nchunks = T > 0 ? ceil_div(T, C) : 0;
    L.ldp = L.tc ? ((V + 7) / 8) * 8 : V;
    L.nvt = ceil_div(V, kVT);
    size_t o = 0;
    L.lse = o; o = up256(o + sizeof(float) * static_cast<size_t>(T));
    L.lossrow = o; o = up256(o + sizeof(float) * static_cast<size_t>(T));
    L.zlab = o; o = up256(o + sizeof(float) * static_cast<size_t>(T));
    L.hdr = o; o = up256(o + sizeof(Hdr));
    // the labels with bad ones replaced by ignore_index (the entry points that do not wait)
    L.labs = o; o = up256(o + sizeof(int64_t) * static_cast<size_t>(T));
    // every chunk's sorted label keys and start table, made in one pass before the chunks
    L.keys = o; o = up256(o + (L.tc ? sizeof(unsigned long long) * static_cast<size_t>(std::max<int64_t>(T, 1)) : 0));
    L.lstart = o; o = up256(o + (L.tc ? sizeof(int) * static_cast<size_t>(ceil_div(std::max<int64_t>(T, 1), L.seg) * (V + 1)) : 0));
    L.part = o; o = up256(o + (L.tc ? sizeof(float2) * static_cast<size_t>(C * L.nvt) : 0));
    L.scr = o; o = up256(o + static_cast<size_t>(C) * static_cast<size_t>(L.ldp) * (L.tc ? 2 : 4));
    const bool need_acc = L.nchunks > 1 && dtype == LIGER_BF16;
    L.acc = o; o = up256(o + (need_acc ? sizeof(float) * static_cast<size_t>(V * H) : 0));
    const bool dx_slabs = L.tc && dx_slab(V) < V;
    L.dxacc = o; o = up256(o + (dx_slabs ? sizeof(float) * static_cast<size_t>(C * H) : 0));
    L.total = o;
    return L;
}

// Workspace of the waiting tensor-core entry points, which run their GEMMs on the
// tokens that are not ignored only: the ordinary layout's lse, loss_row and header
// first (lse and loss_row of every token, as documented), then the region the
// variant runs in for those tokens (at most the ordinary layout's size), then
// their X rows, their dX rows, their labels and the index maps.
struct CompactLayout {
    size_t core, xc, dxc, labc, idx, inv, cnt, total;
};

constexpr int kCompactBlock = 1024;   // tokens per block of the compaction's index pass

// core_at: where the ordinary layout's per-call part ends (after lse, loss_row, z_label
// and the header); core_total: the ordinary layout's size for all T tokens
CompactLayout compact_regions(size_t core_at, size_t core_total, int64_t T, int64_t H, size_t esz) {
    const size_t t = static_cast<size_t>(std::max<int64_t>(T, 1));
    CompactLayout C{};
    size_t o = core_at;
    C.core = o; o = up256(o + core_total);
    C.xc = o; o = up256(o + t * static_cast<size_t>(H) * esz);
    C.dxc = o; o = up256(o + t * static_cast<size_t>(H) * esz);
    C.labc = o; o = up256(o + t * sizeof(int64_t));
    C.idx = o; o = up256(o + t * sizeof(int64_t));
    C.inv = o; o = up256(o + t * sizeof(int));
    C.cnt = o; o = up256(o + sizeof(int) * static_cast<size_t>(ceil_div(static_cast<int64_t>(t), int64_t{kCompactBlock})));
    C.total = o;
    return C;
}

CompactLayout compact_layout(int64_t T, int64_t H, int64_t V, int64_t chunk, int dtype) {
    const Layout L = layout(T, H, V, chunk, dtype);
    return compact_regions(L.labs, L.total, T, H, dtype == LIGER_F32 ? 4 : 2);
}

// ---------------------------------------------------------------- kernels
// ---- compaction of the tokens that are not ignored (stable: their order is kept)
__global__ void __launch_bounds__(kCompactBlock) compact_count(const int64_t* __restrict__ labels, int64_t T,
                                                               int64_t ignore, int* __restrict__ cnt) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kCompactBlock + threadIdx.x;
    const int c = __syncthreads_count(t < T && labels[t] != ignore);
    if (threadIdx.x == 0) cnt[blockIdx.x] = c;
}

// cnt[0, nb) -> exclusive prefix sums, in place (one block of 1024 threads)
__global__ void __launch_bounds__(1024) compact_scan(int* cnt, int64_t nb) {
    __shared__ int sums[1024];
    const int64_t per = (nb + 1023) / 1024;
    const int64_t b0 = threadIdx.x * per, b1 = min(nb, b0 + per);
    int s = 0;
    for (int64_t b = b0; b < b1; ++b) s += cnt[b];
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
        const int v = threadIdx.x >= o ? sums[threadIdx.x - o] : 0;
        __syncthreads();
        sums[threadIdx.x] += v;
        __syncthreads();
    }
    int run = threadIdx.x ? sums[threadIdx.x - 1] : 0;
    for (int64_t b = b0; b < b1; ++b) {
        const int c = cnt[b];
        cnt[b] = run;
        run += c;
    }
}

// idx[p] = t and lab_c[p] = labels[t] for the p-th token that is not ignored; inv[t] = p, or -1
__global__ void __launch_bounds__(kCompactBlock) compact_index(const int64_t* __restrict__ labels, int64_t T,
                                                               int64_t ignore, const int* __restrict__ off,
                                                               int64_t* __restrict__ idx, int* __restrict__ inv,
                                                               int64_t* __restrict__ lab_c) {
    __shared__ int wsum[kCompactBlock / 32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kCompactBlock + threadIdx.x;
    const int64_t y = t < T ? labels[t] : ignore;
    const bool v = t < T && y != ignore;
    const unsigned m = __ballot_sync(0xffffffffu, v);
    if (lane == 0) wsum[wid] = __popc(m);
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wid; ++w) before += wsum[w];
    const int p = off[blockIdx.x] + before + __popc(m & ((1u << lane) - 1u));
    if (v) {
        idx[p] = t;
        lab_c[p] = y;
    }
    if (t < T) inv[t] = v ? p : -1;
}

// rows (16-byte vectors, hv per row): dst[r] = src[idx[r]], r < n
__global__ void gather_rows(const uint4* __restrict__ src, const int64_t* __restrict__ idx, int64_t n, int64_t hv,
                            uint4* __restrict__ dst) {
    for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
        const uint4* s = src + idx[r] * hv;
        uint4* d = dst + r * hv;
        for (int64_t v = threadIdx.x; v < hv; v += blockDim.x) d[v] = ldg16_nc(s + v);
    }
}

// dst = the rows of src, those of ignored tokens as zeros
__global__ void masked_rows(const uint4* src, const int64_t* labels, int64_t ignore, int64_t T, int64_t hv,
                            uint4* __restrict__ dst) {
    wait_for_stream();
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const bool keep = labels[t] != ignore;
        for (int64_t v = threadIdx.x; v < hv; v += blockDim.x)
            dst[t * hv + v] = keep ? ldg16(src + t * hv + v) : make_uint4(0, 0, 0, 0);
    }
}

// rows back in place: dst[t] = src[inv[t]], or +0 where inv[t] < 0 (an ignored token)
__global__ void scatter_rows(const uint4* __restrict__ src, const int* __restrict__ inv, int64_t T, int64_t hv,
                             uint4* __restrict__ dst) {
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const int p = inv[t];
        uint4* d = dst + t * hv;
        if (p < 0) {
            for (int64_t v = threadIdx.x; v < hv; v += blockDim.x) d[v] = make_uint4(0, 0, 0, 0);
        } else {
            const uint4* s = src + static_cast<int64_t>(p) * hv;
            for (int64_t v = threadIdx.x; v < hv; v += blockDim.x) d[v] = ldg16_nc(s + v);
        }
    }
}

// lse and loss_row of every token from those of the tokens that were run (+0 where ignored),
// and the run's kernel error word into the entry point's header
__global__ void scatter_rowvals(const float* __restrict__ lse_c, const float* __restrict__ loss_c,
                                const int* __restrict__ inv, int64_t T, float* __restrict__ lse,
                                float* __restrict__ loss, const int* core_err, int* err) {
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < T;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int p = inv[t];
        lse[t] = p < 0 ? 0.f : lse_c[p];
        loss[t] = p < 0 ? 0.f : loss_c[p];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && *core_err != 0) atomicExch(err, *core_err);
}

// the run's kernel error word into the entry point's header
__global__ void take_err(const int* core_err, int* err) {
    if (*core_err != 0) atomicExch(err, *core_err);
}

// Counts the labels that are not ignore_index and flags any outside [0, V).  With
// lab_out set, also writes the labels with every bad one replaced by ignore_index
// (and not counted), so that no later kernel indexes with it.
__global__ void label_scan(const int64_t* __restrict__ labels, int64_t T, int64_t V, int64_t ignore, Hdr* hdr,
                           int64_t* __restrict__ lab_out) {
    unsigned long long cnt = 0;
    int bad = 0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < T;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        int64_t y = labels[t];
        if (y != ignore && (y < 0 || y >= V)) {
            bad = 1;
            if (lab_out != nullptr) y = ignore;
        }
        if (lab_out != nullptr) lab_out[t] = y;
        if (y != ignore) ++cnt;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
        bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    if ((threadIdx.x & 31) == 0) {
        if (cnt) atomicAdd(&hdr->n_valid, cnt);
        if (bad) atomicOr(&hdr->bad, 1);
    }
}

// The gradient scale from the device-side count: grad_scale / n_valid (mean; 0 when
// nothing is valid) or grad_scale (sum)
__global__ void ce_scale(Hdr* hdr, int reduction, float grad_scale) {
    const unsigned long long n = hdr->n_valid;
    hdr->scale = reduction == 0 ? (n > 0 ? static_cast<float>(static_cast<double>(grad_scale) / static_cast<double>(n))
                                         : 0.0f)
                                : grad_scale;
}

template <int NT>
__device__ __forceinline__ float block_reduce(float v, bool is_max, float* sh) {
    v = is_max ? warp_max(v) : warp_sum(v);
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    __syncthreads();
    if (l == 0) sh[w] = v;
    __syncthreads();
    float r = is_max ? -INFINITY : 0.f;
    for (int i = 0; i < NT / 32; ++i) r = is_max ? fmaxf(r, sh[i]) : r + sh[i];
    return r;
}

// Sort the (label << 32 | token) keys of each segment of seg tokens (ignored
// tokens -> ~0) for the one-hot correction of the dW epilogue.  Segment b covers
// tokens [b*seg, min(n, (b+1)*seg)) and its sorted keys go to out[b*seg ...]; the
// token index in a key is absolute (b*seg + i) or relative to the segment (i).
// By ranks: a block finds how many keys of the segment (blockIdx.y) stand before each
// of 32 keys, one per lane, its warps counting over an eighth of the segment each,
// four labels a load from shared memory (2741 keys: 6.6 us, 52 sorted by one block).
constexpr int kRankThreads = 256;
__global__ void __launch_bounds__(kRankThreads) sort_label_keys(const int64_t* labels, int64_t n, int seg,
                                                                int64_t ignore, int absolute,
                                                                unsigned long long* __restrict__ out) {
    __shared__ __align__(16) uint32_t lab[kMaxSortKeys];
    __shared__ int before[kRankThreads / 32][32];
    const int64_t b0 = static_cast<int64_t>(blockIdx.y) * seg;
    const int cnt = static_cast<int>(n - b0 < seg ? n - b0 : seg);
    const int i0 = blockIdx.x * 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_stream();
    if (i0 >= cnt) return;
    const int quads = (cnt + 3) / 4;
    for (int i = threadIdx.x; i < quads * 4; i += kRankThreads) {
        const int64_t y = i < cnt ? labels[b0 + i] : ignore;
        lab[i] = y == ignore ? 0xFFFFFFFFu : static_cast<uint32_t>(y);   // labels are below 2^30
    }
    __syncthreads();
    // in the order of label, then token: labels up to this key's ahead of the 32, below it behind them
    const int i = i0 + lane;
    const uint32_t y = i < cnt ? lab[i] : 0u;
    const uint4* l4 = reinterpret_cast<const uint4*>(lab);
    int k = 0;
    for (int j = warp; j < i0 / 4; j += kRankThreads / 32) {
        const uint4 v = l4[j];
        k += (v.x <= y) + (v.y <= y) + (v.z <= y) + (v.w <= y);
    }
    for (int j = (i0 + 32) / 4 + warp; j < quads; j += kRankThreads / 32) {   // its padding is below no label
        const uint4 v = l4[j];
        k += (v.x < y) + (v.y < y) + (v.z < y) + (v.w < y);
    }
    if (warp == 0)
        for (int j = i0; j < min(cnt, i0 + 32); ++j) k += lab[j] < y || (lab[j] == y && j < i);
    before[warp][lane] = k;
    __syncthreads();
    if (warp != 0 || i >= cnt) return;
    int rank = 0;
    for (int w = 0; w < kRankThreads / 32; ++w) rank += before[w][lane];
    const unsigned token = (absolute ? static_cast<unsigned>(b0) : 0u) + static_cast<unsigned>(i);
    out[b0 + rank] = y == 0xFFFFFFFFu ? ~0ull : (static_cast<unsigned long long>(y) << 32) | token;
}

// Start tables of every segment (blockIdx.y): lstart[s*(V+1) + v] = first index
// of label v among segment s's sorted keys, v in [0, V], plus s*seg when the
// indices are absolute -- so the tokens of segment s labelled v are
// keys[lstart[v] .. lstart[v+1]) of the array the table's indices refer to.
__global__ void label_starts(const unsigned long long* keys, int64_t n, int seg, int V, int absolute,
                             int* __restrict__ lstart) {
    const int64_t b0 = static_cast<int64_t>(blockIdx.y) * seg;
    const int cnt = static_cast<int>(n - b0 < seg ? n - b0 : seg);
    const unsigned long long* k = keys + b0;
    int* ls = lstart + static_cast<int64_t>(blockIdx.y) * (V + 1);
    const int base = absolute ? static_cast<int>(b0) : 0;
    wait_for_stream();
    for (int v = blockIdx.x * blockDim.x + threadIdx.x; v <= V; v += gridDim.x * blockDim.x) {
        const unsigned long long key = static_cast<unsigned long long>(v) << 32;
        int lo = 0, hi = cnt;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (k[mid] < key) lo = mid + 1;
            else hi = mid;
        }
        ls[v] = base + lo;
    }
}

// Sorted keys and start tables of all nseg segments of seg tokens, in two launches.
int sort_labels(const int64_t* labels, int64_t n, int seg, int64_t ignore, int V, bool absolute,
                unsigned long long* keys, int* lstart, cudaStream_t st) {
    const int64_t nseg = ceil_div(n, static_cast<int64_t>(seg));
    if (nseg <= 0) return LIGER_OK;
    const dim3 ranks(static_cast<unsigned>(ceil_div(std::min<int64_t>(n, seg), int64_t{32})), static_cast<unsigned>(nseg));
    if (int rc = launch_early("sort_label_keys", sort_label_keys, ranks, kRankThreads, 0, st, labels, n, seg, ignore,
                              absolute ? 1 : 0, keys))
        return rc;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(V + 1, 256), 2 * sm_count())),
                    static_cast<unsigned>(nseg));
    return launch_early("label_starts", label_starts, grid, 256, 0, st, keys, n, seg, V, absolute ? 1 : 0, lstart);
}

// Merge the per-tile (m, s) of one chunk row into lse and rewrite P in place
// into the softmax part of D, scale * P * exp(m_tile - lse) (the one-hot part
// is applied exactly, in fp32, by the dX / dW GEMM epilogues).  P null: lse
// and the loss term only.
constexpr int kRowThreads = 256;
__global__ void __launch_bounds__(kRowThreads) dlogits_bf16(const int64_t* __restrict__ labels, int64_t ignore,
                                                            const float2* __restrict__ part, int nvt,
                                                            const float* __restrict__ zlab, __nv_bfloat16* P,
                                                            int64_t ldp, int V, float scale,
                                                            const float* __restrict__ scale_dev,
                                                            float* __restrict__ lse, float* __restrict__ lossrow) {
    extern __shared__ float fac[];   // [nvt]
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const int64_t y = labels[row];
    __nv_bfloat16* prow = P + row * ldp;
    const int nv8 = (V + 7) / 8;
    if (y == ignore) {
        if (P != nullptr)
            for (int k = threadIdx.x; k < nv8; k += kRowThreads)
                stg16(prow + static_cast<int64_t>(k) * 8, make_uint4(0, 0, 0, 0));
        if (threadIdx.x == 0) {
            lse[row] = 0.f;
            lossrow[row] = 0.f;
        }
        return;
    }
    const float2* pr = part + row * nvt;
    float m = -INFINITY;
    for (int j = threadIdx.x; j < nvt; j += kRowThreads) m = fmaxf(m, pr[j].x);
    m = block_reduce<kRowThreads>(m, true, red);
    float s = 0.f;
    for (int j = threadIdx.x; j < nvt; j += kRowThreads) {
        const float2 p = pr[j];
        s += p.y * expf(p.x - m);
    }
    s = block_reduce<kRowThreads>(s, false, red);
    const float l = m + logf(s);
    const float sc = scale_dev != nullptr ? *scale_dev : scale;   // scale_dev: formed on the device
    for (int j = threadIdx.x; j < nvt; j += kRowThreads) fac[j] = sc * expf(pr[j].x - l);
    if (threadIdx.x == 0) {
        lse[row] = l;
        lossrow[row] = l - zlab[row];
    }
    if (P == nullptr) return;   // lse and the loss term only
    __syncthreads();
    for (int k = threadIdx.x; k < nv8; k += kRowThreads) {
        const int col = k * 8;
        const float f = fac[col / kVT];
        float v[8];
        unpack(ldg16(prow + col), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= f;
        stg16(prow + col, pack(v));
    }
}

// fp32 path: z row -> lse, loss term, D (fp32, in place).
__global__ void __launch_bounds__(kRowThreads) dlogits_f32(const int64_t* __restrict__ labels, int64_t ignore,
                                                           float* Z, int64_t ldz, int V, float scale,
                                                           const float* __restrict__ scale_dev,
                                                           float* __restrict__ lse, float* __restrict__ lossrow) {
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const int64_t y = labels[row];
    float* z = Z + row * ldz;
    if (y == ignore) {
        for (int v = threadIdx.x; v < V; v += kRowThreads) z[v] = 0.f;
        if (threadIdx.x == 0) {
            lse[row] = 0.f;
            lossrow[row] = 0.f;
        }
        return;
    }
    float m = -INFINITY;
    for (int v = threadIdx.x; v < V; v += kRowThreads) m = fmaxf(m, z[v]);
    m = block_reduce<kRowThreads>(m, true, red);
    float s = 0.f;
    for (int v = threadIdx.x; v < V; v += kRowThreads) s += expf(z[v] - m);
    s = block_reduce<kRowThreads>(s, false, red);
    const float l = m + logf(s);
    const float zy = z[y];
    __syncthreads();   // every thread has read z[y] before it is overwritten
    if (threadIdx.x == 0) {
        lse[row] = l;
        lossrow[row] = l - zy;
    }
    const float sc = scale_dev != nullptr ? *scale_dev : scale;   // scale_dev: formed on the device
    for (int v = threadIdx.x; v < V; v += kRowThreads) z[v] = sc * (expf(z[v] - l) - (v == y ? 1.0f : 0.0f));
}

// ------------------------------------------------ policy loss and label log-probabilities
// The same products with another loss on top (liger_train.h): a token's term depends on its label's
// log-probability only, so D_t = c_t (softmax - onehot) with a scale c_t for each token in place of
// the cross-entropy's one scale.
struct Policy {
    const float *old_logp, *ref_logp, *adv;   // [T] by original token; adv [B] or, per token, [T]
    int adv_per_token, reduction;
    float lo, hi, beta, grad_scale;           // the ratio is held to [lo, hi]
    const int* seq;                           // [T] sequence of a token, -1: not valid
    const int* n_seq;                         // [B] valid tokens of a sequence
    const Hdr* hdr;                           // n_valid
    int64_t B;
    float* coef;                              // [tokens run] the scale c_t, in the order the GEMMs run them
    float *term, *kl, *clip;                  // [T] w l, kl and 1 where clipped, by original token
    float* logp;                              // [T] by original token, or NULL
    float* kpart;                             // dX: the split tiles' sums
    __nv_bfloat16* xpad;                      // [kPadRows][H]
    __nv_bfloat16* xclean;                    // [T][H] for X without the tokens that are not valid (NULL: all are)
    int zero_logp;                            // the row pass writes logp of the tokens that are not valid (all rows are run)
};

// exp(d) - d - 1 without the cancellation of small d: its Taylor series (terms d^2 / 2! to d^9 / 9!,
// the next one below 2^-24 of the sum for |d| < 0.5), else expm1
__device__ __forceinline__ float kl_term(float d) {
    if (fabsf(d) < 0.5f) {
        float s = 1.f / 362880.f;
        s = fmaf(s, d, 1.f / 40320.f);
        s = fmaf(s, d, 1.f / 5040.f);
        s = fmaf(s, d, 1.f / 720.f);
        s = fmaf(s, d, 1.f / 120.f);
        s = fmaf(s, d, 1.f / 24.f);
        s = fmaf(s, d, 1.f / 6.f);
        s = fmaf(s, d, 0.5f);
        return s * d * d;
    }
    return expm1f(d) - d;
}

// The scale c_t of a valid token with label log-probability lp; writes its terms when `write`.
// NaN in old_logp, ref_logp or adv makes them NaN.
__device__ float policy_token(const Policy& p, int64_t t, float lp, bool write) {
    const int b = p.seq[t];
    const float A = p.adv[p.adv_per_token ? t : b];
    const float r = expf(lp - p.old_logp[t]);
    const bool stop = (A > 0.f && r > p.hi) || (A < 0.f && r < p.lo);
    const float ra = A == 0.f ? 0.f : r * A;
    float l = stop ? -(A > 0.f ? p.hi : p.lo) * A : -ra;
    float slope = stop ? 0.f : -ra;
    float kl = 0.f;
    if (p.ref_logp != nullptr) {
        const float d = p.ref_logp[t] - lp;
        kl = kl_term(d);
        if (p.beta != 0.f) {
            l = fmaf(p.beta, kl, l);
            slope = fmaf(-p.beta, expm1f(d), slope);
        }
    }
    float wf = 1.f;
    if (p.reduction == 0) wf = 1.f / static_cast<float>(p.hdr->n_valid);
    if (p.reduction == 2) wf = 1.f / (static_cast<float>(p.B) * static_cast<float>(p.n_seq[b]));
    if (write) {
        p.term[t] = wf * l;
        p.kl[t] = kl;
        p.clip[t] = stop ? 1.f : 0.f;
    }
    return -(slope * wf) * p.grad_scale;
}

// One thread per token: its sequence (binary search in cu_seqlens), whether it is valid, and the label
// that the later kernels index with (ignore_index where it is not valid); counts the valid tokens of
// each sequence and of all.  bad: bit 0 a label outside [0, V), bit 1 bad cu_seqlens (then no token is
// valid, which the first loop of every block finds by itself).  Without cu_seqlens one sequence.
// logp, term, kl, clip become 0 where a token is not valid (logp NaN at a bad label if bad_nan).
__global__ void __launch_bounds__(256) policy_scan(const int64_t* __restrict__ labels, const int32_t* __restrict__ cu,
                                                   int64_t T, int64_t V, int64_t B, int64_t ignore, Hdr* hdr,
                                                   int64_t* __restrict__ lab_out, int* __restrict__ seq, int* n_seq,
                                                   float* logp, float* term, float* kl, float* clip, int bad_nan) {
    __shared__ int cu_bad;
    if (threadIdx.x == 0) cu_bad = 0;
    __syncthreads();
    if (cu != nullptr)
        for (int64_t b = threadIdx.x; b < B; b += blockDim.x)
            if (cu[b] < 0 || cu[b] > cu[b + 1] || cu[b + 1] > T) cu_bad = 1;
    __syncthreads();
    if (cu_bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hdr->bad, 2);
    const int lane = threadIdx.x & 31;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.x; t0 < T; t0 += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = t0 + threadIdx.x;
        int s = -1;
        int64_t y = ignore;
        bool bad = false;
        if (t < T && !cu_bad) {
            y = labels[t];
            s = 0;
            if (cu != nullptr) {   // the last sequence that starts at or before t
                int64_t lo = 0, hi = B;   // cu[lo] <= t < cu[hi] once both hold
                if (t < cu[0] || t >= cu[B]) {
                    s = -1;
                } else {
                    while (hi - lo > 1) {
                        const int64_t mid = (lo + hi) >> 1;
                        if (cu[mid] <= t) lo = mid;
                        else hi = mid;
                    }
                    s = static_cast<int>(lo);
                }
            }
            if (s < 0 || y == ignore) {
                s = -1;
                y = ignore;
            } else if (y < 0 || y >= V) {
                bad = true;
                s = -1;
                y = ignore;
            }
        }
        if (t < T) {
            lab_out[t] = y;
            if (seq != nullptr) seq[t] = s;
            if (s < 0) {
                if (logp != nullptr) logp[t] = bad && bad_nan ? __int_as_float(0x7FC00000) : 0.f;
                if (term != nullptr) term[t] = kl[t] = clip[t] = 0.f;
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&hdr->bad, 1);
        // integer counts: the order of the atomics does not matter
        const unsigned live = __ballot_sync(0xffffffffu, s >= 0);
        if (live == 0) continue;
        if (lane == 0) atomicAdd(&hdr->n_valid, static_cast<unsigned long long>(__popc(live)));
        if (n_seq != nullptr) {
            const unsigned mates = __match_any_sync(0xffffffffu, s);
            if (s >= 0 && lane == __ffs(mates) - 1) atomicAdd(n_seq + s, __popc(mates));
        }
    }
}

// The row pass of the bf16 path: lse from the (m, s) partials, the token's terms and scale, and P
// rewritten in place into the softmax part of D, c_t P exp(m_tile - lse).  P null: lse and logp only.
// idx: original token of a row (null: t0 + row).  run_err: the error word of the GEMMs of this run (with compacted
// tokens a header of its own, which the entry point's takes over at the end).
// HBM-bound, P read and written once.  blockIdx.y takes a run of `piece` 16-byte vectors of the row, each
// repeating the lse from the row's few KB of partials, four vectors a thread in flight: 2741 rows of
// 128256 218 us in runs of 8192, 0.95 of the copy rate (4096: 222, 2048: 253, 237 a whole row at a time with one
// vector in flight); 8 rows 6 us in runs of 2048 (8192: 10).
__global__ void __launch_bounds__(kRowThreads) policy_rows_bf16(const int64_t* labels, int64_t ignore, const float2* part,
                                                                int nvt, const float* zlab, __nv_bfloat16* P, int64_t ldp,
                                                                int V, const Policy pol, const int64_t* idx, int64_t t0,
                                                                float* __restrict__ coef, int piece, const int* run_err) {
    extern __shared__ float fac[];   // a factor for each vocabulary tile of the piece
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    __nv_bfloat16* prow = P + row * ldp;
    const int k0 = blockIdx.y * piece, k1 = min((V + 7) / 8, k0 + piece);
    const bool write = threadIdx.x == 0 && blockIdx.y == 0;   // the token's values
    wait_for_stream();
    if (labels[row] == ignore) {
        if (P != nullptr) {
            for (int k = k0 + threadIdx.x; k < k1; k += kRowThreads)
                stg16(prow + static_cast<int64_t>(k) * 8, make_uint4(0, 0, 0, 0));
            if (write) coef[row] = 0.f;
        }
        if (write && pol.zero_logp && pol.logp != nullptr) pol.logp[t0 + row] = 0.f;
        return;
    }
    const float2* pr = part + row * nvt;
    float m = -INFINITY;
    for (int j = threadIdx.x; j < nvt; j += kRowThreads) m = fmaxf(m, pr[j].x);
    m = block_reduce<kRowThreads>(m, true, red);
    float s = 0.f;
    for (int j = threadIdx.x; j < nvt; j += kRowThreads) {
        const float2 p = pr[j];
        s += p.y * expf(p.x - m);
    }
    s = block_reduce<kRowThreads>(s, false, red);
    const float l = m + logf(s);
    float lp = zlab[row] - l;
    if (*run_err != 0) lp = __int_as_float(0x7FC00000);   // the GEMM that made the partials gave up on a bounded wait
    const int64_t t = idx != nullptr ? idx[row] : t0 + row;
    if (pol.logp != nullptr && write) pol.logp[t] = lp;
    if (P == nullptr) return;
    const float sc = policy_token(pol, t, lp, write);
    if (write) coef[row] = sc;
    const int f0 = k0 * 8 / kVT, f1 = (k1 * 8 - 1) / kVT;   // the piece's vocabulary tiles
    for (int j = f0 + threadIdx.x; j <= f1; j += kRowThreads) fac[j - f0] = sc * expf(pr[j].x - l);
    __syncthreads();
    constexpr int U = 4;
    for (int kk = k0 + threadIdx.x; kk < k1; kk += U * kRowThreads) {
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (kk + u * kRowThreads < k1) w[u] = ldg16_cs(prow + static_cast<int64_t>(kk + u * kRowThreads) * 8);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = kk + u * kRowThreads;
            if (k >= k1) continue;
            const float f = fac[k * 8 / kVT - f0];
            float v[8];
            unpack(w[u], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= f;
            stg16(prow + static_cast<int64_t>(k) * 8, pack(v));
        }
    }
}

// fp32 path: z row -> lse, the token's terms and scale, D in place (log-probability only: z is left)
__global__ void __launch_bounds__(kRowThreads) policy_rows_f32(const int64_t* labels, int64_t ignore, float* Z, int64_t ldz,
                                                               int V, int with_d, const Policy pol, const int64_t* idx,
                                                               int64_t t0) {
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    wait_for_stream();
    const int64_t y = labels[row];
    float* z = Z + row * ldz;
    if (y == ignore) {
        if (with_d)
            for (int v = threadIdx.x; v < V; v += kRowThreads) z[v] = 0.f;
        if (threadIdx.x == 0 && pol.zero_logp && pol.logp != nullptr) pol.logp[t0 + row] = 0.f;
        return;
    }
    float m = -INFINITY;
    for (int v = threadIdx.x; v < V; v += kRowThreads) m = fmaxf(m, z[v]);
    m = block_reduce<kRowThreads>(m, true, red);
    float s = 0.f;
    for (int v = threadIdx.x; v < V; v += kRowThreads) s += expf(z[v] - m);
    s = block_reduce<kRowThreads>(s, false, red);
    const float l = m + logf(s);
    const float lp = (z[y] - m) - logf(s);
    const int64_t t = idx != nullptr ? idx[row] : t0 + row;
    if (pol.logp != nullptr && threadIdx.x == 0) pol.logp[t] = lp;
    if (!with_d) return;
    __syncthreads();   // every thread has read z[y] before it is overwritten
    const float sc = policy_token(pol, t, lp, threadIdx.x == 0);
    for (int v = threadIdx.x; v < V; v += kRowThreads) z[v] = sc * (expf(z[v] - l) - (v == y ? 1.0f : 0.0f));
}

// loss and stats: the tokens' terms added in a fixed order; NaN if a kernel recorded an error or the
// scan found a bad label or bad sequences.  A warp adds its tokens in fp32 with the rounding errors
// carried along (fp64 adds run at a small fraction of the fp32 rate: 16 us for 4096 tokens in fp64), the
// warps' sums are joined in fp64.
__device__ __forceinline__ void add_with_error(float v, float& sum, float& err) {
    const float t = sum + v, b = t - sum;
    err += (sum - (t - b)) + (v - b);
    sum = t;
}
constexpr int kFinalThreads = 1024;   // 256 are launched for few tokens
__global__ void __launch_bounds__(kFinalThreads) policy_final(const float* term, const float* kl, const float* clip, int64_t T,
                                                              const Hdr* hdr, float* loss, float* stats) {
    __shared__ double red[3][32];
    const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float s[3] = {0.f, 0.f, 0.f}, e[3] = {0.f, 0.f, 0.f};
    wait_for_stream();
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < T; t += nt) {
        add_with_error(term[t], s[0], e[0]);
        add_with_error(kl[t], s[1], e[1]);
        add_with_error(clip[t], s[2], e[2]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float e2 = __shfl_xor_sync(0xffffffffu, e[i], o);
            add_with_error(__shfl_xor_sync(0xffffffffu, s[i], o), s[i], e[i]);
            e[i] += e2;
        }
        // an infinity's error term is NaN: the plain sum stands for it
        if (lane == 0)
            red[i][warp] = isfinite(s[i]) ? static_cast<double>(s[i]) + static_cast<double>(e[i]) : static_cast<double>(s[i]);
    }
    __syncthreads();
    if (warp < 3) {
        const int i = warp;
        double tot = lane < nt / 32 ? red[i][lane] : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
        const double n = static_cast<double>(hdr->n_valid);
        float r = static_cast<float>(i == 0 ? tot : n > 0.0 ? tot / n : 0.0);
        if (hdr->err != 0 || hdr->bad != 0) r = __int_as_float(0x7fc00000);
        if (lane != 0) return;
        if (i == 0) *loss = r;
        else if (stats != nullptr) stats[i - 1] = r;
    }
}

// loss = sum of the row terms (fixed order, fp64) / n_valid; NaN if a
// tensor-core kernel recorded an error.
// dev_denom 0: divide by denom; 1 (mean) / 2 (sum): the denominator from the device-side
// count, and NaN when a label was bad
__global__ void __launch_bounds__(1024) loss_final(const float* __restrict__ lossrow, int64_t T, double denom,
                                                   const Hdr* hdr, float* loss, int dev_denom) {
    __shared__ double red[32];
    double s = 0.0;
    for (int64_t t = threadIdx.x; t < T; t += 1024) s += static_cast<double>(lossrow[t]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double tot = 0.0;
        for (int i = 0; i < 32; ++i) tot += red[i];
        if (dev_denom != 0) denom = dev_denom == 1 ? static_cast<double>(hdr->n_valid) : 1.0;
        float r = denom > 0.0 ? static_cast<float>(tot / denom) : 0.0f;
        if (hdr->err != 0 || (dev_denom != 0 && hdr->bad != 0)) r = __int_as_float(0x7fc00000);
        *loss = r;
    }
}

// Generic SIMT GEMM, C[m, n] = sum_k A(m, k) B(k, n), fp32 accumulation.
// A(m, k) = A[m*sam + k*sak], B(k, n) = B[k*sbk + n*sbn].
//  mode 0: outf[m, n]  = acc          mode 2: outf[m, n] += acc
//  mode 1: outT[m, n]  = acc          mode 3: outT[m, n]  = acc + outf[m, n]
// mode 1 writes +0 on rows whose label is ignore_index (labels may be NULL).
// SBT x SBT output tiles (64, or 32 when 64-wide tiles would leave SMs idle), 256
// threads each holding (SBT/16)^2 of them; k steps of SKT (16, or 64 with the small
// tiles: fewer load-then-synchronise rounds, more loads in flight in each).
constexpr int SB = 64, SK = 16;
template <typename TA, typename TB, typename TO, int MODE, int SBT, int SKT>
__global__ void __launch_bounds__(256) simt_gemm(int M, int N, int K, const TA* __restrict__ A, int64_t sam,
                                                 int64_t sak, const TB* __restrict__ B, int64_t sbk, int64_t sbn,
                                                 float* outf, TO* outT, int64_t ldo, const int64_t* __restrict__ labels,
                                                 int64_t ignore) {
    constexpr int RT = SBT / 16;
    __shared__ float As[SKT][SBT + 1], Bs[SKT][SBT + 1];
    const int m0 = blockIdx.y * SBT, n0 = blockIdx.x * SBT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[RT][RT] = {};
    const bool ak = sak == 1, bn = sbn == 1;
    for (int k0 = 0; k0 < K; k0 += SKT) {
        // consecutive threads take consecutive elements of each operand's contiguous
        // dimension (k when sak == 1, else m; n when sbn == 1, else k), so the loads coalesce
        // whichever operand is transposed
        for (int i = threadIdx.x; i < SBT * SKT; i += 256) {
            const int mm = ak ? i / SKT : i % SBT, kk = ak ? i % SKT : i / SBT;
            const int gm = m0 + mm, gk = k0 + kk;
            As[kk][mm] = (gm < M && gk < K) ? ldf(A + gm * sam + gk * sak) : 0.f;
            const int nn = bn ? i % SBT : i / SKT, kb = bn ? i / SBT : i % SKT;
            const int gn = n0 + nn, gk2 = k0 + kb;
            Bs[kb][nn] = (gn < N && gk2 < K) ? ldf(B + gk2 * sbk + gn * sbn) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < SKT; ++kk) {
            float a[RT], b[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) a[i] = As[kk][ty * RT + i], b[i] = Bs[kk][tx * RT + i];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int gm = m0 + ty * RT + i;
        if (gm >= M) continue;
        const bool zero = MODE == 1 && labels != nullptr && labels[gm] == ignore;
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int gn = n0 + tx * RT + j;
            if (gn >= N) continue;
            const int64_t o = static_cast<int64_t>(gm) * ldo + gn;
            if (MODE == 0) outf[o] = acc[i][j];
            else if (MODE == 1) stf(outT + o, zero ? 0.f : acc[i][j]);
            else if (MODE == 2) outf[o] += acc[i][j];
            else stf(outT + o, acc[i][j] + outf[o]);
        }
    }
}

template <typename TA, typename TB, typename TO, int MODE>
int simt(int M, int N, int K, const TA* A, int64_t sam, int64_t sak, const TB* B, int64_t sbk, int64_t sbn,
         float* outf, TO* outT, int64_t ldo, const int64_t* labels, int64_t ignore, cudaStream_t st) {
    if (M == 0 || N == 0) return LIGER_OK;
    const int64_t tiles64 = ceil_div(N, SB) * ceil_div(M, SB);
    if (tiles64 < sm_count()) {   // too few 64-wide tiles to fill the GPU: 32-wide ones
        dim3 grid(static_cast<unsigned>(ceil_div(N, SB / 2)), static_cast<unsigned>(ceil_div(M, SB / 2)));
        simt_gemm<TA, TB, TO, MODE, SB / 2, 4 * SK><<<grid, 256, 0, st>>>(M, N, K, A, sam, sak, B, sbk, sbn, outf, outT, ldo,
                                                                  labels, ignore);
        return check_launch("simt_gemm");
    }
    dim3 grid(static_cast<unsigned>(ceil_div(N, SB)), static_cast<unsigned>(ceil_div(M, SB)));
    if (grid.y > 65535) return fail(LIGER_ERR_SHAPE, "linear_ce: SIMT grid too large");
    simt_gemm<TA, TB, TO, MODE, SB, SK><<<grid, 256, 0, st>>>(M, N, K, A, sam, sak, B, sbk, sbn, outf, outT, ldo, labels,
                                                          ignore);
    return check_launch("simt_gemm");
}

// ----------------------------------------------------------- orchestration
// Waits for the label scan and says whether the call goes on (LIGER_OK), ends without work (kNothing) or fails.
// A reference to the caller's lambda: nothing is allocated, and nothing can throw across the C entry.
struct Check {
    int (*call)(void*);
    void* self;
    int operator()() const { return call(self); }
};
template <typename F>
Check check_of(F& f) {
    return Check{[](void* p) { return (*static_cast<F*>(p))(); }, &f};
}
constexpr int kNothing = 1;

struct Args {
    const void* X;
    const void* W;
    const int64_t* labels;
    int64_t T, H, V, ignore;
    int reduction;
    float grad_scale;
    float* loss;
    void* dX;
    void* dW;
    uint8_t* ws;
    int dtype;
    cudaStream_t st;
    const float* scale_dev;   // non-null: the gradient scale is read from the device (no host wait)
    const Policy* pol;        // non-null: the policy loss in place of the cross-entropy
    const int64_t* idx;       // policy loss: original token of a row (null: the row itself)
    const Check* check;       // policy loss: non-null: called once before anything but the workspace is written
};

template <typename TI>
int run_simt(const Args& a, const Layout& L, float scale) {
    const TI* X = static_cast<const TI*>(a.X);
    const TI* W = static_cast<const TI*>(a.W);
    TI* dX = static_cast<TI*>(a.dX);
    TI* dW = static_cast<TI*>(a.dW);
    float* lse = reinterpret_cast<float*>(a.ws + L.lse);
    float* lossrow = reinterpret_cast<float*>(a.ws + L.lossrow);
    float* Z = reinterpret_cast<float*>(a.ws + L.scr);
    float* acc = reinterpret_cast<float*>(a.ws + L.acc);
    const bool f32 = a.dtype == LIGER_F32;
    const int H = static_cast<int>(a.H), V = static_cast<int>(a.V);
    int rc;
    for (int64_t c = 0; c < L.nchunks; ++c) {
        const int64_t t0 = c * L.C;
        const int cl = static_cast<int>(std::min(L.C, a.T - t0));
        const bool first = c == 0, last = c == L.nchunks - 1;
        if ((rc = simt<TI, TI, TI, 0>(cl, V, H, X + t0 * H, H, 1, W, 1, H, Z, (TI*)nullptr, V, nullptr, 0, a.st)))
            return rc;
        dlogits_f32<<<cl, kRowThreads, 0, a.st>>>(a.labels + t0, a.ignore, Z, V, V, scale, a.scale_dev, lse + t0,
                                                  lossrow + t0);
        if ((rc = check_launch("dlogits_f32"))) return rc;
        if (dX && (rc = simt<float, TI, TI, 1>(cl, H, V, Z, V, 1, W, H, 1, nullptr, dX + t0 * H, H, a.labels + t0,
                                               a.ignore, a.st)))
            return rc;
        if (dW) {
            const TI* Xc = X + t0 * H;
            if (f32) {
                float* dWf = reinterpret_cast<float*>(dW);
                rc = first ? simt<float, TI, float, 0>(V, H, cl, Z, 1, V, Xc, H, 1, dWf, nullptr, H, nullptr, 0, a.st)
                           : simt<float, TI, float, 2>(V, H, cl, Z, 1, V, Xc, H, 1, dWf, nullptr, H, nullptr, 0, a.st);
            } else if (first && last) {
                rc = simt<float, TI, TI, 1>(V, H, cl, Z, 1, V, Xc, H, 1, nullptr, dW, H, nullptr, 0, a.st);
            } else if (first) {
                rc = simt<float, TI, TI, 0>(V, H, cl, Z, 1, V, Xc, H, 1, acc, nullptr, H, nullptr, 0, a.st);
            } else if (!last) {
                rc = simt<float, TI, TI, 2>(V, H, cl, Z, 1, V, Xc, H, 1, acc, nullptr, H, nullptr, 0, a.st);
            } else {
                rc = simt<float, TI, TI, 3>(V, H, cl, Z, 1, V, Xc, H, 1, acc, dW, H, nullptr, 0, a.st);
            }
            if (rc) return rc;
        }
    }
    return LIGER_OK;
}

// A GEMM over fewer rows of X than this is given them among rows of zeros: every CTA reads the same few
// lines of X at the same time, and over one to fifteen rows they sit in so few L2 slices that this bounds
// it (logits at 4096 x 128256: 1 token 305 us, 9 206, 10 264, 16 181).
constexpr int64_t kPadRows = 16;
int pad_rows(const __nv_bfloat16* X, int64_t n, int64_t H, __nv_bfloat16* pad, cudaStream_t st) {
    const size_t row = static_cast<size_t>(H) * 2;
    if (cudaMemsetAsync(pad + n * H, 0, (kPadRows - n) * row, st) != cudaSuccess ||
        cudaMemcpyAsync(pad, X, n * row, cudaMemcpyDeviceToDevice, st) != cudaSuccess)
        return check_launch("rows of X");
    return LIGER_OK;
}

// Z = X_c W^T for the cl rows at Xc with the logits epilogue e (its labels, zlab,
// part and p_out set for row 0 of the chunk), in launches over rows_in_l2 rows: each
// launch sweeps the whole vocabulary over its rows of X (an 8192-row chunk at hidden
// 4096 takes two launches, reading W twice but each X row once)
// Rows of X past cl up to x_rows (they are there, and are read, but give no output).
int launch_logits(const __nv_bfloat16* Xc, int cl, int H, int V, const CUtensorMap& mW_k, const tc::EpiParams& e,
                  int64_t ldp, int64_t nvt, cudaStream_t st, int64_t x_rows = 0) {
    using namespace tc;
    const int64_t sub = rows_in_l2(H, cl);
    for (int64_t s0 = 0; s0 < cl; s0 += sub) {
        const int sl = static_cast<int>(std::min<int64_t>(sub, cl - s0));
        CUtensorMap mX;
        // A (K-major)
        if (int rc = make_map(&mX, Xc + s0 * H, H, std::max<int64_t>(sl, x_rows), H, BK, BM)) return rc;
        EpiParams f = e;
        f.M = sl;
        f.labels = e.labels + s0;
        f.zlab = e.zlab + s0;
        f.part = e.part + s0 * nvt;
        if (e.p_out != nullptr) f.p_out = e.p_out + s0 * ldp;
        if (int rc = launch_gemm<0, 0, EPI_LOGITS, 1>(mX, mW_k, sl, V, H, f, st)) return rc;
    }
    return LIGER_OK;
}

// ---- dX of the policy loss
// K is the whole vocabulary and the tiles are few (256 tokens at hidden 4096: 16 tiles for 76 CTA
// pairs, 2000 k-blocks each), so the last, partly filled round of tiles, which may be the only one, is
// split along K over the idle pairs, each item leaving fp32 sums that split_join adds up.  Above
// kDxSlabRows vocabulary rows in several rounds the launches go over slabs as for the cross-entropy.
// At hidden 4096, vocabulary 128256, with the split and without: 256 tokens 211 and 619 us, 2741 tokens
// 1618 and 1881 us.
constexpr int kPairs = 80;               // most CTA pairs planned for
constexpr int kDxMinBlocks = 16;         // fewest k-blocks of an item
constexpr int64_t kDxMaxSlabs = 4;       // slabs whose split sums the workspace holds
constexpr int64_t kTileFloats = 256 * 256;

struct DxPlan {
    int64_t slab;     // vocabulary rows per launch
    int slabs, full, rem, splits;   // rem tiles from `full` on are split into `splits` (0: none)
};

DxPlan dx_plan(int64_t rows, int64_t H, int64_t V) {
    DxPlan p{};
    const int64_t pairs = std::min<int64_t>(std::max(1, sm_count() / 2), kPairs);
    const int64_t tiles = ceil_div(rows, int64_t{256}) * ceil_div(H, int64_t{256});
    p.slab = tiles <= pairs ? V : dx_slab(V);
    p.slabs = static_cast<int>(ceil_div(V, p.slab));
    p.rem = static_cast<int>(tiles % pairs);
    p.full = static_cast<int>(tiles) - p.rem;
    if (p.rem > 0 && p.slabs <= kDxMaxSlabs)
        p.splits = static_cast<int>(std::min<int64_t>(pairs / p.rem, ceil_div(p.slab, int64_t{tc::BK}) / kDxMinBlocks));
    if (p.splits < 2) p.splits = 0;
    return p;
}

// dX of the cl rows of the chunk at t0: D = P [cl, V], e as set up for the chunk
int policy_dx(const Args& a, const Layout& L, const __nv_bfloat16* P, const tc::EpiParams& e, int64_t t0, int cl) {
    using namespace tc;
    const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.W);
    const int H = static_cast<int>(a.H);
    const int64_t V = a.V;
    const DxPlan p = dx_plan(cl, H, V);
    float* dxacc = reinterpret_cast<float*>(a.ws + L.dxacc);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dX) + t0 * H;
    const int items = p.rem * p.splits;
    int rc;
    for (int64_t v0 = 0; v0 < V; v0 += p.slab) {
        const int vl = static_cast<int>(std::min<int64_t>(p.slab, V - v0));
        const bool first = v0 == 0, last = v0 + vl >= V;
        CUtensorMap mD, mW;
        if ((rc = make_map(&mD, P + v0, vl, cl, L.ldp, BK, BM))) return rc;        // A: D[:, slab] (K-major)
        if ((rc = make_map(&mW, W + v0 * H, H, vl, H, MN_BOX, BK))) return rc;     // B: W[slab, :] (MN-major)
        EpiParams d = e;
        d.p_out = nullptr;
        d.M = cl;
        d.N = H;
        d.raster = RASTER_N_GROUPS;
        d.hint_a = HINT_NORMAL;
        d.hint_b = HINT_NORMAL;
        d.acc = dxacc;
        d.lda = H;
        d.acc_read = first ? 0 : 1;
        d.acc_write = last ? 0 : 1;
        d.out_write = last ? 1 : 0;
        d.out = out;
        d.ldo = H;
        d.keys = nullptr;
        d.corr_src = last ? W : nullptr;
        d.ld_corr = H;
        if (p.splits > 0) {
            d.full_tiles = p.full;
            d.ksplits = p.splits;
            d.kpart_rows = TileCfg<1>::TM;
            d.kpart = a.pol->kpart + (v0 / p.slab) * items * kTileFloats;
        }
        if ((rc = launch_gemm<0, 1, EPI_ACCUM, 1, MODE_TOKENS>(mD, mW, cl, H, vl, d, a.st))) return rc;
    }
    if (p.splits == 0) return LIGER_OK;
    const SplitJoin j{a.pol->kpart, p.rem, p.splits, p.slabs, p.full, TileCfg<1>::TM, static_cast<int>(ceil_div(cl, 256)),
                      static_cast<int>(ceil_div(H, 256)), a.labels + t0, a.ignore, e.tok_scale, W, out, cl, H};
    return launch_early("linear_policy dX", split_join, dim3(static_cast<unsigned>(p.rem), TileCfg<1>::TM / 8), 256, 0, a.st, j);
}

int run_tc(const Args& a, const Layout& L, float scale) {
    using namespace tc;
    const __nv_bfloat16* X = static_cast<const __nv_bfloat16*>(a.X);
    const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.W);
    float* lse = reinterpret_cast<float*>(a.ws + L.lse);
    float* lossrow = reinterpret_cast<float*>(a.ws + L.lossrow);
    float* zlab = reinterpret_cast<float*>(a.ws + L.zlab);
    Hdr* hdr = reinterpret_cast<Hdr*>(a.ws + L.hdr);
    float2* part = reinterpret_cast<float2*>(a.ws + L.part);
    __nv_bfloat16* P = reinterpret_cast<__nv_bfloat16*>(a.ws + L.scr);
    float* acc = reinterpret_cast<float*>(a.ws + L.acc);
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(a.ws + L.keys);
    int* lstart = reinterpret_cast<int*>(a.ws + L.lstart);
    const int H = static_cast<int>(a.H), V = static_cast<int>(a.V);
    int rc;
    if (a.pol != nullptr && a.idx == nullptr && a.dW != nullptr && a.pol->xclean != nullptr) {
        // dW = D^T X sums over all tokens: a zero of D times whatever stands in X at a token that is
        // not valid is NaN if that is no finite number (4096 tokens of 4096: 10 us)
        if ((rc = launch_early("masked_rows", masked_rows, dim3(static_cast<unsigned>(std::min<int64_t>(a.T, 8 * sm_count()))),
                               256, 0, a.st, reinterpret_cast<const uint4*>(X), a.labels, a.ignore, a.T, a.H * 2 / 16,
                               reinterpret_cast<uint4*>(a.pol->xclean))))
            return rc;
        X = a.pol->xclean;
    }
    CUtensorMap mW_k, mW_mn;
    if ((rc = make_map(&mW_k, W, H, V, H, BK, B_BOX_ROWS))) return rc;          // B of Z = X W^T  (K-major)
    if ((rc = make_map(&mW_mn, W, H, V, H, MN_BOX, BK))) return rc;     // B of dX = D W   (MN-major)
    const size_t fac_smem = sizeof(float) * static_cast<size_t>(L.nvt);
    // label keys: one segment per chunk (indices relative to the chunk) up to 8192 rows, else
    // 8192-token segments with absolute indices, several per chunk
    const bool rel = L.seg == L.C;
    if (a.dW && (rc = sort_labels(a.labels, a.T, L.seg, a.ignore, V, !rel, keys, lstart, a.st))) return rc;
    for (int64_t c = 0; c < L.nchunks; ++c) {
        const int64_t t0 = c * L.C;
        const int cl = static_cast<int>(std::min(L.C, a.T - t0));
        const bool first = c == 0, last = c == L.nchunks - 1;
        const __nv_bfloat16* Xc = X + t0 * H;
        CUtensorMap mX_mn, mD_k, mD_mn;
        if ((rc = make_map(&mX_mn, Xc, H, cl, H, MN_BOX, BK))) return rc;  // B of dW (MN-major)
        if ((rc = make_map(&mD_k, P, V, cl, L.ldp, BK, BM))) return rc;  // A of dX (K-major)
        if ((rc = make_map(&mD_mn, P, V, cl, L.ldp, MN_BOX, BK))) return rc;  // A of dW (MN-major)

        EpiParams e{};
        e.err = &hdr->err;
        e.early = a.pol != nullptr ? 1 : 0;
        e.ignore_index = a.ignore;
        e.labels = a.labels + t0;
        // 1. logits -> P, (m, s) partials, z at label
        e.M = cl;
        e.N = V;
        e.raster = RASTER_M_FASTEST;
        e.hint_a = HINT_EVICT_LAST;    // X_c: reused by every vocab tile, keep in L2
        e.hint_b = HINT_EVICT_FIRST;   // W: streamed once per chunk
        e.p_out = P;
        e.ldp = L.ldp;
        e.part = part;
        e.nvt = static_cast<int>(L.nvt);
        e.zlab = zlab + t0;
        if (a.pol != nullptr && cl < kPadRows) {
            if ((rc = pad_rows(Xc, cl, H, a.pol->xpad, a.st))) return rc;
            rc = launch_logits(a.pol->xpad, cl, H, V, mW_k, e, L.ldp, L.nvt, a.st, kPadRows);
        } else {
            rc = launch_logits(Xc, cl, H, V, mW_k, e, L.ldp, L.nvt, a.st);
        }
        if (rc) return rc;
        if (a.check != nullptr && first && (rc = (*a.check)())) return rc;
        // 2. lse, loss terms, P -> D in place (policy loss: long runs of a row where they fill the GPU)
        const int piece = cl * ceil_div(V, 8 * 8192) >= 8 * sm_count() ? 8192 : 2048;
        if (a.pol != nullptr) {
            const dim3 grid(cl, static_cast<unsigned>(ceil_div(ceil_div(V, 8), piece)));
            const size_t piece_smem = sizeof(float) * static_cast<size_t>(piece * 8 / kVT + 1);
            rc = launch_early("linear_policy rows", policy_rows_bf16, grid, kRowThreads, piece_smem, a.st, a.labels + t0, a.ignore,
                              part, static_cast<int>(L.nvt), zlab + t0, P, L.ldp, V, *a.pol,
                              a.idx != nullptr ? a.idx + t0 : nullptr, t0, a.pol->coef + t0, piece, &hdr->err);
        } else {
            dlogits_bf16<<<cl, kRowThreads, fac_smem, a.st>>>(a.labels + t0, a.ignore, part, static_cast<int>(L.nvt),
                                                              zlab + t0, P, L.ldp, V, scale, a.scale_dev, lse + t0,
                                                              lossrow + t0);
            rc = check_launch("dlogits_bf16");
        }
        if (rc) return rc;
        if (a.pol != nullptr) e.tok_scale = a.pol->coef + t0;
        // 3. dX_c = D W, minus scale * W[label] in fp32
        if (a.dX && a.pol != nullptr) {
            if ((rc = policy_dx(a, L, P, e, t0, cl))) return rc;
        } else if (a.dX && dx_slab(V) < V) {
            // over vocabulary slabs, summed in fp32; the last slab subtracts scale * W[label]
            // and writes dX in bf16
            float* dxacc = reinterpret_cast<float*>(a.ws + L.dxacc);
            const int64_t slab = dx_slab(V);
            for (int64_t v0 = 0; v0 < V; v0 += slab) {
                const int vl = static_cast<int>(std::min<int64_t>(slab, V - v0));
                const bool s_first = v0 == 0, s_last = v0 + vl >= V;
                CUtensorMap mDs_k, mWs_mn;
                if ((rc = make_map(&mDs_k, P + v0, vl, cl, L.ldp, BK, BM))) return rc;     // A: D[:, slab] (K-major)
                if ((rc = make_map(&mWs_mn, W + v0 * H, H, vl, H, MN_BOX, BK))) return rc;  // B: W[slab, :] (MN-major)
                EpiParams d = e;
                d.p_out = nullptr;
                d.M = cl;
                d.N = H;
                d.raster = RASTER_N_GROUPS;
                d.hint_a = HINT_NORMAL;
                d.hint_b = HINT_NORMAL;
                d.acc = dxacc;
                d.lda = H;
                d.acc_read = s_first ? 0 : 1;
                d.acc_write = s_last ? 0 : 1;
                d.out_write = s_last ? 1 : 0;
                d.out = static_cast<__nv_bfloat16*>(a.dX) + t0 * H;
                d.ldo = H;
                d.keys = nullptr;
                d.corr_src = s_last ? W : nullptr;
                d.ld_corr = H;
                d.corr_scale = scale;
                d.scale_ptr = a.scale_dev;
                if ((rc = launch_gemm<0, 1, EPI_ACCUM, 1>(mDs_k, mWs_mn, cl, H, vl, d, a.st))) return rc;
            }
        } else if (a.dX) {
            EpiParams d = e;
            d.M = cl;
            d.N = H;
            d.out = static_cast<__nv_bfloat16*>(a.dX) + t0 * H;
            d.ldo = H;
            d.raster = RASTER_N_GROUPS;
            d.hint_a = HINT_NORMAL;        // D and W: reused within a wave of tiles
            d.hint_b = HINT_NORMAL;
            d.corr_src = W;
            d.ld_corr = H;
            d.corr_scale = scale;
            d.scale_ptr = a.scale_dev;
            if ((rc = launch_gemm<0, 1, EPI_STORE, 1>(mD_k, mW_mn, cl, H, V, d, a.st))) return rc;
        }
        // 4. dW (+)= D^T X_c, minus scale * X_t in fp32 for each token t labelled with the row
        if (a.dW) {
            EpiParams d = e;
            d.ld_corr = H;
            d.corr_scale = scale;
            d.scale_ptr = a.scale_dev;
            d.nkeys = cl;
            if (rel) {
                d.corr_src = Xc;
                d.keys = keys + t0;               // this chunk's keys (token indices relative to the chunk)
                d.lstart = lstart + c * (V + 1);
            } else {
                d.corr_src = X;                   // absolute token indices
                if (a.pol != nullptr) d.tok_scale = a.pol->coef;
                d.keys = keys;
                d.lstart = lstart + (t0 / L.seg) * (V + 1);
                d.nseg = static_cast<int>(ceil_div(static_cast<int64_t>(cl), static_cast<int64_t>(L.seg)));
                d.lstride = V + 1;
            }
            d.M = V;
            d.N = H;
            // n fastest touches all of X_c in every wave: fine while X_c stays in L2 (up to
            // 32 MiB), above that groups of 8 column blocks of it do (at the price of reading
            // each D block once per group)
            d.raster = static_cast<int64_t>(cl) * H * 2 > (int64_t{32} << 20) ? RASTER_N_GROUPS : RASTER_N_FASTEST;
            d.hint_a = HINT_NORMAL;        // D^T (evict-first measured ~1 % slower with CTA-pair tiles)
            d.hint_b = HINT_EVICT_LAST;    // X_c: reused by every vocab row block, keep in L2
            d.labels = nullptr;
            d.acc = acc;
            d.lda = H;
            d.out = static_cast<__nv_bfloat16*>(a.dW);
            d.ldo = H;
            d.acc_read = first ? 0 : 1;
            d.acc_write = last ? 0 : 1;
            d.out_write = last ? 1 : 0;
            rc = a.pol != nullptr ? launch_gemm<1, 1, EPI_ACCUM, 1, MODE_TOKENS>(mD_mn, mX_mn, V, H, cl, d, a.st)
                                  : launch_gemm<1, 1, EPI_ACCUM, 1>(mD_mn, mX_mn, V, H, cl, d, a.st);
            if (rc) return rc;
        }
    }
    return LIGER_OK;
}

// Where a layout keeps its per-token lse and loss terms and its header.
struct RowVals {
    size_t lse, lossrow, hdr;
};

// A variant's GEMMs on the tokens that are not ignored only (n_valid of T, known on
// the host from the label scan): an ignored token has D = 0, so it adds nothing to
// dW and its dX row, lse and loss term are 0; its logits, which the GEMMs would
// otherwise compute, are not needed.  The tokens are compacted in order (their X
// rows and labels gathered), run_core runs the variant on them in the region C.core
// (its own layout for n_valid tokens, whose lse, loss terms and header sit at cv),
// and dX, lse and the loss terms are put back in place (tv: the full layout's).
template <typename RunCore>
int run_compacted(const Args& a, int64_t n_valid, const CompactLayout& C, const RowVals& tv, const RowVals& cv,
                  RunCore run_core) {
    uint8_t* w8 = a.ws;
    int* cnt = reinterpret_cast<int*>(w8 + C.cnt);
    int64_t* idx = reinterpret_cast<int64_t*>(w8 + C.idx);
    int* inv = reinterpret_cast<int*>(w8 + C.inv);
    int64_t* labc = reinterpret_cast<int64_t*>(w8 + C.labc);
    const int64_t nb = ceil_div(a.T, static_cast<int64_t>(kCompactBlock));
    compact_count<<<static_cast<unsigned>(nb), kCompactBlock, 0, a.st>>>(a.labels, a.T, a.ignore, cnt);
    compact_scan<<<1, 1024, 0, a.st>>>(cnt, nb);
    compact_index<<<static_cast<unsigned>(nb), kCompactBlock, 0, a.st>>>(a.labels, a.T, a.ignore, cnt, idx, inv, labc);
    const int64_t hv = a.H * 2 / 16;   // 16-byte vectors per bf16 row (H is a multiple of 8 on this path)
    const int rgrid = static_cast<int>(std::min<int64_t>(std::max<int64_t>(n_valid, 1), 8 * sm_count()));
    gather_rows<<<rgrid, 256, 0, a.st>>>(static_cast<const uint4*>(a.X), idx, n_valid, hv,
                                         reinterpret_cast<uint4*>(w8 + C.xc));
    if (int rc = check_launch("linear_ce compaction")) return rc;
    Hdr* hc = reinterpret_cast<Hdr*>(w8 + C.core + cv.hdr);
    if (cudaMemsetAsync(hc, 0, sizeof(Hdr), a.st) != cudaSuccess) return check_launch("linear_ce memset");
    Args b = a;
    b.X = w8 + C.xc;
    b.labels = labc;
    b.idx = idx;
    b.T = n_valid;
    b.dX = a.dX ? static_cast<void*>(w8 + C.dxc) : nullptr;
    b.ws = w8 + C.core;
    if (int rc = run_core(b)) return rc;
    if (a.dX) {
        const int tgrid = static_cast<int>(std::min<int64_t>(a.T, 8 * sm_count()));
        scatter_rows<<<tgrid, 256, 0, a.st>>>(reinterpret_cast<const uint4*>(w8 + C.dxc), inv, a.T, hv,
                                              static_cast<uint4*>(a.dX));
    }
    if (a.pol != nullptr) {   // its row pass wrote the tokens' values in place already
        take_err<<<1, 1, 0, a.st>>>(&hc->err, &reinterpret_cast<Hdr*>(w8 + tv.hdr)->err);
        return check_launch("linear_policy scatter");
    }
    const int vgrid = static_cast<int>(std::min<int64_t>(ceil_div(a.T, int64_t{256}), 4 * sm_count()));
    scatter_rowvals<<<vgrid, 256, 0, a.st>>>(reinterpret_cast<const float*>(w8 + C.core + cv.lse),
                                             reinterpret_cast<const float*>(w8 + C.core + cv.lossrow), inv, a.T,
                                             reinterpret_cast<float*>(w8 + tv.lse),
                                             reinterpret_cast<float*>(w8 + tv.lossrow), &hc->err,
                                             &reinterpret_cast<Hdr*>(w8 + tv.hdr)->err);
    return check_launch("linear_ce scatter");
}

// The token-chunked path on the tokens that are not ignored only.
int run_tc_compact(const Args& a, int64_t n_valid, int64_t chunk, float scale) {
    const Layout Lt = layout(a.T, a.H, a.V, chunk, a.dtype);   // the documented lse / loss_row of every token
    const Layout Lc = layout(n_valid, a.H, a.V, chunk, a.dtype);
    if (Lc.total > Lt.total) return run_tc(a, Lt, scale);   // the region holds any layout of fewer tokens
    return run_compacted(a, n_valid, compact_layout(a.T, a.H, a.V, chunk, a.dtype), RowVals{Lt.lse, Lt.lossrow, Lt.hdr},
                         RowVals{Lc.lse, Lc.lossrow, Lc.hdr}, [&](const Args& b) { return run_tc(b, Lc, scale); });
}

// --------------------------------------- two-pass (vocab-chunked) variant
// The same loss and gradients with no [tokens x vocab] buffer at all: pass 1
// computes only lse (the logits GEMM keeps per-tile (m, s) partials, token
// chunk by token chunk); pass 2 recomputes the logits one vocabulary chunk of
// Vc rows at a time for all T tokens, writes the softmax part of D for that
// chunk ([T x Vc] bf16), accumulates dX += D_c W_c in an fp32 [T x H]
// buffer and writes the finished rows dW_c = D_c^T X.  8 T H V flops (the
// logits twice) against 6 T H V for the token-chunked path, and a workspace
// of O(T (H + Vc)) instead of O(C V + V H).
constexpr int64_t kAutoVChunk = 8192;

struct Layout2 {
    int64_t C, nvt, Vc, ldc, nvchunks, nseg;
    size_t lse, lossrow, zlab, hdr, labs, keys, lstart, part, dscr, acc, total;
};

Layout2 layout2(int64_t T, int64_t H, int64_t V, int64_t vchunk) {
    Layout2 L{};
    L.C = std::max<int64_t>(1, std::min<int64_t>(kAutoChunkTC, T));
    L.nvt = ceil_div(V, kVT);
    L.Vc = std::min<int64_t>(vchunk > 0 ? vchunk : kAutoVChunk, V);
    L.ldc = ((L.Vc + 7) / 8) * 8;
    L.nvchunks = ceil_div(V, L.Vc);
    L.nseg = T > 0 ? ceil_div(T, static_cast<int64_t>(kMaxSortKeys)) : 0;
    size_t o = 0;
    L.lse = o; o = up256(o + sizeof(float) * static_cast<size_t>(T));
    L.lossrow = o; o = up256(o + sizeof(float) * static_cast<size_t>(T));
    L.zlab = o; o = up256(o + sizeof(float) * static_cast<size_t>(T));
    L.hdr = o; o = up256(o + sizeof(Hdr));
    // the labels with bad ones replaced by ignore_index (the entry points that do not wait)
    L.labs = o; o = up256(o + sizeof(int64_t) * static_cast<size_t>(T));
    L.keys = o; o = up256(o + sizeof(unsigned long long) * static_cast<size_t>(T));
    L.lstart = o; o = up256(o + sizeof(int) * static_cast<size_t>(L.nseg * (V + 1)));
    L.part = o; o = up256(o + sizeof(float2) * static_cast<size_t>(L.C * L.nvt));
    L.dscr = o; o = up256(o + 2 * static_cast<size_t>(T) * static_cast<size_t>(L.ldc));
    L.acc = o; o = up256(o + (L.nvchunks > 1 ? sizeof(float) * static_cast<size_t>(T * H) : 0));
    L.total = o;
    return L;
}

int run_two_pass(const Args& a, const Layout2& L, float scale) {
    using namespace tc;
    const __nv_bfloat16* X = static_cast<const __nv_bfloat16*>(a.X);
    const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.W);
    float* lse = reinterpret_cast<float*>(a.ws + L.lse);
    float* lossrow = reinterpret_cast<float*>(a.ws + L.lossrow);
    float* zlab = reinterpret_cast<float*>(a.ws + L.zlab);
    Hdr* hdr = reinterpret_cast<Hdr*>(a.ws + L.hdr);
    float2* part = reinterpret_cast<float2*>(a.ws + L.part);
    __nv_bfloat16* D = reinterpret_cast<__nv_bfloat16*>(a.ws + L.dscr);
    float* acc = reinterpret_cast<float*>(a.ws + L.acc);
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(a.ws + L.keys);
    int* lstart = reinterpret_cast<int*>(a.ws + L.lstart);
    const int H = static_cast<int>(a.H), V = static_cast<int>(a.V), T = static_cast<int>(a.T);
    int rc;
    CUtensorMap mW_k;
    if ((rc = make_map(&mW_k, W, H, V, H, BK, B_BOX_ROWS))) return rc;
    // pass 1: lse and the loss terms, token chunk by token chunk (the chunk's X stays in L2)
    const size_t fac_smem = sizeof(float) * static_cast<size_t>(L.nvt);
    for (int64_t t0 = 0; t0 < a.T; t0 += L.C) {
        const int cl = static_cast<int>(std::min(L.C, a.T - t0));
        EpiParams e{};
        e.err = &hdr->err;
        e.ignore_index = a.ignore;
        e.labels = a.labels + t0;
        e.M = cl;
        e.N = V;
        e.raster = RASTER_M_FASTEST;
        e.hint_a = HINT_EVICT_LAST;
        e.hint_b = HINT_EVICT_FIRST;
        e.p_out = nullptr;   // partials and the label logit only
        e.part = part;
        e.nvt = static_cast<int>(L.nvt);
        e.zlab = zlab + t0;
        if ((rc = launch_logits(X + t0 * H, cl, H, V, mW_k, e, 0, L.nvt, a.st))) return rc;
        dlogits_bf16<<<cl, kRowThreads, fac_smem, a.st>>>(a.labels + t0, a.ignore, part, static_cast<int>(L.nvt),
                                                          zlab + t0, nullptr, 0, V, scale, a.scale_dev, lse + t0,
                                                          lossrow + t0);
        if ((rc = check_launch("dlogits_bf16"))) return rc;
    }
    // label keys of all tokens, sorted in segments of kMaxSortKeys, one start table per segment
    if (a.dW && (rc = sort_labels(a.labels, a.T, kMaxSortKeys, a.ignore, V, true, keys, lstart, a.st))) return rc;
    // pass 2: per vocabulary chunk, recompute the logits, D_c, dX +=, dW_c
    CUtensorMap mX_all, mX_mn;
    if ((rc = make_map(&mX_all, X, H, T, H, BK, BM))) return rc;     // A of the recompute (K-major)
    if ((rc = make_map(&mX_mn, X, H, T, H, MN_BOX, BK))) return rc;  // B of dW_c (MN-major)
    for (int64_t c = 0; c < L.nvchunks; ++c) {
        const int64_t c0 = c * L.Vc;
        const int vl = static_cast<int>(std::min(L.Vc, a.V - c0));
        const bool last = c == L.nvchunks - 1;
        const __nv_bfloat16* Wc = W + c0 * H;
        CUtensorMap mWc_k, mWc_mn, mD_k, mD_mn;
        if ((rc = make_map(&mWc_k, Wc, H, vl, H, BK, B_BOX_ROWS))) return rc;
        if ((rc = make_map(&mWc_mn, Wc, H, vl, H, MN_BOX, BK))) return rc;
        if ((rc = make_map(&mD_k, D, vl, T, L.ldc, BK, BM))) return rc;
        if ((rc = make_map(&mD_mn, D, vl, T, L.ldc, MN_BOX, BK))) return rc;
        EpiParams e{};
        e.err = &hdr->err;
        e.ignore_index = a.ignore;
        e.labels = a.labels;
        // a. D_c = scale * softmax part, from the recomputed logits and lse
        e.M = T;
        e.N = vl;
        // groups of 8 column blocks of W_c (16 MB) stay in L2 while X streams past once per
        // group (n fastest needs all 67 MB of W_c in every wave); X reused within a wave
        e.raster = RASTER_N_GROUPS;
        e.hint_a = HINT_NORMAL;
        e.hint_b = HINT_EVICT_LAST;    // W_c: reused by every token block
        e.lse = lse;
        e.corr_scale = scale;
        e.scale_ptr = a.scale_dev;
        e.out = D;
        e.ldo = L.ldc;
        if ((rc = launch_gemm<0, 0, EPI_SOFTMAX, 1>(mX_all, mWc_k, T, vl, H, e, a.st))) return rc;
        // b. dX (+)= D_c W_c in fp32, the one-hot part subtracted once (first chunk)
        if (a.dX) {
            EpiParams d{};
            d.err = &hdr->err;
            d.ignore_index = a.ignore;
            d.labels = a.labels;
            d.corr_src = c == 0 ? W : nullptr;
            d.ld_corr = H;
            d.corr_scale = scale;
            d.scale_ptr = a.scale_dev;
            d.M = T;
            d.N = H;
            d.raster = RASTER_N_GROUPS;
            d.acc = acc;
            d.lda = H;
            d.acc_read = c > 0 ? 1 : 0;
            d.acc_write = last ? 0 : 1;
            d.out_write = last ? 1 : 0;
            d.out = static_cast<__nv_bfloat16*>(a.dX);
            d.ldo = H;
            if ((rc = launch_gemm<0, 1, EPI_ACCUM, 1>(mD_k, mWc_mn, T, H, vl, d, a.st))) return rc;
        }
        // c. dW_c = D_c^T X, minus scale * X_t for the tokens labelled with each row
        if (a.dW) {
            EpiParams d{};
            d.err = &hdr->err;
            d.ignore_index = a.ignore;
            d.corr_src = X;
            d.ld_corr = H;
            d.corr_scale = scale;
            d.scale_ptr = a.scale_dev;
            d.keys = keys;
            d.nkeys = T;
            d.lstart = lstart + c0;
            d.nseg = static_cast<int>(L.nseg);
            d.lstride = V + 1;
            d.M = vl;
            d.N = H;
            d.raster = RASTER_N_FASTEST;
            d.out_write = 1;
            d.out = static_cast<__nv_bfloat16*>(a.dW) + c0 * H;
            d.ldo = H;
            if ((rc = launch_gemm<1, 1, EPI_ACCUM, 1>(mD_mn, mX_mn, vl, H, T, d, a.st))) return rc;
        }
    }
    return LIGER_OK;
}

CompactLayout compact_layout2(int64_t T, int64_t H, int64_t V, int64_t vchunk) {
    const Layout2 L = layout2(T, H, V, vchunk);
    return compact_regions(L.labs, L.total, T, H, 2);
}

// The two-pass path on the tokens that are not ignored only (both passes skip the
// ignored tokens' logits).
int run_two_pass_compact(const Args& a, int64_t n_valid, int64_t vchunk, float scale) {
    const Layout2 Lt = layout2(a.T, a.H, a.V, vchunk);
    const Layout2 Lc = layout2(n_valid, a.H, a.V, vchunk);
    if (Lc.total > Lt.total) return run_two_pass(a, Lt, scale);
    return run_compacted(a, n_valid, compact_layout2(a.T, a.H, a.V, vchunk), RowVals{Lt.lse, Lt.lossrow, Lt.hdr},
                         RowVals{Lc.lse, Lc.lossrow, Lc.hdr}, [&](const Args& b) { return run_two_pass(b, Lc, scale); });
}

}  // namespace
}  // namespace liger

using namespace liger;

extern "C" size_t liger_linear_ce_workspace(int64_t T, int64_t H, int64_t V, int64_t chunk, int dtype) {
    if (T < 0 || H <= 0 || V <= 0 || chunk < 0 || (dtype != LIGER_F32 && dtype != LIGER_BF16)) return 0;
    if (use_tc(H, V, dtype)) return compact_layout(T, H, V, chunk, dtype).total;
    return layout(T, H, V, chunk, dtype).total;
}

namespace liger {
namespace {

struct CommonLayout {
    size_t lse, lossrow, hdr, labs, total;
};

// A pinned host copy of the header for this thread (allocated on first use, kept for
// the thread's lifetime; pinned memory is visible to every device's context).
int pinned_hdr(Hdr** out) {
    thread_local Hdr* buf = nullptr;
    if (buf == nullptr) {
        void* p = nullptr;
        if (cudaMallocHost(&p, sizeof(Hdr)) != cudaSuccess) return check_launch("linear_ce pinned header");
        buf = static_cast<Hdr*>(p);
    }
    *out = buf;
    return LIGER_OK;
}

// Shared tail of both entry points: pointer and workspace checks, the label
// scan (bad labels -> LIGER_ERR_LABEL before any other work), the all-ignored
// case, the gradient scale, the variant's GEMMs, the final loss.
// sync = false: no host wait (capturable in a CUDA graph); bad labels are replaced by
// ignore_index in a workspace copy, the scale and the mean's count stay on the device,
// and the loss is NaN if a label was bad.
template <typename Run>
int ce_entry(const char* who, const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H, int64_t V,
             int64_t ignore_index, int reduction, float grad_scale, float* loss, void* dX, void* dW, void* ws,
             size_t ws_bytes, int dtype, void* stream, const CommonLayout& CL, Run run, bool sync = true) {
    if (!X || !W || !loss || (T > 0 && !labels)) return fail(LIGER_ERR_NULL, "%s: X, W, labels, loss required", who);
    if (!aligned16(X) || !aligned16(W) || (dX && !aligned16(dX)) || (dW && !aligned16(dW)) ||
        (reinterpret_cast<uintptr_t>(loss) & 3) || (reinterpret_cast<uintptr_t>(labels) & 7))
        return fail(LIGER_ERR_ALIGN, "%s: X, W, dX, dW must be 16-byte aligned", who);
    if (!ws || ws_bytes < CL.total || (reinterpret_cast<uintptr_t>(ws) & 255))
        return fail(LIGER_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) required, got %zu", who,
                    CL.total, ws_bytes);
    cudaStream_t st = as_stream(stream);
    uint8_t* w8 = static_cast<uint8_t*>(ws);
    Hdr* hdr = reinterpret_cast<Hdr*>(w8 + CL.hdr);
    if (cudaMemsetAsync(hdr, 0, sizeof(Hdr), st) != cudaSuccess) return check_launch("linear_ce memset");
    if (!sync && T > 0) {
        int64_t* labs = reinterpret_cast<int64_t*>(w8 + CL.labs);
        const int grid = static_cast<int>(std::min<int64_t>(ceil_div(T, 256), 4 * sm_count()));
        label_scan<<<grid, 256, 0, st>>>(labels, T, V, ignore_index, hdr, labs);
        if (int rc = check_launch("label_scan")) return rc;
        ce_scale<<<1, 1, 0, st>>>(hdr, reduction, grad_scale);
        if (int rc = check_launch("ce_scale")) return rc;
        Args a{X, W, labs, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, w8, dtype, st, &hdr->scale};
        if (int rc = run(a, 0.0f, int64_t{-1})) return rc;   // the count stays on the device
        loss_final<<<1, 1024, 0, st>>>(reinterpret_cast<float*>(w8 + CL.lossrow), T, 0.0, hdr, loss,
                                       reduction == 0 ? 1 : 2);
        return check_launch("loss_final");
    }
    Hdr h{};
    if (T > 0) {
        const int grid = static_cast<int>(std::min<int64_t>(ceil_div(T, 256), 4 * sm_count()));
        label_scan<<<grid, 256, 0, st>>>(labels, T, V, ignore_index, hdr, nullptr);
        if (int rc = check_launch("label_scan")) return rc;
        // read through a pinned buffer of this thread: a copy into pageable memory takes the
        // driver's staging path, which can wait behind other copies in flight
        Hdr* hp = nullptr;
        if (int rc = pinned_hdr(&hp)) return rc;
        if (cudaMemcpyAsync(hp, hdr, sizeof(Hdr), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
            cudaStreamSynchronize(st) != cudaSuccess)
            return check_launch("linear_ce label scan");
        h = *hp;
        if (h.bad) return fail(LIGER_ERR_LABEL, "%s: a label is outside [0, %lld) and is not %lld", who,
                               (long long)V, (long long)ignore_index);
    }
    const int64_t n_valid = static_cast<int64_t>(h.n_valid);
    const size_t esz = dtype == LIGER_F32 ? 4 : 2;
    if (n_valid == 0) {
        // nothing to learn from: loss 0, zero gradients (PyTorch would give NaN for the mean)
        bool ok = cudaMemsetAsync(loss, 0, sizeof(float), st) == cudaSuccess;
        if (dX) ok = ok && cudaMemsetAsync(dX, 0, static_cast<size_t>(T * H) * esz, st) == cudaSuccess;
        if (dW) ok = ok && cudaMemsetAsync(dW, 0, static_cast<size_t>(V * H) * esz, st) == cudaSuccess;
        if (T > 0) ok = ok && cudaMemsetAsync(w8 + CL.lse, 0, sizeof(float) * static_cast<size_t>(T), st) == cudaSuccess;
        if (T > 0)
            ok = ok && cudaMemsetAsync(w8 + CL.lossrow, 0, sizeof(float) * static_cast<size_t>(T), st) == cudaSuccess;
        return ok ? LIGER_OK : check_launch("linear_ce memset");
    }
    const float scale = reduction == 0 ? static_cast<float>(static_cast<double>(grad_scale) / static_cast<double>(n_valid))
                                       : grad_scale;
    Args a{X, W, labels, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, w8, dtype, st, nullptr};
    if (int rc = run(a, scale, n_valid)) return rc;
    const double denom = reduction == 0 ? static_cast<double>(n_valid) : 1.0;
    loss_final<<<1, 1024, 0, st>>>(reinterpret_cast<float*>(w8 + CL.lossrow), T, denom, hdr, loss, 0);
    return check_launch("loss_final");
}

}  // namespace
}  // namespace liger

namespace {
int linear_ce_impl(const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H, int64_t V,
                   int64_t ignore_index, int reduction, float grad_scale, float* loss, void* dX, void* dW, void* ws,
                   size_t ws_bytes, int64_t chunk, int dtype, void* stream, bool sync) {
    clear_error();
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "linear_ce: dtype %d", dtype);
    if (T < 0 || H <= 0 || V <= 0 || chunk < 0 || H > (1 << 30) || V > (1 << 30) || T > (int64_t{1} << 31) ||
        (reduction != 0 && reduction != 1))
        return fail(LIGER_ERR_SHAPE, "linear_ce: T=%lld H=%lld V=%lld chunk=%lld reduction=%d", (long long)T,
                    (long long)H, (long long)V, (long long)chunk, reduction);
    const Layout L = layout(T, H, V, chunk, dtype);
    const size_t total = L.tc ? compact_layout(T, H, V, chunk, dtype).total : L.total;
    const CommonLayout CL{L.lse, L.lossrow, L.hdr, L.labs, total};
    return ce_entry(
        "linear_ce", X, W, labels, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, ws, ws_bytes, dtype,
        stream, CL,
        [&](const Args& a, float scale, int64_t n_valid) {
            if (L.tc) {
                // some tokens ignored, and their count known on the host: run the others only
                if (n_valid > 0 && n_valid < a.T) return run_tc_compact(a, n_valid, chunk, scale);
                return run_tc(a, L, scale);
            }
            if (dtype == LIGER_F32) return run_simt<float>(a, L, scale);
            return run_simt<__nv_bfloat16>(a, L, scale);
        },
        sync);
}
}  // namespace

extern "C" int liger_linear_ce_fwd_bwd(const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H,
                                       int64_t V, int64_t ignore_index, int reduction, float grad_scale, float* loss,
                                       void* dX, void* dW, void* ws, size_t ws_bytes, int64_t chunk, int dtype,
                                       void* stream) {
    return linear_ce_impl(X, W, labels, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, ws, ws_bytes,
                          chunk, dtype, stream, true);
}

extern "C" int liger_linear_ce_fwd_bwd_async(const void* X, const void* W, const int64_t* labels, int64_t T,
                                             int64_t H, int64_t V, int64_t ignore_index, int reduction,
                                             float grad_scale, float* loss, void* dX, void* dW, void* ws,
                                             size_t ws_bytes, int64_t chunk, int dtype, void* stream) {
    return linear_ce_impl(X, W, labels, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, ws, ws_bytes,
                          chunk, dtype, stream, false);
}

extern "C" size_t liger_linear_ce_two_pass_workspace(int64_t T, int64_t H, int64_t V, int64_t vchunk) {
    if (T < 0 || H <= 0 || V <= 0 || vchunk < 0) return 0;
    return compact_layout2(T, H, V, vchunk).total;
}

namespace {
int linear_ce_two_pass_impl(const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H, int64_t V,
                            int64_t ignore_index, int reduction, float grad_scale, float* loss, void* dX, void* dW,
                            void* ws, size_t ws_bytes, int64_t vchunk, int dtype, void* stream, bool sync) {
    clear_error();
    if (dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "linear_ce_two_pass: bf16 only (tensor-core path)");
    if (T < 0 || H < 64 || H % 8 || V < 256 || vchunk < 0 || (vchunk % 8) || H > (1 << 30) || V > (1 << 30) ||
        T > (int64_t{1} << 31) - 1 || (reduction != 0 && reduction != 1))
        return fail(LIGER_ERR_SHAPE, "linear_ce_two_pass: T=%lld H=%lld V=%lld vchunk=%lld reduction=%d "
                    "(H >= 64 and a multiple of 8, V >= 256, vchunk a multiple of 8)", (long long)T, (long long)H,
                    (long long)V, (long long)vchunk, reduction);
    const Layout2 L = layout2(T, H, V, vchunk);
    const CommonLayout CL{L.lse, L.lossrow, L.hdr, L.labs, compact_layout2(T, H, V, vchunk).total};
    return ce_entry(
        "linear_ce_two_pass", X, W, labels, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, ws, ws_bytes,
        dtype, stream, CL,
        [&](const Args& a, float scale, int64_t n_valid) {
            // some tokens ignored, and their count known on the host: run the others only
            if (n_valid > 0 && n_valid < a.T) return run_two_pass_compact(a, n_valid, vchunk, scale);
            return run_two_pass(a, L, scale);
        },
        sync);
}
}  // namespace

extern "C" int liger_linear_ce_two_pass_fwd_bwd(const void* X, const void* W, const int64_t* labels, int64_t T,
                                                int64_t H, int64_t V, int64_t ignore_index, int reduction,
                                                float grad_scale, float* loss, void* dX, void* dW, void* ws,
                                                size_t ws_bytes, int64_t vchunk, int dtype, void* stream) {
    return linear_ce_two_pass_impl(X, W, labels, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, ws,
                                   ws_bytes, vchunk, dtype, stream, true);
}

extern "C" int liger_linear_ce_two_pass_fwd_bwd_async(const void* X, const void* W, const int64_t* labels, int64_t T,
                                                      int64_t H, int64_t V, int64_t ignore_index, int reduction,
                                                      float grad_scale, float* loss, void* dX, void* dW, void* ws,
                                                      size_t ws_bytes, int64_t vchunk, int dtype, void* stream) {
    return linear_ce_two_pass_impl(X, W, labels, T, H, V, ignore_index, reduction, grad_scale, loss, dX, dW, ws,
                                   ws_bytes, vchunk, dtype, stream, false);
}

// ------------------------------------------------ policy loss and label log-probabilities
namespace liger {
namespace {

// Workspace of the policy loss: the cross-entropy's, then its own per-token arrays.
struct PolicyLayout {
    Layout L;
    size_t seq, n_seq, coef, term, kl, clip, split, kpart, xpad, total;
};

// Tokens per chunk of the policy loss on the tensor-core path when the caller leaves it open: up to
// 8192 at once, so that a batch of up to that needs no fp32 [V x H] sum of dW across chunks (reading
// and writing it took 0.6 of 6.9 ms at 4096 x 4096 x 128256) and the dX tiles fill their waves better.
int64_t policy_chunk(int64_t T, int64_t H, int64_t V, int64_t chunk, int dtype) {
    return chunk > 0 || !use_tc(H, V, dtype) ? chunk : std::max<int64_t>(1, std::min<int64_t>(T, kAutoChunkTC));
}

PolicyLayout policy_layout(int64_t T, int64_t H, int64_t V, int64_t B, int64_t chunk, int dtype) {
    PolicyLayout P{};
    chunk = policy_chunk(T, H, V, chunk, dtype);
    P.L = layout(T, H, V, chunk, dtype);
    size_t o = up256(P.L.tc ? compact_layout(T, H, V, chunk, dtype).total : P.L.total);
    const size_t per_token = up256(sizeof(float) * static_cast<size_t>(std::max<int64_t>(T, 1)));
    P.seq = o; o += per_token;
    P.coef = o; o += per_token;
    P.term = o; o += per_token;
    P.kl = o; o += per_token;
    P.clip = o; o += per_token;
    P.n_seq = o; o = up256(o + sizeof(int) * static_cast<size_t>(B));
    P.split = o; o += P.L.tc ? 0 : sizeof(float) * static_cast<size_t>(kSplitFloats);
    // items of one launch: at most as many as CTA pairs
    P.kpart = o; o += P.L.tc ? sizeof(float) * static_cast<size_t>(kPairs * kTileFloats * std::min(kDxMaxSlabs, ceil_div(V, dx_slab(V)))) : 0;
    P.xpad = o; o += P.L.tc ? up256(2 * static_cast<size_t>(kPadRows * H)) : 0;
    P.total = o;
    return P;
}

constexpr int64_t kFewParts = 4 * 2048;   // partials of the few-token path

// Workspace of the log-probabilities.  Tensor-core path: header, labels, z at the label, the row
// partials of a chunk; then, for the form that drops ignored tokens, their X rows and index maps.
struct LogpLayout {
    bool tc;
    int64_t C, nvt;
    size_t hdr, labs, zlab, part, scr, split, total;
    CompactLayout comp;
};

LogpLayout logp_layout(int64_t T, int64_t H, int64_t V, int dtype) {
    LogpLayout P{};
    P.tc = use_tc(H, V, dtype);
    P.nvt = ceil_div(V, kVT);
    P.C = P.tc ? kAutoChunkTC : std::max<int64_t>(128, (int64_t{1} << 26) / V);   // as layout()
    P.C = std::max<int64_t>(1, std::min(P.C, T));
    const size_t t = static_cast<size_t>(std::max<int64_t>(T, 1));
    size_t o = 0;
    P.hdr = o; o = up256(o + sizeof(Hdr));
    P.labs = o; o = up256(o + sizeof(int64_t) * t);
    P.zlab = o; o = up256(o + sizeof(float) * t);
    // (few tokens: 4 tokens times at most 2048 blocks)
    P.part = o; o = up256(o + (P.tc ? sizeof(float2) * static_cast<size_t>(std::max<int64_t>(P.C * P.nvt, kFewParts)) : 0));
    P.scr = o; o = up256(o + (P.tc ? 0 : sizeof(float) * static_cast<size_t>(P.C * V)));
    P.split = o; o += P.tc ? 0 : sizeof(float) * static_cast<size_t>(kSplitFloats);
    P.comp = compact_regions(o, 0, std::max(T, kPadRows), H, 2);
    P.total = P.tc ? P.comp.total : o;
    return P;
}

// Logits of at most NT tokens, W read once: the tensor-core GEMM would spend a 256-row tile on
// them (305 us for one token at 4096 x 128256, where reading W takes 155 us; 158 us here).
// A warp takes R rows of W at a time, its lanes the rows' 16-byte vectors, 8 loads of a row in
// flight (4 KB of it side by side: one row at a time 158 us, four rows with two loads each 174), the
// tokens' vectors from shared memory; products of two bf16 values are exact in fp32.
// Lane t keeps token t's running maximum and sum of exponentials over the warp's rows; the block
// writes one (m, s) per token, as the GEMM's epilogue does per tile, and the logit at the label.
// HBM-bound up to 4 tokens (167 us); 8 are bound by the multiply-adds (322 us).
template <int NT, int R>
__global__ void __launch_bounds__(256) logp_few(const __nv_bfloat16* X, const __nv_bfloat16* W, const int64_t* labels, int n,
                                                int H, int V, float2* __restrict__ part, int nparts,
                                                float* __restrict__ zlab) {
    extern __shared__ uint4 xs[];   // [NT][H / 8]
    __shared__ float2 ms[8][NT];
    const int nv = H / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_stream();
    for (int i = threadIdx.x; i < NT * nv; i += 256)
        xs[i] = i < n * nv ? ldg16(X + static_cast<int64_t>(i) * 8) : make_uint4(0, 0, 0, 0);
    const int64_t y = lane < n ? labels[lane] : -1;
    __syncthreads();
    float m = -INFINITY, s = 0.f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * R;
    for (int64_t v0 = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * R; v0 < V; v0 += step) {
        const __nv_bfloat16* wr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) wr[r] = W + min(v0 + r, static_cast<int64_t>(V) - 1) * H;
        float2 acc[NT][R];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[t][r] = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int j = lane; j < nv; j += 32) {
            uint4 w[R];
#pragma unroll
            for (int r = 0; r < R; ++r) w[r] = ldg16_cs(wr[r] + static_cast<int64_t>(j) * 8);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 x = xs[t * nv + j];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][r] = fma_bf2(word(x, e), word(w[r], e), acc[t][r]);
            }
        }
        float z[R];   // of this lane's token
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float v = warp_sum(acc[t][r].x + acc[t][r].y);
                if (lane == t) z[r] = v;
            }
        if (lane < n) {
            float top = m;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (v0 + r < V) top = fmaxf(top, z[r]);
            const float base = top == -INFINITY ? 0.f : top;   // only -inf so far: exp(-inf) = 0, not NaN
            float add = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (v0 + r < V) {
                    add += expf(z[r] - base);
                    if (v0 + r == y) zlab[lane] = z[r];
                }
            s = s * expf(m - base) + add;
            m = top;
        }
    }
    if (lane < NT) ms[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x < n) {
        float top = -INFINITY, sum = 0.f;
        for (int w = 0; w < 8; ++w) top = fmaxf(top, ms[w][threadIdx.x].x);
        for (int w = 0; w < 8; ++w) {
            const float2 p = ms[w][threadIdx.x];
            if (p.y != 0.f) sum += p.y * expf(p.x - top);   // a warp without rows has s = 0; NaN is passed on
        }
        part[static_cast<int64_t>(threadIdx.x) * nparts + blockIdx.x] = make_float2(top, sum);
    }
}

constexpr int kFewTokens = 4;
constexpr size_t kFewSmem = 96u * 1024u;   // the tokens' vectors: two blocks per SM

template <int NT, int R>
int launch_logp_few(const __nv_bfloat16* X, const __nv_bfloat16* W, const int64_t* labs, int n, int H, int V, float2* part,
                    float* zlab, int64_t most_parts, int& nparts, cudaStream_t st) {
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return check_launch("logp_few device");
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(logp_few<NT, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kFewSmem)) !=
            cudaSuccess)
            return check_launch("logp_few attribute");
        done[dev].store(true, std::memory_order_release);
    }
    const size_t smem = static_cast<size_t>(NT) * H * 2;
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, logp_few<NT, R>, 256, smem);
    // every block has rows, and no more blocks than the workspace holds partials for
    nparts = static_cast<int>(std::min<int64_t>({ceil_div(V, 8 * R), static_cast<int64_t>(sm_count()) * std::max(1, per_sm), most_parts}));
    return launch_early("logp_few", logp_few<NT, R>, dim3(nparts), 256, smem, st, X, W, labs, n, H, V, part, nparts, zlab);
}

// Reads the header of the scan back: post() queues the copy, wait() waits for it alone (work queued in
// between does not have to end first).
// The copy has landed when the object goes (the pinned buffer is this thread's, for its next call).
struct HdrRead {
    Hdr* host = nullptr;
    cudaEvent_t done = nullptr;
    bool pending = false;

    int post(const char* who, const Hdr* hdr, cudaStream_t st) {
        thread_local cudaEvent_t events[64] = {};   // per device, kept as the pinned buffer is
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return check_launch(who);
        if (events[dev] == nullptr && cudaEventCreateWithFlags(&events[dev], cudaEventDisableTiming) != cudaSuccess)
            return check_launch(who);
        done = events[dev];
        if (int rc = pinned_hdr(&host)) return rc;
        if (cudaMemcpyAsync(host, hdr, sizeof(Hdr), cudaMemcpyDeviceToHost, st) != cudaSuccess) return check_launch(who);
        if (cudaEventRecord(done, st) != cudaSuccess) {
            cudaStreamSynchronize(st);
            return check_launch(who);
        }
        pending = true;
        return LIGER_OK;
    }
    int wait(const char* who, Hdr* out) {
        pending = false;
        if (cudaEventSynchronize(done) != cudaSuccess) return check_launch(who);
        *out = *host;
        return LIGER_OK;
    }
    ~HdrRead() {
        if (pending) cudaEventSynchronize(done);
    }
};

// Whether dropping the tokens that are not valid saves a row tile of the GEMMs; if it does not, the
// tokens run as they are (seven launches fewer).
bool worth_compacting(int64_t n, int64_t T) { return ceil_div(n, int64_t{256}) < ceil_div(T, int64_t{256}); }
// Whether that is known before the valid tokens are counted (off the tensor cores none are dropped).  The
// call then queues the logits, which only the workspace sees, before it waits for the count, so that the
// GPU has work while the host wakes up (one token's log-probability at 4096 x 128256 165 us, 170 without;
// policy loss of 3 tokens at 256 x 44779 91 us, 96).
bool never_compacted(bool tc, int64_t T) { return !tc || T <= 256; }

unsigned scan_grid(int64_t T) { return static_cast<unsigned>(std::min<int64_t>(ceil_div(T, 256), 4 * sm_count())); }

// Z = X_c W^T of cl rows off the tensor cores
template <typename TI>
int simt_logits(const TI* Xc, const TI* W, float* Z, int cl, int H, int V, float* split, cudaStream_t st) {
    HeadGemm g{};
    g.M = cl;
    g.N = V;
    g.K = H;
    g.sam = H;
    g.sak = 1;
    g.sbk = 1;
    g.sbn = H;
    g.ldo = V;
    return launch_head_gemm(Xc, W, Z, g, split, st);
}

// The policy loss off the tensor cores, in token chunks of L.C rows.
template <typename TI>
int run_policy_simt(const Args& a, const Layout& L, float* split) {
    const TI *X = static_cast<const TI*>(a.X), *W = static_cast<const TI*>(a.W);
    TI *dX = static_cast<TI*>(a.dX), *dW = static_cast<TI*>(a.dW);
    float* Z = reinterpret_cast<float*>(a.ws + L.scr);
    float* acc = reinterpret_cast<float*>(a.ws + L.acc);
    const int H = static_cast<int>(a.H), V = static_cast<int>(a.V);
    int rc;
    for (int64_t c = 0; c < L.nchunks; ++c) {
        const int64_t t0 = c * L.C;
        const int cl = static_cast<int>(std::min(L.C, a.T - t0));
        const bool first = c == 0, last = c == L.nchunks - 1;
        if ((rc = simt_logits(X + t0 * H, W, Z, cl, H, V, split, a.st))) return rc;
        if (a.check != nullptr && first && (rc = (*a.check)())) return rc;
        if ((rc = launch_early("linear_policy rows", policy_rows_f32, dim3(cl), kRowThreads, 0, a.st, a.labels + t0, a.ignore,
                               Z, V, V, 1, *a.pol, nullptr, t0)))
            return rc;
        if (dX) {   // dX_c = D W
            HeadGemm g{};
            g.M = cl;
            g.N = H;
            g.K = V;
            g.sam = V;
            g.sak = 1;
            g.sbk = H;
            g.sbn = 1;
            g.ldo = H;
            g.labels = a.labels + t0;
            g.ignore = a.ignore;
            if ((rc = launch_head_gemm(Z, W, dX + t0 * H, g, split, a.st))) return rc;
        }
        if (dW) {   // dW (+)= D^T X_c; bf16 with several chunks: the sum in fp32, rounded with the last
            HeadGemm g{};
            g.M = V;
            g.N = H;
            g.K = cl;
            g.sam = 1;
            g.sak = V;
            g.sbk = H;
            g.sbn = 1;
            g.ldo = H;
            g.klabels = a.labels + t0;
            g.ignore = a.ignore;
            const bool f32 = a.dtype == LIGER_F32;
            g.add = !first && (f32 || !last) ? 1 : 0;
            if (f32 || last) {
                if (!f32 && !first) g.base = acc;
                rc = launch_head_gemm(Z, X + t0 * H, dW, g, split, a.st);
            } else {
                rc = launch_head_gemm(Z, X + t0 * H, acc, g, split, a.st);
            }
            if (rc) return rc;
        }
    }
    return LIGER_OK;
}

// The log-probabilities of n rows at X with labels labs; idx: original token of a row (null: the row)
int run_logp_tc(const __nv_bfloat16* X, const __nv_bfloat16* W, const int64_t* labs, const int64_t* idx, int64_t n, int H,
                int V, int64_t ignore, float* logp, uint8_t* w8, const LogpLayout& L, cudaStream_t st, const Check* check) {
    using namespace tc;
    CUtensorMap mW_k;
    int rc;
    if ((rc = make_map(&mW_k, W, H, V, H, BK, B_BOX_ROWS))) return rc;
    Policy pol{};
    pol.logp = logp;
    pol.zero_logp = check != nullptr ? 1 : 0;
    int* err = &reinterpret_cast<Hdr*>(w8 + L.hdr)->err;
    float2* part = reinterpret_cast<float2*>(w8 + L.part);
    float* zlab = reinterpret_cast<float*>(w8 + L.zlab);
    if (n <= kFewTokens && kFewTokens * static_cast<size_t>(H) * 2 <= kFewSmem) {
        int np = 0;
        const int nn = static_cast<int>(n);
        const int64_t most = kFewParts / kFewTokens;
        rc = nn == 1   ? launch_logp_few<1, 1>(X, W, labs, nn, H, V, part, zlab, most, np, st)
             : nn == 2 ? launch_logp_few<2, 1>(X, W, labs, nn, H, V, part, zlab, most, np, st)
                       : launch_logp_few<4, 2>(X, W, labs, nn, H, V, part, zlab, most, np, st);
        if (rc || (check != nullptr && (rc = (*check)()))) return rc;
        return launch_early("linear_logp rows", policy_rows_bf16, dim3(nn), kRowThreads, 0, st, labs, ignore, part, np, zlab,
                            nullptr, 0, V, pol, idx, 0, nullptr, 0, err);
    }
    int64_t x_rows = 0;
    if (n < kPadRows) {
        __nv_bfloat16* pad = reinterpret_cast<__nv_bfloat16*>(w8 + L.comp.dxc);
        if ((rc = pad_rows(X, n, H, pad, st))) return rc;
        X = pad;
        x_rows = kPadRows;
    }
    for (int64_t t0 = 0; t0 < n; t0 += L.C) {
        const int cl = static_cast<int>(std::min(L.C, n - t0));
        EpiParams e{};
        e.err = err;
        e.early = 1;
        e.ignore_index = ignore;
        e.labels = labs + t0;
        e.M = cl;
        e.N = V;
        e.raster = RASTER_M_FASTEST;
        e.hint_a = HINT_EVICT_LAST;
        e.hint_b = HINT_EVICT_FIRST;
        e.p_out = nullptr;
        e.part = part;
        e.nvt = static_cast<int>(L.nvt);
        e.zlab = zlab + t0;
        if ((rc = launch_logits(X + t0 * H, cl, H, V, mW_k, e, 0, L.nvt, st, x_rows))) return rc;
        if (check != nullptr && t0 == 0 && (rc = (*check)())) return rc;
        if ((rc = launch_early("linear_logp rows", policy_rows_bf16, dim3(cl), kRowThreads, 0, st, labs + t0, ignore, part,
                               static_cast<int>(L.nvt), zlab + t0, nullptr, 0, V, pol, idx != nullptr ? idx + t0 : nullptr, t0,
                               nullptr, 0, err)))
            return rc;
    }
    return LIGER_OK;
}

template <typename TI>
int run_logp_simt(const void* X, const void* W, const int64_t* labs, int64_t T, int H, int V, int64_t ignore, float* logp,
                  uint8_t* w8, const LogpLayout& L, cudaStream_t st, const Check* check) {
    float* Z = reinterpret_cast<float*>(w8 + L.scr);
    Policy pol{};
    pol.logp = logp;
    pol.zero_logp = check != nullptr ? 1 : 0;
    for (int64_t t0 = 0; t0 < T; t0 += L.C) {
        const int cl = static_cast<int>(std::min(L.C, T - t0));
        if (int rc = simt_logits(static_cast<const TI*>(X) + t0 * H, static_cast<const TI*>(W), Z, cl, H, V,
                                 reinterpret_cast<float*>(w8 + L.split), st))
            return rc;
        if (check != nullptr && t0 == 0)
            if (int rc = (*check)()) return rc;
        if (int rc = launch_early("linear_logp rows", policy_rows_f32, dim3(cl), kRowThreads, 0, st, labs + t0, ignore, Z, V, V,
                                  0, pol, nullptr, t0))
            return rc;
    }
    return LIGER_OK;
}

// Off the tensor cores the products' tiles limit the rows of a chunk and the vocabulary.
bool head_shape_ok(int64_t T, int64_t H, int64_t V, int dtype, int64_t chunk = 0) {
    if (!(T >= 0 && H > 0 && V > 0 && H <= (1 << 30) && V <= (1 << 30) && T <= (int64_t{1} << 31) - 1)) return false;
    return use_tc(H, V, dtype) || (V <= kHeadRows && std::min(T, layout(T, H, V, chunk, dtype).C) <= kHeadRows);
}

int logp_impl(const char* who, const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H, int64_t V,
              int64_t ignore, float* logp, void* ws, size_t ws_bytes, int dtype, void* stream, bool sync) {
    clear_error();
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (!head_shape_ok(T, H, V, dtype))
        return fail(LIGER_ERR_SHAPE, "%s: T=%lld H=%lld V=%lld", who, (long long)T, (long long)H, (long long)V);
    if (T == 0) return LIGER_OK;
    if (!X || !W || !labels || !logp) return fail(LIGER_ERR_NULL, "%s: X, W, labels, logp required", who);
    if (!aligned16(X) || !aligned16(W) || (reinterpret_cast<uintptr_t>(logp) & 3) ||
        (reinterpret_cast<uintptr_t>(labels) & 7))
        return fail(LIGER_ERR_ALIGN, "%s: X and W must be 16-byte aligned, labels 8, logp 4", who);
    const LogpLayout L = logp_layout(T, H, V, dtype);
    if (!ws || ws_bytes < L.total || (reinterpret_cast<uintptr_t>(ws) & 255))
        return fail(LIGER_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) required, got %zu", who, L.total,
                    ws_bytes);
    cudaStream_t st = as_stream(stream);
    uint8_t* w8 = static_cast<uint8_t*>(ws);
    Hdr* hdr = reinterpret_cast<Hdr*>(w8 + L.hdr);
    int64_t* labs = reinterpret_cast<int64_t*>(w8 + L.labs);
    if (cudaMemsetAsync(hdr, 0, sizeof(Hdr), st) != cudaSuccess) return check_launch("linear_logp memset");
    // the waiting form leaves logp alone until it knows that the labels are good
    policy_scan<<<scan_grid(T), 256, 0, st>>>(labels, nullptr, T, V, 1, ignore, hdr, labs, nullptr, nullptr,
                                              sync ? nullptr : logp, nullptr, nullptr, nullptr, 1);
    if (int rc = check_launch("linear_logp scan")) return rc;
    int64_t n = T;
    HdrRead scan;
    const Check* before_rows = nullptr;
    auto settle = [&]() -> int {
        Hdr h{};
        if (int rc = scan.wait("linear_logp scan", &h)) return rc;
        if (h.bad) return fail(LIGER_ERR_LABEL, "%s: a label is outside [0, %lld) and is not %lld", who, (long long)V,
                               (long long)ignore);
        n = static_cast<int64_t>(h.n_valid);
        if (n < T && (n == 0 || before_rows == nullptr) &&
            cudaMemsetAsync(logp, 0, sizeof(float) * static_cast<size_t>(T), st) != cudaSuccess)
            return check_launch("linear_logp memset");
        return n == 0 ? kNothing : LIGER_OK;
    };
    const Check check = check_of(settle);
    if (sync) {
        if (int rc = scan.post("linear_logp scan", hdr, st)) return rc;
        if (never_compacted(L.tc, T)) before_rows = &check;
        else if (int rc = check()) return rc == kNothing ? LIGER_OK : rc;
    }
    if (!L.tc || before_rows != nullptr) {
        const int rc =
            L.tc ? run_logp_tc(static_cast<const __nv_bfloat16*>(X), static_cast<const __nv_bfloat16*>(W), labs, nullptr, T, (int)H,
                               (int)V, ignore, logp, w8, L, st, before_rows)
            : dtype == LIGER_F32
                ? run_logp_simt<float>(X, W, labs, T, (int)H, (int)V, ignore, logp, w8, L, st, before_rows)
                : run_logp_simt<__nv_bfloat16>(X, W, labs, T, (int)H, (int)V, ignore, logp, w8, L, st, before_rows);
        return rc == kNothing ? LIGER_OK : rc;
    }
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16*>(X), *w = static_cast<const __nv_bfloat16*>(W);
    const int64_t* idx = nullptr;
    if (n < T && !worth_compacting(n, T)) n = T;
    if (n < T) {   // only the tokens that are not ignored, in order
        int* cnt = reinterpret_cast<int*>(w8 + L.comp.cnt);
        int64_t* at = reinterpret_cast<int64_t*>(w8 + L.comp.idx);
        int64_t* labc = reinterpret_cast<int64_t*>(w8 + L.comp.labc);
        __nv_bfloat16* xc = reinterpret_cast<__nv_bfloat16*>(w8 + L.comp.xc);
        const int64_t nb = ceil_div(T, static_cast<int64_t>(kCompactBlock));
        compact_count<<<static_cast<unsigned>(nb), kCompactBlock, 0, st>>>(labs, T, ignore, cnt);
        compact_scan<<<1, 1024, 0, st>>>(cnt, nb);
        compact_index<<<static_cast<unsigned>(nb), kCompactBlock, 0, st>>>(labs, T, ignore, cnt, at,
                                                                           reinterpret_cast<int*>(w8 + L.comp.inv), labc);
        gather_rows<<<static_cast<int>(std::min<int64_t>(n, 8 * sm_count())), 256, 0, st>>>(
            static_cast<const uint4*>(X), at, n, H * 2 / 16, reinterpret_cast<uint4*>(xc));
        if (int rc = check_launch("linear_logp compaction")) return rc;
        x = xc;
        labs = labc;
        idx = at;
    }
    return run_logp_tc(x, w, labs, idx, n, (int)H, (int)V, ignore, logp, w8, L, st, nullptr);
}

int policy_impl(const char* who, const void* X, const void* W, const int64_t* labels, const int32_t* cu,
                const float* old_logp, const float* ref_logp, const float* adv, int64_t T, int64_t H, int64_t V, int64_t B,
                int64_t ignore, int reduction, int flags, float eps_low, float eps_high, float beta, float grad_scale,
                float* loss, float* stats, float* logp, void* dX, void* dW, void* ws, size_t ws_bytes, int64_t chunk,
                int dtype, void* stream, bool sync) {
    clear_error();
    if (dtype != LIGER_F32 && dtype != LIGER_BF16) return fail(LIGER_ERR_DTYPE, "%s: dtype %d", who, dtype);
    if (chunk < 0 || !head_shape_ok(T, H, V, dtype, chunk) || B < 1 || B > (1 << 30) || reduction < 0 || reduction > 2 ||
        (flags & ~LIGER_POLICY_ADV_PER_TOKEN))
        return fail(LIGER_ERR_SHAPE, "%s: T=%lld H=%lld V=%lld B=%lld chunk=%lld reduction=%d flags=%d", who, (long long)T,
                    (long long)H, (long long)V, (long long)B, (long long)chunk, reduction, flags);
    if (!cu && B != 1) return fail(LIGER_ERR_NULL, "%s: cu_seqlens is required with B=%lld", who, (long long)B);
    if (!(eps_low >= 0.f && eps_low <= 1.f) || !(eps_high >= 0.f) || !(beta == beta) || !(grad_scale == grad_scale))
        return fail(LIGER_ERR_SHAPE, "%s: eps_low=%g (0 to 1) eps_high=%g (>= 0) beta=%g grad_scale=%g", who, eps_low,
                    eps_high, beta, grad_scale);
    if (!W || !loss || (T > 0 && (!X || !labels || !old_logp || !adv || (beta != 0.f && !ref_logp))))
        return fail(LIGER_ERR_NULL, "%s: X, W, labels, old_logp, adv, loss (and ref_logp with beta) required", who);
    const auto off = [](const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; };
    if (off(X, 16) || off(W, 16) || off(dX, 16) || off(dW, 16) || off(labels, 8) || off(cu, 4) || off(old_logp, 4) ||
        off(ref_logp, 4) || off(adv, 4) || off(loss, 4) || off(stats, 4) || off(logp, 4))
        return fail(LIGER_ERR_ALIGN, "%s: X, W, dX, dW must be 16-byte aligned, labels 8, the others 4", who);
    const PolicyLayout PL = policy_layout(T, H, V, B, chunk, dtype);
    chunk = policy_chunk(T, H, V, chunk, dtype);
    if (!ws || ws_bytes < PL.total || (reinterpret_cast<uintptr_t>(ws) & 255))
        return fail(LIGER_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) required, got %zu", who, PL.total,
                    ws_bytes);
    // logp is written while other blocks still read the old and the reference policy's
    const auto overlaps = [&](const float* p, int64_t n) {
        const auto a = reinterpret_cast<uintptr_t>(logp), b = reinterpret_cast<uintptr_t>(p);
        return a < b + static_cast<size_t>(n) * sizeof(float) && b < a + static_cast<size_t>(T) * sizeof(float);
    };
    if (logp && T > 0 && (overlaps(old_logp, T) || (ref_logp && overlaps(ref_logp, T)) ||
                          overlaps(adv, flags & LIGER_POLICY_ADV_PER_TOKEN ? T : B)))
        return fail(LIGER_ERR_SHAPE, "%s: logp overlaps old_logp, ref_logp or adv", who);
    cudaStream_t st = as_stream(stream);
    uint8_t* w8 = static_cast<uint8_t*>(ws);
    Hdr* hdr = reinterpret_cast<Hdr*>(w8 + PL.L.hdr);
    int64_t* labs = reinterpret_cast<int64_t*>(w8 + PL.L.labs);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(w8 + at); };
    // few sequences: their counts behind the header, in the 256 bytes that it has, zeroed with it
    const bool near = B <= 48;
    static_assert(sizeof(Hdr) <= 64, "counts from byte 64 on");
    int *seq = reinterpret_cast<int*>(w8 + PL.seq), *n_seq = reinterpret_cast<int*>(w8 + (near ? PL.L.hdr + 64 : PL.n_seq));
    if (cudaMemsetAsync(hdr, 0, near ? 256 : sizeof(Hdr), st) != cudaSuccess ||
        (!near && cudaMemsetAsync(n_seq, 0, sizeof(int) * static_cast<size_t>(B), st) != cudaSuccess))
        return check_launch("linear_policy memset");
    int64_t n = T;
    if (T > 0) {
        policy_scan<<<scan_grid(T), 256, 0, st>>>(labels, cu, T, V, B, ignore, hdr, labs, seq, n_seq, sync ? nullptr : logp,
                                                  f32(PL.term), f32(PL.kl), f32(PL.clip), 0);
        if (int rc = check_launch("linear_policy scan")) return rc;
    }
    HdrRead scan;
    const Check* before_rows = nullptr;
    auto settle = [&]() -> int {
        Hdr h{};
        if (int rc = scan.wait("linear_policy scan", &h)) return rc;
        if (h.bad & 2) return fail(LIGER_ERR_SHAPE, "%s: cu_seqlens descends or leaves [0, %lld]", who, (long long)T);
        if (h.bad) return fail(LIGER_ERR_LABEL, "%s: a label is outside [0, %lld) and is not %lld", who, (long long)V,
                               (long long)ignore);
        n = static_cast<int64_t>(h.n_valid);
        if (logp && n < T && (n == 0 || before_rows == nullptr) &&
            cudaMemsetAsync(logp, 0, sizeof(float) * static_cast<size_t>(T), st) != cudaSuccess)
            return check_launch("linear_policy memset");
        return n == 0 ? kNothing : LIGER_OK;
    };
    const Check check = check_of(settle);
    int rc = T == 0 ? kNothing : LIGER_OK;
    if (sync && T > 0) {
        if ((rc = scan.post("linear_policy scan", hdr, st))) return rc;
        if (never_compacted(PL.L.tc, T)) before_rows = &check;
        else rc = check();
        if (rc < 0) return rc;
    }
    const Policy pol{old_logp, ref_logp, adv, flags & LIGER_POLICY_ADV_PER_TOKEN, reduction, 1.f - eps_low, 1.f + eps_high,
                     beta, grad_scale, seq, n_seq, hdr, B, f32(PL.coef), f32(PL.term), f32(PL.kl), f32(PL.clip), logp, f32(PL.kpart),
                     reinterpret_cast<__nv_bfloat16*>(w8 + PL.xpad),
                     PL.L.tc && (!sync || before_rows != nullptr || n < T) ? reinterpret_cast<__nv_bfloat16*>(w8 + compact_layout(T, H, V, chunk, dtype).xc)
                                                  : nullptr,
                     before_rows != nullptr ? 1 : 0};
    const Args a{X, W, labs, T, H, V, ignore, reduction, grad_scale, loss, dX, dW, w8, dtype, st, nullptr, &pol, nullptr,
                 before_rows};
    if (rc == LIGER_OK) {
        if (PL.L.tc) rc = n < T && worth_compacting(n, T) ? run_tc_compact(a, n, chunk, 0.f) : run_tc(a, PL.L, 0.f);
        else rc = dtype == LIGER_F32 ? run_policy_simt<float>(a, PL.L, f32(PL.split)) : run_policy_simt<__nv_bfloat16>(a, PL.L, f32(PL.split));
    }
    if (rc == kNothing) {   // nothing to learn from
        const size_t esz = dtype == LIGER_F32 ? 4 : 2;
        bool ok = cudaMemsetAsync(loss, 0, sizeof(float), st) == cudaSuccess;
        if (stats) ok = ok && cudaMemsetAsync(stats, 0, 2 * sizeof(float), st) == cudaSuccess;
        if (dX) ok = ok && cudaMemsetAsync(dX, 0, static_cast<size_t>(T * H) * esz, st) == cudaSuccess;
        if (dW) ok = ok && cudaMemsetAsync(dW, 0, static_cast<size_t>(V * H) * esz, st) == cudaSuccess;
        return ok ? LIGER_OK : check_launch("linear_policy memset");
    }
    if (rc) return rc;
    return launch_early("linear_policy", policy_final, dim3(1), T <= 1024 ? 256 : kFinalThreads, 0, st, f32(PL.term),
                        f32(PL.kl), f32(PL.clip), T, hdr, loss, stats);
}

}  // namespace
}  // namespace liger

extern "C" size_t liger_linear_logp_workspace(int64_t T, int64_t H, int64_t V, int dtype) {
    if ((dtype != LIGER_F32 && dtype != LIGER_BF16) || !head_shape_ok(T, H, V, dtype)) return 0;
    return logp_layout(T, H, V, dtype).total;
}

extern "C" int liger_linear_logp_fwd(const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H, int64_t V,
                                     int64_t ignore_index, float* logp, void* ws, size_t ws_bytes, int dtype,
                                     void* stream) {
    return logp_impl("linear_logp", X, W, labels, T, H, V, ignore_index, logp, ws, ws_bytes, dtype, stream, true);
}

extern "C" int liger_linear_logp_fwd_async(const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H,
                                           int64_t V, int64_t ignore_index, float* logp, void* ws, size_t ws_bytes,
                                           int dtype, void* stream) {
    return logp_impl("linear_logp_async", X, W, labels, T, H, V, ignore_index, logp, ws, ws_bytes, dtype, stream, false);
}

extern "C" size_t liger_linear_policy_workspace(int64_t T, int64_t H, int64_t V, int64_t B, int64_t chunk, int dtype) {
    if ((dtype != LIGER_F32 && dtype != LIGER_BF16) || B < 1 || chunk < 0 || !head_shape_ok(T, H, V, dtype, chunk)) return 0;
    return policy_layout(T, H, V, B, chunk, dtype).total;
}

extern "C" int liger_linear_policy_fwd_bwd(const void* X, const void* W, const int64_t* labels, const int32_t* cu_seqlens,
                                           const float* old_logp, const float* ref_logp, const float* adv, int64_t T,
                                           int64_t H, int64_t V, int64_t B, int64_t ignore_index, int reduction, int flags,
                                           float eps_low, float eps_high, float beta, float grad_scale, float* loss,
                                           float* stats, float* logp, void* dX, void* dW, void* ws, size_t ws_bytes,
                                           int64_t chunk, int dtype, void* stream) {
    return policy_impl("linear_policy", X, W, labels, cu_seqlens, old_logp, ref_logp, adv, T, H, V, B, ignore_index,
                       reduction, flags, eps_low, eps_high, beta, grad_scale, loss, stats, logp, dX, dW, ws, ws_bytes,
                       chunk, dtype, stream, true);
}

extern "C" int liger_linear_policy_fwd_bwd_async(const void* X, const void* W, const int64_t* labels,
                                                 const int32_t* cu_seqlens, const float* old_logp, const float* ref_logp,
                                                 const float* adv, int64_t T, int64_t H, int64_t V, int64_t B,
                                                 int64_t ignore_index, int reduction, int flags, float eps_low,
                                                 float eps_high, float beta, float grad_scale, float* loss, float* stats,
                                                 float* logp, void* dX, void* dW, void* ws, size_t ws_bytes, int64_t chunk,
                                                 int dtype, void* stream) {
    return policy_impl("linear_policy_async", X, W, labels, cu_seqlens, old_logp, ref_logp, adv, T, H, V, B, ignore_index,
                       reduction, flags, eps_low, eps_high, beta, grad_scale, loss, stats, logp, dX, dW, ws, ws_bytes,
                       chunk, dtype, stream, false);
}
