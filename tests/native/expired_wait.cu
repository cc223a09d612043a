// The policy loss of compacted tokens as the library runs it, with the error word that its GEMMs would set on an expired
// wait set (or not) in stream order, behind the run's own reset of its header and ahead of its first GEMM.
#include <stddef.h>

#include "linear_ce.cu"

extern "C" int policy_compacted(const void* X, const void* W, const int64_t* labels, const float* old_logp, const float* adv,
                                int64_t T, int64_t H, int64_t V, int64_t n, float* loss, float* stats, float* logp, void* dX,
                                void* dW, void* ws, size_t ws_bytes, int expired, void* stream) {
    const int dtype = LIGER_BF16;
    const int64_t ignore = -100, chunk = policy_chunk(T, H, V, 0, dtype);
    const PolicyLayout P = policy_layout(T, H, V, 1, 0, dtype);
    const Layout Lt = layout(T, H, V, chunk, dtype), Lc = layout(n, H, V, chunk, dtype);
    if (!P.L.tc || ws_bytes < P.total || n < 1 || n >= T || Lc.total > Lt.total) return -100;
    cudaStream_t st = as_stream(stream);
    uint8_t* w8 = static_cast<uint8_t*>(ws);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(w8 + at); };
    Hdr* hdr = reinterpret_cast<Hdr*>(w8 + P.L.hdr);
    int64_t* labs = reinterpret_cast<int64_t*>(w8 + P.L.labs);
    int *seq = reinterpret_cast<int*>(w8 + P.seq), *n_seq = reinterpret_cast<int*>(w8 + P.L.hdr + 64);
    if (cudaMemsetAsync(hdr, 0, 256, st) != cudaSuccess) return -101;
    policy_scan<<<scan_grid(T), 256, 0, st>>>(labels, nullptr, T, V, 1, ignore, hdr, labs, seq, n_seq, logp, f32(P.term),
                                              f32(P.kl), f32(P.clip), 0);
    const Policy pol{old_logp, nullptr, adv, 0, 0, 0.8f, 1.2f, 0.f, 1.f, seq, n_seq, hdr, 1, f32(P.coef), f32(P.term),
                     f32(P.kl), f32(P.clip), logp, f32(P.kpart), reinterpret_cast<__nv_bfloat16*>(w8 + P.xpad), nullptr, 0};
    const Args a{X, W, labs, T, H, V, ignore, 0, 1.f, loss, dX, dW, w8, dtype, st, nullptr, &pol, nullptr, nullptr};
    const int rc = run_compacted(a, n, compact_layout(T, H, V, chunk, dtype), RowVals{Lt.lse, Lt.lossrow, Lt.hdr},
                                 RowVals{Lc.lse, Lc.lossrow, Lc.hdr}, [&](const Args& b) {
                                     if (expired && cudaMemsetAsync(b.ws + Lc.hdr + offsetof(Hdr, err), 1, sizeof(int), st) !=
                                                        cudaSuccess)
                                         return -102;
                                     return run_tc(b, Lc, 0.f);
                                 });
    if (rc) return rc;
    policy_final<<<1, 256, 0, st>>>(f32(P.term), f32(P.kl), f32(P.clip), T, hdr, loss, stats);
    return check_launch("policy_final");
}
