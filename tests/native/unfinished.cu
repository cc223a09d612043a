// What the epilogue warps of the CTA-pair products write after an expired wait, for every warp of a range of tiles (or of a split
// tile's items), without the product: block t of the grid is tile t (its row block t / num_n), its warps the eight of the pair.
#include "tc_gemm.cuh"

namespace liger {
namespace tc {
namespace {
__global__ void rows(float* sums, int items, __nv_bfloat16* out, __half* pre, int64_t ldo, int M, int N, int num_n) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x;
    const int m0 = t / num_n * TileCfg<1>::TM, n0 = t % num_n * BN;
    if (sums == nullptr) unfinished_rows(nullptr, out, pre, ldo, M, N, m0, warp * 32, n0, lane);
    for (int i = 0; sums != nullptr && i < items; ++i)
        unfinished_rows(sums + (static_cast<int64_t>(t) * items + i) * TileCfg<1>::TM * BN, out, pre, ldo, M, N, m0, warp * 32, n0, lane);
}
}  // namespace
}  // namespace tc
}  // namespace liger

// sums: [tiles][items][TM][BN] or NULL; out, pre [M, ldo]
extern "C" int unfinished(float* sums, int items, void* out, void* pre, int64_t ldo, int M, int N, void* stream) {
    using namespace liger::tc;
    const int num_n = (N + BN - 1) / BN, tiles = (M + TileCfg<1>::TM - 1) / TileCfg<1>::TM * num_n;
    rows<<<tiles, 256, 0, static_cast<cudaStream_t>(stream)>>>(sums, items, static_cast<__nv_bfloat16*>(out), static_cast<__half*>(pre), ldo, M,
                                                              N, num_n);
    return static_cast<int>(cudaGetLastError());
}
