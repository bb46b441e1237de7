// experts_wgrad.cu -- the weights' and bias gradients (experts.cuh).
#include "experts.cuh"

namespace moe {

cudaError_t launch_expert_wgrad(const moe_rows *G, const void *dy, int N, const void *x, int K, void *dw, void *db,
                                int fp32, cudaStream_t s)
{
    if (G->rows == 0) {
        const size_t n = (size_t)G->E * N * (fp32 ? 4 : 2);
        const cudaError_t err = db ? cudaMemsetAsync(db, 0, n, s) : cudaSuccess;
        return err == cudaSuccess ? cudaMemsetAsync(dw, 0, n * K, s) : err;
    }
    Params p = {};
    p.offsets = G->offsets;
    p.ws = G->ws;
    p.E = G->E;
    p.rows = G->rows;
    p.M = N;
    p.N = K;
    p.fp32 = fp32;
    p.dw = dw;
    p.db = db;
    const Cut cut = wgrad_cut(N, K, G->rows, G->E);
    cudaError_t err = encode_window(&p.ma, dy, N, G->rows, 2, &p.whole_a);
    if (err == cudaSuccess) err = encode_window(&p.mb, x, K, G->rows, cut.bn / cut.cg / 64, &p.whole_b);
    if (err == cudaSuccess && !fp32) {
        const uint64_t d[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)G->E}, st[2] = {(uint64_t)K, (uint64_t)N * K};
        const uint32_t b[3] = {32, 32, 1};
        err = encode(&p.mo, false, dw, 3, d, st, b, CU_TENSOR_MAP_SWIZZLE_64B);
    }
    if (err != cudaSuccess) return err;
    return launch_cut<kWgrad, kBf16>(p, cut, s);
}

}  // namespace moe
