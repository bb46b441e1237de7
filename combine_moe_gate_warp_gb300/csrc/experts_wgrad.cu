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
    p.sectors = !fp32 && K % 16 == 0 && reinterpret_cast<uintptr_t>(dw) % 32 == 0;
    p.db = db;
    const Cut cut = pick(N, K, G->E, true, (G->rows / G->E + 63) / 64, false);
    cudaError_t err = encode_mn(&p.ma, dy, N, G->rows, 1, 2, &p.whole_a);
    if (err == cudaSuccess) err = encode_mn(&p.mb, x, K, G->rows, 1, cut.bn / cut.cg / 64, &p.whole_b);
    if (err != cudaSuccess) return err;
    return launch_cut<kWgrad, false>(p, cut, s);
}

}  // namespace moe
