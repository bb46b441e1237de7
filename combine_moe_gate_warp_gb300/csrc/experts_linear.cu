// experts_linear.cu -- the expert products from bf16 rows (experts.cuh).
#include "experts.cuh"

namespace moe {

cudaError_t launch_expert_linear(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                                 const float *w_scales, int N, const void *bias, int act, const void *residual,
                                 void *y, void *saved, void *saved_scales, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    if (x_scales)
        return launch_expert_linear_e4m3(G, x, x_scales, K, w, w_scales, N, bias, act, residual, y, saved, saved_scales, s);
    return linear<kBf16>(G, x, x_scales, K, w, w_scales, N, bias, act, residual, y, saved, saved_scales, s);
}

}  // namespace moe
