// experts_linear_fp4.cu -- the expert products from rows and weights in 4 bits
// (experts.cuh).
#include "experts.cuh"

namespace moe {

cudaError_t launch_expert_linear_fp4(const moe_rows *G, const void *x, const void *x_scales, int K, const void *w,
                                     const void *w_scales, int N, const void *bias, int act, const void *residual,
                                     void *y, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    return linear<kFp4>(G, x, x_scales, K, w, w_scales, N, bias, act, residual, y, nullptr, nullptr, s);
}

}  // namespace moe
