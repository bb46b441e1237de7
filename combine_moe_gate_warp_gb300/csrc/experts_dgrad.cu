// experts_dgrad.cu -- the rows' gradients (experts.cuh).
#include "experts.cuh"

namespace moe {

cudaError_t launch_expert_dgrad(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                                const void *saved, const void *saved_scales, void *dx, void *a, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    if (act != MOE_ACT_NONE)
        return launch_expert_dgrad_saved(G, dy, N, w, K, act, saved, saved_scales, dx, a, s);
    return dgrad<kDgrad>(G, dy, N, w, K, act, saved, saved_scales, dx, a, s);
}

}  // namespace moe
