// experts_dgrad_saved.cu -- the rows' gradients through a saved layer (experts.cuh).
#include "experts.cuh"

namespace moe {

cudaError_t launch_expert_dgrad_saved(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                                      const void *saved, const void *saved_scales, void *dx, void *a, cudaStream_t s)
{
    return dgrad<kDgradSaved>(G, dy, N, w, K, act, saved, saved_scales, dx, a, s);
}

}  // namespace moe
