// experts.h -- launchers of the expert products (include/moe_experts.h).
#pragma once

#include "common.cuh"
#include "moe_experts.h"

namespace moe {
cudaError_t launch_expert_linear(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                                 const float *w_scales, int N, const void *bias, int act, const void *residual,
                                 void *y, void *saved, void *saved_scales, cudaStream_t s);
cudaError_t launch_expert_linear_e4m3(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                                      const float *w_scales, int N, const void *bias, int act, const void *residual,
                                      void *y, void *saved, void *saved_scales, cudaStream_t s);
cudaError_t launch_expert_dgrad(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                                const void *saved, const void *saved_scales, void *dx, void *a, cudaStream_t s);
cudaError_t launch_expert_dgrad_saved(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                                      const void *saved, const void *saved_scales, void *dx, void *a, cudaStream_t s);
cudaError_t launch_expert_wgrad(const moe_rows *G, const void *dy, int N, const void *x, int K, void *dw, void *db,
                                int fp32, cudaStream_t s);
cudaError_t launch_act_backward(const moe_rows *G, const void *dy, int N, int act, const void *saved,
                                const void *saved_scales, void *du, void *a, cudaStream_t s);
}  // namespace moe
