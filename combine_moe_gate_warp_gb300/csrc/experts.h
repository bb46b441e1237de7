// experts.h -- launchers of the expert products (include/moe_experts.h).
#pragma once

#include "common.cuh"
#include "moe_experts.h"

namespace moe {
// How a product is cut: SMs of a tile (2: a pair, 256 of m; 1: 128), columns
// of n per tile, and blocks that share a tile's k.
struct Cut {
    int cg, bn, split;
};
// linear and dgrad: m output columns of `rows` rows, k_stages of 128 bytes
Cut rows_cut(int m, int rows, int E, long long k_stages);
// rows and weights in 4 bits: scales take the tensor memory of a wider tile
constexpr int kFp4Wide = 224;
Cut rows_cut_fp4(int m, int rows, int E, long long k_stages);
Cut wgrad_cut(int N, int K, int rows, int E);

cudaError_t launch_expert_linear(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                                 const float *w_scales, int N, const void *bias, int act, const void *residual,
                                 void *y, void *saved, void *saved_scales, cudaStream_t s);
cudaError_t launch_expert_linear_e4m3(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                                      const float *w_scales, int N, const void *bias, int act, const void *residual,
                                      void *y, void *saved, void *saved_scales, cudaStream_t s);
cudaError_t launch_expert_linear_fp4(const moe_rows *G, const void *x, const void *x_scales, int K, const void *w,
                                     const void *w_scales, int N, const void *bias, int act, const void *residual,
                                     void *y, cudaStream_t s);
cudaError_t launch_expert_dgrad(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                                const void *saved, const void *saved_scales, void *dx, void *a, cudaStream_t s);
cudaError_t launch_expert_dgrad_saved(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                                      const void *saved, const void *saved_scales, void *dx, void *a, cudaStream_t s);
cudaError_t launch_expert_wgrad(const moe_rows *G, const void *dy, int N, const void *x, int K, void *dw, void *db,
                                int fp32, cudaStream_t s);
cudaError_t launch_act_backward(const moe_rows *G, const void *dy, int N, int act, const void *saved,
                                const void *saved_scales, void *du, void *a, cudaStream_t s);
cudaError_t launch_quantize_fp4(const moe_rows *G, const void *rows, int K, void *codes, void *scales, cudaStream_t s);
cudaError_t launch_dequantize_fp4(const moe_rows *G, const void *codes, const void *scales, int K, void *rows,
                                  cudaStream_t s);
}  // namespace moe
