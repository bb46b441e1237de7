/*
 * moe_experts.h -- C ABI of libmoeroute's expert products, what stands
 * between moe_dispatch and moe_combine:
 *
 *     moe_dispatch -> moe_expert_linear (in) -> moe_expert_linear (out) -> moe_combine
 *
 * matrix products grouped by expert over the packed rows, with bias,
 * activation and residual in the epilogue, their gradients, and the hidden
 * layer saved in 8 bits between the passes.  A single group of rows gives
 * the shared experts' plain products.
 *
 * Conventions: those of moe_route.h (device pointers owned by the caller,
 * 16-byte aligned; asynchronous on `stream`; argument errors found on the
 * host before anything is enqueued; device-detected problems recorded in the
 * workspace and read with moe_get_status()).  Row-major, contiguous.  Sums
 * are held in fp32 and rounded once, to nearest even, as they are written.
 *
 * Supported range: 1 <= E <= 256, 0 <= rows < 2^30, K and N multiples of 8
 * up to 2^20 (K a multiple of 16 for e4m3; N a multiple of 16 with
 * MOE_ACT_SWIGLU; a saved layer's columns a multiple of 32, 64 with
 * MOE_ACT_SWIGLU), E * N < 2^31.  Anything else is MOE_ERR_UNSUPPORTED.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations.  A product with N columns gives N output columns, and N / 2
 * with MOE_ACT_SWIGLU, whose columns are F = N / 2 gates and then F ups. */
#define MOE_ACT_NONE 0
#define MOE_ACT_SILU 1   /* u / (1 + exp(-u)) */
#define MOE_ACT_GELU 2   /* u (1 + erf(u / sqrt 2)) / 2 */
#define MOE_ACT_SWIGLU 3 /* silu(gate) * up */

/*
 * The rows of a call: rows offsets[e] .. offsets[e+1]-1 belong to expert e,
 * as moe_dispatch_layout leaves them (R = offsets[E] <= rows; an expert may
 * have none).  offsets == NULL: all `rows` rows are one group (E == 1).
 * Row buffers hold `rows` rows; rows >= R are neither read for a result nor
 * written.  An expert whose offsets are negative, pass `rows`, decrease or
 * start below an earlier offset is treated as empty, and recorded as
 * MOE_ERR_DEVICE_DATA.
 */
typedef struct moe_rows {
    int32_t rows, E;
    const int32_t *offsets; /* [E+1] device, or NULL */
    void *ws;               /* a workspace (its status word): >= 8192 bytes, moe_workspace_init() */
} moe_rows;

/*
 * moe_expert_linear -- for the rows r of each expert e:
 *     u[r, n] = sum_k x[r, k] * w[e, n, k] + bias[e, n]
 *     y[r]    = act(u[r]) + residual[r]
 *
 *   x         [rows, K] bf16, or uint8 e4m3 codes with x_scales [rows, 2] fp32
 *             (scale, zero), as moe_dispatch packs them (x_scales != NULL):
 *             x = zero + scale * code.
 *   w         [E, N, K] bf16, or (with x_scales) uint8 e4m3 codes with
 *             w_scales [E, N, 2] fp32: w = scale * code, and sum = the sum
 *             over k of scale * code.  Then u = xs*(ws*acc) + zero*sum with
 *             acc = sum_k of the codes' products.
 *   bias      [E, N] bf16 or NULL.
 *   residual  [rows, out] bf16 or NULL, out = N, or N / 2 with MOE_ACT_SWIGLU.
 *   y     out [rows, out] bf16.
 *   saved, saved_scales  out, or both NULL: u in 8 bits, for the backward
 *             pass: uint8 e4m3 codes [rows, N] and scale bytes [rows, N/32].
 *             32 consecutive columns of a row share the scale 2^(byte - 127),
 *             the smallest power of two (not below 2^-127) with
 *             max |u| <= 448 * scale; code = e4m3 RNE(u / scale).  Byte 255:
 *             the block holds a NaN or an infinity and decodes as NaN.
 */
moe_status moe_expert_linear(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                             const float *w_scales, int N, const void *bias, int act, const void *residual, void *y,
                             void *saved, void *saved_scales, moe_stream_t stream);

/*
 * moe_expert_dgrad -- the gradient with respect to the rows:
 *     d[r, k] = sum_n dy[r, n] * w[e, n, k]
 *   dy [rows, N] bf16, w [E, N, K] bf16.
 *   act == MOE_ACT_NONE: dx out [rows, K] bf16 = d; saved and a are NULL.
 *   else: the product's input was act(u) with u saved (saved [rows, C],
 *   saved_scales [rows, C/32]; C = K, or 2K with MOE_ACT_SWIGLU), and the
 *   gradient goes on through it: dx out [rows, C] bf16 = d * act'(u) (d in
 *   fp32), a out (or NULL) [rows, K] bf16 = act(u).
 */
moe_status moe_expert_dgrad(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                            const void *saved, const void *saved_scales, void *dx, void *a, moe_stream_t stream);

/*
 * moe_expert_wgrad -- the gradients with respect to weights and bias:
 *     dw[e, n, k] = sum over the expert's rows of dy[r, n] * x[r, k]
 *     db[e, n]    = sum over the expert's rows of dy[r, n]
 *   dy [rows, N] bf16, x [rows, K] bf16; dw out [E, N, K], db out [E, N] or
 *   NULL, both bf16, or fp32 if `fp32`.  An expert without rows gets zeros.
 *   The order of the sums depends on the sizes only.
 */
moe_status moe_expert_wgrad(const moe_rows *G, const void *dy, int N, const void *x, int K, void *dw, void *db,
                            int fp32, moe_stream_t stream);

/*
 * moe_act_backward -- the gradient through an activation whose input was
 * saved: du[r] = dy[r] * act'(u[r]), and a[r] = act(u[r]) (or NULL).
 *   dy [rows, out] bf16, saved [rows, N], saved_scales [rows, N/32],
 *   du out [rows, N] bf16, a out [rows, out] bf16.
 */
moe_status moe_act_backward(const moe_rows *G, const void *dy, int N, int act, const void *saved,
                            const void *saved_scales, void *du, void *a, moe_stream_t stream);

/*
 * moe_expert_cut -- how the product of these sizes is cut on the current
 * device, for tests and for tuning; nothing is launched.
 *   cut  out [3], on the host: SMs of a tile (2: a pair), packed rows per
 *        tile (wgrad: columns of x), blocks that share a tile's sums; zeros
 *        without rows.
 */
#define MOE_EXPERT_LINEAR 0
#define MOE_EXPERT_DGRAD 1
#define MOE_EXPERT_WGRAD 2
moe_status moe_expert_cut(int product, int e4m3, int rows, int E, int K, int N, int32_t *cut);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
