// act_backward.cu -- beside the expert products: the gradient through
// an activation whose input was saved in 8 bits, where no product precedes it
// to take it into its epilogue.  Bound by HBM: each value is read once and
// written once.
#include "activation.cuh"
#include "experts.h"
#include "launchers.h"

namespace moe {

namespace {

// Rows in use: offsets[E], checked against the buffers.
__device__ __forceinline__ int rows_in_use(const int32_t *offsets, int E, int rows, void *ws)
{
    if (!offsets) return rows;
    const int R = offsets[E];
    if (R < 0 || R > rows) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_status(ws, MOE_ERR_DEVICE_DATA);
        return 0;
    }
    return R;
}

// A thread takes 8 consecutive output columns of a row (16 bytes of dy, 8
// codes) and walks rows and columns by the grid's stride.
__global__ void __launch_bounds__(256) act_backward_kernel(const __nv_bfloat16 *dy, int out, int act,
                                                           const uint8_t *saved, const uint8_t *scales,
                                                           __nv_bfloat16 *du, __nv_bfloat16 *a,
                                                           const int32_t *offsets, int E, int rows, void *ws)
{
    const int R = rows_in_use(offsets, E, rows, ws);
    const bool glu = act == MOE_ACT_SWIGLU;
    const int vecs = out / 8, N = glu ? 2 * out : out;
    const long long step = (long long)gridDim.x * 256;
    const int drow = (int)(step / vecs), dcol = (int)(step % vecs);
    const long long first = (long long)blockIdx.x * 256 + threadIdx.x;
    int row = (int)(first / vecs), col = (int)(first % vecs);
    while (row < R) {
        const size_t at = (size_t)row * out + col * 8, sat = (size_t)row * N + col * 8;
        const uint4 d4 = *reinterpret_cast<const uint4 *>(dy + at);
        const float d[8] = {bf16lo(d4.x), bf16hi(d4.x), bf16lo(d4.y), bf16hi(d4.y),
                            bf16lo(d4.z), bf16hi(d4.z), bf16lo(d4.w), bf16hi(d4.w)};
        const uint8_t *b = scales + (size_t)row * (N / 32) + col / 4;
        const uint2 c = *reinterpret_cast<const uint2 *>(saved + sat);
        float u[8], g[8], v[8];
        saved_decode4(c.x, saved_scale(b[0]), u);
        saved_decode4(c.y, saved_scale(b[0]), u + 4);
        if (glu) {
            const uint2 c2 = *reinterpret_cast<const uint2 *>(saved + sat + out);
            const float s2 = saved_scale(b[out / 32]);
            float up[8], gup[8];
            saved_decode4(c2.x, s2, up);
            saved_decode4(c2.y, s2, up + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = logistic(u[i]), silu = u[i] * q;
                g[i] = d[i] * up[i] * (q * (1.0f + u[i] * (1.0f - q)));
                gup[i] = d[i] * silu;
                v[i] = silu * up[i];
            }
            const uint2 lo = pack_bf16x4(gup), hi = pack_bf16x4(gup + 4);
            *reinterpret_cast<uint4 *>(du + sat + out) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[i] = d[i] * act_slope(u[i], act);
                v[i] = act_value(u[i], act);
            }
        }
        uint2 lo = pack_bf16x4(g), hi = pack_bf16x4(g + 4);
        *reinterpret_cast<uint4 *>(du + sat) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        if (a) {
            lo = pack_bf16x4(v);
            hi = pack_bf16x4(v + 4);
            *reinterpret_cast<uint4 *>(a + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        row += drow;
        col += dcol;
        if (col >= vecs) {
            col -= vecs;
            ++row;
        }
    }
}

}  // namespace

cudaError_t launch_act_backward(const moe_rows *G, const void *dy, int N, int act, const void *saved,
                                const void *saved_scales, void *du, void *a, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    const int out = act == MOE_ACT_SWIGLU ? N / 2 : N;
    long long blocks = ((long long)G->rows * (out / 8) + 255) / 256;
    const int most = resident_grid(reinterpret_cast<const void *>(act_backward_kernel), 256, 0);
    if (blocks > most) blocks = most;
    act_backward_kernel<<<(unsigned)blocks, 256, 0, s>>>(
        static_cast<const __nv_bfloat16 *>(dy), out, act, static_cast<const uint8_t *>(saved),
        static_cast<const uint8_t *>(saved_scales), static_cast<__nv_bfloat16 *>(du),
        static_cast<__nv_bfloat16 *>(a), G->offsets, G->E, G->rows, G->ws);
    return cudaGetLastError();
}

}  // namespace moe
