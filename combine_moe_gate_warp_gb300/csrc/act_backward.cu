// act_backward.cu -- beside the expert products: the gradient through
// an activation whose input was saved in 8 bits, where no product precedes it
// to take it into its epilogue.  Bound by HBM: each value is read once and
// written once.
#include "activation.cuh"
#include "experts.h"
#include "launchers.h"

namespace moe {

namespace {

// The rows that belong to an expert, by the same rules as in the products.
// Where the offsets rise and stay inside the buffers they are one span.
// Where not, the experts that break a rule are empty, and a row is looked up
// among the others.
struct Members {
    int lo[MOE_MAX_EXPERTS], hi[MOE_MAX_EXPERTS];
};
// First and last row to look at; true if every row between them is a member.
// For the whole block of at least MOE_MAX_EXPERTS threads.
__device__ __forceinline__ bool members(const int32_t *offsets, int E, int rows, void *ws, Members &m, int &first,
                                        int &last)
{
    first = 0;
    last = rows;
    if (!offsets) return true;
    const int e = threadIdx.x;
    int lo = 0, hi = 0;
    if (e < E) {
        lo = offsets[e];
        hi = offsets[e + 1];
    }
    if (__syncthreads_and(e >= E || (lo >= 0 && hi >= lo && hi <= rows))) {
        first = offsets[0];
        last = offsets[E];
        return true;
    }
    if (e < E) {
        int before = 0;  // rows below the largest offset so far are an earlier expert's
        for (int i = 0; i <= e; ++i) before = max(before, offsets[i]);
        if (lo < before || hi < lo || hi > rows) {
            if (blockIdx.x == 0) record_status(ws, MOE_ERR_DEVICE_DATA);
            lo = hi = 0;
        }
        m.lo[e] = lo;
        m.hi[e] = hi;
    }
    __syncthreads();
    return false;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float *f)
{
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo(w[i]);
        f[2 * i + 1] = bf16hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float *f)
{
    const uint2 lo = pack_bf16x4(f), hi = pack_bf16x4(f + 4);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// A thread takes 16 consecutive output columns of a row (32 bytes of dy, 16
// codes: half of a block) and walks rows and columns by the grid's stride.
// 5000 rows of 4096 silu columns, 103 MB: 18.7 us (5.5 TB/s).
__global__ void __launch_bounds__(256) act_backward_kernel(const __nv_bfloat16 *dy, int out, int act,
                                                           const uint8_t *saved, const uint8_t *scales,
                                                           __nv_bfloat16 *du, __nv_bfloat16 *a,
                                                           const int32_t *offsets, int E, int rows, void *ws)
{
    static_assert(MOE_MAX_EXPERTS <= 256, "a thread looks at an expert");
    __shared__ Members m;
    int start, last;
    const bool all = members(offsets, E, rows, ws, m, start, last);
    const bool glu = act == MOE_ACT_SWIGLU;
    const int vecs = out / 16, N = glu ? 2 * out : out;
    const long long step = (long long)gridDim.x * 256;
    const int drow = (int)(step / vecs), dcol = (int)(step % vecs);
    const long long first = (long long)blockIdx.x * 256 + threadIdx.x;
    int row = start + (int)(first / vecs), col = (int)(first % vecs);
    const auto advance = [&] {
        row += drow;
        col += dcol;
        if (col >= vecs) {
            col -= vecs;
            ++row;
        }
    };
    for (; row < last; advance()) {
        if (!all) {
            bool mine = false;
            for (int e = 0; e < E; ++e) mine |= row >= m.lo[e] && row < m.hi[e];
            if (!mine) continue;
        }
        const size_t at = (size_t)row * out + col * 16, sat = (size_t)row * N + col * 16;
        const uint8_t *b = scales + (size_t)row * (N / 32) + col / 2;
        const uint4 d0 = *reinterpret_cast<const uint4 *>(dy + at), d1 = *reinterpret_cast<const uint4 *>(dy + at + 8);
        const uint4 c = *reinterpret_cast<const uint4 *>(saved + sat);
        uint4 c2 = make_uint4(0, 0, 0, 0);
        unsigned b2 = 0;
        if (glu) {
            c2 = *reinterpret_cast<const uint4 *>(saved + sat + out);
            b2 = b[out / 32];
        }
        const float s = saved_scale(b[0]), s2 = saved_scale(b2);
        const unsigned cw[4] = {c.x, c.y, c.z, c.w}, cw2[4] = {c2.x, c2.y, c2.z, c2.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float d[8], u[8], g[8], v[8];
            unpack8(h ? d1 : d0, d);
            saved_decode4(cw[2 * h], s, u);
            saved_decode4(cw[2 * h + 1], s, u + 4);
            if (glu) {
                float up[8], gup[8];
                saved_decode4(cw2[2 * h], s2, up);
                saved_decode4(cw2[2 * h + 1], s2, up + 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float q = logistic(u[i]), silu = u[i] * q;
                    g[i] = d[i] * up[i] * (q * (1.0f + u[i] * (1.0f - q)));
                    gup[i] = d[i] * silu;
                    v[i] = silu * up[i];
                }
                *reinterpret_cast<uint4 *>(du + sat + out + h * 8) = pack8(gup);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    g[i] = d[i] * act_slope(u[i], act);
                    v[i] = a ? act_value(u[i], act) : 0.0f;
                }
            }
            *reinterpret_cast<uint4 *>(du + sat + h * 8) = pack8(g);
            if (a) *reinterpret_cast<uint4 *>(a + at + h * 8) = pack8(v);
        }
    }
}

}  // namespace

cudaError_t launch_act_backward(const moe_rows *G, const void *dy, int N, int act, const void *saved,
                                const void *saved_scales, void *du, void *a, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    const int out = act == MOE_ACT_SWIGLU ? N / 2 : N;
    long long blocks = ((long long)G->rows * (out / 16) + 255) / 256;
    const int most = resident_grid(reinterpret_cast<const void *>(act_backward_kernel), 256, 0);
    if (blocks > most) blocks = most;
    act_backward_kernel<<<(unsigned)blocks, 256, 0, s>>>(
        static_cast<const __nv_bfloat16 *>(dy), out, act, static_cast<const uint8_t *>(saved),
        static_cast<const uint8_t *>(saved_scales), static_cast<__nv_bfloat16 *>(du),
        static_cast<__nv_bfloat16 *>(a), G->offsets, G->E, G->rows, G->ws);
    return cudaGetLastError();
}

}  // namespace moe
