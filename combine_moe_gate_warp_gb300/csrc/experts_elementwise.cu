// experts_elementwise.cu -- beside the expert products: the gradient through
// an activation whose input was saved in 8 bits, and the bias gradient.  Both
// are bound by HBM: each value is read once and written once.
#include "activation.cuh"
#include "experts.h"
#include "launchers.h"
#include "umma.cuh"

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

// db[e, n] = sum of dy[r, n] over the expert's rows.  A cluster of 8 blocks
// takes 256 columns of one expert: each warp adds every 64th row (8 columns
// per lane), the block adds its warps, block 0 of the cluster adds the blocks
// over distributed shared memory.  The order is fixed by the sizes.
constexpr int kSumBlocks = 8;
__global__ void __cluster_dims__(kSumBlocks, 1, 1) __launch_bounds__(256)
    row_sums_kernel(const __nv_bfloat16 *dy, int N, void *db, int fp32, const int32_t *offsets, int E, int rows,
                    void *ws)
{
    __shared__ float part[8][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_cta_rank(), e = blockIdx.y, col0 = (int)(blockIdx.x / kSumBlocks) * 256;
    int lo = offsets ? offsets[e] : 0, hi = offsets ? offsets[e + 1] : rows;
    // an offset below an earlier one would give rows to two experts
    const bool low = offsets && (int)threadIdx.x <= e && lo < max(0, offsets[threadIdx.x]);
    if (__syncthreads_or(low) || hi < lo || hi > rows) {
        if (threadIdx.x == 0) record_status(ws, MOE_ERR_DEVICE_DATA);
        lo = hi = 0;
    }
    const int col = col0 + lane * 8;
    float s[8] = {};
    if (col < N) {
#pragma unroll 4
        for (int r = lo + rank * 8 + warp; r < hi; r += 8 * kSumBlocks) {
            const uint4 v = *reinterpret_cast<const uint4 *>(dy + (size_t)r * N + col);
            s[0] += bf16lo(v.x);
            s[1] += bf16hi(v.x);
            s[2] += bf16lo(v.y);
            s[3] += bf16hi(v.y);
            s[4] += bf16lo(v.z);
            s[5] += bf16hi(v.z);
            s[6] += bf16lo(v.w);
            s[7] += bf16hi(v.w);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][lane * 8 + i] = s[i];
    __syncthreads();
    float sum = 0.0f;
    for (int i = 0; i < 8; ++i) sum += part[i][threadIdx.x];
    __syncthreads();
    part[0][threadIdx.x] = sum;
    cluster_sync_all();
    if (rank == 0 && col0 + (int)threadIdx.x < N) {
        sum = 0.0f;
        for (int i = 0; i < kSumBlocks; ++i) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(v)
                         : "r"(cluster_addr(&part[0][threadIdx.x], (uint32_t)i))
                         : "memory");
            sum += v;
        }
        const size_t at = (size_t)e * N + col0 + threadIdx.x;
        if (fp32) static_cast<float *>(db)[at] = sum;
        else static_cast<__nv_bfloat16 *>(db)[at] = __float2bfloat16_rn(sum);
    }
    __syncwarp();
    cluster_sync_all();  // the peers' shared memory stays until it has been read
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

cudaError_t launch_row_sums(const moe_rows *G, const void *dy, int N, void *db, int fp32, cudaStream_t s)
{
    if (G->rows == 0) return cudaMemsetAsync(db, 0, (size_t)G->E * N * (fp32 ? 4 : 2), s);
    const dim3 grid((unsigned)((N + 255) / 256 * kSumBlocks), (unsigned)G->E);
    row_sums_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(dy), N, db, fp32, G->offsets, G->E,
                                         G->rows, G->ws);
    return cudaGetLastError();
}

}  // namespace moe
