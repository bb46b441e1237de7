// experts.cu -- the experts' matrix products over the packed rows, on the
// tcgen05 tensor cores (include/moe_experts.h).
//
// One kernel serves the three products of a layer.  Every product is
// D[m, n] = sum_k A[m, k] * B[n, k]:
//
//                m                n               k
//   linear       output column    packed row      input column     (A = w, B = x)
//   dgrad        input column     packed row      output column    (A = w^T, B = dy)
//   wgrad        output column    input column    packed row       (A = dy^T, B = x^T)
//
// The ragged axis (an expert's rows) is n for the first two.  A matrix
// instruction takes any n that is a multiple of 16 (32 for a pair of SMs), so
// the last tile of an expert costs what its rows need, where rows on the m
// axis would fill 128 or 256.  For the same reason a decode step, a few rows
// per expert, runs the same way with a small n.
//
// A block is persistent: warp 0 loads tiles of 128 bytes of k with TMA into
// a ring of stages, warp 1 issues the matrix instructions into one of two
// accumulators in tensor memory, warps 4-7 drain the other one.  The blocks
// walk the tiles in a fixed order, derived from the offsets on the device;
// no result depends on timing.
#include <cudaTypedefs.h>
#include <stdint.h>

#include <atomic>

#include "activation.cuh"
#include "experts.h"
#include "launchers.h"
#include "umma.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kEpiWarp = 4;      // first epilogue warp
constexpr int kTileM = 128;      // rows of A per block
constexpr int kChunk = 16;       // accumulator columns staged at a time
constexpr int kStageA = kTileM * 128;  // bytes

constexpr int kLinear = 0, kDgrad = 1, kWgrad = 2;

__host__ __device__ constexpr int stage_bytes(int CG, int BN) { return kStageA + BN / CG * 128; }
constexpr int kStaging = 2 * kChunk * kTileM * 4;  // bytes
constexpr int kControl = 4096;
// ring depth: what is left of 227 KB beside the staging buffers, the barriers
// and tile counts, and the alignment to 1 KB; at most 12 stages
__host__ __device__ constexpr int stages(int CG, int BN)
{
    const int n = (227 * 1024 - kStaging - kControl - 1024) / stage_bytes(CG, BN);
    return n > 12 ? 12 : n;
}
__host__ __device__ constexpr int smem_bytes(int CG, int BN)
{
    return 1024 + stages(CG, BN) * stage_bytes(CG, BN) + kStaging + kControl;
}
__host__ __device__ constexpr int tmem_cols(int BN) { return 2 * BN < 32 ? 32 : 2 * BN; }

struct Params {
    CUtensorMap ma, mb;
    const int32_t *offsets;
    void *ws;
    int E, rows;
    int M;         // extent of m
    int N;         // wgrad: extent of n
    int K;         // linear, dgrad: extent of k, in bytes
    int act, glu;  // glu: A's rows alternate gate and up columns
    int fp32;
    const __nv_bfloat16 *bias, *residual;
    const float2 *x_scales, *w_scales;
    __nv_bfloat16 *y, *a;
    void *dw;
    uint8_t *saved, *saved_scales;
};

struct Control {
    uint64_t full[12], empty[12], acc_full[2], acc_empty[2], tail;
    uint32_t tmem;
    int abort;
    int part[8];
    int row0[MOE_MAX_EXPERTS], rows[MOE_MAX_EXPERTS];  // of each expert, checked
    int tile0[MOE_MAX_EXPERTS + 1];                    // its first tile
};
static_assert(sizeof(Control) <= kControl, "barriers and tile counts");

// Wait for phase `parity`, at most kSpinLimitNs.  False once the limit has
// passed or another role of the block has given up; then every role leaves
// its loop.
__device__ __forceinline__ bool poll(uint64_t *bar, uint32_t parity, Control *c, void *ws)
{
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    for (;;) {
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return true;
        if (*(volatile int *)&c->abort) return false;
        if (global_timer_ns() - t0 > kSpinLimitNs) {
            *(volatile int *)&c->abort = 1;
            record_status(ws, MOE_ERR_TIMEOUT);
            return false;
        }
    }
}

// The same for a whole warp, which goes on together.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Control *c, void *ws)
{
    return __all_sync(0xFFFFFFFFu, poll(bar, parity, c, ws));
}

struct Tile {
    int e, m, n, rows;  // expert, tile of m, tile of n, the expert's rows
    int row0;
};

// The tiles of a block pair in order.  Within an expert the tiles go through
// groups of 8 tiles of m, all tiles of n for each: the ~76 tiles in flight
// then share 8 panels of A and about 9 of B, near the least traffic.
struct Walk {
    const Control *c;
    int E, tm;  // tiles of m
    int tile, step, e;
    __device__ Walk(const Control *c_, int E_, int tm_, int first, int step_)
        : c(c_), E(E_), tm(tm_), tile(first), step(step_), e(0)
    {
    }
    __device__ bool next(Tile &t)
    {
        if (tile >= c->tile0[E]) return false;
        while (tile >= c->tile0[e + 1]) ++e;
        const int local = tile - c->tile0[e];
        const int tn = (c->tile0[e + 1] - c->tile0[e]) / tm;
        const int g = local / (8 * tn), in = local - g * 8 * tn;
        const int gm = min(8, tm - g * 8);
        t.e = e;
        t.n = in / gm;
        t.m = g * 8 + in - t.n * gm;
        t.row0 = c->row0[e];
        t.rows = c->rows[e];
        tile += step;
        return true;
    }
};

// Largest magnitude over 2^STEPS lanes, as bit patterns with the sign cleared
// (a NaN is then larger than any value).
template <int STEPS>
__device__ __forceinline__ unsigned lane_max(unsigned bits)
{
#pragma unroll
    for (int i = 0; i < STEPS; ++i) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1 << i));
    return bits;
}
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What one lane keeps for the 4 accumulator rows (columns of the output) it
// finishes in every row of a tile.
struct LaneColumns {
    int col;        // first output column (linear: of u; swiglu: of the gates)
    bool on;
    float bias[4];
    float ws[4], wsum[4];
};

// --------------------------------------------------------------------------
// linear: one output row r, four values of u (swiglu: gate, up, gate, up)
// --------------------------------------------------------------------------
template <bool FP8>
__device__ __forceinline__ void finish_linear(const Params &p, const LaneColumns &lc, int r, float4 v, int lane)
{
    float u[4] = {v.x, v.y, v.z, v.w};
    if (FP8) {
        const float2 xs = p.x_scales[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = fmaf(xs.x, lc.ws[i] * u[i], xs.y * lc.wsum[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] += lc.bias[i];
    const int out = p.glu ? p.M / 2 : p.M;
    if (p.saved) {
        if (p.glu) {  // 32 gates (and their ups) lie in 16 lanes
            const unsigned bg = saved_byte(lane_max<4>(lc.on ? max(mag(u[0]), mag(u[2])) : 0u));
            const unsigned bu = saved_byte(lane_max<4>(lc.on ? max(mag(u[1]), mag(u[3])) : 0u));
            if (lc.on) {
                const float ig = saved_inverse(bg), iu = saved_inverse(bu);
                uint8_t *s = p.saved + (size_t)r * p.M + lc.col;
                *reinterpret_cast<uint16_t *>(s) = (uint16_t)e4m3_pair(u[0] * ig, u[2] * ig);
                *reinterpret_cast<uint16_t *>(s + out) = (uint16_t)e4m3_pair(u[1] * iu, u[3] * iu);
                if ((lane & 15) == 0) {
                    uint8_t *b = p.saved_scales + (size_t)r * (p.M / 32) + lc.col / 32;
                    b[0] = (uint8_t)bg;
                    b[out / 32] = (uint8_t)bu;
                }
            }
        } else {
            const unsigned m4 = max(max(mag(u[0]), mag(u[1])), max(mag(u[2]), mag(u[3])));
            const unsigned by = saved_byte(lane_max<3>(lc.on ? m4 : 0u));
            if (lc.on) {
                const float inv = saved_inverse(by);
                *reinterpret_cast<unsigned *>(p.saved + (size_t)r * p.M + lc.col) =
                    e4m3_pair(u[0] * inv, u[1] * inv) | (e4m3_pair(u[2] * inv, u[3] * inv) << 16);
                if ((lane & 7) == 0) p.saved_scales[(size_t)r * (p.M / 32) + lc.col / 32] = (uint8_t)by;
            }
        }
    }
    if (!lc.on) return;
    const size_t at = (size_t)r * out + lc.col;
    if (p.glu) {
        float y0 = act_value(u[0], MOE_ACT_SILU) * u[1], y1 = act_value(u[2], MOE_ACT_SILU) * u[3];
        if (p.residual) {
            const unsigned q = *reinterpret_cast<const unsigned *>(p.residual + at);
            y0 += bf16lo(q);
            y1 += bf16hi(q);
        }
        *reinterpret_cast<unsigned *>(p.y + at) = pack_bf16(y0, y1);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = act_value(u[i], p.act);
        if (p.residual) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p.residual + at);
            u[0] += bf16lo(q.x);
            u[1] += bf16hi(q.x);
            u[2] += bf16lo(q.y);
            u[3] += bf16hi(q.y);
        }
        *reinterpret_cast<uint2 *>(p.y + at) = pack_bf16x4(u);
    }
}

// --------------------------------------------------------------------------
// dgrad: one row r, four columns of d, plain or through the saved layer
// --------------------------------------------------------------------------
__device__ __forceinline__ void finish_dgrad(const Params &p, const LaneColumns &lc, int r, float4 v)
{
    if (!lc.on) return;
    const float d[4] = {v.x, v.y, v.z, v.w};
    const size_t at = (size_t)r * p.M + lc.col;
    if (p.act == MOE_ACT_NONE) {
        *reinterpret_cast<uint2 *>(p.y + at) = pack_bf16x4(d);
        return;
    }
    const size_t C = p.act == MOE_ACT_SWIGLU ? 2 * (size_t)p.M : p.M;
    const uint8_t *s = p.saved + r * C + lc.col;
    const uint8_t *b = p.saved_scales + r * (C / 32) + lc.col / 32;
    __nv_bfloat16 *o = p.y + r * C + lc.col;
    float u[4], du[4], av[4];
    saved_decode4(*reinterpret_cast<const unsigned *>(s), saved_scale(b[0]), u);
    if (p.act == MOE_ACT_SWIGLU) {
        float up[4], dup[4];
        saved_decode4(*reinterpret_cast<const unsigned *>(s + p.M), saved_scale(b[p.M / 32]), up);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float q = logistic(u[i]), silu = u[i] * q;
            du[i] = d[i] * up[i] * (q * (1.0f + u[i] * (1.0f - q)));
            dup[i] = d[i] * silu;
            av[i] = silu * up[i];
        }
        *reinterpret_cast<uint2 *>(o + p.M) = pack_bf16x4(dup);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            du[i] = d[i] * act_slope(u[i], p.act);
            av[i] = act_value(u[i], p.act);
        }
    }
    *reinterpret_cast<uint2 *>(o) = pack_bf16x4(du);
    if (p.a) *reinterpret_cast<uint2 *>(p.a + at) = pack_bf16x4(av);
}

// --------------------------------------------------------------------------
// the kernel
// --------------------------------------------------------------------------
template <int CG, int BN, int MODE, bool FP8>
__global__ void __launch_bounds__(kThreads, 1) experts_kernel(const __grid_constant__ Params p)
{
    constexpr int kStages = stages(CG, BN);
    constexpr int kStage = stage_bytes(CG, BN);
    constexpr int kHalfN = BN / CG;  // rows of B per block
    constexpr int kBM = kTileM * CG;
    constexpr bool kMnA = MODE != kLinear, kMnB = MODE == kWgrad;
    constexpr int kStepN = CG == 2 ? 32 : 16;
    constexpr int kElems = FP8 ? 128 : 64;  // values of k per stage

    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    float *stg = reinterpret_cast<float *>(smem + kStages * kStage);
    Control *c = reinterpret_cast<Control *>(smem + kStages * kStage + kStaging);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0u;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&c->full[i], CG);
            mbar_init(&c->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c->acc_full[i], 1);
            mbar_init(&c->acc_empty[i], 4 * CG);
        }
        mbar_init(&c->tail, 1);
        c->abort = 0;
        mbar_fence_init();
        tmap_prefetch(&p.ma);
        tmap_prefetch(&p.mb);
    }
    if (warp == 2) tmem_alloc<CG>(&c->tmem, tmem_cols(BN));

    // rows and first tile of every expert: thread e looks at expert e
    const int tm = (p.M + kBM - 1) / kBM;
    {
        int lo = 0, hi = 0, tiles = 0;
        if (tid < p.E) {
            lo = p.offsets ? p.offsets[tid] : 0;
            hi = p.offsets ? p.offsets[tid + 1] : p.rows;
        }
        // the largest offset so far: rows below it belong to an earlier
        // expert, and two experts never write the same row
        int top = max(lo, hi);
#pragma unroll
        for (int i = 1; i < 32; i *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, top, i);
            if (lane >= i) top = max(top, v);
        }
        int before = __shfl_up_sync(0xFFFFFFFFu, top, 1);
        if (lane == 0) before = 0;
        if (lane == 31) c->part[warp] = top;
        __syncthreads();
        for (int i = 0; i < warp; ++i) before = max(before, c->part[i]);
        __syncthreads();
        if (tid < p.E) {
            if (lo < before || hi < lo || hi > p.rows) {
                if (blockIdx.x == 0) record_status(p.ws, MOE_ERR_DEVICE_DATA);
                lo = hi = 0;
            }
            tiles = tm * (((MODE == kWgrad ? p.N : hi - lo) + BN - 1) / BN);
            c->row0[tid] = lo;
            c->rows[tid] = hi - lo;
        }
        int sum = tiles;
#pragma unroll
        for (int i = 1; i < 32; i *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, i);
            if (lane >= i) sum += v;
        }
        if (lane == 31) c->part[warp] = sum;
        __syncthreads();
        for (int i = 0; i < warp; ++i) sum += c->part[i];
        if (tid < p.E) c->tile0[tid + 1] = sum;
        if (tid == 0) c->tile0[0] = 0;
    }
    __syncwarp();
    tc_fence_before();
    if (CG == 2) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem;

    Walk walk(c, p.E, tm, blockIdx.x / CG, gridDim.x / CG);
    Tile t;
    const auto iterations = [&](const Tile &q) {
        return MODE == kWgrad ? (q.rows + 63) / 64 : (p.K + 127) / 128;
    };
    // columns of the accumulator in use: what is left of the ragged axis
    const auto width = [&](const Tile &q) {
        const int left = (MODE == kWgrad ? p.N : q.rows) - q.n * BN;
        return min(BN, (left + kStepN - 1) / kStepN * kStepN);
    };

    if (warp == 0) {
        // ---- loads -------------------------------------------------------
        int s = 0;
        uint32_t ph = 0, tail_ph = 0;
        bool ok = true;
        while (ok && walk.next(t)) {
            const int iters = iterations(t);
            const int m0 = t.m * kBM + (int)rank * kTileM;
            const int n0 = t.n * BN + (int)rank * (width(t) / CG);
            for (int i = 0; i < iters; ++i) {
                ok = wait(&c->empty[s], ph ^ 1, c, p.ws);
                if (!ok) break;
                // the last rows of an expert do not fill 64 of k: the rows
                // after them are another expert's (or nobody's, with any
                // bits), and are zeroed in both tiles once they have landed
                const int keep = MODE == kWgrad ? t.rows - i * 64 : 64;
                const bool tail = keep < 64;
                unsigned char *sa = smem + s * kStage, *sb = sa + kStageA;
                const uint32_t full = cluster_addr(&c->full[s], 0);
                if (lane == 0) {
                    uint32_t bar = full;
                    if (tail) {
                        mbar_arrive_expect_tx(&c->tail, kStage);
                        bar = cluster_addr(&c->tail, rank);
                    } else {
                        mbar_arrive_expect_tx_cluster(full, kStage);
                    }
                    const int k0 = i * kElems;
                    if (MODE == kLinear) {
                        tma_load_4d<CG>(sa, &p.ma, k0, 0, p.glu ? m0 / 2 : m0, t.e, bar);
                        tma_load_2d<CG>(sb, &p.mb, k0, t.row0 + n0, bar);
                    } else if (MODE == kDgrad) {
                        for (int j = 0; j < 2; ++j)
                            tma_load_4d<CG>(sa + j * 8192, &p.ma, m0 + 64 * j, k0, t.e, 0, bar);
                        tma_load_2d<CG>(sb, &p.mb, k0, t.row0 + n0, bar);
                    } else {
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d<CG>(sa + j * 8192, &p.ma, m0 + 64 * j, t.row0 + k0, bar);
                        for (int j = 0; j < kHalfN / 64; ++j)
                            tma_load_2d<CG>(sb + j * 8192, &p.mb, n0 + 64 * j, t.row0 + k0, bar);
                    }
                }
                __syncwarp();
                if (MODE == kWgrad && tail) {
                    ok = wait(&c->tail, tail_ph, c, p.ws);
                    if (!ok) break;
                    tail_ph ^= 1;
                    // row k of a tile is the 128 bytes at 128 * k of each 8 KB
                    for (int j = 0; j < 2 + kHalfN / 64; ++j)
                        for (int o = keep * 128 + lane * 16; o < 8192; o += 512)
                            *reinterpret_cast<uint4 *>(sa + j * 8192 + o) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(full);
                }
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        // every stage read: no copy and no arrival is on its way to this
        // block's shared memory when it ends
        for (int i = 0; ok && i < kStages; ++i) {
            ok = wait(&c->empty[s], ph ^ 1, c, p.ws);
            if (++s == kStages) {
                s = 0;
                ph ^= 1;
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---- matrix instructions ------------------------------------------
        constexpr uint32_t kLeadA = kMnA ? 8192 : 16, kLeadB = kMnB ? 8192 : 16;
        constexpr uint32_t kStepA = (kMnA ? 2048 : 32) >> 4, kStepB = (kMnB ? 2048 : 32) >> 4;
        int s = 0, acc = 0;
        uint32_t ph = 0, aph = 0;
        bool ok = true;
        while (ok && walk.next(t)) {
            const int iters = iterations(t);
            if (iters == 0) continue;
            const uint32_t idesc = mma_idesc(FP8, kMnA, kMnB, kBM, width(t));
            ok = wait(&c->acc_empty[acc], aph ^ 1, c, p.ws);
            if (!ok) break;
            tc_fence_after();
            for (int i = 0; i < iters; ++i) {
                ok = wait(&c->full[s], ph, c, p.ws);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t sa = smem_addr(smem + s * kStage);
                    const uint64_t da = smem_desc(sa, kLeadA, 1024), db = smem_desc(sa + kStageA, kLeadB, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss<CG, FP8>(tmem + acc * BN, da + k * kStepA, db + k * kStepB, idesc, (i | k) != 0);
                    mma_commit<CG>(&c->empty[s]);
                    if (i == iters - 1) mma_commit<CG>(&c->acc_full[acc]);
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            acc ^= 1;
            aph ^= acc == 0;
        }
    } else if (warp >= kEpiWarp) {
        // ---- epilogue ------------------------------------------------------
        const int q = warp - kEpiWarp;  // == warp % 4: the lanes of tensor memory it may read
        int acc = 0, buf = 0;
        uint32_t aph = 0;
        while (walk.next(t)) {
            const int iters = iterations(t);
            const int m0 = t.m * kBM + (int)rank * kTileM, n0 = t.n * BN;
            const int cols = min(BN, (MODE == kWgrad ? p.N : t.rows) - n0);
            if (iters != 0) {
                // all four warps go on, or none
                const bool ok = wait(&c->acc_full[acc], aph, c, p.ws);
                int all;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                             "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(all)
                             : "r"((int)ok)
                             : "memory");
                if (!all) break;
                tc_fence_after();
            }
            const uint32_t from = tmem + ((uint32_t)(q * 32) << 16) + acc * BN;
            LaneColumns lc;
            if (MODE != kWgrad) {
                lc.col = p.glu ? m0 / 2 + 2 * lane : m0 + 4 * lane;
                const int half = p.M / 2;
                lc.on = lc.col < (p.glu ? half : p.M);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = p.glu ? (i & 1) * half + lc.col + (i >> 1) : lc.col + i;
                    const size_t at = (size_t)t.e * p.M + row;
                    lc.bias[i] = MODE == kLinear && p.bias && lc.on ? __bfloat162float(p.bias[at]) : 0.0f;
                    const float2 w = FP8 && lc.on ? p.w_scales[at] : make_float2(0.0f, 0.0f);
                    lc.ws[i] = w.x;
                    lc.wsum[i] = w.y;
                }
            }
            for (int c0 = 0; c0 < cols; c0 += kChunk) {
                uint32_t v[kChunk];
                if (iters != 0) {
                    tmem_ld16(from + c0, v);
                    tmem_wait_ld();
                    if (c0 + kChunk >= cols) {  // the accumulator is free again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(cluster_addr(&c->acc_empty[acc], 0));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[i] = 0u;
                }
                if (MODE == kWgrad) {
                    // lane = one row of dw, 16 consecutive values of it
                    const int m = m0 + q * 32 + lane;
                    if (m < p.M) {
                        const size_t at = ((size_t)t.e * p.M + m) * p.N + n0 + c0;
#pragma unroll
                        for (int j = 0; j < kChunk; j += 8) {
                            if (c0 + j >= cols) break;
                            float f[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[j + i]);
                            if (p.fp32) {
                                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.dw) + at + j);
                                o[0] = make_float4(f[0], f[1], f[2], f[3]);
                                o[1] = make_float4(f[4], f[5], f[6], f[7]);
                            } else {
                                const uint2 lo = pack_bf16x4(f), hi = pack_bf16x4(f + 4);
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.dw) + at + j) =
                                    make_uint4(lo.x, lo.y, hi.x, hi.y);
                            }
                        }
                    }
                } else {
                    // lane = one column of the output, 16 rows: transposed
                    // through shared memory, then a warp finishes whole rows
                    float *b = stg + buf * (kChunk * kTileM);
                    buf ^= 1;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) b[i * kTileM + q * 32 + lane] = __uint_as_float(v[i]);
                    asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
                    for (int i = q; i < kChunk && c0 + i < cols; i += 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(b + i * kTileM + lane * 4);
                        const int r = t.row0 + n0 + c0 + i;
                        if (MODE == kLinear) finish_linear<FP8>(p, lc, r, u, lane);
                        else finish_dgrad(p, lc, r, u);
                    }
                }
            }
            if (iters != 0) {
                acc ^= 1;
                aph ^= acc == 0;
            }
        }
    }
    __syncwarp();
    if (*(volatile int *)&c->abort) {
        // given up: leave the copies and products in flight time to land
        const unsigned long long t0 = global_timer_ns();
        for (int i = 0; i < 100000 && global_timer_ns() - t0 < 1000000ull; ++i) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    if (CG == 2) cluster_sync_all();
    else __syncthreads();
    if (warp == 2) tmem_free<CG>(tmem, tmem_cols(BN));
}

// --------------------------------------------------------------------------
// host side
// --------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::atomic<void *> cached{nullptr};
    void *f = cached.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// A map of `rank` axes, innermost first; strides in values, of axes 1 and up.
cudaError_t encode(CUtensorMap *m, bool fp8, const void *base, int rank, const uint64_t *dims,
                   const uint64_t *strides, const uint32_t *box)
{
    const auto fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t d[4], st[3];
    cuuint32_t b[4], one[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i) st[i - 1] = strides[i - 1] * (fp8 ? 1 : 2);
    }
    const CUresult r =
        fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
           const_cast<void *>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_rows(CUtensorMap *m, bool fp8, const void *base, int cols, int rows, int box_cols, int box_rows)
{
    const uint64_t d[2] = {(uint64_t)cols, (uint64_t)rows}, st[1] = {(uint64_t)cols};
    const uint32_t b[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
    return encode(m, fp8, base, 2, d, st, b);
}

template <int CG, int BN, int MODE, bool FP8>
cudaError_t launch(const Params &p, cudaStream_t s)
{
    // No programmatic dependent launch here: the kernel takes whole SMs and
    // their tensor memory, so the next one has nowhere to start early.
    const auto fn = experts_kernel<CG, BN, MODE, FP8>;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(fn), smem_bytes(CG, BN));
    if (err != cudaSuccess) return err;
    // the most tiles that offsets over these rows can give
    const long long tm = (p.M + kTileM * CG - 1) / (kTileM * CG);
    const long long tn = MODE == kWgrad ? (long long)p.E * ((p.N + BN - 1) / BN)
                                        : p.rows / BN + (p.rows < p.E ? p.rows : p.E);
    long long blocks = device_sm_count() / CG;
    if (tm * tn < blocks) blocks = tm * tn;
    if (blocks < 1) blocks = 1;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * CG));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(CG, BN);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

// Tile width along the ragged axis: the rows an expert has on average.
int pick_width(int rows, int E)
{
    const int mean = rows / E;
    return mean <= 32 ? 32 : mean <= 128 ? 128 : 256;
}

}  // namespace

cudaError_t launch_expert_linear(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                                 const float *w_scales, int N, const void *bias, int act, const void *residual,
                                 void *y, void *saved, void *saved_scales, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    const bool fp8 = x_scales != nullptr;
    Params p = {};
    p.offsets = G->offsets;
    p.ws = G->ws;
    p.E = G->E;
    p.rows = G->rows;
    p.M = N;
    p.K = fp8 ? K : 2 * K;
    p.act = act;
    p.glu = act == MOE_ACT_SWIGLU;
    p.bias = static_cast<const __nv_bfloat16 *>(bias);
    p.residual = static_cast<const __nv_bfloat16 *>(residual);
    p.x_scales = reinterpret_cast<const float2 *>(x_scales);
    p.w_scales = reinterpret_cast<const float2 *>(w_scales);
    p.y = static_cast<__nv_bfloat16 *>(y);
    p.saved = static_cast<uint8_t *>(saved);
    p.saved_scales = static_cast<uint8_t *>(saved_scales);
    const int bn = pick_width(G->rows, G->E), cg = bn == 256 ? 2 : 1, elems = fp8 ? 128 : 64;
    // w as [E][N/halves][halves][K] with the halves inside: one load brings
    // gate and up rows alternating, so that a pair of them ends in one lane
    const uint64_t h = p.glu ? 2 : 1, n = (uint64_t)N / h;
    const uint64_t d[4] = {(uint64_t)K, h, n, (uint64_t)G->E};
    const uint64_t st[3] = {n * K, (uint64_t)K, (uint64_t)N * K};
    const uint32_t b[4] = {(uint32_t)elems, (uint32_t)h, (uint32_t)(kTileM / h), 1};
    cudaError_t err = encode(&p.ma, fp8, w, 4, d, st, b);
    if (err == cudaSuccess) err = encode_rows(&p.mb, fp8, x, K, G->rows, elems, bn / cg);
    if (err != cudaSuccess) return err;
    if (fp8)
        return bn == 32    ? launch<1, 32, kLinear, true>(p, s)
               : bn == 128 ? launch<1, 128, kLinear, true>(p, s)
                           : launch<2, 256, kLinear, true>(p, s);
    return bn == 32    ? launch<1, 32, kLinear, false>(p, s)
           : bn == 128 ? launch<1, 128, kLinear, false>(p, s)
                       : launch<2, 256, kLinear, false>(p, s);
}

cudaError_t launch_expert_dgrad(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                                const void *saved, const void *saved_scales, void *dx, void *a, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    Params p = {};
    p.offsets = G->offsets;
    p.ws = G->ws;
    p.E = G->E;
    p.rows = G->rows;
    p.M = K;
    p.K = 2 * N;
    p.act = act;
    p.y = static_cast<__nv_bfloat16 *>(dx);
    p.a = static_cast<__nv_bfloat16 *>(a);
    p.saved = static_cast<uint8_t *>(const_cast<void *>(saved));
    p.saved_scales = static_cast<uint8_t *>(const_cast<void *>(saved_scales));
    const int bn = pick_width(G->rows, G->E), cg = bn == 256 ? 2 : 1;
    const uint64_t d[4] = {(uint64_t)K, (uint64_t)N, (uint64_t)G->E, 1};
    const uint64_t st[3] = {(uint64_t)K, (uint64_t)N * K, (uint64_t)N * K};
    const uint32_t b[4] = {64, 64, 1, 1};
    cudaError_t err = encode(&p.ma, false, w, 4, d, st, b);
    if (err == cudaSuccess) err = encode_rows(&p.mb, false, dy, N, G->rows, 64, bn / cg);
    if (err != cudaSuccess) return err;
    return bn == 32    ? launch<1, 32, kDgrad, false>(p, s)
           : bn == 128 ? launch<1, 128, kDgrad, false>(p, s)
                       : launch<2, 256, kDgrad, false>(p, s);
}

cudaError_t launch_expert_wgrad(const moe_rows *G, const void *dy, int N, const void *x, int K, void *dw, int fp32,
                                cudaStream_t s)
{
    if (G->rows == 0) return cudaMemsetAsync(dw, 0, (size_t)G->E * N * K * (fp32 ? 4 : 2), s);
    Params p = {};
    p.offsets = G->offsets;
    p.ws = G->ws;
    p.E = G->E;
    p.rows = G->rows;
    p.M = N;
    p.N = K;
    p.fp32 = fp32;
    p.dw = dw;
    cudaError_t err = encode_rows(&p.ma, false, dy, N, G->rows, 64, 64);
    if (err == cudaSuccess) err = encode_rows(&p.mb, false, x, K, G->rows, 64, 64);
    if (err != cudaSuccess) return err;
    // few tiles: one SM per tile of half the size keeps more of them busy
    const long long pairs = (long long)G->E * ((N + 255) / 256) * ((K + 255) / 256);
    return pairs * 2 <= device_sm_count() ? launch<1, 128, kWgrad, false>(p, s) : launch<2, 256, kWgrad, false>(p, s);
}

}  // namespace moe
