// experts.cuh -- the experts' matrix products over the packed rows, on the
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
// accumulators in tensor memory, and two groups of four warps (4-11) drain the
// other one.  The blocks walk the tiles in a fixed order, derived from the
// offsets on the device; no result depends on timing.
//
// What bounds it, on a GB300 (single launches; cards differ by up to 6 %):
//   linear, 56902 rows, 32 experts, 2048 -> 2 x 1024 swiglu   257-267 us, tensor
//     pipe 87 % busy, 1.8 PFLOP/s: the matrix instructions.  Back to back for
//     seconds the power limit lowers the clock: 306 us and more
//   dgrad, 31918 rows, 16 experts, 5120 -> 2560               450-477 us, 86 %
//   wgrad, the same                                           460 us, 85 %
//   linear, 128 rows, 32 experts, 2048 -> 2 x 1024            47 us, 5.7 TB/s:
//     the weights' bytes (and 6 us to start and to finish)
//   linear in 4 bits, 65536 rows, 16 experts, 5120 -> 2 x 2048 swiglu  465 us,
//     5.9 PFLOP/s (432 us in a row on two sets of inputs, 6.4); one expert, 8192
//     -> 8192: 1270 us, 6.9 PFLOP/s: the matrix instructions and the way of
//     their scales; below some 3000 of k the epilogue: 224 us at 256, 232 at
//     1024, 262 at 2048
//   linear in 4 bits, 128 rows, 32 experts, 2048 -> 2 x 2048   29 us, 4.9 TB/s
//   linear, 512 rows, 8 experts, 512 -> 2 x 256               6 us from the
//     first instruction to the last: 0.8 for offsets and barriers, 1 until the
//     first bytes, 2 for 8 stages, 1.5 for the epilogue
#pragma once

#include <cudaTypedefs.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "activation.cuh"
#include "experts.h"
#include "launchers.h"
#include "umma.cuh"

namespace moe {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarp = 4;            // first epilogue warp; two groups of four follow
constexpr int kTileM = 128;            // rows of A per block
constexpr int kStageA = kTileM * 128;  // bytes

constexpr int kLinear = 0, kDgrad = 1, kWgrad = 2, kDgradSaved = 3;
// what the operands are: bf16, e4m3 (whose scales the epilogue applies), or
// e2m1 with a power of two for 32 values of k, which the matrix instructions
// apply (linear only)
constexpr int kBf16 = 0, kE4m3 = 1, kFp4 = 2;

// accumulator columns (packed rows) that an epilogue group takes at a time
__host__ __device__ constexpr int chunk(int MODE) { return MODE == kDgradSaved ? 16 : 32; }

// Shared memory of one epilogue group.  A row of 128 output columns is padded
// by 16 bytes (by 32 where it has 64, for swiglu), so that neighbouring rows
// start in other banks.
constexpr int kPitch = 272, kPitchGlu = 160, kPitchCode = 144;
constexpr int kOutBytes = 32 * kPitch;
constexpr int kCodeBytes = 32 * kPitchCode;
constexpr int kOnes = 2048;          // wgrad: the bias sums' ones, then
constexpr int kDwBytes = 32 * 32 * 2;  // for each epilogue warp 32 rows of 32 values of dw
__host__ __device__ constexpr int group_bytes(int MODE, int KIND)
{
    return KIND == kFp4          ? kOutBytes
           : MODE == kWgrad      ? kOnes / 2 + 4 * kDwBytes
           : MODE == kDgradSaved ? 3 * 16 * kPitch + 2 * 16 * kPitchCode + 512
                                 : kOutBytes + kCodeBytes + 256 + 1024 + 512;
}
constexpr int kControl = 4096;

// kFp4: a stage's scales, as tensor memory takes them: 512 bytes for 128 rows
// and 128 values of k (lane i: rows i, i + 32, i + 64, i + 96, 4 bytes each);
// A's 128 rows, and all of B's rows in both blocks of a pair
constexpr int kScaleAtom = 512;
__host__ __device__ constexpr int scale_atoms(int BN) { return (BN + 127) / 128; }
__host__ __device__ constexpr int scale_bytes(int BN) { return 2 * (1 + scale_atoms(BN)) * kScaleAtom; }
__host__ __device__ constexpr int stage_bytes(int CG, int BN, int KIND)
{
    return kStageA + BN / CG * 128 + (KIND == kFp4 ? scale_bytes(BN) : 0);
}
// the other blocks' sums of a tile whose k is split over a cluster
__host__ __device__ constexpr int join_bytes(bool SPLIT, int BN) { return SPLIT ? BN * kTileM * 4 : 0; }
// ring depth: what is left of 227 KB beside the epilogue, the barriers and tile
// counts, and the alignment to 1 KB; at most 12 stages
__host__ __device__ constexpr int stages(int CG, int BN, int MODE, int KIND, bool SPLIT)
{
    const int n = (227 * 1024 - 2 * group_bytes(MODE, KIND) - join_bytes(SPLIT, BN) - kControl - 1024) / stage_bytes(CG, BN, KIND);
    return n > 12 ? 12 : n;
}
__host__ __device__ constexpr int smem_bytes(int CG, int BN, int MODE, int KIND, bool SPLIT)
{
    return 1024 + stages(CG, BN, MODE, KIND, SPLIT) * stage_bytes(CG, BN, KIND) + 2 * group_bytes(MODE, KIND) +
           join_bytes(SPLIT, BN) + kControl;
}
// Tensor memory: two accumulators, and for kFp4 sets of a stage's scales behind
// them (4 columns an atom).  A copy of scales runs before the products that are
// issued after it, but nothing holds it back behind the products that are
// issued before it and may still be queued: it must not touch what they read.
// With a set for each stage of the ring, the stage's barriers see to that.  The
// widest pair has room for two sets, and waits for the products of the stage
// two back (65536 rows, 16 experts, 5120 -> 2 x 2048: 465 us, without 440; with
// a wait that polls, or by the issuing thread alone, 472 to 513).
__host__ __device__ constexpr int scale_cols(int BN) { return 8 * (1 + scale_atoms(BN)); }
__host__ __device__ constexpr int scale_sets(int BN, int stages)
{
    const int room = (512 - 2 * BN) / scale_cols(BN);
    return room < stages ? room : stages;
}
__host__ __device__ constexpr int tmem_cols(int BN, int sets)
{
    const int need = 2 * BN + sets * scale_cols(BN);
    return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}

struct Params {
    CUtensorMap ma, mb, mb32, mo;  // mb32: 32 rows of B at a time, for an expert's last tile; mo: bf16 dw
    const int32_t *offsets;
    void *ws;
    int E, rows;
    int M;         // extent of m
    int N;         // wgrad: extent of n
    int K;         // linear, dgrad: extent of k, in bytes
    int act, glu;  // glu: A's rows alternate gate and up columns
    int fp32;
    int whole_a, whole_b;  // an MN-major operand whose columns are whole blocks of 64
    int bn;        // columns of n per tile, at most BN
    int split;     // blocks that share a tile's k (a cluster of 2, 4 or 8), or 1
    const __nv_bfloat16 *bias, *residual;
    const float2 *x_scales, *w_scales;
    const uint8_t *x_bytes, *w_bytes;  // kFp4: scale bytes of rows and weights
    int pitch, valid_scales;           // their bytes per row, and how many hold scales
    int sectors;                       // rows of scales start at multiples of 32 bytes
    __nv_bfloat16 *y, *a;
    void *dw, *db;
    uint8_t *saved, *saved_scales;
};

struct Control {
    uint64_t full[12], empty[12], acc_full[2], acc_empty[2], joined, taken;
    uint32_t tmem;
    int abort;
    unsigned skip;  // the injected failure
    unsigned long long limit;  // of every wait, ns
    int part[12];
    int row0[MOE_MAX_EXPERTS], rows[MOE_MAX_EXPERTS];  // of each expert, checked
    int tile0[MOE_MAX_EXPERTS + 1];                    // its first tile
};
static_assert(sizeof(Control) <= kControl, "barriers and tile counts");

// A wait may have to outlast a whole tile: the epilogue's for the products, and
// what waits for it.  A stage takes 0.3 us on its SM, and 48 KB for each of
// 152 SMs are 1.1 us of HBM's time; 2^28 rows of one expert are 4 million
// stages of one tile of wgrad.
constexpr unsigned long long kStageLimitNs = 2000;

// Wait for phase `parity`, at most the block's limit.  False once the limit has
// passed or another role of the block has given up; then every role leaves
// its loop.  CLUSTER: another block's mbar_hand_over arrives there.
template <bool CLUSTER>
__device__ __forceinline__ bool poll(uint64_t *bar, uint32_t parity, Control *c, void *ws)
{
    const auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    for (int i = 0; i < 64; ++i)
        if (done()) return true;
    const unsigned long long t0 = global_timer_ns();
    for (;;) {
        for (int i = 0; i < 16; ++i)
            if (done()) return true;
        if (*(volatile int *)&c->abort) return false;
        if (global_timer_ns() - t0 > c->limit) {
            *(volatile int *)&c->abort = 1;
            record_status(ws, MOE_ERR_TIMEOUT);
            return false;
        }
    }
}

// The same for a whole warp, which goes on together.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Control *c, void *ws)
{
    return __all_sync(0xFFFFFFFFu, poll<CLUSTER>(bar, parity, c, ws));
}

// a / b for 0 <= a < 2^30 and b > 0 with a quotient below 2^22: the rounded
// quotient is off by one at most, which the remainder shows.  A third of the
// integer division's time, which every role spends three times on a tile.
__device__ __forceinline__ int quotient(int a, int b)
{
    int q = (int)__fdividef((float)a, (float)b);
    const int r = a - q * b;
    if (r < 0) --q;
    else if (r >= b) ++q;
    return q;
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
        const int tn = quotient(c->tile0[e + 1] - c->tile0[e], tm);
        const int g = quotient(local, 8 * tn), in = local - g * 8 * tn;
        const int gm = min(8, tm - g * 8);
        t.e = e;
        t.n = quotient(in, gm);
        t.m = g * 8 + in - t.n * gm;
        t.row0 = c->row0[e];
        t.rows = c->rows[e];
        tile += step;
        return true;
    }
};

// 32 bytes, read once, with one request
__device__ __forceinline__ u32x8 load_sector(const void *at)
{
    u32x8 v;
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.lo.x), "=r"(v.lo.y), "=r"(v.lo.z), "=r"(v.lo.w), "=r"(v.hi.x), "=r"(v.hi.y), "=r"(v.hi.z),
                   "=r"(v.hi.w)
                 : "l"(at));
    return v;
}

__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ void group_sync(int g)
{
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + g) : "memory");
}

__device__ __forceinline__ void st_shared_bf16(unsigned char *p, float v)
{
    *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
}

// `rows` rows of `units` 16-byte vectors from shared memory (row pitch
// `pitch`) to global memory (row pitch `gpitch` bytes); vectors from `on` up
// lie past the last column.  128 threads, tid in 0..127, at most ROWS rows.
template <int UNITS, int ROWS>
__device__ __forceinline__ void copy_out(const unsigned char *s, int pitch, void *gbase, size_t gpitch, int rows,
                                         int on, int tid)
{
    unsigned char *g = static_cast<unsigned char *>(gbase);
    const int c = tid % UNITS;
#pragma unroll
    for (int i = 0; i < (ROWS * UNITS + 127) / 128; ++i) {
        const int r = tid / UNITS + i * (128 / UNITS);
        if (r < rows && c < on)
            *reinterpret_cast<uint4 *>(g + (size_t)r * gpitch + c * 16) =
                *reinterpret_cast<const uint4 *>(s + r * pitch + c * 16);
    }
}
// The other way, into registers (zeros past the edges), and on to shared memory.
template <int UNITS, int ROWS>
__device__ __forceinline__ void fetch(uint4 *v, const void *gbase, size_t gpitch, int rows, int on, int tid)
{
    const unsigned char *g = static_cast<const unsigned char *>(gbase);
    const int c = tid % UNITS;
#pragma unroll
    for (int i = 0; i < (ROWS * UNITS + 127) / 128; ++i) {
        const int r = tid / UNITS + i * (128 / UNITS);
        v[i] = r < rows && c < on ? *reinterpret_cast<const uint4 *>(g + (size_t)r * gpitch + c * 16)
                                  : make_uint4(0, 0, 0, 0);
    }
}
template <int UNITS, int ROWS>
__device__ __forceinline__ void place(const uint4 *v, unsigned char *s, int pitch, int tid)
{
    const int c = tid % UNITS;
#pragma unroll
    for (int i = 0; i < (ROWS * UNITS + 127) / 128; ++i)
        *reinterpret_cast<uint4 *>(s + (tid / UNITS + i * (128 / UNITS)) * pitch + c * 16) = v[i];
}

// --------------------------------------------------------------------------
// linear and plain dgrad.  A lane holds one accumulator row, i.e. one column
// of u (swiglu: even lanes a gate, odd lanes its up), for 32 packed rows, so
// bias, weight scale and activation need no memory in the loop.  Results go
// through shared memory as bf16 and leave in whole row segments.
// --------------------------------------------------------------------------
template <int KIND>
struct LinearEpilogue {
    static constexpr bool FP8 = KIND == kE4m3;
    const Params &p;
    unsigned char *out, *codes;
    float2 *xs;
    unsigned *top;   // [4 warps][gates, ups][32 rows], largest magnitudes
    float *inverse;  // [4 blocks][32 rows], 1 / scale
    int g, q, lane, tid;
    // of a tile
    int col0, cols;  // first output column of the block's tile, how many exist
    float bias, ws, wsum;
    uint4 res[4];

    __device__ LinearEpilogue(const Params &p_, unsigned char *base, int g_, int q_, int lane_)
        : p(p_), out(base), codes(base + kOutBytes), xs(reinterpret_cast<float2 *>(base + kOutBytes + kCodeBytes)),
          top(reinterpret_cast<unsigned *>(base + kOutBytes + kCodeBytes + 256)),
          inverse(reinterpret_cast<float *>(base + kOutBytes + kCodeBytes + 256 + 1024)), g(g_), q(q_), lane(lane_),
          tid(q_ * 32 + lane_)
    {
    }
    __device__ __forceinline__ int out_cols() const { return p.glu ? p.M / 2 : p.M; }

    __device__ __forceinline__ void tile(int e, int m0)
    {
        const int n = out_cols();
        col0 = p.glu ? m0 / 2 : m0;
        cols = min(p.glu ? 64 : 128, n - col0);
        const int c = p.glu ? q * 16 + lane / 2 : q * 32 + lane;
        const size_t at = (size_t)e * p.M + (p.glu ? (lane & 1) * n : 0) + col0 + c;
        bias = ws = wsum = 0.0f;
        if (c < cols) {
            if (p.bias) bias = __bfloat162float(p.bias[at]);
            if (FP8) {
                const float2 w = p.w_scales[at];
                ws = w.x;
                wsum = w.y;
            }
        }
    }
    // residual rows of a chunk, ahead of their use
    __device__ __forceinline__ void ahead(int row, int rows)
    {
        if (!p.residual || rows <= 0) return;
        const __nv_bfloat16 *at = p.residual + (size_t)row * out_cols() + col0;
        if (p.glu) fetch<8, 32>(res, at, 2 * (size_t)out_cols(), rows, cols / 8, tid);
        else fetch<16, 32>(res, at, 2 * (size_t)out_cols(), rows, cols / 8, tid);
    }
    __device__ __forceinline__ void finish(uint32_t (&v)[32], int row, int rows, int next_rows)
    {
        const int pitch = p.glu ? kPitchGlu : kPitch;
        if (p.residual || FP8) {
            if (p.residual) {
                if (p.glu) place<8, 32>(res, out, pitch, tid);
                else place<16, 32>(res, out, pitch, tid);
                ahead(row + 64, next_rows);
            }
            if (FP8 && q == 0 && lane < rows) xs[lane] = p.x_scales[row + lane];
            group_sync(g);
        }
        float u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            u[i] = __uint_as_float(v[i]);
            if (FP8) {
                const float2 x = xs[i];
                u[i] = fmaf(x.x, ws * u[i], x.y * wsum);
            }
            u[i] += bias;
        }
        if constexpr (KIND != kFp4)
            if (p.saved) save(u, row, rows);
        if constexpr (KIND == kFp4) {
            apply(u, pitch);
        } else if (p.glu) {
            // lanes 2i and 2i+1 hold gate and up of a column: of each two
            // rows the even lane finishes the first, the odd lane the second
            const bool odd = lane & 1;
            unsigned char *o = out + (odd ? pitch : 0) + (q * 16 + lane / 2) * 2;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                if (i % 8 == 0 && i >= rows) break;  // few rows: nothing is done for the others
                const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? u[i] : u[i + 1], 1);
                const float gate = odd ? got : u[i], up = odd ? u[i + 1] : got;
                float y = gate * logistic(gate) * up;
                if (p.residual) y += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(o + i * pitch));
                st_shared_bf16(o + i * pitch, y);
            }
        } else {
            unsigned char *o = out + (q * 32 + lane) * 2;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                if (j >= rows) break;  // few rows: nothing is done for the others
                if (p.act == MOE_ACT_SILU) {
#pragma unroll
                    for (int i = j; i < j + 8; ++i) u[i] = act_value(u[i], MOE_ACT_SILU);
                } else if (p.act == MOE_ACT_GELU) {
#pragma unroll
                    for (int i = j; i < j + 8; ++i) u[i] = act_value(u[i], MOE_ACT_GELU);
                }
#pragma unroll
                for (int i = j; i < j + 8; ++i) {
                    if (p.residual)
                        u[i] += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(o + i * kPitch));
                    st_shared_bf16(o + i * kPitch, u[i]);
                }
            }
        }
        group_sync(g);
        const size_t n = out_cols();
        __nv_bfloat16 *y = p.y + (size_t)row * n + col0;
        if (p.glu) copy_out<8, 32>(out, kPitchGlu, y, 2 * n, rows, cols / 8, tid);
        else copy_out<16, 32>(out, kPitch, y, 2 * n, rows, cols / 8, tid);
        if (KIND != kFp4 && p.saved) {
            uint8_t *s = p.saved + (size_t)row * p.M + col0;
            if (p.glu) {
                copy_out<4, 32>(codes, kPitchCode, s, p.M, rows, cols / 16, tid);
                copy_out<4, 32>(codes + 64, kPitchCode, s + n, p.M, rows, cols / 16, tid);
            } else {
                copy_out<8, 32>(codes, kPitchCode, s, p.M, rows, cols / 16, tid);
            }
        }
        group_sync(g);
    }
    // Activation, residual and rounding of a chunk for kFp4, whose products may
    // be shorter than this: each step for all rows before the next, nothing
    // tested in between.  65536 rows, 256 -> 2 x 2048: 229 us, with the tests
    // and the residual's load beside each store (as in finish) 306 us; 5120 ->
    // 2 x 2048: 408 and 445 us.
    __device__ __forceinline__ void apply(float (&u)[32], int pitch)
    {
        const bool odd = p.glu && (lane & 1);
        unsigned char *const o = out + (p.glu ? (odd ? pitch : 0) + (q * 16 + lane / 2) * 2 : (q * 32 + lane) * 2);
        if (p.glu) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? u[i] : u[i + 1], 1);
                const float gate = odd ? got : u[i], up = odd ? u[i + 1] : got;
                u[i] = gate * logistic(gate) * up;
            }
        } else if (p.act == MOE_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = act_value(u[i], MOE_ACT_SILU);
        } else if (p.act == MOE_ACT_GELU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = act_value(u[i], MOE_ACT_GELU);
        }
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!p.glu || i % 2 == 0)
                    u[i] += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(o + i * pitch));
        }
        if (p.glu) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) st_shared_bf16(o + i * kPitchGlu, u[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) st_shared_bf16(o + i * kPitch, u[i]);
        }
    }
    // u in 8 bits: the 32 columns of a block are the 32 lanes of a warp, or
    // for swiglu every other lane of two warps
    __device__ __forceinline__ void save(const float (&u)[32], int row, int rows)
    {
        if (p.glu) {
            const bool odd = lane & 1;
            unsigned gates = 0, ups = 0;  // of row `lane`
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const unsigned m = mag(u[i]);
                const unsigned mg = __reduce_max_sync(0xFFFFFFFFu, odd ? 0u : m);
                const unsigned mu = __reduce_max_sync(0xFFFFFFFFu, odd ? m : 0u);
                if (lane == i) {
                    gates = mg;
                    ups = mu;
                }
            }
            top[q * 64 + lane] = gates;
            top[q * 64 + 32 + lane] = ups;
            group_sync(g);
            // 2 blocks of gates and 2 of ups for 32 rows: one a thread
            const int r = tid & 31, b = tid >> 5, half = b >> 1, side = b & 1;
            const unsigned *t = top + half * 128 + side * 32 + r;
            const unsigned byte = saved_byte(max(t[0], t[64]));
            inverse[tid] = saved_inverse(byte);
            if (r < rows && half * 32 < cols)
                p.saved_scales[(size_t)(row + r) * (p.M / 32) + (side * out_cols() + col0) / 32 + half] = (uint8_t)byte;
            group_sync(g);
            const float2 *inv = reinterpret_cast<const float2 *>(inverse + ((q & 2) + (lane & 1)) * 32);
            uint8_t *c = codes + (odd ? 64 : 0) + q * 16 + lane / 2;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 f = inv[i / 2];
                const unsigned two = e4m3_pair(u[i] * f.x, u[i + 1] * f.y);
                c[i * kPitchCode] = (uint8_t)two;
                c[(i + 1) * kPitchCode] = (uint8_t)(two >> 8);
            }
        } else {
            unsigned keep = 0;  // of row `lane`
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const unsigned m = __reduce_max_sync(0xFFFFFFFFu, mag(u[i]));
                if (lane == i) keep = m;
            }
            const unsigned byte = saved_byte(keep);
            if (lane < rows && q * 32 < cols)
                p.saved_scales[(size_t)(row + lane) * (p.M / 32) + col0 / 32 + q] = (uint8_t)byte;
            float *mine = inverse + q * 32;  // read by this warp alone
            mine[lane] = saved_inverse(byte);
            __syncwarp();
            uint8_t *c = codes + q * 32 + lane;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 f = *reinterpret_cast<const float2 *>(mine + i);
                const unsigned two = e4m3_pair(u[i] * f.x, u[i + 1] * f.y);
                c[i * kPitchCode] = (uint8_t)two;
                c[(i + 1) * kPitchCode] = (uint8_t)(two >> 8);
            }
        }
    }
};

// --------------------------------------------------------------------------
// dgrad through a saved layer.  A lane holds one column of d for 16 packed
// rows; the codes of that column come through shared memory, and up to three
// results (du, for swiglu of gate and up, and the activation) leave through it.
// --------------------------------------------------------------------------
struct SavedEpilogue {
    const Params &p;
    unsigned char *out, *codes;
    float *scale;  // [16 rows][4 gate blocks, 4 up blocks]
    int g, q, lane, tid;
    int col0, cols;
    uint4 pre[2];
    unsigned pre_scale;

    __device__ SavedEpilogue(const Params &p_, unsigned char *base, int g_, int q_, int lane_)
        : p(p_), out(base), codes(base + 3 * 16 * kPitch), scale(reinterpret_cast<float *>(base + 3 * 16 * kPitch + 2 * 16 * kPitchCode)),
          g(g_), q(q_), lane(lane_), tid(q_ * 32 + lane_)
    {
    }
    __device__ __forceinline__ bool glu() const { return p.act == MOE_ACT_SWIGLU; }
    __device__ __forceinline__ size_t saved_cols() const { return glu() ? 2 * (size_t)p.M : p.M; }
    __device__ __forceinline__ void tile(int, int m0)
    {
        col0 = m0;
        cols = min(128, p.M - m0);
    }
    __device__ __forceinline__ void ahead(int row, int rows)
    {
        if (rows <= 0) return;
        const size_t C = saved_cols();
        const uint8_t *s = p.saved + (size_t)row * C + col0;
        fetch<8, 16>(pre, s, C, rows, cols / 16, tid);
        if (glu()) fetch<8, 16>(pre + 1, s + p.M, C, rows, cols / 16, tid);
        const int r = tid >> 3, b = tid & 3, up = (tid >> 2) & 1;
        pre_scale = 0;
        if (r < rows && b * 32 < cols && (glu() || !up))
            pre_scale = p.saved_scales[(size_t)(row + r) * (C / 32) + (up * p.M + col0) / 32 + b];
    }
    __device__ __forceinline__ void finish(uint32_t (&v)[16], int row, int rows, int next_rows)
    {
        place<8, 16>(pre, codes, kPitchCode, tid);
        if (glu()) place<8, 16>(pre + 1, codes + 16 * kPitchCode, kPitchCode, tid);
        scale[tid] = saved_scale(pre_scale);
        ahead(row + 32, next_rows);
        group_sync(g);
        const uint8_t *c = codes + q * 32 + lane;
        unsigned char *o = out + (q * 32 + lane) * 2;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            if (i % 8 == 0 && i >= rows) break;
            const float2 x = e4m3_decode2(c[i * kPitchCode] | ((unsigned)c[(i + 1) * kPitchCode] << 8));
            const float u[2] = {x.x * scale[i * 8 + q], x.y * scale[i * 8 + 8 + q]};
            const float d[2] = {__uint_as_float(v[i]), __uint_as_float(v[i + 1])};
            if (glu()) {
                const uint8_t *cu = c + 16 * kPitchCode;
                const float2 z = e4m3_decode2(cu[i * kPitchCode] | ((unsigned)cu[(i + 1) * kPitchCode] << 8));
                const float up[2] = {z.x * scale[i * 8 + 4 + q],
                                     z.y * scale[i * 8 + 12 + q]};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float s = logistic(u[j]), silu = u[j] * s;
                    unsigned char *at = o + (i + j) * kPitch;
                    st_shared_bf16(at, d[j] * up[j] * (s * (1.0f + u[j] * (1.0f - s))));
                    st_shared_bf16(at + 16 * kPitch, d[j] * silu);
                    if (p.a) st_shared_bf16(at + 32 * kPitch, silu * up[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    unsigned char *at = o + (i + j) * kPitch;
                    st_shared_bf16(at, d[j] * act_slope(u[j], p.act));
                    if (p.a) st_shared_bf16(at + 32 * kPitch, act_value(u[j], p.act));
                }
            }
        }
        group_sync(g);
        const size_t C = saved_cols();
        __nv_bfloat16 *y = p.y + (size_t)row * C + col0;
        copy_out<16, 16>(out, kPitch, y, 2 * C, rows, cols / 8, tid);
        if (glu()) copy_out<16, 16>(out + 16 * kPitch, kPitch, y + p.M, 2 * C, rows, cols / 8, tid);
        if (p.a)
            copy_out<16, 16>(out + 32 * kPitch, kPitch, p.a + (size_t)row * p.M + col0, 2 * (size_t)p.M, rows,
                             cols / 8, tid);
        group_sync(g);
    }
};

// 32 consecutive values of a row of dw, `n` of them (a multiple of 8) inside it.
__device__ __forceinline__ void store_row(const Params &p, size_t at, const uint32_t (&v)[32], int n)
{
    if (p.fp32) {
        float *o = static_cast<float *>(p.dw) + at;
#pragma unroll
        for (int j = 0; j < 32; j += 4)
            if (j < n) *reinterpret_cast<uint4 *>(o + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        return;
    }
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.dw) + at;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j * 8 < n)
            *reinterpret_cast<uint4 *>(o + j * 8) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// The warp's 32 rows of 32 values as one tile copy: rows of 64 bytes in
// shared memory (64-byte swizzle: no bank conflicts), written out by the copy
// engine.  32 lanes' own stores to 32 rows cost the load/store unit four times
// as much, which bounded experts with few rows.
__device__ __forceinline__ void store_tile(const Params &p, unsigned char *buf, const uint32_t (&v)[32], int lane, int col,
                                           int row, int e)
{
    if (lane == 0) bulk_wait_group_read<0>();  // the last tile has left the buffer
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
        *reinterpret_cast<uint4 *>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row < p.M) {
        tma_store_3d(&p.mo, buf, col, row, e);
        bulk_commit_group();
    }
}

// --------------------------------------------------------------------------
// the kernel
// --------------------------------------------------------------------------
template <int CG, int BN, int MODE, int KIND, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) experts_kernel(const __grid_constant__ Params p)
{
    constexpr bool FP8 = KIND == kE4m3, FP4 = KIND == kFp4;
    constexpr bool kHandOver = FP4 && CG == 2;  // the second block's scales, to the first's copy of them
    constexpr int kStages = stages(CG, BN, MODE, KIND, SPLIT);
    constexpr int kStage = stage_bytes(CG, BN, KIND);
    constexpr int kSets = FP4 ? scale_sets(BN, kStages) : 0, kColumns = tmem_cols(BN, kSets);
    constexpr int kGroup = group_bytes(MODE, KIND);
    constexpr int kScales = kStageA + BN / CG * 128;  // kFp4: where a stage's scales start
    constexpr int kBM = kTileM * CG;
    constexpr bool kMnA = MODE != kLinear, kMnB = MODE == kWgrad;
    constexpr int kStepN = MODE == kWgrad ? 64 * CG : CG == 2 ? 32 : 16;
    constexpr int kElems = KIND == kBf16 ? 64 : 128;  // k of a stage, in units of the tensor maps

    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *stg = smem + kStages * kStage;
    float *join = reinterpret_cast<float *>(stg + 2 * kGroup);
    Control *c = reinterpret_cast<Control *>(stg + 2 * kGroup + join_bytes(SPLIT, BN));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    static_assert(CG == 1 || !SPLIT, "a pair does not share its k");
    constexpr bool kCluster = CG == 2 || SPLIT;
    const uint32_t self = kCluster ? cluster_cta_rank() : 0u;
    const uint32_t rank = CG == 2 ? self : 0u;   // of the pair: which half of m
    const uint32_t lead = CG == 2 ? 0u : self;   // whose barriers the matrix instructions wait on
    const int split = SPLIT ? p.split : 1;

    int lo = 0, hi = 0;  // read first: the tiles wait for them
    if (tid < p.E) {
        lo = p.offsets ? p.offsets[tid] : 0;
        hi = p.offsets ? p.offsets[tid + 1] : p.rows;
    }
    WsHeader *const header = static_cast<WsHeader *>(p.ws);
    if (tid == 0) {
        const unsigned skip = blockIdx.x == 0 ? *(volatile unsigned *)&header->inject_skip_load : 0u;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&c->full[i], FP4 ? 1 + CG : 1);  // the copies, and each block's scales
            mbar_init(&c->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c->acc_full[i], 1);
            mbar_init(&c->acc_empty[i], 8 * CG);
        }
        mbar_init(&c->joined, 8 * split);
        mbar_init(&c->taken, 8 * split);
        c->abort = 0;
        c->limit = kSpinLimitNs + (MODE == kWgrad ? p.rows / 64 : p.K / 128) * kStageLimitNs;
        c->skip = skip;
        if (skip) header->inject_skip_load = 0;
        mbar_fence_init();
        tmap_prefetch(&p.ma);
        tmap_prefetch(&p.mb);
    }
    if (warp == 2) tmem_alloc<CG>(&c->tmem, kColumns);
    if (MODE == kWgrad && tid < 128) {
        // the bias sums' B operand: 2 KB of bf16 ones (any layout of them is the same)
        reinterpret_cast<uint4 *>(stg)[tid] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        fence_proxy_async_smem();
    }

    // rows and first tile of every expert: thread e looks at expert e
    const int tm = (p.M + kBM - 1) / kBM;
    {
        const auto tiles_of = [&](int rows) {
            return tm * (((MODE == kWgrad ? p.N : rows) + p.bn - 1) / p.bn + (MODE == kWgrad && p.db ? 1 : 0));
        };
        const auto scan = [&](int v) {  // inclusive, over a warp
#pragma unroll
            for (int i = 1; i < 32; i *= 2) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, v, i);
                if (lane >= i) v += u;
            }
            return v;
        };
        int sum = scan(tid < p.E ? tiles_of(max(hi - lo, 0)) : 0);
        if (lane == 31) c->part[warp] = sum;
        // offsets that only rise and stay inside the rows need no second look
        if (!__syncthreads_and(tid >= p.E || (lo >= 0 && hi >= lo && hi <= p.rows))) {
            // the largest offset so far: rows below it belong to an earlier
            // expert, and two experts never write the same row
            int before = 0;
            if (p.offsets)
                for (int i = 0; i <= tid && i < p.E; ++i) before = max(before, p.offsets[i]);
            if (tid < p.E && (lo < before || hi < lo || hi > p.rows)) {
                if (blockIdx.x == 0) record_status(p.ws, MOE_ERR_DEVICE_DATA);
                lo = hi = 0;
            }
            sum = scan(tid < p.E ? tiles_of(hi - lo) : 0);
            if (lane == 31) c->part[warp] = sum;
            __syncthreads();
        }
        for (int i = 0; i < warp; ++i) sum += c->part[i];
        if (tid < p.E) {
            c->row0[tid] = lo;
            c->rows[tid] = hi - lo;
            c->tile0[tid + 1] = sum;
        }
        if (tid == 0) c->tile0[0] = 0;
    }
    __syncwarp();
    tc_fence_before();
    if (kCluster) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem;

    const int chunks_b = MODE == kWgrad ? p.bn / CG / 64 : 0;  // 64 columns each
    const int sharers = CG == 2 ? 2 : split;  // blocks of a cluster
    Walk walk(c, p.E, tm, blockIdx.x / sharers, gridDim.x / sharers);
    Tile t;
    // this block's part of a tile's k, in stages
    struct Span {
        int first, count;
        bool last;
    };
    const auto span = [&](const Tile &q) {
        const int all = MODE == kWgrad ? (q.rows + 63) / 64 : (p.K + 127) / 128;
        if (!SPLIT) return Span{0, all, true};
        const int lo_k = all * (int)self / split, hi_k = all * ((int)self + 1) / split;
        return Span{lo_k, hi_k - lo_k, hi_k == all};
    };
    // wgrad: the tile after the last of n is the bias gradient's, the product
    // of dy^T with ones: no rows of x to load, 16 columns (32 for a pair)
    const int tn_bias = MODE == kWgrad ? (p.N + p.bn - 1) / p.bn : -1;
    const auto is_bias = [&](const Tile &q) { return MODE == kWgrad && q.n == tn_bias; };
    // columns of the accumulator in use: what is left of the ragged axis
    const auto width = [&](const Tile &q) {
        if (is_bias(q)) return 16 * CG;
        const int left = (MODE == kWgrad ? p.N : q.rows) - q.n * p.bn;
        return min(p.bn, (left + kStepN - 1) / kStepN * kStepN);
    };

    if (warp == 0) {
        // ---- loads -------------------------------------------------------
        // As below: the warp walks together and one thread issues.  What it
        // does for a stage bounds narrow tiles, so an operand whose columns
        // are whole blocks of 64 comes with one instruction.
        const bool one = elect_one();
        const uint32_t load_bytes = kStageA + (MODE == kWgrad ? chunks_b * 8192 : p.bn / CG * 128);
        int s = 0;
        uint32_t ph = 1;
        bool ok = true, ready = false, skip = c->skip != 0;
        while (ok && walk.next(t)) {
            const Span part = span(t);
            const int m0 = t.m * kBM + (int)rank * kTileM;
            const int n0 = t.n * p.bn + (int)rank * (width(t) / CG);
            const bool no_b = is_bias(t);
            // a narrow last tile loads the rows it has, by 32
            const int few = MODE == kWgrad ? 0 : (width(t) / CG + 31) / 32;
            const bool some = few * 32 < p.bn / CG;
            const uint32_t bytes = no_b ? kStageA : MODE != kWgrad && some ? kStageA + few * 4096 : load_bytes;
            for (int i = part.first; i < part.first + part.count; ++i) {
                ok = ready || wait(&c->empty[s], ph, c, p.ws);
                if (!ok) break;
                const int now = s;
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
                const bool next = mbar_test_wait(&c->empty[s], ph);
                if (one && !skip) {
                    unsigned char *sa = smem + now * kStage, *sb = sa + kStageA;
                    const int k0 = i * kElems;
                    uint32_t bar = smem_addr(&c->full[now]);
                    // the pair's first block expects the bytes of both
                    if (CG == 1 || self == 0) mbar_arrive_expect_tx(&c->full[now], CG * bytes);
                    else bar = cluster_addr(&c->full[now], 0);
                    if constexpr (MODE == kWgrad) {
                        // The last rows of an expert rarely fill 64 of k; the
                        // rows after them are another expert's, or nobody's
                        // with any bits in them.  The window of a tail starts
                        // before its first row: zeros come first, the tail's
                        // rows last (encode_window).
                        const int row = t.row0 + k0, from = min(t.rows - k0 - 64, 0);
                        if (p.whole_a) {
                            tma_load_4d<CG>(sa, &p.ma, 0, from, row, m0 / 64, bar);
                        } else {
                            for (int j = 0; j < 2; ++j)
                                tma_load_4d<CG>(sa + j * 8192, &p.ma, m0 + 64 * j, from, row, 0, bar);
                        }
                        if (!no_b) {
                            if (p.whole_b) {
                                tma_load_4d<CG>(sb, &p.mb, 0, from, row, n0 / 64, bar);
                            } else {
                                for (int j = 0; j < chunks_b; ++j)
                                    tma_load_4d<CG>(sb + j * 8192, &p.mb, n0 + 64 * j, from, row, 0, bar);
                            }
                        }
                    } else {
                        if constexpr (MODE == kLinear) {
                            tma_load_4d<CG>(sa, &p.ma, k0, 0, p.glu ? m0 / 2 : m0, t.e, bar);
                        } else if (p.whole_a) {
                            tma_load_4d<CG>(sa, &p.ma, 0, k0, m0 / 64, t.e, bar);
                        } else {
                            for (int j = 0; j < 2; ++j)
                                tma_load_4d<CG>(sa + j * 8192, &p.ma, m0 + 64 * j, k0, 0, t.e, bar);
                        }
                        if (!some) {
                            tma_load_2d<CG>(sb, &p.mb, k0, t.row0 + n0, bar);
                        } else {
                            for (int j = 0; j < few; ++j)
                                tma_load_2d<CG>(sb + j * 4096, &p.mb32, k0, t.row0 + n0 + 32 * j, bar);
                        }
                    }
                }
                skip = false;
                __syncwarp();
                ready = __all_sync(0xFFFFFFFFu, next);
            }
        }
        // every stage read: no copy and no arrival is on its way to this
        // block's shared memory when it ends
        for (int i = 0; ok && i < kStages; ++i) {
            ok = wait(&c->empty[s], ph, c, p.ws);
            if (++s == kStages) {
                s = 0;
                ph ^= 1;
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---- matrix instructions ------------------------------------------
        // One elected thread issues; the warp walks the loop together, so that
        // descriptors and addresses stay in uniform registers.  The next
        // stage's barrier is looked at before the current stage's
        // instructions: the answer is there when their issue, which blocks
        // while the tensor cores' queue is full, has gone through.
        {
            constexpr uint32_t kLeadA = kMnA ? 8192 : 16, kLeadB = kMnB ? 8192 : 16;
            constexpr uint32_t kStepA = (kMnA ? 2048 : 32) >> 4, kStepB = (kMnB ? 2048 : 32) >> 4;
            const uint64_t da0 = smem_desc(smem_addr(smem), kLeadA, 1024);
            const uint64_t db0 = smem_desc(smem_addr(smem) + kStageA, kLeadB, 1024);
            const uint64_t ones = smem_desc(smem_addr(stg), kLeadB, 1024);
            const uint64_t ds0 = scale_desc(smem_addr(smem) + kScales);
            const bool one = elect_one();
            int s = 0, acc = 0, set = 0, begun = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true, ready = false, more = walk.next(t);
            while (more) {
                const int iters = span(t).count;
                if (iters == 0) {
                    more = walk.next(t);
                    continue;
                }
                const uint32_t idesc =
                    FP4 ? mma_idesc_fp4(kBM, width(t)) : mma_idesc(FP8, kMnA, kMnB, kBM, width(t));
                const uint32_t d = tmem + acc * BN;
                const bool wide = FP4 && width(t) > 128;
                const bool bias = is_bias(t);
                // the steps of 16 rows that a tail fills, the stage's last
                const int last_steps = MODE == kWgrad && span(t).last ? ((t.rows & 63) + 15) / 16 : 0;
                ok = wait(&c->acc_empty[acc], aph ^ 1, c, p.ws);
                if (!ok) break;
                tc_fence_after();
                for (int i = 0; i < iters; ++i) {
                    ok = ready || wait<kHandOver>(&c->full[s], ph, c, p.ws);
                    if (!ok) break;
                    if (kHandOver) take_over();
                    if (FP4 && kSets < kStages) {  // the products that read this set of scales
                        if (begun == kSets) {
                            ok = wait(&c->empty[s >= kSets ? s - kSets : s - kSets + kStages], s >= kSets ? ph : ph ^ 1, c,
                                      p.ws);
                            if (!ok) break;
                        } else {
                            ++begun;
                        }
                        set = set + 1 >= kSets ? 0 : set + 1;
                    } else {
                        set = s;
                    }
                    tc_fence_after();
                    const int now = s;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    const bool next =
                        kHandOver ? mbar_test_wait_cluster(&c->full[s], ph) : mbar_test_wait(&c->full[s], ph);
                    const uint64_t da = da0 + (uint64_t)(now * (kStage >> 4)), db = db0 + (uint64_t)(now * (kStage >> 4));
                    const int from = MODE == kWgrad && last_steps != 0 && i == iters - 1 ? 4 - last_steps : 0;
                    if (one) {
                        if constexpr (FP4) {
                            // the scales to tensor memory, then four products of
                            // 64 values of k; two of them share the scales of 128
                            const uint32_t sfa = tmem + 2 * BN + set * scale_cols(BN), sfb = sfa + 8;
                            const uint64_t ds = ds0 + (uint64_t)(now * (kStage >> 4));
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                scales_to_tmem<CG>(sfa + w * 4, ds + w * (kScaleAtom >> 4));
#pragma unroll
                                for (int h = 0; h < scale_atoms(BN); ++h)
                                    if (h == 0 || wide)
                                        scales_to_tmem<CG>(sfb + (w * scale_atoms(BN) + h) * 4,
                                                           ds + (2 + w * scale_atoms(BN) + h) * (kScaleAtom >> 4));
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_fp4<CG>(d, da + k * kStepA, db + k * kStepB, idesc | mma_scale_id(k & 1),
                                            sfa + (k >> 1) * 4, sfb + (k >> 1) * (4 * scale_atoms(BN)), i != 0 || k != 0);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (MODE != kWgrad || k >= from)
                                    mma_ss<CG, FP8>(d, da + k * kStepA, bias ? ones : db + k * kStepB, idesc, i != 0 || k != from);
                        }
                        mma_commit<CG>(&c->empty[now]);
                    }
                    __syncwarp();
                    if (i == 0) more = walk.next(t);  // the divisions of the next tile hide behind this one
                    ready = __all_sync(0xFFFFFFFFu, next);
                }
                if (!ok) break;
                if (one) mma_commit<CG>(&c->acc_full[acc]);
                __syncwarp();
                acc ^= 1;
                aph ^= acc == 0;
            }
        }
        __syncwarp();
    } else if (FP4 && (warp == 2 || warp == 3)) {
        // ---- scales ---------------------------------------------------------
        // The rows' scales lie in row order, tensor memory wants 4 bytes of 4
        // rows side by side, and no copy engine turns pieces of 4 bytes around.
        // So a lane reads 8 kSpan bytes (of four stages: a whole sector) of the
        // rows lane, lane + 32, .. of both operands, and stores 4 bytes of 4
        // rows with one instruction.  The two warps take every other kSpan
        // stages: a stage takes one of them about 780 cycles, its products
        // 530.  65536 rows, 16 experts, 5120 -> 2 x 2048: 445 us (before the
        // epilogue below); a sector with two requests 465 us; the rows' bytes through a ring in shared memory
        // 513 us; a warp for each operand, four stages ahead in registers and
        // unrolled for that, 860 us: 270 KB of instructions, and the block
        // waits for them.  Without any loads here 410 us.
        // A warp does not wait for the stages that it leaves out.  Its last wait
        // told it that the ring has been read up to kStages before that stage;
        // a parity asked for more than kStages later could be that of an
        // earlier round and let it overwrite what is still to be read.
        constexpr int kRowsB = (BN + 31) / 32, kRows = 4 + kRowsB, kSpan = kStages > 4 ? 4 : 2;
        static_assert(!FP4 || kSpan + 1 <= kStages, "the ring is as long as the way from wait to wait");
        int s = 0, turn = 0;
        uint32_t ph = 1;
        bool ok = true;
        const auto step = [&](int n) {
            s += n;
            if (s >= kStages) {
                s -= kStages;
                ph ^= 1;
            }
        };
        while (ok && walk.next(t)) {
            const Span part = span(t);
            const int end = part.first + part.count, m0 = t.m * kBM + (int)rank * kTileM, n0 = t.n * p.bn;
            const uint8_t *at[kRows];
#pragma unroll
            for (int r = 0; r < 4; ++r) {  // glu: A's rows alternate gate and up columns
                const int row = r * 32 + lane, half = p.glu ? p.M / 2 : p.M, col = p.glu ? (m0 + row) / 2 : m0 + row;
                at[r] = col < half ? p.w_bytes + ((size_t)t.e * p.M + (p.glu ? (row & 1) * half : 0) + col) * p.pitch
                                   : nullptr;
            }
#pragma unroll
            for (int r = 0; r < kRowsB; ++r) {
                const int row = r * 32 + lane;
                at[4 + r] = row < min(p.bn, t.rows - n0) ? p.x_bytes + (size_t)(t.row0 + n0 + row) * p.pitch : nullptr;
            }
            for (int i = part.first; ok && i < end;) {
                const int span0 = i / kSpan * kSpan, next = min(span0 + kSpan, end);
                if ((turn++ & 1) != (warp & 1)) {
                    step(next - i);
                    i = next;
                    continue;
                }
                const int left = p.valid_scales - span0 * 8;  // scale bytes of a row from here on
                uint32_t v[kRows][2 * kSpan];
                if (kSpan == 4 && p.sectors) {
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const u32x8 q = at[r] ? load_sector(at[r] + span0 * 8) : u32x8{};
                        const uint32_t w[8] = {q.lo.x, q.lo.y, q.lo.z, q.lo.w, q.hi.x, q.hi.y, q.hi.z, q.hi.w};
#pragma unroll
                        for (int k = 0; k < 2 * kSpan; ++k) v[r][k] = w[k];
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
#pragma unroll
                        for (int h = 0; h < kSpan / 2; ++h) {
                            const uint4 q = at[r] && h * 16 < left
                                                ? __ldg(reinterpret_cast<const uint4 *>(at[r] + span0 * 8 + h * 16))
                                                : make_uint4(0u, 0u, 0u, 0u);
                            v[r][4 * h] = q.x;
                            v[r][4 * h + 1] = q.y;
                            v[r][4 * h + 2] = q.z;
                            v[r][4 * h + 3] = q.w;
                        }
                }
                if (left < 8 * kSpan)  // nothing past a row's scales
#pragma unroll
                    for (int k = 0; k < 2 * kSpan; ++k) {
                        const int n = left - 4 * k;
                        const uint32_t keep = n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
#pragma unroll
                        for (int r = 0; r < kRows; ++r) v[r][k] &= keep;
                    }
#pragma unroll
                for (int q = 0; q < kSpan; ++q) {
                    if (span0 + q < i || span0 + q >= next) continue;
                    ok = ok && wait(&c->empty[s], ph, c, p.ws);
                    if (!ok) break;
                    unsigned char *to = smem + s * kStage + kScales + lane * 16;
                    const auto word = [&](int r, int end_r, int w) { return r < end_r ? v[r < kRows ? r : 0][2 * q + w] : 0u; };
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        *reinterpret_cast<uint4 *>(to + w * kScaleAtom) =
                            make_uint4(word(0, 4, w), word(1, 4, w), word(2, 4, w), word(3, 4, w));
#pragma unroll
                        for (int h = 0; h < scale_atoms(BN); ++h)
                            *reinterpret_cast<uint4 *>(to + (2 + w * scale_atoms(BN) + h) * kScaleAtom) =
                                make_uint4(word(4 * h + 4, kRows, w), word(4 * h + 5, kRows, w),
                                           word(4 * h + 6, kRows, w), word(4 * h + 7, kRows, w));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    // The first block's thread starts the copy that reads the
                    // second's scales, so they are released at cluster scope:
                    // what lies in shared memory alone, which takes no time
                    // that could be measured (440 us, with an arrival of the
                    // block's own scope 438).  A fence of all memory takes
                    // 1900 cycles a stage (1230 us against 513 at the time).
                    if (lane == 0) {
                        const uint32_t full = cluster_addr(&c->full[s], lead);
                        if (kHandOver) mbar_hand_over(full);
                        else mbar_arrive_remote(full);
                    }
                    step(1);
                }
                i = next;
            }
        }
    } else if (warp >= kEpiWarp) {
        // ---- epilogue ------------------------------------------------------
        // Two groups of four warps take the chunks of a tile in turn.
        constexpr int kChunk = chunk(MODE);
        const int q = warp & 3, g = (warp - kEpiWarp) >> 2;  // q: the lanes of tensor memory a warp may read
        unsigned char *const dw_tile = stg + kOnes + (warp - kEpiWarp) * kDwBytes;  // wgrad
        int acc = 0, turn = 0;
        uint32_t aph = 0;
        using Epilogue = std::conditional_t<MODE == kDgradSaved, SavedEpilogue, LinearEpilogue<KIND>>;
        Epilogue ep(p, stg + g * kGroup, g, q, lane);
        // all four warps of the group go on, or none
        const auto agree = [&](bool ok) {
            int all;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                         "barrier.cta.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(all)
                         : "r"((int)ok), "r"(1 + g)
                         : "memory");
            return all != 0;
        };
        // `n` finished columns of the accumulator, from column c0 of the tile on
        const auto finish = [&](uint32_t(&v)[kChunk], int m0, int n0, int c0, int n, int next) {
            if constexpr (MODE == kWgrad) {
                // lane = one row of dw, consecutive values of it
                const int m = m0 + q * 32 + lane;
                const size_t r = (size_t)t.e * p.M + m;
                if (m < p.M) {
                    if (is_bias(t)) {
                        if (p.fp32) static_cast<float *>(p.db)[r] = __uint_as_float(v[0]);
                        else static_cast<__nv_bfloat16 *>(p.db)[r] = __float2bfloat16_rn(__uint_as_float(v[0]));
                    } else if (SPLIT || p.fp32) {
                        store_row(p, r * p.N + n0 + c0, v, n);
                    }
                }
                if (!SPLIT && !p.fp32 && !is_bias(t)) store_tile(p, dw_tile, v, lane, n0 + c0, m0 + q * 32, t.e);
                __syncwarp();
            } else {
                ep.finish(v, t.row0 + n0 + c0, n, next);
            }
        };
        while (walk.next(t)) {
            const int iters = span(t).count;
            const int m0 = t.m * kBM + (int)rank * kTileM, n0 = t.n * p.bn;
            const int cols = is_bias(t) ? 1 : min(p.bn, (MODE == kWgrad ? p.N : t.rows) - n0);
            const uint32_t from = tmem + ((uint32_t)(q * 32) << 16) + acc * BN;
            const auto release = [&] {  // this warp's last look at the accumulator
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(cluster_addr(&c->acc_empty[acc], lead));
            };
            if constexpr (!SPLIT) {
                const int c_first = ((g + turn) & 1) * kChunk;
                turn += (cols + kChunk - 1) / kChunk;
                if (MODE != kWgrad) {
                    ep.tile(t.e, m0);
                    ep.ahead(t.row0 + n0 + c_first, min(kChunk, cols - c_first));
                }
                if (iters != 0) {
                    if (!agree(wait(&c->acc_full[acc], aph, c, p.ws))) break;
                    tc_fence_after();
                    if (c_first >= cols) release();
                }
                for (int c0 = c_first; c0 < cols; c0 += 2 * kChunk) {
                    uint32_t v[kChunk];
                    if (iters != 0) {
                        tmem_ld(from + c0, v);
                        tmem_wait_ld();
                        if (c0 + 2 * kChunk >= cols) release();
                    } else {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) v[i] = 0u;
                    }
                    finish(v, m0, n0, c0, min(kChunk, cols - c0), min(kChunk, cols - c0 - 2 * kChunk));
                }
            } else {
                // Every block has sums over its part of k for all columns; it
                // finishes BN / split of the columns.  Each sends the others'
                // columns to them and adds what arrives in the order of k.
                const int w = BN / split, shift = __ffs(w) - 1, mine = (int)self * w, own = min(w, cols - mine);
                if (MODE != kWgrad) {
                    ep.tile(t.e, m0);
                    ep.ahead(t.row0 + n0 + mine + g * kChunk, min(kChunk, own - g * kChunk));
                }
                bool ok = iters == 0 || wait(&c->acc_full[acc], aph, c, p.ws);
                ok = wait(&c->taken, turn ^ 1, c, p.ws) && ok;  // the last tile's sums have been read
                if (!agree(ok)) break;
                tc_fence_after();
                for (int c0 = g * kChunk; c0 < cols; c0 += 2 * kChunk) {
                    uint32_t v[kChunk];
                    if (iters != 0) {
                        tmem_ld(from + c0, v);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        const int col = c0 + i;
                        if (col >= cols) break;
                        st_cluster(cluster_addr(join + ((int)self * w + (col & (w - 1))) * kTileM + q * 32 + lane,
                                                col >> shift),
                                   iters != 0 ? v[i] : 0u);
                    }
                }
                if (iters != 0) release();
                fence_cluster();
                __syncwarp();
                if (lane < split) mbar_arrive_remote(cluster_addr(&c->joined, lane));
                if (!agree(wait(&c->joined, turn, c, p.ws))) break;
                fence_cluster();
                for (int c0 = g * kChunk; c0 < own; c0 += 2 * kChunk) {
                    uint32_t v[kChunk];
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        float sum = 0.0f;
                        if (c0 + i < own)
                            for (int o = 0; o < split; ++o) sum += join[(o * w + c0 + i) * kTileM + q * 32 + lane];
                        v[i] = __float_as_uint(sum);
                    }
                    finish(v, m0, n0, mine + c0, min(kChunk, own - c0), min(kChunk, own - c0 - 2 * kChunk));
                }
                fence_cluster();
                __syncwarp();
                if (lane < split) mbar_arrive_remote(cluster_addr(&c->taken, lane));
                turn ^= 1;
            }
            if (iters != 0) {
                acc ^= 1;
                aph ^= acc == 0;
            }
        }
        if (MODE == kWgrad && lane == 0) bulk_wait_group<0>();  // written, and out of shared memory
    }
    __syncwarp();
    if (*(volatile int *)&c->abort) {
        // given up: leave the copies and products in flight time to land
        const unsigned long long t0 = global_timer_ns();
        for (int i = 0; i < 100000 && global_timer_ns() - t0 < 1000000ull; ++i) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    if (kCluster) cluster_sync_all();
    else __syncthreads();
    if (warp == 2) tmem_free<CG>(tmem, kColumns);
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
                   const uint64_t *strides, const uint32_t *box,
                   CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B)
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
           const_cast<void *>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_rows(CUtensorMap *m, bool fp8, const void *base, int cols, int rows, int box_cols, int box_rows)
{
    const uint64_t d[2] = {(uint64_t)cols, (uint64_t)rows}, st[1] = {(uint64_t)cols};
    const uint32_t b[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
    return encode(m, fp8, base, 2, d, st, b);
}

// An MN-major operand: `cols` columns (the m or n of the product) of `rows`
// rows (its k), E of them.  A stage takes 64 rows and `blocks` blocks of 64
// columns, each block to 8 KB of its own: with one load where the columns
// are whole blocks, else one load for each.
cudaError_t encode_mn(CUtensorMap *m, const void *base, int cols, int rows, int E, int blocks, int *whole)
{
    const uint64_t per = E > 1 ? (uint64_t)cols * rows : cols;  // unused for one
    *whole = cols % 64 == 0;
    if (*whole) {
        const uint64_t d[4] = {64, (uint64_t)rows, (uint64_t)cols / 64, (uint64_t)E};
        const uint64_t st[3] = {(uint64_t)cols, 64, per};
        const uint32_t b[4] = {64, 64, (uint32_t)blocks, 1};
        return encode(m, false, base, 4, d, st, b);
    }
    const uint64_t d[4] = {(uint64_t)cols, (uint64_t)rows, 1, (uint64_t)E}, st[3] = {(uint64_t)cols, per, per};
    const uint32_t b[4] = {64, 64, 1, 1};
    return encode(m, false, base, 4, d, st, b);
}

// The same for wgrad, whose k are packed rows: the window axis before the rows
// slides over them (both have the row's stride), so that value (c, i, r) is
// column c of row r + i for 0 <= i < 64.  A load that starts at i = -z gets z
// rows of zeros and then rows r .. r + 63 - z, whatever follows those.  Only
// rows that the load asks for are read: r + i stays below `rows`.
cudaError_t encode_window(CUtensorMap *m, const void *base, int cols, int rows, int blocks, int *whole)
{
    const uint64_t pitch = (uint64_t)cols, r = (uint64_t)rows;
    *whole = cols % 64 == 0;
    if (*whole) {
        const uint64_t d[4] = {64, 64, r, pitch / 64}, st[3] = {pitch, pitch, 64};
        const uint32_t b[4] = {64, 64, 1, (uint32_t)blocks};
        return encode(m, false, base, 4, d, st, b);
    }
    const uint64_t d[4] = {pitch, 64, r, 1}, st[3] = {pitch, pitch, pitch};
    const uint32_t b[4] = {64, 64, 1, 1};
    return encode(m, false, base, 4, d, st, b);
}

template <int CG, int BN, int MODE, int KIND, bool SPLIT>
cudaError_t launch(const Params &p, cudaStream_t s)
{
    // No programmatic dependent launch: do not add it.  With it (tensor memory
    // allocated before the wait for the predecessor) a sequence of the
    // elementwise gradient, dgrad, wgrad and a column sum stopped for good
    // after some passes, outside every bounded wait, and the cause was not
    // found.  Without it no block starts before the kernels ahead of it on
    // its stream are complete, and the waits that have no limit end:
    //   tcgen05.alloc: no other block of these kernels fits on the SM (below),
    //     so its tensor memory is free, or held by a kernel of another stream
    //     that gives it back without waiting for this one;
    //   the cluster barriers: the first comes before any other wait; every
    //     role's loop ends, by its tiles or by a limit, and meets the second;
    //   an epilogue group's barriers: its four warps decide together (agree)
    //     and walk the same chunks;
    //   bulk_wait_group, tcgen05.wait::ld: copies and loads already issued,
    //     which depend on nothing else.
    static_assert(2 * (smem_bytes(CG, BN, MODE, KIND, SPLIT) + 1024) > 228 * 1024, "one block on an SM");
    const auto fn = experts_kernel<CG, BN, MODE, KIND, SPLIT>;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(fn), smem_bytes(CG, BN, MODE, KIND, SPLIT));
    if (err != cudaSuccess) return err;
    // the most tiles that offsets over these rows can give
    const long long tm = (p.M + kTileM * CG - 1) / (kTileM * CG);
    const long long tn = MODE == kWgrad ? (long long)p.E * ((p.N + p.bn - 1) / p.bn + 1)
                                            : p.rows / p.bn + (p.rows < p.E ? p.rows : p.E);
    const int cluster = SPLIT ? p.split : CG;

    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(CG, BN, MODE, KIND, SPLIT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    cfg.gridDim = dim3((unsigned)cluster);
    long long blocks = device_sm_count() / cluster;
    if (cluster > 2) {
        // how many such clusters the GPCs hold at once: asked once per device and size
        static std::atomic<int> held[64][2];
        int dev = 0;
        err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        int n = dev < 64 ? held[dev][cluster / 8].load(std::memory_order_relaxed) : 0;
        if (n == 0) {
            err = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
            if (err != cudaSuccess) return err;
            if (dev < 64) held[dev][cluster / 8].store(n, std::memory_order_relaxed);
        }
        if (n < blocks) blocks = n;
    }
    if (tm * tn < blocks) blocks = tm * tn;
    if (blocks < 1) blocks = 1;
    cfg.gridDim = dim3((unsigned)(blocks * cluster));
    return cudaLaunchKernelEx(&cfg, fn, p);
}

template <int MODE, int KIND>
cudaError_t launch_cut(Params &p, const Cut &c, cudaStream_t s)
{
    p.bn = c.bn;
    p.split = c.split;
    if (c.cg == 2) return launch<2, KIND == kFp4 ? kFp4Wide : 256, MODE, KIND, false>(p, s);
    if constexpr (MODE != kWgrad)
        if (c.bn == 32)
            return c.split > 1 ? launch<1, 32, MODE, KIND, true>(p, s) : launch<1, 32, MODE, KIND, false>(p, s);
    return c.split > 1 ? launch<1, 128, MODE, KIND, true>(p, s) : launch<1, 128, MODE, KIND, false>(p, s);
}

template <int KIND>
cudaError_t linear(const moe_rows *G, const void *x, const void *x_scales, int K, const void *w, const void *w_scales,
                   int N, const void *bias, int act, const void *residual, void *y, void *saved, void *saved_scales,
                   cudaStream_t s)
{
    Params p = {};
    p.offsets = G->offsets;
    p.ws = G->ws;
    p.E = G->E;
    p.rows = G->rows;
    p.M = N;
    p.act = act;
    p.glu = act == MOE_ACT_SWIGLU;
    p.bias = static_cast<const __nv_bfloat16 *>(bias);
    p.residual = static_cast<const __nv_bfloat16 *>(residual);
    if (KIND == kE4m3) {
        p.x_scales = static_cast<const float2 *>(x_scales);
        p.w_scales = static_cast<const float2 *>(w_scales);
    } else if (KIND == kFp4) {
        p.x_bytes = static_cast<const uint8_t *>(x_scales);
        p.w_bytes = static_cast<const uint8_t *>(w_scales);
        p.pitch = MOE_FP4_PITCH(K);
        p.valid_scales = K / 32;
        p.sectors = p.pitch % 32 == 0 && reinterpret_cast<uintptr_t>(x_scales) % 32 == 0 &&
                    reinterpret_cast<uintptr_t>(w_scales) % 32 == 0;
    }
    p.y = static_cast<__nv_bfloat16 *>(y);
    p.saved = static_cast<uint8_t *>(saved);
    p.saved_scales = static_cast<uint8_t *>(saved_scales);
    const bool bytes = KIND != kBf16;  // the tensor maps' unit; two values of kFp4
    const int cols = KIND == kFp4 ? K / 2 : K, elems = bytes ? 128 : 64;
    p.K = bytes ? cols : 2 * cols;
    const Cut cut = KIND == kFp4 ? rows_cut_fp4(N, G->rows, G->E, (cols + 127) / 128)
                                 : rows_cut(N, G->rows, G->E, (cols + elems - 1) / elems);
    // w as [E][N/halves][halves][K] with the halves inside: one load brings
    // gate and up rows alternating, so that a pair of them ends in one lane
    const uint64_t h = p.glu ? 2 : 1, n = (uint64_t)N / h, k = (uint64_t)cols;
    const uint64_t d[4] = {k, h, n, (uint64_t)G->E};
    const uint64_t st[3] = {n * k, k, (uint64_t)N * k};
    const uint32_t b[4] = {(uint32_t)elems, (uint32_t)h, (uint32_t)(kTileM / h), 1};
    cudaError_t err = encode(&p.ma, bytes, w, 4, d, st, b);
    if (err == cudaSuccess) err = encode_rows(&p.mb, bytes, x, cols, G->rows, elems, cut.bn / cut.cg);
    if (err == cudaSuccess && cut.bn > 32) err = encode_rows(&p.mb32, bytes, x, cols, G->rows, elems, 32);
    if (err != cudaSuccess) return err;
    return launch_cut<kLinear, KIND>(p, cut, s);
}

template <int MODE>
cudaError_t dgrad(const moe_rows *G, const void *dy, int N, const void *w, int K, int act, const void *saved,
                  const void *saved_scales, void *dx, void *a, cudaStream_t s)
{
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
    const Cut cut = rows_cut(K, G->rows, G->E, (N + 63) / 64);
    cudaError_t err = encode_mn(&p.ma, w, K, N, G->E, 2, &p.whole_a);
    if (err == cudaSuccess) err = encode_rows(&p.mb, false, dy, N, G->rows, 64, cut.bn / cut.cg);
    if (err == cudaSuccess && cut.bn > 32) err = encode_rows(&p.mb32, false, dy, N, G->rows, 64, 32);
    if (err != cudaSuccess) return err;
    return launch_cut<MODE, kBf16>(p, cut, s);
}

}  // namespace
}  // namespace moe
