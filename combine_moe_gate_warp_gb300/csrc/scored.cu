// scored.cu -- routing by scores (moe_gate_scored) and its gradient.
//
// The score s_e of an expert is the sigmoid of its logit or its share in the
// softmax of all.  A bias is added for the selection only; groups of
// consecutive experts are ranked by the sum of their one or two best
// v_e = s_e + bias_e, and the k best experts of the best groups are taken.
//
// Which of two experts is the better one is decided as 64 bits decide it:
// two scores that fp32 cannot tell apart, or tells apart by its own rounding,
// are common (8 of 256 experts: a few tokens in a thousand), and a selection
// that depended on the order of some sum would not be one that a test, a
// second run elsewhere or a backward pass could repeat.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "gate_stats.cuh"
#include "launchers.h"
#include "tma.cuh"

namespace moe {
namespace {

constexpr float kTiny = 1e-20f;  // beside the sum of the selected scores

struct GateArgs {
    const float *logits;
    int T, E, k;
    moe_scoring S;
    int32_t *idx;
    float *gates;
    int32_t *counts;
    double *aux, *ent;
    void *ws;
};

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The values v_e of a row in 64 bits, for a whole warp: the one definition that
// every selection in 64 bits goes by, the division by the softmax's sum too:
// scores that differ by less than it rounds are a tie.  Among experts without a
// bias the undivided exp(l - top) has the same order wherever `clear` says so,
// and the sum is left out there (50021 tokens, 60 experts: 28.8 us, with it
// 29.8).  `at_once`: divided from the start.
struct Row64 {
    double top, sum;
    bool divided;
    __device__ Row64(const float *row, const GateArgs &a, int lane, bool at_once) : top(0.0), sum(1.0), divided(true)
    {
        if (a.S.score != MOE_SCORE_SOFTMAX) return;
        float t = -INFINITY;
        for (int e = lane; e < a.E; e += 32) t = fmaxf(t, row[e]);
        top = warp_max(t);
        divided = false;
        if (a.S.bias || at_once) divide(row, a, lane);
    }
    __device__ void divide(const float *row, const GateArgs &a, int lane)
    {
        sum = 0.0;
        for (int e = lane; e < a.E; e += 32) sum += exp((double)row[e] - top);
        sum = warp_sum(sum);
        divided = true;
    }
    __device__ double value(const float *row, const GateArgs &a, int e) const
    {
        const double l = row[e];
        double v = a.S.score == MOE_SCORE_SOFTMAX ? exp(l - top) / sum : 1.0 / (1.0 + exp(-l));
        if (a.S.bias) v += (double)a.S.bias[e];
        return v == v ? v : -INFINITY;  // a NaN is reported as bad data; the ids stay valid
    }
    // Whether the order of exp(l - top) is that of the scores, whatever the
    // rounding of the division: two logits of this size are equal, or 2^-46
    // apart, and the quotients are not subnormal (the sum is at most 256).
    __device__ bool clear(float l) const { return fabsf(l) >= 0x1p-23f && (double)l - top > -600.0; }
};

// --------------------------------------------------------------------------
// One token in 64 bits, by a whole warp: lane j < k gets slot j's expert.
// --------------------------------------------------------------------------
struct Scratch {
    double *v, *group;    // [E], [groups]
    unsigned char *kept;  // [groups]
    static __host__ __device__ int bytes(int E, int G) { return 8 * E + 9 * G; }
    __device__ Scratch(void *p, int E, int G)
        : v(static_cast<double *>(p)), group(v + E), kept(reinterpret_cast<unsigned char *>(group + G))
    {
    }
};

__device__ __noinline__ int select64(const float *row, const GateArgs &a, void *memory, int lane)
{
    const int E = a.E, per = E / a.S.groups;
    const Scratch s(memory, E, a.S.groups);
    const Row64 r(row, a, lane, true);
    unsigned mine = 0;  // experts lane, lane + 32, ... still to choose from
    for (int e = lane, i = 0; e < E; e += 32, ++i) {
        s.v[e] = r.value(row, a, e);
        mine |= 1u << i;
    }
    __syncwarp();
    if (a.S.top_groups < a.S.groups) {
        for (int g = lane; g < a.S.groups; g += 32) {
            double first = -INFINITY, second = -INFINITY;
            for (int e = g * per; e < (g + 1) * per; ++e) {
                const double v = s.v[e];
                second = fmax(second, fmin(first, v));
                first = fmax(first, v);
            }
            s.group[g] = a.S.group_top == 2 ? first + second : first;
        }
        __syncwarp();
        for (int g = lane; g < a.S.groups; g += 32) {
            const double v = s.group[g];
            int before = 0;
            for (int h = 0; h < a.S.groups; ++h) before += s.group[h] > v || (s.group[h] == v && h < g);
            s.kept[g] = before < a.S.top_groups;
        }
        __syncwarp();
        for (int e = lane, i = 0; e < E; e += 32, ++i)
            if (!s.kept[e / per]) mine &= ~(1u << i);
    }
    int slot = 0;
    for (int j = 0; j < a.k; ++j) {
        double best = 0.0;
        int id = -1;
        for (int e = lane, i = 0; e < E; e += 32, ++i)
            if ((mine >> i & 1u) && (id < 0 || s.v[e] > best)) {
                best = s.v[e];
                id = e;
            }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const double v = __shfl_xor_sync(0xffffffffu, best, d);
            const int o = __shfl_xor_sync(0xffffffffu, id, d);
            if (o >= 0 && (id < 0 || v > best || (v == best && o < id))) {
                best = v;
                id = o;
            }
        }
        if ((id & 31) == lane) mine &= ~(1u << (id >> 5));
        if (lane == j) slot = id;
    }
    __syncwarp();
    return slot;
}

__device__ __forceinline__ double warp_max(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// The kept groups, where those between `low` and `high` are ordered in 64 bits,
// by a whole warp: those above, and the best of these.  False if there are more
// than 32 of these.
__device__ __noinline__ bool groups_near(const float *row, const GateArgs &a, const unsigned *values, int low, int high,
                                         unsigned *kept, int lane)
{
    const int G = a.S.groups, per = a.E / G;
    int n = 0, above = 0, mine = -1;  // lane b: the border's group b
    for (int g0 = 0; g0 < G; g0 += 32) {
        const int g = g0 + lane, v = g < G ? (int)(values[g] >> 8) : 0;
        const unsigned over = __ballot_sync(0xffffffffu, g < G && v > high);
        if (g < G && v > high) kept[above + __popc(over & ((1u << lane) - 1u))] = (unsigned)g;
        above += __popc(over);
        const unsigned who = __ballot_sync(0xffffffffu, g < G && v >= low && v <= high);
        const int c = __popc(who);
        // the (lane - n)-th of them
        if (lane >= n && lane < n + c) mine = g0 + __fns(who, 0, lane - n + 1);
        n += c;
    }
    if (n > 32) return false;
    const Row64 r(row, a, lane, true);
    double value = 0.0;
    for (int b = 0; b < n; ++b) {
        const int g = __shfl_sync(0xffffffffu, mine, b);
        double first = -INFINITY, second = -INFINITY;
        for (int i = lane; i < per; i += 32) {
            const double v = r.value(row, a, g * per + i);
            second = fmax(second, fmin(first, v));
            first = fmax(first, v);
        }
        const double m = warp_max(first);
        double sum = m;
        if (a.S.group_top == 2) {
            const int who = __ffs(__ballot_sync(0xffffffffu, first == m)) - 1;
            sum += warp_max(lane == who ? second : first);
        }
        if (lane == b) value = sum;
    }
    int before = 0;
    for (int b = 0; b < n; ++b) {
        const double v = __shfl_sync(0xffffffffu, value, b);
        const int g = __shfl_sync(0xffffffffu, mine, b);
        before += v > value || (v == value && g < mine);
    }
    if (lane < n && above + before < a.S.top_groups) kept[above + before] = (unsigned)mine;
    __syncwarp();
    return true;
}

struct Kept {
    const unsigned *keys;    // of the token's experts
    const unsigned *groups;  // its kept groups
    int per, count;          // experts of a group, and of all kept ones
};

// The k best of a token's candidates in 64 bits, by a whole warp: the k ids in
// sel, and the other kept experts whose key is at most `near` steps behind the
// last one's.  The rest are behind for certain.  One candidate a lane; false
// (and nothing done) if there are more.
__device__ __noinline__ bool select_near(const float *row, const GateArgs &a, const Kept &kept, unsigned last, int near,
                                         unsigned *sel, unsigned *list, int lane)
{
    int n = a.k;
    if (lane < n) list[lane] = sel[lane];
    for (int m0 = 0; m0 < kept.count; m0 += 32) {
        const int m = m0 + lane, g = m / kept.per;
        const int e = m < kept.count ? (int)kept.groups[g] * kept.per + m - g * kept.per : 0;
        const unsigned key = m < kept.count ? kept.keys[e] : 0u;
        const bool also = key != 0u && key < last && (int)(key >> 9) >= (int)(last >> 9) - near;
        const unsigned who = __ballot_sync(0xffffffffu, also);
        const int at = n + __popc(who & ((1u << lane) - 1u));
        if (also && at < 32) list[at] = (unsigned)e;
        n += __popc(who);
    }
    if (n > 32) return false;
    __syncwarp();
    const int id = lane < n ? (int)list[lane] : 0;
    Row64 r(row, a, lane, false);
    double v = r.value(row, a, id);
    if (!r.divided && !__all_sync(0xffffffffu, lane >= n || r.clear(row[id]))) {
        r.divide(row, a, lane);
        v = r.value(row, a, id);
    }
    int before = 0;
    for (int c = 0; c < n; ++c) {
        const double o = __shfl_sync(0xffffffffu, v, c);
        const int oid = __shfl_sync(0xffffffffu, id, c);
        before += o > v || (o == v && oid < id);
    }
    if (lane < n && before < a.k) sel[before] = (unsigned)id;
    __syncwarp();
    return true;
}

__device__ __forceinline__ float sigmoid(float l)
{
    const float e = expf(-fabsf(l));  // no overflow, and digits down to the subnormals
    const float q = __frcp_rn(1.0f + e);
    return l < 0.0f ? e * q : q;
}

// --------------------------------------------------------------------------
// The selection on 32-bit keys.  L lanes share a token.  A value v becomes a
// whole number q of 23 bits, q = (v - lowest) * steps, and with the expert's
// id below it one key: largest key first means largest value, then lowest id,
// and a comparison with its exchange is two instructions, min and max.  Lists
// of KL keys are sorted by Batcher's networks, merged, and merged across the
// lanes of a token.
//
// What bounds it: the latency of its instructions, of which 16 warps an SM (128
// registers a thread) issue 0.46 a cycle and scheduler; alone the 109 a token
// at 64 experts would take 23 us.  HBM is at a fifth.  262144 tokens, 64
// experts in 8 groups, top-8 of 4 groups: 62 us; 16384 tokens, 256 experts in
// 16 groups: 26 us; a few tokens: 8 us, by the host.  All of it in 64 bits, a
// warp for each token, took 2994, 430 and 17 us.
//
// The time depends on the values: q has steps of the whole span of scores and
// biases, and whatever lies within a few of them goes to 64 bits.  262144
// tokens as above, L2 flushed: logits of spread 1 and 3 without a bias 66 and
// 68 us, 4 79, 6 (half of the tokens have scores that round alike) 248, 8 609;
// one expert's bias at -1: 68 us, at -100 136, at -10000 1408, at -10^6 and
// below 7327.
//
// What q does not decide is found and decided elsewhere: with the bound on
// q's error below, neighbours in the order that are at most `near` apart, and
// groups at the border between kept and dropped that are, may be the other
// way round.  Equal logits with equal biases are equal values, and rightly in
// the order of their ids.  Whatever else is that close is settled in 64 bits by
// the whole warp: the groups of the border and the candidates alone
// (groups_near, select_near) or, where those are too many, the token anew
// (select64).
//
// A warp copies its tokens' logits to shared memory, and the keys take their
// place there.  With several lanes to a token the rows start in other banks:
// row pitch = L modulo 32.  With one lane the rows lie as in memory, and the
// lanes whose rows start in the same bank start at different experts.
// --------------------------------------------------------------------------
constexpr float kSteps = 8388600.0f;  // of q, below 2^23

// q's error in steps.  The exponential (ex2.approx, 2 steps of 2^-23) with its
// argument's rounding and the reciprocal (1 step) leave a sigmoid within
// 1.25 * 2^-22 of its value, 2.5 steps for values that span 1 or more; the
// bias less the lowest, the bias term and the sum are rounded: 0.5 each.  4
// in all, 8 for two values.
constexpr int kNearSigmoid = 10;
// Softmax: exp(l - max) (expf, 2 steps of 2^-23, and its argument's rounding)
// is within 1.2 * 2^-22 of it, 2.4 steps, and 1.5 as above: 8 for two.  The sum
// of E terms, in 8 parts or more, and its reciprocal are within 42 * 2^-24;
// they scale all scores alike and matter where a bias is added: 21 steps more.
constexpr int kNearSoftmax = 10, kNearSoftmaxBias = 32;

__device__ __forceinline__ unsigned make_key(float steps, int e)  // steps in [2^23, 2^24)
{
    return (__float_as_uint(steps) << 9) + (unsigned)(511 - e);
}
__device__ __forceinline__ int key_id(unsigned key) { return 511 - (int)(key & 511u); }

template <int KL>
__device__ __forceinline__ void order(unsigned (&x)[KL], int i, int j)  // larger first
{
    const unsigned a = max(x[i], x[j]), b = min(x[i], x[j]);
    x[i] = a;
    x[j] = b;
}
// Batcher's odd-even merge sort
template <int KL>
__device__ __forceinline__ void sort_keys(unsigned (&x)[KL])
{
#pragma unroll
    for (int p = 1; p < KL; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j <= KL - 1 - q; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < KL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order(x, i + j, i + j + q);
}
// The KL largest of two sorted lists, sorted; `rest`: the largest of those left out.
template <int KL>
__device__ __forceinline__ void merge_keys(unsigned (&x)[KL], const unsigned (&y)[KL], unsigned &rest)
{
#pragma unroll
    for (int i = 0; i < KL; ++i) {
        rest = max(rest, min(x[i], y[KL - 1 - i]));
        x[i] = max(x[i], y[KL - 1 - i]);
    }
#pragma unroll
    for (int q = KL / 2; q >= 1; q /= 2)
#pragma unroll
        for (int i = 0; i < KL; ++i)
            if (!(i & q)) order(x, i, i + q);
}

template <int L, typename F>
__device__ __forceinline__ F lanes_max(F v)
{
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}
template <int L, typename F>
__device__ __forceinline__ F lanes_sum(F v)
{
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
template <int L>
__device__ __forceinline__ unsigned lanes_min(unsigned v)
{
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kGateWarps = 4;

__host__ __device__ inline int row_pitch(int E, int L)
{
    return L == 1 || L == 32 ? E : (E + 31 - L) / 32 * 32 + L;
}
// Words of shared memory of a warp: keys, where select64 works once the lists
// are made; groups' values, and in their place the ids that select_near and
// select64 find; kept groups; a list for select_near.
__host__ __device__ inline int up16(int n) { return (n + 15) / 16 * 16; }
__host__ __device__ inline int key_words(int E, int G, int L)
{
    const int keys = 32 / L * row_pitch(E, L), work = (Scratch::bytes(E, G) + 3) / 4;
    return up16(keys > work ? keys : work);
}
__host__ __device__ inline int group_pitch(int G, int k) { return (G > k ? G : k) | 1; }
__host__ __device__ inline int warp_words(int E, int G, int top, int k, int L)
{
    return key_words(E, G, L) + up16(32 / L * (group_pitch(G, k) + (top | 1))) + 32;
}

__device__ __forceinline__ unsigned lds_u32(unsigned at)
{
    unsigned v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ void copy_async4(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_async16(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_async_all()
{
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

template <int KL, int L>
__global__ void __launch_bounds__(32 * kGateWarps, 4) gate_scored_kernel(const __grid_constant__ GateArgs a)
{
    constexpr int kTokens = 32 / L;
    constexpr unsigned kAll = L == 32 ? ~0u : (1u << L) - 1u;  // the lanes of the first token
    extern __shared__ __align__(64) unsigned s_dyn[];
    __shared__ float s_bias[MOE_MAX_EXPERTS];  // less the lowest, in steps + 2^23 (sigmoid)
    __shared__ unsigned s_hist[MOE_MAX_EXPERTS];
    __shared__ float s_low[kGateWarps], s_high[kGateWarps];
    __shared__ int s_last;
    WsHeader *ws = static_cast<WsHeader *>(a.ws);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L, tok = lane / L;
    const int E = a.E, k = a.k, G = a.S.groups, per = E / G, pitch = row_pitch(E, L);
    const bool softmax = a.S.score == MOE_SCORE_SOFTMAX, grouped = a.S.top_groups < G;
    const int top = a.S.top_groups;
    unsigned *const rows = s_dyn + warp * warp_words(E, G, top, k, L);
    const int gp = group_pitch(G, k);
    unsigned *const groups = rows + key_words(E, G, L), *const kept_groups = groups + kTokens * gp;
    unsigned *const list = groups + up16(kTokens * (gp + (top | 1)));
    unsigned *const mine = rows + tok * pitch, *const mk = kept_groups + tok * (top | 1);
    unsigned *const mg = groups + tok * gp;   // values of the groups of this lane's token
    unsigned *const sel = mg;                 // [k] its ids, later
    // the kept experts: those of `top` groups, or all
    const Kept kept = {mine, mk, grouped ? per : E, grouped ? top * per : E};
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_hist[e] = 0u;
    pdl_wait();
    pdl_launch_dependents();

    // L == 1: where this lane starts in its row (see above)
    const int common = E & -E & 31 ? E & -E : 32, turn = L == 1 ? lane * common / 32 : 0;
    const int turn_group = turn / kept.per, turn_in = turn - turn_group * kept.per;
    // the logits of a warp's tokens; zeros past the last
    const auto load = [&](long long t0) {
        const int tokens = (int)min((long long)kTokens, a.T - t0);
        const float *const tile = a.logits + t0 * E;
        if (L == 1) {
            const int there = tokens * E, whole = there & ~3;
#pragma unroll 4
            for (int i = 4 * lane; i < 32 * E; i += 128)
                if (i < whole || i >= there) copy_async16(rows + i, i < whole ? tile + i : tile, i < whole);
            if (whole != there && lane < 4) {
                const int i = whole + lane;
                copy_async4(rows + i, tile + (i < there ? i : 0), i < there);
            }
        } else if (L % 4 == 0 && (E & 3) == 0) {
            for (int r = 0; r < kTokens; ++r)
                for (int e = 4 * lane; e < E; e += 128)
                    copy_async16(rows + r * pitch + e, tile + (r < tokens ? r * E + e : 0), r < tokens);
        } else if (E >= 32) {
            for (int r = 0; r < kTokens; ++r)
                for (int e = lane; e < E; e += 32)
                    copy_async4(rows + r * pitch + e, tile + (r < tokens ? r * E + e : 0), r < tokens);
        } else {  // the rows lie one after the other: a flat copy
            int r = lane / E, c = lane - r * E;
            const int dr = 32 / E, dc = 32 - dr * E;
            for (int i = lane; i < kTokens * E; i += 32) {
                copy_async4(rows + r * pitch + c, tile + (i < tokens * E ? i : 0), i < tokens * E);
                r += dr;
                c += dc;
                if (c >= E) {
                    c -= E;
                    ++r;
                }
            }
        }
    };
    const long long first_token = ((long long)blockIdx.x * kGateWarps + warp) * kTokens;
    if (first_token < a.T) load(first_token);  // while the biases are looked at
    float check = 0.0f;  // stays 0 over finite values
    float low = 0.0f, high = 0.0f;
    if (a.S.bias) {
        low = INFINITY;
        high = -INFINITY;
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            const float b = a.S.bias[e];
            check = fmaf(b, 0.0f, check);
            low = fminf(low, b);
            high = fmaxf(high, b);
        }
        high = warp_max(high);
        low = -warp_max(-low);
        if (lane == 0) {
            s_low[warp] = low;
            s_high[warp] = high;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kGateWarps; ++w) {
            low = fminf(low, s_low[w]);
            high = fmaxf(high, s_high[w]);
        }
    }
    const float span = high - low;
    const float steps = softmax ? 1.0f : kSteps / (1.0f + span);
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const float b = a.S.bias ? a.S.bias[e] - low : 0.0f;
        s_bias[e] = softmax ? b : fmaf(b, steps, 8388608.0f);
    }
    __syncthreads();
    const int near = softmax ? (a.S.bias ? kNearSoftmaxBias : kNearSoftmax) : kNearSigmoid;

    const long long stride = (long long)gridDim.x * kGateWarps * kTokens;
    for (long long t0 = first_token; t0 < a.T; t0 += stride) {
        const int tokens = (int)min((long long)kTokens, a.T - t0);
        const float *const tile = a.logits + t0 * E;
        const bool on = tok < tokens;
        const float *const row = tile + (on ? tok : 0) * E;  // of this lane's token
        copy_async_all();
        __syncwarp();

        // keys in place of the logits
        float total = 1.0f, peak = 0.0f, unit = 1.0f, scale = 1.0f;
        if (softmax) {
            // a lane's n-th expert
            const auto nth = [&](int n) { return L == 1 ? (n + turn >= E ? n + turn - E : n + turn) : sub + n * L; };
            const int each = L == 1 ? E : (E - sub + L - 1) / L;
            peak = -INFINITY;
#pragma unroll 8
            for (int n = 0; n < each; ++n) peak = fmaxf(peak, __uint_as_float(mine[nth(n)]));
            peak = lanes_max<L>(peak);
            float part[8] = {};
            for (int n0 = 0; n0 < each; n0 += 8) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (n0 + u < each) {
                        const int e = nth(n0 + u);
                        const float l = __uint_as_float(mine[e]);
                        check = fmaf(l, 0.0f, check);
                        const float x = expf(l - peak);
                        part[u] += x;
                        mine[e] = __float_as_uint(x);
                    }
                }
            }
            total = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
            total = lanes_sum<L>(total);
            // without a bias the order is that of exp(l - peak)
            const float inv = a.S.bias ? reciprocal_fast(total) : 1.0f;
            unit = kSteps / (inv + span);
            scale = inv * unit;
        }
        // the key of the value (softmax: exp(l - peak), else the logit) at x[i],
        // expert e0 + i
        const auto key = [&](auto soft, const unsigned *x, const float *bias, int e0, int i) {
            const float v = __uint_as_float(x[i]);
            if constexpr (decltype(soft)::value)
                return make_key(fmaf(v, scale, fmaf(bias[i], unit, 8388608.0f)), e0 + i);
            check = fmaf(v, 0.0f, check);
            return make_key(fmaf(reciprocal_fast(1.0f + exp2_fast(v * -kLog2e)), steps, bias[i]), e0 + i);
        };
        bool unsure = false, unsure_groups = false;
        const auto same = [&](int e, int o) {  // equal values for certain
            return row[e] == row[o] && (!a.S.bias || a.S.bias[e] == a.S.bias[o]);
        };
        if (grouped) {
            const bool two = a.S.group_top == 2;
            const auto best = [&](int g, unsigned &first, unsigned &second) {
                // lanes of a token start at different experts: other banks
                const unsigned *const x = mine + g * per;
                first = second = 0u;
                int i = L == 1 ? 0 : sub % per;
                for (int n = 0; n < per; ++n) {
                    const unsigned v = x[i];
                    second = max(second, min(first, v));
                    first = max(first, v);
                    if (++i == per) i = 0;
                }
            };
            if (L == 1) {
                const auto fill = [&](auto soft) {
                    int g = turn_group;
                    for (int n = 0; n < G; ++n) {
                        unsigned first = 0u, second = 0u;
                        unsigned *const x = mine + g * per;
                        const float *const bias = s_bias + g * per;
                        int i = turn_in;
#pragma unroll 8
                        for (int m = 0; m < per; ++m) {
                            const unsigned v = key(soft, x, bias, g * per, i);
                            x[i] = v;
                            second = max(second, min(first, v));
                            first = max(first, v);
                            i = i + 1 == per ? 0 : i + 1;
                        }
                        mg[g] = ((first >> 9) + (two ? second >> 9 : 0u)) << 8 | (unsigned)(255 - g);
                        g = g + 1 == G ? 0 : g + 1;
                    }
                };
                if (softmax) fill(std::true_type());
                else fill(std::false_type());
            } else {
                const auto fill = [&](auto soft) {
#pragma unroll 4
                    for (int e = sub; e < E; e += L) mine[e] = key(soft, mine, s_bias, 0, e);
                };
                if (softmax) fill(std::true_type());
                else fill(std::false_type());
                __syncwarp();
                for (int g = sub; g < G; g += L) {
                    unsigned first, second;
                    best(g, first, second);
                    mg[g] = ((first >> 9) + (two ? second >> 9 : 0u)) << 8 | (unsigned)(255 - g);
                }
                __syncwarp();
            }
            unsigned least = ~0u, most = 0u;  // kept, dropped
            if (G <= (L == 1 ? 16 : 64)) {
                // few groups: each one's place among all
                for (int g = sub; g < G; g += L) {
                    const unsigned v = mg[g];
                    int before = 0;
#pragma unroll 8
                    for (int h = 0; h < G; ++h) before += mg[h] > v;
                    if (before < top) {
                        least = min(least, v);
                        mk[before] = (unsigned)g;
                    } else {
                        most = max(most, v);
                    }
                }
            } else {
                // many: a value between the last kept and the first dropped, by
                // halving.  The values differ, so there is one.  169897 tokens,
                // 112 experts in 56 groups: 160 us, by the places 253; with 8
                // lanes 21757 tokens, 192 experts in 96 groups: 80 and 90 us,
                // 87590 tokens, 82 experts in 41 groups: 115 and 101.
                unsigned lo = ~0u, hi = 0u;
                for (int g = sub; g < G; g += L) {
                    lo = min(lo, mg[g]);
                    hi = max(hi, mg[g]);
                }
                lo = lanes_min<L>(lo) - 1u;  // all are above lo, none above hi
                hi = lanes_max<L>(hi);
                unsigned cut = lo;
                bool found = false;
                while (!__all_sync(0xffffffffu, found)) {
                    const unsigned mid = lo + (hi - lo) / 2u;
                    int n = 0;
#pragma unroll 8
                    for (int g = sub; g < G; g += L) n += mg[g] > mid;
                    n = lanes_sum<L>(n);
                    if (n == top) {
                        cut = mid;
                        found = true;
                    }
                    if (n > top) lo = mid;
                    else hi = mid;
                }
                int at = 0;
                for (int g0 = 0; g0 < G; g0 += L) {
                    const int g = g0 + sub;
                    const unsigned v = g < G ? mg[g] : 0u;
                    const bool in = g < G && v > cut;
                    const unsigned who = __ballot_sync(0xffffffffu, in) >> (tok * L) & kAll;
                    if (in) {
                        mk[at + __popc(who & ((1u << sub) - 1u))] = (unsigned)g;
                        least = min(least, v);
                    } else if (g < G) {
                        most = max(most, v);
                    }
                    at += __popc(who);
                }
            }
            least = lanes_min<L>(least);
            most = lanes_max<L>(most);
            const int far = two ? 2 * near : near;
            if ((int)(least >> 8) - (int)(most >> 8) <= far) {
                // Groups near the border are in order only if they are equal:
                // the best of each, whose lead over the rest is certain.
                unsigned r1, r2;
                best(255 - (int)(least & 255u), r1, r2);
                const int a1 = key_id(r1), a2 = key_id(r2);
                for (int g = sub; g < G; g += L) {
                    const int v = (int)(mg[g] >> 8);
                    if (v > (int)(most >> 8) + far || v < (int)(least >> 8) - far) continue;
                    unsigned f1, f2;
                    best(g, f1, f2);
                    const int b1 = key_id(f1), b2 = key_id(f2);
                    unsure_groups |=
                        two ? !((same(a1, b1) && same(a2, b2)) || (same(a1, b2) && same(a2, b1))) : !same(a1, b1);
                    const unsigned last = two ? f2 : f1;
                    for (int i = g * per; i < (g + 1) * per; ++i)
                        if (mine[i] < last && (int)(mine[i] >> 9) >= (int)(last >> 9) - near)
                            // one that equals the second, and with it may be above a near first
                            unsure_groups |= !same(i, key_id(last)) ||
                                             (two && (int)(f1 >> 9) - (int)(f2 >> 9) <= near && !same(b1, b2));
                }
            }
            unsigned ask = __ballot_sync(0xffffffffu, on && unsure_groups);
            unsure_groups = false;
            while (ask != 0u) {
                const int who = (__ffs(ask) - 1) / L;
                ask &= ~(kAll << (who * L));
                const int low = (int)(__shfl_sync(0xffffffffu, least, who * L) >> 8) - far;
                const int high = (int)(__shfl_sync(0xffffffffu, most, who * L) >> 8) + far;
                __syncwarp();
                if (!groups_near(tile + who * E, a, groups + who * gp, low, high, kept_groups + who * (top | 1), lane))
                    unsure_groups |= tok == who;
            }
        } else {
            const auto fill = [&](auto soft) {
                int e = L == 1 ? turn : sub;
#pragma unroll 8
                for (int n = sub; n < E; n += L) {
                    mine[e] = key(soft, mine, s_bias, 0, e);
                    e += L;
                    if (L == 1 && e == E) e = 0;
                }
            };
            if (softmax) fill(std::true_type());
            else fill(std::false_type());
            if (sub == 0) mk[0] = 0u;
        }
        __syncwarp();

        // The largest keys of the kept experts.  A lane takes every L-th of
        // them, group after group.
        unsigned lst[KL], rest = 0u;
        if (L == 1 && kept.per % KL == 0) {
            // whole lists at a time.  The lanes take a list's keys in different
            // orders: other banks
            const unsigned from = (unsigned)(lane & (KL - 1)) * 4u;
#pragma unroll
            for (int u = 0; u < KL; ++u) lst[u] = 0u;
            int n = 0, c = 0;
            for (int done = 0; done < kept.count; done += KL) {
                unsigned x[KL];
                const unsigned at = smem_addr(mine + mk[n] * kept.per + c) + from;
#pragma unroll
                for (int u = 0; u < KL; ++u) x[u] = lds_u32(at ^ (4u * u));
                sort_keys(x);
                if (done == 0) {
#pragma unroll
                    for (int u = 0; u < KL; ++u) lst[u] = x[u];
                } else {
                    merge_keys(lst, x, rest);
                }
                c += KL;
                if (c == kept.per) {
                    c = 0;
                    ++n;
                }
            }
        } else {
            int m = sub, i = sub, n = 0;
            const unsigned *base = mine;
            const auto move = [&] {  // to the group that expert m of the kept lies in
                while (i >= kept.per) {
                    i -= kept.per;
                    ++n;
                }
                if (m < kept.count) base = mine + mk[n] * kept.per;
            };
            move();
            const auto take = [&] {
                const unsigned v = m < kept.count ? base[i] : 0u;
                m += L;
                i += L;
                if (i >= kept.per) move();
                return v;
            };
#pragma unroll
            for (int u = 0; u < KL; ++u) lst[u] = take();
            sort_keys(lst);
            for (int done = KL * L; done < kept.count; done += KL * L) {
                unsigned x[KL];
#pragma unroll
                for (int u = 0; u < KL; ++u) x[u] = take();
                sort_keys(x);
                merge_keys(lst, x, rest);
            }
        }
#pragma unroll
        for (int d = 1; d < L; d *= 2) {
            unsigned x[KL];
#pragma unroll
            for (int u = 0; u < KL; ++u) x[u] = __shfl_xor_sync(0xffffffffu, lst[u], d);
            rest = max(rest, __shfl_xor_sync(0xffffffffu, rest, d));
            merge_keys(lst, x, rest);
        }
        // neighbours that may be the other way round
        unsigned last = 0u, after = rest;  // of the selected, and the best of the others
        bool close = false;
#pragma unroll
        for (int u = 0; u < KL; ++u) {
            if (u + 1 < KL)
                if (u + 1 < k && (int)(lst[u] >> 9) - (int)(lst[u + 1] >> 9) <= near) close = true;
            if (u == k - 1) last = lst[u];
            if (u == k) after = lst[u];
        }
        const bool edge = after != 0u && (int)(last >> 9) - (int)(after >> 9) <= near;
        if (close) {
#pragma unroll
            for (int u = 0; u + 1 < KL; ++u)
                if (u + 1 < k && (int)(lst[u] >> 9) - (int)(lst[u + 1] >> 9) <= near)
                    unsure |= !same(key_id(lst[u]), key_id(lst[u + 1]));
        }
        if (edge)
            for (int m = sub; m < kept.count; m += L) {
                const int e = (int)mk[m / kept.per] * kept.per + m % kept.per;
                if (mine[e] < last && (int)(mine[e] >> 9) >= (int)(last >> 9) - near) unsure |= !same(e, key_id(last));
            }
        constexpr int kMine = KL > L ? KL / L : 1;  // slots of a lane: sub, sub + L, ..
        int id[kMine];
#pragma unroll
        for (int u = 0; u < KL; ++u)
            if (u % L == sub) id[u / L] = key_id(lst[u]);
        unsure = (unsure || unsure_groups) && on;
        const unsigned any = __ballot_sync(0xffffffffu, unsure);
        const unsigned by_group = __ballot_sync(0xffffffffu, on && unsure_groups);
        if (any != 0u) {
#pragma unroll
            for (int u = 0; u < kMine; ++u)
                if (sub + u * L < k) sel[sub + u * L] = (unsigned)id[u];
            __syncwarp();
            unsigned full = 0u;
            for (unsigned todo = any; todo != 0u;) {
                const int who = (__ffs(todo) - 1) / L;
                const unsigned theirs = kAll << (who * L);
                todo &= ~theirs;
                if (!(by_group & theirs)) {
                    const Kept their = {rows + who * pitch, kept_groups + who * (top | 1), kept.per, kept.count};
                    const unsigned edge_key = __shfl_sync(0xffffffffu, last, who * L);
                    if (select_near(tile + who * E, a, their, edge_key, near, groups + who * gp, list, lane)) continue;
                }
                full |= theirs;
            }
            // these use the memory of the keys
            while (full != 0u) {
                const int who = (__ffs(full) - 1) / L;
                full &= ~(kAll << (who * L));
                const int got = select64(tile + who * E, a, rows, lane);
                if (lane < k) groups[who * gp + lane] = (unsigned)got;
            }
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kMine; ++u)
                if (sub + u * L < k) id[u] = (int)sel[sub + u * L];
        }

        __syncwarp();
        if (t0 + stride < a.T) load(t0 + stride);  // the keys are done with

        // the gates
        const float part_of = __frcp_rn(total);
        float g[kMine], sum = 0.0f;
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            g[u] = 0.0f;
            if (on && sub + u * L < k) {
                const float l = __ldg(row + id[u]);
                g[u] = softmax ? expf(l - peak) * part_of : sigmoid(l);
                atomicAdd(&s_hist[id[u]], 1u);
            }
            sum += g[u];
        }
        const float norm = a.S.renorm ? __frcp_rn(lanes_sum<L>(sum) + kTiny) : 1.0f;
        if (on) {
            int32_t *const oi = a.idx + (t0 + tok) * k;
            float *const og = a.gates + (t0 + tok) * k;
#pragma unroll
            for (int u = 0; u < kMine; ++u) g[u] = g[u] * norm * a.S.scale;
            if (L == 1 && kMine % 4 == 0 && k == KL) {
#pragma unroll
                for (int u = 0; u + 3 < kMine; u += 4) {
                    *reinterpret_cast<int4 *>(oi + u) = make_int4(id[u], id[u + 1], id[u + 2], id[u + 3]);
                    *reinterpret_cast<float4 *>(og + u) = make_float4(g[u], g[u + 1], g[u + 2], g[u + 3]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kMine; ++u)
                    if (sub + u * L < k) {
                        oi[sub + u * L] = id[u];
                        og[sub + u * L] = g[u];
                    }
            }
        }
        __syncwarp();
    }
    if (check != 0.0f) record_status(ws, MOE_ERR_DEVICE_DATA);  // a NaN is not 0 either
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        if (s_hist[e]) atomicAdd(&ws->gate_counts[e], s_hist[e]);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = (atomicAdd(&ws->gate_ticket, 1u) == gridDim.x - 1);
    __syncthreads();
    if (!s_last) return;
    publish_stats(ws, a.T, k, E, a.counts, a.aux, a.ent, [&](int e, unsigned c) {
        if (!a.S.bias_next) return;
        const long long have = (long long)c * E, mean = (long long)a.T * k;
        const float sign = have < mean ? 1.0f : have > mean ? -1.0f : 0.0f;
        a.S.bias_next[e] = __fadd_rn(a.S.bias ? a.S.bias[e] : 0.0f, __fmul_rn(a.S.bias_rate, sign));
    });
}

template <int KL, int L>
cudaError_t launch_scored(const GateArgs &a, cudaStream_t s)
{
    const auto fn = gate_scored_kernel<KL, L>;
    const int smem = kGateWarps * warp_words(a.E, a.S.groups, a.S.top_groups, a.k, L) * 4;
    cudaError_t err = allow_dynamic_smem(reinterpret_cast<const void *>(fn), smem);
    if (err != cudaSuccess) return err;
    const int res = resident_grid(reinterpret_cast<const void *>(fn), 32 * kGateWarps, smem);
    const long long per_block = kGateWarps * (32 / L);
    long long blocks = ((long long)a.T + per_block - 1) / per_block;
    if (blocks > res) blocks = res;
    if (blocks < 1) blocks = 1;
    return launch_pdl(fn, dim3((unsigned)blocks), dim3(32 * kGateWarps), (size_t)smem, s, a);
}

// Lanes of a token.  One, where the tokens alone keep the SMs busy: the lists
// are not merged across lanes.  The more experts, the longer a lane takes and
// the more shared memory its row.  Measured with one lane and with eight:
// 262144 tokens, 60 experts 71 and 141 us; 65536, 32 experts 18 and 27; 40000,
// 64 experts 23 and 21; 262144, 128 experts 113 and 131; 65536, 128 experts 63
// and 37; 16384, 256 experts 40 and 26.  32 lanes for the least latency of few
// tokens.
int scored_lanes(int T, int E)
{
    const int sms = device_sm_count();
    if ((E <= 64 && T >= sms * 256) || (E <= 128 && T >= sms * 768)) return 1;
    return T >= sms * 32 ? 8 : 32;
}

template <int KL>
cudaError_t launch_scored_lanes(const GateArgs &a, cudaStream_t s)
{
    const int lanes = scored_lanes(a.T, a.E);
    if (lanes == 1) return launch_scored<KL, 1>(a, s);
    if (lanes == 8) return launch_scored<KL, 8>(a, s);
    return launch_scored<KL, 32>(a, s);
}

// --------------------------------------------------------------------------
// The gradient.  With N = sum of the selected scores + tiny (renorm) or 1,
// D = sum_j d_j s_j and c the scale,
//   ds_j = c (d_j - D / N) / N     (renorm)     ds_j = c d_j     (else)
//   sigmoid: dl[sel_j] = ds_j s_j (1 - s_j), others 0
//   softmax: dl[e] = s_e ([e = sel_j] ds_j - X),  X = sum_j ds_j s_j;
//            renorm: X = c (D / N) (tiny / N), without the difference of
//            two nearly equal sums
// A group of G lanes per token; lane i of it has the units i, i + G, .. of VEC
// experts (4 where E is a multiple of 4; up to 16 experts a lane, so that a
// warp's sums serve several tokens) and, if i < k, slot i.  The row is written
// without its selected experts, which slot i's lane then writes: comparing
// every expert with every slot took half of the instructions.  Sigmoid reads
// the selected logits only.  Bound by HBM: d_logits is written whole.  131072
// tokens, 128 experts, softmax, 138 MB: 24.3 us (5.7 TB/s; 52 us before).
// --------------------------------------------------------------------------
constexpr int kBwdThreads = 256;

template <int G, typename F>
__device__ __forceinline__ F group_sum(F v)
{
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

template <bool SOFTMAX, int G, int EPL, int VEC>
__global__ void __launch_bounds__(kBwdThreads)
gate_scored_bwd_kernel(const float *__restrict__ logits, const int32_t *__restrict__ idx,
                       const float *__restrict__ d_gates, long long T, int E, int k, int renorm, float scale,
                       float *d_logits, void *ws)
{
    constexpr int kTokens = 32 / G, N = EPL * VEC;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane & (G - 1);
    const long long step = (long long)gridDim.x * (kBwdThreads / 32) * kTokens;
    for (long long t0 = ((long long)blockIdx.x * (kBwdThreads / 32) + (threadIdx.x >> 5)) * kTokens; t0 < T; t0 += step) {
        const long long t = t0 + lane / G;
        const bool valid = t < T;
        int sel = -1;
        float d = 0.0f, l = 0.0f;
        if (valid && sub < k) {
            sel = __ldg(idx + t * k + sub);
            d = __ldg(d_gates + t * k + sub);
        }
        float out[N];
        if (SOFTMAX) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = (sub + G * i) * VEC;
                const float *at = logits + t * E + e;
                if constexpr (VEC == 4) {
                    const float4 v = valid && e < E ? __ldg(reinterpret_cast<const float4 *>(at))
                                                    : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    out[4 * i] = v.x;
                    out[4 * i + 1] = v.y;
                    out[4 * i + 2] = v.z;
                    out[4 * i + 3] = v.w;
                } else {
                    out[i] = valid && e < E ? __ldg(at) : -INFINITY;
                }
            }
        }
        if (valid && sub < k) {
            if (sel < 0 || sel >= E) {
                record_status(ws, MOE_ERR_DEVICE_DATA);
                sel = -1;
                d = 0.0f;
            } else {
                l = __ldg(logits + t * E + sel);
            }
        }
        float s = 0.0f, slope = 0.0f;
        if (SOFTMAX) {
            float m = -INFINITY, z = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) m = fmaxf(m, out[i]);
            m = group_max<G>(m);
            if (!valid) m = 0.0f;  // exp(-inf - 0) = 0, as past the last expert
#pragma unroll
            for (int i = 0; i < N; ++i) {
                out[i] = expf(out[i] - m);
                z += out[i];
            }
            z = __fdiv_rn(1.0f, group_sum<G>(z));
#pragma unroll
            for (int i = 0; i < N; ++i) out[i] *= z;
            if (sel >= 0) s = expf(l - m) * z;
        } else if (sel >= 0) {
            const float e = expf(-fabsf(l)), q = __fdiv_rn(1.0f, 1.0f + e);  // s (1 - s) = e / (1 + e)^2
            s = l < 0.0f ? e * q : q;
            slope = e * q * q;
        }
        float ds = d * scale, all = group_sum<G>(ds * s);
        if (renorm) {
            const float n = __fdiv_rn(1.0f, group_sum<G>(s) + kTiny);
            ds = (ds - all * n) * n;
            all = all * n * (kTiny * n);
        }
        const float own = sel < 0 ? 0.0f : ds * (SOFTMAX ? s : slope);
        float sum = SOFTMAX ? -s * all : 0.0f;  // of the expert's slots, in their order
        for (int j = 0; j < k; ++j) {
            const int ej = __shfl_sync(0xffffffffu, sel, j, G);
            const float oj = __shfl_sync(0xffffffffu, own, j, G);
            if (ej == sel) sum += oj;
        }
        if (valid)
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = (sub + G * i) * VEC;
                float *at = d_logits + t * E + e;
                if (e < E) {
                    if constexpr (VEC == 4)
                        *reinterpret_cast<float4 *>(at) =
                            SOFTMAX ? make_float4(-out[4 * i] * all, -out[4 * i + 1] * all, -out[4 * i + 2] * all,
                                                  -out[4 * i + 3] * all)
                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    else
                        *at = SOFTMAX ? -out[i] * all : 0.0f;
                }
            }
        __syncwarp();  // the row before its selected experts
        if (sel >= 0) d_logits[t * E + sel] = sum;
    }
}

struct BwdArgs {
    const float *logits;
    const int32_t *idx;
    const float *d_gates;
    int T, E, k, renorm;
    float scale;
    float *d_logits;
    void *ws;
};

template <bool SOFTMAX, int G, int EPL, int VEC>
cudaError_t launch_bwd(const BwdArgs &a, cudaStream_t s)
{
    const auto fn = gate_scored_bwd_kernel<SOFTMAX, G, EPL, VEC>;
    const long long per_block = (kBwdThreads / 32) * (32 / G);
    const long long need = ((long long)a.T + per_block - 1) / per_block;
    const int res = resident_grid(reinterpret_cast<const void *>(fn), kBwdThreads, 0);
    return launch_pdl(fn, dim3((unsigned)(need < res ? need : res)), dim3(kBwdThreads), 0, s, a.logits, a.idx, a.d_gates,
                      (long long)a.T, a.E, a.k, a.renorm, a.scale, a.d_logits, a.ws);
}

template <bool SOFTMAX, int G>
cudaError_t launch_bwd_units(const BwdArgs &a, int each, cudaStream_t s)
{
    if (each <= 1) return launch_bwd<SOFTMAX, G, 1, 4>(a, s);
    if (each <= 2) return launch_bwd<SOFTMAX, G, 2, 4>(a, s);
    return launch_bwd<SOFTMAX, G, 4, 4>(a, s);
}

template <bool SOFTMAX>
cudaError_t launch_bwd_e(const BwdArgs &a, cudaStream_t s)
{
    if (a.E % 4 == 0) {  // up to 4 units a lane, and a lane for every slot
        const int units = a.E / 4, lanes = (units + 3) / 4 > a.k ? (units + 3) / 4 : a.k;
        if (lanes <= 4) return launch_bwd_units<SOFTMAX, 4>(a, (units + 3) / 4, s);
        if (lanes <= 8) return launch_bwd_units<SOFTMAX, 8>(a, (units + 7) / 8, s);
        return launch_bwd_units<SOFTMAX, 16>(a, (units + 15) / 16, s);
    }
    const int lanes = a.E;  // k <= E
    if (lanes <= 8) return launch_bwd<SOFTMAX, 8, 1, 1>(a, s);
    if (lanes <= 32) return launch_bwd<SOFTMAX, 16, 2, 1>(a, s);
    if (lanes <= 64) return launch_bwd<SOFTMAX, 16, 4, 1>(a, s);
    if (lanes <= 128) return launch_bwd<SOFTMAX, 16, 8, 1>(a, s);
    return launch_bwd<SOFTMAX, 32, 8, 1>(a, s);
}

}  // namespace

cudaError_t launch_gate_scored(const float *logits, int T, int E, int k, const moe_scoring *S, int32_t *idx,
                               float *gates, int32_t *counts, double *aux, double *ent, void *ws, cudaStream_t s)
{
    GateArgs a = {logits, T, E, k, *S, idx, gates, counts, aux, ent, ws};
    // Groups by their best expert, as many as slots or more: the k best experts
    // of all are in them.  (Groups before the one of such an expert have an
    // expert each that comes before it, fewer than k.)
    if (S->group_top == 1 && k <= S->top_groups) a.S.groups = a.S.top_groups = 1;
    if (k <= 4) return launch_scored_lanes<4>(a, s);
    if (k <= 8) return launch_scored_lanes<8>(a, s);
    return launch_scored_lanes<16>(a, s);
}

cudaError_t launch_gate_scored_backward(const float *logits, const int32_t *idx, const float *d_gates, int T, int E,
                                        int k, const moe_scoring *S, float *d_logits, void *ws, cudaStream_t s)
{
    if (T == 0) return cudaSuccess;
    const BwdArgs a = {logits, idx, d_gates, T, E, k, S->renorm, S->scale, d_logits, ws};
    return S->score == MOE_SCORE_SOFTMAX ? launch_bwd_e<true>(a, s) : launch_bwd_e<false>(a, s);
}

}  // namespace moe
