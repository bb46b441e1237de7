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

#include "common.cuh"
#include "gate_stats.cuh"
#include "launchers.h"

namespace moe {
namespace {

constexpr int kWarps = 4;
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

// --------------------------------------------------------------------------
// One token in 64 bits, by a whole warp: lane j < k gets slot j's expert.
// --------------------------------------------------------------------------
struct Scratch {
    double v[MOE_MAX_EXPERTS], group[MOE_MAX_EXPERTS];
    unsigned char kept[MOE_MAX_EXPERTS];
};

__device__ __noinline__ int select64(const float *row, const GateArgs &a, Scratch &s, int lane)
{
    const int E = a.E, per = E / a.S.groups;
    double m = 0.0, inv = 0.0;
    if (a.S.score == MOE_SCORE_SOFTMAX) {
        float top = -INFINITY;
        for (int e = lane; e < E; e += 32) top = fmaxf(top, row[e]);
        m = warp_max(top);
        double sum = 0.0;
        for (int e = lane; e < E; e += 32) sum += exp((double)row[e] - m);
        inv = 1.0 / warp_sum(sum);
    }
    unsigned mine = 0;  // experts lane, lane + 32, ... still to choose from
    for (int e = lane, i = 0; e < E; e += 32, ++i) {
        const double l = row[e];
        double v = a.S.score == MOE_SCORE_SOFTMAX ? exp(l - m) * inv : 1.0 / (1.0 + exp(-l));
        if (a.S.bias) v += (double)a.S.bias[e];
        s.v[e] = v == v ? v : -INFINITY;  // reported as bad data; the ids stay valid
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

__device__ __forceinline__ float sigmoid(float l)
{
    const float e = expf(-fabsf(l));  // no overflow, and digits down to the subnormals
    return __fdiv_rn(l < 0.0f ? e : 1.0f, 1.0f + e);
}

// --------------------------------------------------------------------------
// A warp per token.
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(32 * kWarps) gate_scored_kernel(const GateArgs a)
{
    __shared__ Scratch s_scratch[kWarps];
    __shared__ unsigned s_hist[MOE_MAX_EXPERTS];
    __shared__ int s_last;
    WsHeader *ws = static_cast<WsHeader *>(a.ws);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) s_hist[e] = 0u;
    pdl_wait();
    pdl_launch_dependents();
    bool finite = true;
    if (a.S.bias)
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) finite &= isfinite(a.S.bias[e]);
    __syncthreads();
    for (long long t = (long long)blockIdx.x * kWarps + warp; t < a.T; t += (long long)gridDim.x * kWarps) {
        const float *row = a.logits + t * a.E;
        float m = -INFINITY, sum = 0.0f;
        for (int e = lane; e < a.E; e += 32) {
            finite &= isfinite(row[e]);
            m = fmaxf(m, row[e]);
        }
        const int id = select64(row, a, s_scratch[warp], lane);
        float g = 0.0f;
        if (a.S.score == MOE_SCORE_SOFTMAX) {
            m = warp_max(m);
            for (int e = lane; e < a.E; e += 32) sum += expf(row[e] - m);
            sum = warp_sum(sum);
            if (lane < a.k) g = __fdiv_rn(expf(row[id] - m), sum);
        } else if (lane < a.k) {
            g = sigmoid(row[id]);
        }
        if (a.S.renorm) g = __fdiv_rn(g, warp_sum(g) + kTiny);
        if (lane < a.k) {
            a.idx[t * a.k + lane] = id;
            a.gates[t * a.k + lane] = g * a.S.scale;
            atomicAdd(&s_hist[id], 1u);
        }
    }
    if (!finite) record_status(ws, MOE_ERR_DEVICE_DATA);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        if (s_hist[e]) atomicAdd(&ws->gate_counts[e], s_hist[e]);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = (atomicAdd(&ws->gate_ticket, 1u) == gridDim.x - 1);
    __syncthreads();
    if (!s_last) return;
    publish_stats(ws, a.T, a.k, a.E, a.counts, a.aux, a.ent, [&](int e, unsigned c) {
        if (!a.S.bias_next) return;
        const long long have = (long long)c * a.E, mean = (long long)a.T * a.k;
        const float sign = have < mean ? 1.0f : have > mean ? -1.0f : 0.0f;
        a.S.bias_next[e] = __fadd_rn(a.S.bias ? a.S.bias[e] : 0.0f, __fmul_rn(a.S.bias_rate, sign));
    });
}

// --------------------------------------------------------------------------
// The gradient.  With N = sum of the selected scores + tiny (renorm) or 1,
// D = sum_j d_j s_j and c the scale,
//   ds_j = c (d_j - D / N) / N     (renorm)     ds_j = c d_j     (else)
//   sigmoid: dl[sel_j] = ds_j s_j (1 - s_j), others 0
//   softmax: dl[e] = s_e ([e = sel_j] ds_j - X),  X = sum_j ds_j s_j;
//            renorm: X = c (D / N) (tiny / N), without the difference of
//            two nearly equal sums
// A group of G lanes per token (E rounded up to a power of two, at most 32),
// lane i of it has experts i, i + G, ... and, if i < k, slot i.  Sigmoid reads
// the selected logits only.  Bound by HBM: d_logits is written whole.
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

template <bool SOFTMAX, int G, int EPL>
__global__ void __launch_bounds__(kBwdThreads)
gate_scored_bwd_kernel(const float *__restrict__ logits, const int32_t *__restrict__ idx,
                       const float *__restrict__ d_gates, long long T, int E, int k, int renorm, float scale,
                       float *__restrict__ d_logits, void *ws)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane & (G - 1);
    constexpr int kTokens = 32 / G;  // of a warp
    const long long step = (long long)gridDim.x * (kBwdThreads / 32) * kTokens;
    for (long long t0 = ((long long)blockIdx.x * (kBwdThreads / 32) + (threadIdx.x >> 5)) * kTokens; t0 < T; t0 += step) {
        const long long t = t0 + lane / G;
        const bool valid = t < T;
        int sel = -1;
        float d = 0.0f, l = 0.0f;
        if (valid && sub < k) {
            sel = __ldg(idx + t * k + sub);
            d = __ldg(d_gates + t * k + sub);
            if (sel < 0 || sel >= E) {
                record_status(ws, MOE_ERR_DEVICE_DATA);
                sel = -1;
                d = 0.0f;
            } else {
                l = __ldg(logits + t * E + sel);
            }
        }
        float out[EPL], s = 0.0f, slope = 0.0f;
        if (SOFTMAX) {
            float m = -INFINITY, z = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                out[i] = valid && sub + G * i < E ? __ldg(logits + t * E + sub + G * i) : -INFINITY;
                m = fmaxf(m, out[i]);
            }
            m = group_max<G>(m);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                out[i] = valid && sub + G * i < E ? expf(out[i] - m) : 0.0f;
                z += out[i];
            }
            z = __fdiv_rn(1.0f, group_sum<G>(z));
#pragma unroll
            for (int i = 0; i < EPL; ++i) out[i] *= z;
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
#pragma unroll
        for (int i = 0; i < EPL; ++i) out[i] = SOFTMAX ? -out[i] * all : 0.0f;
        for (int j = 0; j < k; ++j) {
            const int ej = __shfl_sync(0xffffffffu, sel, j, G);
            const float oj = __shfl_sync(0xffffffffu, own, j, G);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (ej == sub + G * i) out[i] += oj;
        }
        if (valid)
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (sub + G * i < E) d_logits[t * E + sub + G * i] = out[i];
    }
}

template <bool SOFTMAX, int G, int EPL>
cudaError_t launch_bwd(const float *logits, const int32_t *idx, const float *d_gates, int T, int E, int k, int renorm,
                       float scale, float *d_logits, void *ws, cudaStream_t s)
{
    const auto fn = gate_scored_bwd_kernel<SOFTMAX, G, EPL>;
    const long long per_block = (kBwdThreads / 32) * (32 / G);
    const long long need = ((long long)T + per_block - 1) / per_block;
    const int res = resident_grid(reinterpret_cast<const void *>(fn), kBwdThreads, 0);
    return launch_pdl(fn, dim3((unsigned)(need < res ? need : res)), dim3(kBwdThreads), 0, s, logits, idx, d_gates,
                      (long long)T, E, k, renorm, scale, d_logits, ws);
}

template <bool SOFTMAX>
cudaError_t launch_bwd_e(const float *logits, const int32_t *idx, const float *d_gates, int T, int E, int k,
                         int renorm, float scale, float *d_logits, void *ws, cudaStream_t s)
{
#define MOE_BWD(G, EPL) return launch_bwd<SOFTMAX, G, EPL>(logits, idx, d_gates, T, E, k, renorm, scale, d_logits, ws, s)
    if (E <= 1) MOE_BWD(1, 1);
    if (E <= 2) MOE_BWD(2, 1);
    if (E <= 4) MOE_BWD(4, 1);
    if (E <= 8) MOE_BWD(8, 1);
    if (E <= 16) MOE_BWD(16, 1);
    switch ((E + 31) / 32) {
    case 1: MOE_BWD(32, 1);
    case 2: MOE_BWD(32, 2);
    case 3: MOE_BWD(32, 3);
    case 4: MOE_BWD(32, 4);
    case 5: MOE_BWD(32, 5);
    case 6: MOE_BWD(32, 6);
    case 7: MOE_BWD(32, 7);
    default: MOE_BWD(32, 8);
    }
#undef MOE_BWD
}

}  // namespace

cudaError_t launch_gate_scored(const float *logits, int T, int E, int k, const moe_scoring *S, int32_t *idx,
                               float *gates, int32_t *counts, double *aux, double *ent, void *ws, cudaStream_t s)
{
    const GateArgs a = {logits, T, E, k, *S, idx, gates, counts, aux, ent, ws};
    const int res = resident_grid(reinterpret_cast<const void *>(gate_scored_kernel), 32 * kWarps, 0);
    long long blocks = ((long long)T + kWarps - 1) / kWarps;
    if (blocks > res) blocks = res;
    if (blocks < 1) blocks = 1;
    return launch_pdl(gate_scored_kernel, dim3((unsigned)blocks), dim3(32 * kWarps), 0, s, a);
}

cudaError_t launch_gate_scored_backward(const float *logits, const int32_t *idx, const float *d_gates, int T, int E,
                                        int k, const moe_scoring *S, float *d_logits, void *ws, cudaStream_t s)
{
    if (T == 0) return cudaSuccess;
    return S->score == MOE_SCORE_SOFTMAX
               ? launch_bwd_e<true>(logits, idx, d_gates, T, E, k, S->renorm, S->scale, d_logits, ws, s)
               : launch_bwd_e<false>(logits, idx, d_gates, T, E, k, S->renorm, S->scale, d_logits, ws, s);
}

}  // namespace moe
