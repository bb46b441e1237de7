// gate_stats.cuh -- what the last block of a gate kernel does: the rows of
// each expert, and the aux loss and entropy that follow from them.
#pragma once

#include <math.h>

#include "common.cuh"

namespace moe {

constexpr int kStatsMaxThreads = 256;

// log2 of a positive, finite double: exact binary exponent plus log2f of the
// mantissa in [1, 2) (absolute error ~1e-7), avoiding fp64 transcendentals.
__device__ __forceinline__ double log2_via_mantissa(double x)
{
    const long long bits = __double_as_longlong(x);
    const int ex = (int)((bits >> 52) & 0x7FF) - 1023;
    const double m = __longlong_as_double((bits & 0x000FFFFFFFFFFFFFll) | 0x3FF0000000000000ll);
    return (double)ex + (double)log2f((float)m);
}

// 1/x for a positive double: the fp32 reciprocal refined by two
// Newton-Raphson steps (r <- r (2 - x r); each doubles the correct bits:
// 24 -> 48 -> full double), instead of an fp64 divide.
__device__ __forceinline__ double rcp_newton(double x)
{
    double r = (double)__frcp_rn((float)x);
    r = r * (2.0 - x * r);
    r = r * (2.0 - x * r);
    return r;
}

// For a whole block of at most kStatsMaxThreads threads, the last one of its
// grid, with every other block's counts in ws->gate_counts: publishes and
// clears them.  Either statistic may be left out (NULL); `each` gets every
// expert and its count.
template <typename Each>
__device__ __forceinline__ void publish_stats(WsHeader *ws, int T, int k, int E, int32_t *__restrict__ expert_counts,
                                              double *__restrict__ aux_out, double *__restrict__ ent_out,
                                              const Each &each)
{
    // FP64 units are scarce on this part, so the per-expert work avoids fp64
    // transcendentals:
    //   entropy = -sum_e p_e log2(p_e + eps),  p_e = c_e / N,  N = T*k
    //           = log2(N) * SUM / N - (1/N) sum_e c_e log2(c_e + eps*N),  SUM = sum_e c_e
    // with each log2 of a double taken as exponent + log2f(mantissa) (error
    // ~1e-7 absolute), the products c_e*log2(.) summed exactly in 2^-32
    // fixed point with integer warp shuffles (deterministic), and
    //   aux = E * (sum_e c_e^2) / T^2  from the exact integer sum of squares.
    __threadfence();
    __shared__ long long s_fix[kStatsMaxThreads / 32];
    __shared__ unsigned long long s_sq[kStatsMaxThreads / 32], s_sum[kStatsMaxThreads / 32];
    const double n_assign = (double)T * (double)k;
    const double eps_n = 1e-8 * n_assign;
    long long fix = 0;
    unsigned long long sq = 0ull, sum = 0ull;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const unsigned c = atomicExch(&ws->gate_counts[e], 0u);
        expert_counts[e] = (int32_t)c;
        sq += (unsigned long long)c * c;
        sum += c;
        each(e, c);
        if (c) fix += llrint((double)c * log2_via_mantissa((double)c + eps_n) * 4294967296.0);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        fix += __shfl_xor_sync(0xffffffffu, fix, d);
        sq += __shfl_xor_sync(0xffffffffu, sq, d);
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    if (lane == 0) {
        s_fix[wid] = fix;
        s_sq[wid] = sq;
        s_sum[wid] = sum;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        long long F = 0;
        unsigned long long SQ = 0ull, SUM = 0ull;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
            F += s_fix[w];
            SQ += s_sq[w];
            SUM += s_sum[w];
        }
        double aux = 0.0, ent = 0.0;
        if (T > 0) {
            const double inv_t = rcp_newton((double)T);
            aux = (double)E * ((double)SQ * inv_t * inv_t);
            ent = (log2_via_mantissa(n_assign) * (double)SUM - (double)F * (1.0 / 4294967296.0)) *
                  rcp_newton(n_assign);
        }
        if (aux_out) *aux_out = aux;
        if (ent_out) *ent_out = ent;
        ws->gate_ticket = 0u;
    }
}

}  // namespace moe
