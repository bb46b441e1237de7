// rows.cuh -- which of a call's rows belong to an expert (moe_rows).
#pragma once

#include "common.cuh"

namespace moe {

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

// Whether `row` is one of them, where the rows between the first and the last are not all.
__device__ __forceinline__ bool is_member(const Members &m, int E, int row)
{
    bool mine = false;
    for (int e = 0; e < E; ++e) mine |= row >= m.lo[e] && row < m.hi[e];
    return mine;
}

}  // namespace moe
