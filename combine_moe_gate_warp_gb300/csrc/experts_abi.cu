// experts_abi.cu -- the extern "C" entry points declared in
// include/moe_experts.h: argument checks on the host (nothing is enqueued
// when they are bad), then the launch.
#include "experts.h"

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline moe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline cudaStream_t stream_of(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int kMaxCols = 1 << 20;

inline moe_status check_rows(const moe_rows *G)
{
    if (!G || !G->ws || G->rows < 0) return MOE_ERR_INVALID_ARG;
    if (!aligned16(G->ws)) return MOE_ERR_INVALID_ARG;
    if (G->E < 1 || G->E > MOE_MAX_EXPERTS || G->rows >= (1 << 30)) return MOE_ERR_UNSUPPORTED;
    if (!G->offsets && G->E != 1) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

inline bool cols_ok(int n, int multiple) { return n >= multiple && n <= kMaxCols && n % multiple == 0; }

inline moe_status check_sizes(const moe_rows *G, int K, int N)
{
    if (!cols_ok(K, 8) || !cols_ok(N, 8)) return MOE_ERR_UNSUPPORTED;
    if ((long long)G->E * N >= (1LL << 31) || (long long)G->E * K >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline bool act_ok(int act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_SWIGLU; }
// columns of a saved layer
inline bool saved_cols_ok(int n, int act) { return cols_ok(n, act == MOE_ACT_SWIGLU ? 64 : 32); }

}  // namespace

extern "C" {

moe_status moe_expert_linear(const moe_rows *G, const void *x, const float *x_scales, int K, const void *w,
                             const float *w_scales, int N, const void *bias, int act, const void *residual, void *y,
                             void *saved, void *saved_scales, moe_stream_t stream)
{
    moe_status st = check_rows(G);
    if (st != MOE_OK) return st;
    if (!act_ok(act)) return MOE_ERR_INVALID_ARG;
    st = check_sizes(G, K, N);
    if (st != MOE_OK) return st;
    if ((x_scales == nullptr) != (w_scales == nullptr) || (saved == nullptr) != (saved_scales == nullptr))
        return MOE_ERR_INVALID_ARG;
    if (x_scales && K % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (act == MOE_ACT_SWIGLU && N % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (saved && !saved_cols_ok(N, act)) return MOE_ERR_UNSUPPORTED;
    if (!w || (G->rows > 0 && (!x || !y))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(x_scales) || !aligned16(w) || !aligned16(w_scales) || !aligned16(bias) ||
        !aligned16(residual) || !aligned16(y) || !aligned16(saved) || !aligned16(saved_scales))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(moe::launch_expert_linear(G, x, x_scales, K, w, w_scales, N, bias, act, residual, y, saved,
                                               saved_scales, stream_of(stream)));
}

moe_status moe_expert_dgrad(const moe_rows *G, const void *dy, int N, const void *w, int K, int act,
                            const void *saved, const void *saved_scales, void *dx, void *a, moe_stream_t stream)
{
    moe_status st = check_rows(G);
    if (st != MOE_OK) return st;
    if (!act_ok(act)) return MOE_ERR_INVALID_ARG;
    st = check_sizes(G, K, N);
    if (st != MOE_OK) return st;
    if (!w || (G->rows > 0 && (!dy || !dx))) return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_NONE) {
        if (saved || saved_scales || a) return MOE_ERR_INVALID_ARG;
    } else {
        if (K > kMaxCols / 2 || !saved_cols_ok(act == MOE_ACT_SWIGLU ? 2 * K : K, act)) return MOE_ERR_UNSUPPORTED;
        if (G->rows > 0 && (!saved || !saved_scales)) return MOE_ERR_INVALID_ARG;
    }
    if (!aligned16(dy) || !aligned16(w) || !aligned16(saved) || !aligned16(saved_scales) || !aligned16(dx) ||
        !aligned16(a))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(
        moe::launch_expert_dgrad(G, dy, N, w, K, act, saved, saved_scales, dx, a, stream_of(stream)));
}

moe_status moe_expert_wgrad(const moe_rows *G, const void *dy, int N, const void *x, int K, void *dw, void *db,
                            int fp32, moe_stream_t stream)
{
    moe_status st = check_rows(G);
    if (st != MOE_OK) return st;
    st = check_sizes(G, K, N);
    if (st != MOE_OK) return st;
    if (!dw || (G->rows > 0 && (!dy || !x))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(dw) || !aligned16(db)) return MOE_ERR_INVALID_ARG;
    return from_cuda(moe::launch_expert_wgrad(G, dy, N, x, K, dw, db, fp32 != 0, stream_of(stream)));
}

moe_status moe_act_backward(const moe_rows *G, const void *dy, int N, int act, const void *saved,
                            const void *saved_scales, void *du, void *a, moe_stream_t stream)
{
    moe_status st = check_rows(G);
    if (st != MOE_OK) return st;
    if (!act_ok(act) || act == MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
    if (!saved_cols_ok(N, act)) return MOE_ERR_UNSUPPORTED;
    if (G->rows > 0 && (!dy || !saved || !saved_scales || !du)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(saved) || !aligned16(saved_scales) || !aligned16(du) || !aligned16(a))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(moe::launch_act_backward(G, dy, N, act, saved, saved_scales, du, a, stream_of(stream)));
}

moe_status moe_expert_cut(int product, int e4m3, int rows, int E, int K, int N, int32_t *cut)
{
    if (!cut || rows < 0 || product < MOE_EXPERT_LINEAR || product > MOE_EXPERT_WGRAD) return MOE_ERR_INVALID_ARG;
    if (e4m3 && product != MOE_EXPERT_LINEAR) return MOE_ERR_INVALID_ARG;
    if (E < 1 || E > MOE_MAX_EXPERTS || rows >= (1 << 30) || !cols_ok(K, 8) || !cols_ok(N, 8))
        return MOE_ERR_UNSUPPORTED;
    cut[0] = cut[1] = cut[2] = 0;
    if (rows == 0) return MOE_OK;  // nothing is cut
    const int elems = e4m3 ? 128 : 64;
    const moe::Cut c = product == MOE_EXPERT_LINEAR  ? moe::rows_cut(N, rows, E, (K + elems - 1) / elems)
                       : product == MOE_EXPERT_DGRAD ? moe::rows_cut(K, rows, E, (N + 63) / 64)
                                                     : moe::wgrad_cut(N, K, rows, E);
    cut[0] = c.cg;
    cut[1] = c.bn;
    cut[2] = c.split;
    return MOE_OK;
}

}  // extern "C"
