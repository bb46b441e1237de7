// fp4.cu -- rows brought to 4 bits and back (include/moe_route.h): the
// dispatch in 4 bits, and the same for packed rows.
//
// A block of 32 consecutive columns is the unit of the format, and one
// thread's unit of work: it reads 64 bytes of bf16, finds the largest
// magnitude without a neighbour's help, and writes 16 bytes of codes and one
// scale byte, once for every packed row that the token has.  A warp's 32
// blocks lie side by side, so it moves 2 KB of bf16 in, 512 bytes and 32
// bytes out.  Bound by HBM: each value of x is read once, each code written
// once for each of its rows.  Of 4096 columns: 65536 tokens to 2 experts each
// 130 us (6.3 TB/s; 163 with one block in flight a thread), 131072 packed rows
// to 4 bits 209 us (6.5 TB/s) and back 221 us (6.1 TB/s).
#include "fp4.cuh"
#include "experts.h"
#include "launchers.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// A thread's place in a matrix of `rows` rows of `blocks` units, which it
// walks by the grid's stride.
struct Place {
    long long row;
    int col, dcol, blocks;
    long long drow;
    __device__ Place(int blocks_, long long first_row) : blocks(blocks_)
    {
        const long long step = (long long)gridDim.x * kThreads, at = (long long)blockIdx.x * kThreads + threadIdx.x;
        drow = step / blocks;
        dcol = (int)(step - drow * blocks);
        row = at / blocks;
        col = (int)(at - row * blocks);
        row += first_row;
    }
    __device__ __forceinline__ void advance()
    {
        row += drow;
        col += dcol;
        if (col >= blocks) {
            col -= blocks;
            ++row;
        }
    }
};

struct Block32 {
    uint4 v[4];
};

__device__ __forceinline__ Block32 load32(const __nv_bfloat16 *p, bool wide, uint64_t pol)
{
    Block32 b;
    if (wide) {
        const u32x8 *q = reinterpret_cast<const u32x8 *>(p);
        const u32x8 lo = ld_stream_v8(q, pol), hi = ld_stream_v8(q + 1, pol);
        b.v[0] = lo.lo;
        b.v[1] = lo.hi;
        b.v[2] = hi.lo;
        b.v[3] = hi.hi;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) b.v[i] = ld_stream_v4(reinterpret_cast<const uint4 *>(p) + i, pol);
    }
    return b;
}

// codes of 32 values and their scale byte
__device__ __forceinline__ uint4 encode32(const Block32 &b, unsigned &byte)
{
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned w[4] = {b.v[i].x, b.v[i].y, b.v[i].z, b.v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    }
    byte = fp4_byte(max(m & 0xFFFFu, m >> 16));
    const float inv = fp4_inverse(byte);
    unsigned c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned w[4] = {b.v[i].x, b.v[i].y, b.v[i].z, b.v[i].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = bf16lo(w[j]) * inv;
            f[2 * j + 1] = bf16hi(w[j]) * inv;
        }
        c[i] = byte == 255u ? 0x77777777u : fp4_encode8(f);
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// A block's codes and scale; the last of a row also clears the bytes between
// the row's scales and the next row's.
__device__ __forceinline__ void store32(uint8_t *codes, uint8_t *scales, long long row, int col, int blocks, int pitch,
                                        const uint4 &c, unsigned byte, uint64_t pol)
{
    st_stream_v4(reinterpret_cast<uint4 *>(codes) + row * blocks + col, c, pol);
    uint8_t *s = scales + row * pitch;
    s[col] = (uint8_t)byte;
    if (col == blocks - 1)
        for (int i = blocks; i < pitch; ++i) s[i] = 0;
}

// token rows to their packed rows
__global__ void __launch_bounds__(kThreads)
dispatch_fp4_kernel(const __nv_bfloat16 *__restrict__ x, long long T, int blocks, int pitch, int k,
                    const int32_t *__restrict__ dst_row, int r_max, const int32_t *__restrict__ R_ptr, uint8_t *codes,
                    uint8_t *scales, void *ws, bool wide)
{
    pdl_wait();
    pdl_launch_dependents();
    const uint64_t pol = l2_stream_policy(true);
    const int rows_valid = min(r_max, __ldg(R_ptr));
    const auto pack = [&](const Place &p, const Block32 &b) {
        const int32_t *dst = dst_row + p.row * k;
        unsigned byte;
        const uint4 c = encode32(b, byte);
        for (int j = 0; j < k; ++j) {
            const int r = __ldg(dst + j);
            if (r >= rows_valid) {
                if (p.col == 0) record_status(ws, MOE_ERR_DEVICE_DATA);
            } else if (r >= 0) {
                store32(codes, scales, r, p.col, blocks, pitch, c, byte, pol);
            }
        }
    };
    // two blocks in flight: the way from a token's values to its packed rows is
    // three loads and stores long
    for (Place p(blocks, 0); p.row < T; p.advance()) {
        const Place first = p;
        const Block32 b = load32(x + (p.row * blocks + p.col) * 32, wide, pol);
        p.advance();
        const bool two = p.row < T;
        Block32 c = b;
        if (two) c = load32(x + (p.row * blocks + p.col) * 32, wide, pol);
        pack(first, b);
        if (two) pack(p, c);
    }
}

__global__ void __launch_bounds__(kThreads)
quantize_fp4_kernel(const __nv_bfloat16 *__restrict__ x, int blocks, int pitch, const int32_t *offsets, int E, int rows,
                    uint8_t *codes, uint8_t *scales, void *ws, bool wide)
{
    __shared__ Members m;
    pdl_wait();
    pdl_launch_dependents();
    const uint64_t pol = l2_stream_policy(false);  // a product reads the codes next
    int first, last;
    const bool all = members(offsets, E, rows, ws, m, first, last);
    for (Place p(blocks, first); p.row < last; p.advance()) {
        if (!all && !is_member(m, E, (int)p.row)) continue;
        const Block32 b = load32(x + (p.row * blocks + p.col) * 32, wide, pol);
        unsigned byte;
        const uint4 c = encode32(b, byte);
        store32(codes, scales, p.row, p.col, blocks, pitch, c, byte, pol);
    }
}

__global__ void __launch_bounds__(kThreads)
dequantize_fp4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int blocks, int pitch,
                      const int32_t *offsets, int E, int rows, __nv_bfloat16 *x, void *ws, bool wide)
{
    __shared__ Members m;
    pdl_wait();
    pdl_launch_dependents();
    const uint64_t pol = l2_stream_policy(true);  // measured: 231 -> 221 us
    int first, last;
    const bool all = members(offsets, E, rows, ws, m, first, last);
    for (Place p(blocks, first); p.row < last; p.advance()) {
        if (!all && !is_member(m, E, (int)p.row)) continue;
        const uint4 c = ld_stream_v4(reinterpret_cast<const uint4 *>(codes) + p.row * blocks + p.col, pol);
        const unsigned s = fp4_scale2(scales[p.row * pitch + p.col]);
        const unsigned w[4] = {c.x, c.y, c.z, c.w};
        Block32 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            unsigned o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned two = w[i] >> (8 * j);  // codes of columns 2j and 2j + 1
                o[j] = fp4_decode2((two & 15u) | ((two & 0xF0u) << 12), s);
            }
            b.v[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __nv_bfloat16 *o = x + (p.row * blocks + p.col) * 32;
        if (wide) {
            u32x8 *q = reinterpret_cast<u32x8 *>(o);
            st_stream_v8(q, u32x8{b.v[0], b.v[1]}, pol);
            st_stream_v8(q + 1, u32x8{b.v[2], b.v[3]}, pol);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_stream_v4(reinterpret_cast<uint4 *>(o) + i, b.v[i], pol);
        }
    }
}

bool aligned32(const void *p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

// blocks for `units` threads, at most what the device holds at once
template <typename F>
unsigned grid_for(F fn, long long units)
{
    const long long most = resident_grid(reinterpret_cast<const void *>(fn), kThreads, 0);
    const long long n = (units + kThreads - 1) / kThreads;
    return (unsigned)(n < most ? n : most);
}

}  // namespace

cudaError_t launch_dispatch_fp4(const void *x, int T, int H, const moe_layout *L, void *codes, void *scales,
                                cudaStream_t s)
{
    if (T == 0) return cudaSuccess;
    return launch_pdl(dispatch_fp4_kernel, dim3(grid_for(dispatch_fp4_kernel, (long long)T * (H / 32))), dim3(kThreads),
                      0, s, static_cast<const __nv_bfloat16 *>(x), (long long)T, H / 32, MOE_FP4_PITCH(H), (int)L->k,
                      (const int32_t *)L->dst_row, (int)L->r_max, (const int32_t *)(L->offsets + L->E),
                      static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales), L->ws, aligned32(x));
}

cudaError_t launch_quantize_fp4(const moe_rows *G, const void *rows, int K, void *codes, void *scales, cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    return launch_pdl(quantize_fp4_kernel, dim3(grid_for(quantize_fp4_kernel, (long long)G->rows * (K / 32))),
                      dim3(kThreads), 0, s, static_cast<const __nv_bfloat16 *>(rows), K / 32, MOE_FP4_PITCH(K),
                      G->offsets, (int)G->E, (int)G->rows, static_cast<uint8_t *>(codes),
                      static_cast<uint8_t *>(scales), G->ws, aligned32(rows));
}

cudaError_t launch_dequantize_fp4(const moe_rows *G, const void *codes, const void *scales, int K, void *rows,
                                  cudaStream_t s)
{
    if (G->rows == 0) return cudaSuccess;
    return launch_pdl(dequantize_fp4_kernel, dim3(grid_for(dequantize_fp4_kernel, (long long)G->rows * (K / 32))),
                      dim3(kThreads), 0, s, static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales),
                      K / 32, MOE_FP4_PITCH(K), G->offsets, (int)G->E, (int)G->rows,
                      static_cast<__nv_bfloat16 *>(rows), G->ws, aligned32(rows));
}

}  // namespace moe
