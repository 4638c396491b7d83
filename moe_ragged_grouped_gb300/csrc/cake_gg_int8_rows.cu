// cake_gg_int8_rows.cu -- the 8-bit integer products for few rows.
//
//   Y[m, n] = (sum_k q[r(m), k] W[e(m), n, k]) * ws[e(m), n] * xs[r(m)]
//
// With a handful of rows per expert every weight byte is used a handful of
// times, so the weights' bytes bound the time.  Each warp owns C channels of
// one expert and up to 8 of its rows; its lanes walk K in 16-byte vectors, so
// a warp load covers 512 contiguous bytes of a weight row, and U * C loads are
// in flight per lane before the first is used.  Products are summed four at a
// time in 32-bit integers (exact: K < 2^17 keeps |sum| below 2^31), so the
// order of the sums is free and a row's K can be divided over the warps of a
// block; the result is rounded once, at the end.
#include "cake_gg_int8.h"
#include "cake_gg_ptx.cuh"

namespace cakegg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// 16 weight bytes, read once: not kept in L1.
__device__ __forceinline__ uint4 ld_weights(const int8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int acc)
{
    acc = __dp4a(int(a.x), int(b.x), acc);
    acc = __dp4a(int(a.y), int(b.y), acc);
    acc = __dp4a(int(a.z), int(b.z), acc);
    return __dp4a(int(a.w), int(b.w), acc);
}

__device__ __forceinline__ void store_out(const I8Params &p, int64_t at, float v)
{
    if (p.out_f32) static_cast<float *>(p.Y)[at] = v;
    else static_cast<uint16_t *>(p.Y)[at] = uint16_t(pack_bf16x2(v, 0.0f) & 0xffffu);
}

// Rows [m, m + n_rows) of expert e against the block's channels.  R >= n_rows
// rows are computed (a missing one repeats the first and is not stored).
template <int R, int C, int U>
__device__ __forceinline__ void row_chunk(const I8Params &p, const int8_t *__restrict__ q, int e, int64_t m,
                                          int n_rows, int block_c, int S, int *part)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ks = warp % S, groups = kWarps / S;
    const int n0 = (block_c * groups + warp / S) * C;
    const int nv = p.K / 16;                 // 16-byte vectors of a row
    const int step = 32 * S;
    const bool live = n0 < p.N;              // N is a multiple of 8, so all C channels are
    const int8_t *w = p.W + (int64_t(e) * p.N + (live ? n0 : 0)) * p.K;

    int acc[R][C];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = 0;

    const int8_t *x[R];
    bool ready = false;
    for (int v0 = ks * 32 + lane; __any_sync(0xffffffffu, live && v0 < nv); v0 += U * step) {
        uint4 wv[U][C];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int v = v0 + u * step;
                wv[u][c] = live && v < nv ? ld_weights(w + int64_t(c) * p.K + int64_t(v) * 16) : make_uint4(0, 0, 0, 0);
            }
        if (!ready) {
            // the tokens are complete once the grid before this one is
            grid_dependency_wait();
            ready = true;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                int64_t t = m + (r < n_rows ? r : 0);
                if (p.rows) t = p.rows[t];
                x[r] = q + (t >= 0 && t < p.T ? t : 0) * int64_t(p.K);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u * step < nv ? v0 + u * step : 0;   // past the end: weights are zero
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint4 xv = *reinterpret_cast<const uint4 *>(x[r] + int64_t(v) * 16);
#pragma unroll
                for (int c = 0; c < C; ++c) acc[r][c] = dot16(wv[u][c], xv, acc[r][c]);
            }
        }
    }
    grid_dependency_wait();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int s = __reduce_add_sync(0xffffffffu, acc[r][c]);
            if (lane == 0) part[warp * (R * C) + r * C + c] = s;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < groups * R * C; i += kThreads) {
        const int g = i / (R * C), r = i / C % R, c = i % C;
        const int n = (block_c * groups + g) * C + c;
        if (r >= n_rows || n >= p.N) continue;
        int sum = 0;
        for (int k = 0; k < S; ++k) sum += part[(g * S + k) * (R * C) + r * C + c];
        int64_t t = m + r;
        if (p.rows) t = p.rows[t];
        if (t < 0 || t >= p.T) {
            atomicCAS(p.status, 0, kI8StatusBadRows);
            continue;
        }
        store_out(p, (m + r) * int64_t(p.N) + n, float(sum) * p.ws[int64_t(e) * p.N + n] * p.xs[t]);
    }
}

// blockIdx.x = row * blocks_n + channel block.  The block whose row starts a
// chunk of its expert's rows computes the chunk; the others leave.
__global__ void __launch_bounds__(kThreads)
    i8_rows_kernel(const I8Params p, const int8_t *__restrict__ q, int blocks_n, int S)
{
    __shared__ int part[kWarps * 32];
    __shared__ int found[4];   // expert, its first row, its end, offsets invalid
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();
    const int64_t m = blockIdx.x / unsigned(blocks_n);
    const int block_c = int(blockIdx.x % unsigned(blocks_n));
    if (threadIdx.x == 0) {
        found[0] = p.offsets ? -1 : 0;
        found[1] = 0;
        found[2] = int(p.M);
        found[3] = 0;
    }
    __syncthreads();
    if (p.offsets)
        for (int e = threadIdx.x; e < p.E; e += kThreads) {
            const int a = p.offsets[e], b = p.offsets[e + 1];
            if ((e == 0 && a != 0) || b < a || b > p.M) found[3] = 1;
            else if (a <= m && m < b) {
                found[0] = e;
                found[1] = a;
                found[2] = b;
            }
        }
    __syncthreads();
    const int e = found[0];
    if (found[3] || e < 0 || (m - found[1]) % kI8RowChunk != 0) {
        grid_dependency_wait();
        if (found[3] && threadIdx.x == 0) atomicCAS(p.status, 0, kI8StatusBadOffsets);
        return;
    }
    const int n = int(found[2] - m < kI8RowChunk ? found[2] - m : kI8RowChunk);
    if (n == 1) row_chunk<1, 2, 4>(p, q, e, m, n, block_c, S, part);
    else if (n == 2) row_chunk<2, 2, 4>(p, q, e, m, n, block_c, S, part);
    else if (n <= 4) row_chunk<4, 2, 4>(p, q, e, m, n, block_c, S, part);
    else row_chunk<8, 2, 4>(p, q, e, m, n, block_c, S, part);
}

}  // namespace

cudaError_t launch_i8_rows(const I8Params &p, const int8_t *q, bool pdl, cudaStream_t stream)
{
    const int S = 1, C = 2;
    const int blocks_n = (p.N + kWarps / S * C - 1) / (kWarps / S * C);
    const int64_t blocks = p.M * blocks_n;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, i8_rows_kernel, p, q, blocks_n, S);
}

}  // namespace cakegg
