// cake_gg_combine.cu -- the rows' way back to their tokens, and its gradients.
//
//   y[t] = sum_j w[t, j] r[position[t, j]]           (or without weights)
//   dr[position[t, j]] = w[t, j] dy[t]               (without: tokens to their rows)
//   dw[t, j] = <dy[t], r[position[t, j]]>
//
// Sums are FP32, over j in order, each product rounded with its addition; nothing
// is added by atomics.  A position outside [0, M) is no row: it adds nothing and
// gets nothing.
#include <cstdint>
#include <cstdlib>
#include <type_traits>

#include <cuda_runtime.h>

#include "../../include/cake_gg.h"
#include "cake_gg_ptx.cuh"

namespace cakegg {
int device_sms(int *sms);   // (cake_gg_capi.cu)
}
using namespace cakegg;

namespace {

constexpr int32_t kMaxTop = 32;
constexpr unsigned kFull = 0xffffffffu;

// Eight values of a row in memory, as FP32.  Each is read and written once, so loads
// and stores are the first out of the caches: with that 8191 tokens of 2 x 4096 BF16 take
// 35 us (5.8 TB/s) instead of 38, their gradients 56 instead of 60 (with the loads alone so 68).
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8])
{
    const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8])
{
    __stcs(reinterpret_cast<uint4 *>(p),
           make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}

// Four values, for tokens to FP32 rows.
__device__ __forceinline__ void load4(const uint16_t *p, float (&v)[8], int i)
{
    const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p));
    v[i] = __uint_as_float(w.x << 16), v[i + 1] = __uint_as_float(w.x & 0xffff0000u);
    v[i + 2] = __uint_as_float(w.y << 16), v[i + 3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float *p, float (&v)[8], int i)
{
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
}

__device__ __forceinline__ void store4(float *p, const float (&v)[8], int i)
{
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
}

struct CombineParams {
    const void *rows;         // r [M, K]
    const int32_t *position;  // [T, top_k]
    const float *weight;      // [T, top_k] or null
    void *out;                // y [T, K]
    const void *d_out;        // dy [T, K]
    void *d_rows;             // [M, K]
    float *d_weight;          // [T, top_k] or null
    int64_t T, M;
    int32_t top_k, K;
};

// A block has N tokens and 8 values a thread of a part of their rows, or, of short rows,
// N tokens for each G threads (100000 of 2 x 256 31 us, with blocks of 32 threads 51; but
// 32768 of 4 x 512 35, with blocks of 64 threads 30).  Bound by HBM and by the loads in
// flight: two tokens where one has few rows or short ones.
template <int N, bool SHORT, typename RT, typename OT>
__global__ void __launch_bounds__(256)
    combine_kernel(const CombineParams p, int G)
{
    grid_dependency_wait();
    grid_launch_dependents();
    int64_t t = int64_t(blockIdx.x) * N;
    int thread = int(threadIdx.x);
    if (SHORT) {
        const int mine = __shfl_sync(kFull, thread / G, 0);
        t = (int64_t(blockIdx.x) * (256 / G) + mine) * N;
        thread -= mine * G;
    }
    const int32_t k = int32_t(blockIdx.y * blockDim.x) * 8 + thread * 8;
    if (k >= p.K) return;
    float sum[N][8] = {};
#pragma unroll 4
    for (int j = 0; j < p.top_k; ++j)
#pragma unroll
        for (int h = 0; h < N; ++h) {
            if ((SHORT || h > 0) && t + h >= p.T) continue;
            const int64_t at = (t + h) * p.top_k + j, m = p.position[at];
            const float w = p.weight ? p.weight[at] : 1.0f;
            if (m < 0 || m >= p.M) continue;
            float v[8];
            load8(static_cast<const RT *>(p.rows) + m * p.K + k, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[h][i] = fmaf(w, v[i], sum[h][i]);
        }
#pragma unroll
    for (int h = 0; h < N; ++h)
        if ((!SHORT && h == 0) || t + h < p.T) store8(static_cast<OT *>(p.out) + (t + h) * p.K + k, sum[h]);
}

// A block's 256 threads are one token's or, of short rows, several tokens', G threads
// each.  A thread has C vectors of 8 values of dy at a time, which stay in registers for
// the token's rows, of which U are under way at once.  (DW: with the weights' gradients.)
// With a token a block, of as many threads as its row has vectors, 100000 tokens of 2 x 256
// took 101 us, their gradients 101 (26 and 49 so), 4096 of 8 x 7168 195 (166).  Of more U or
// C hold registers that more blocks would have: 8191 x 2 x 4096 57 us, with U = 4 73.
template <int C, int U, bool DW, typename RT, typename OT>
__global__ void __launch_bounds__(256)
    combine_grad_kernel(const CombineParams p, int G)
{
    // (FP32 rows that are only written: a warp's stores lie side by side, 16 bytes a lane)
    constexpr bool kSplit = !DW && sizeof(RT) == 4;
    __shared__ float part[DW ? kMaxTop : 1][8];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tokens = 256 / G, mine = __shfl_sync(kFull, int(threadIdx.x) / G, 0), thread = int(threadIdx.x) - mine * G;   // (uniform)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, step = G * 8;
    const int64_t t0 = int64_t(blockIdx.x) * tokens, t = t0 + mine;
    const int top_k = t < p.T ? p.top_k : 0;
    const int32_t *position = p.position + t * p.top_k;
    const OT *dy = static_cast<const OT *>(p.d_out) + t * p.K;
    for (int32_t k0 = 0; k0 < p.K; k0 += C * step) {
        const int32_t k = k0 + thread * 8, ka = k0 + (thread & ~31) * 8 + lane * 4;
        float g[C][8] = {};
#pragma unroll
        for (int c = 0; c < C; ++c)
            if constexpr (kSplit) {
                if (top_k > 0 && ka + c * step < p.K) load4(dy + ka + c * step, g[c], 0);
                if (top_k > 0 && ka + c * step + 128 < p.K) load4(dy + ka + c * step + 128, g[c], 4);
            } else if (top_k > 0 && k + c * step < p.K) {
                load8(dy + k + c * step, g[c]);
            }
        for (int j0 = 0; j0 < top_k; j0 += U) {
            int64_t m[U];
            float dot[U] = {}, v[DW ? U : 1][DW ? C : 1][8] = {};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                m[u] = j0 + u < top_k ? position[j0 + u] : -1;
                if (m[u] >= p.M) m[u] = -1;
                if constexpr (DW) {
                    if (m[u] >= 0)
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            if (k + c * step < p.K) load8(static_cast<const RT *>(p.rows) + m[u] * p.K + k + c * step, v[u][c]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (m[u] < 0) continue;
                const float w = p.weight ? p.weight[t * p.top_k + j0 + u] : 1.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float d[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (DW) dot[u] = fmaf(g[c][i], v[u][c][i], dot[u]);
                        d[i] = w * g[c][i];
                    }
                    RT *to = static_cast<RT *>(p.d_rows) + m[u] * p.K + c * step;
                    if constexpr (kSplit) {
                        if (ka + c * step < p.K) store4(to + ka, d, 0);
                        if (ka + c * step + 128 < p.K) store4(to + ka + 128, d, 4);
                    } else if (k + c * step < p.K) {
                        store8(to + k, d);
                    }
                }
            }
            if constexpr (DW) {
#pragma unroll
                for (int s = 16; s; s >>= 1)
#pragma unroll
                    for (int u = 0; u < U; ++u) dot[u] += __shfl_xor_sync(kFull, dot[u], s);
                if (lane == 0)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (j0 + u < top_k) part[j0 + u][warp] = k0 == 0 ? dot[u] : part[j0 + u][warp] + dot[u];
            }
        }
    }
    if constexpr (DW) {
        __syncthreads();
        for (int i = threadIdx.x; i < tokens * p.top_k; i += 256) {
            const int of = i / p.top_k, j = i % p.top_k;
            if (t0 + of >= p.T) break;
            float sum = 0.0f;
            for (int w = 0; w < G / 32; ++w) sum += part[j][of * (G / 32) + w];
            p.d_weight[t0 * p.top_k + i] = sum;
        }
    }
}

// Rows that no position names: a mark for each that one does, then zeros for those
// without, a warp 32 rows.  (All named: 4.4 us for 8191 x 2 rows of 4096 BF16, 4.8 for
// 4096 x 8 of 7168, where zeros in all rows before their gradients take 34 and 116.)
__global__ void __launch_bounds__(256)
    mark_kernel(const int32_t *__restrict__ position, int64_t n, int64_t M, uint8_t *__restrict__ named)
{
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t m = position[i];
    if (m >= 0 && m < M) named[m] = 1;
}
__global__ void __launch_bounds__(256)
    clear_kernel(const uint8_t *__restrict__ named, int64_t M, int32_t pieces, uint4 *__restrict__ rows)
{
    const int lane = threadIdx.x & 31;
    const int64_t m0 = (int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 32;
    unsigned bare = __ballot_sync(kFull, m0 + lane < M && named[m0 + lane] == 0);
    for (; bare; bare &= bare - 1) {
        uint4 *row = rows + (m0 + __ffs(int(bare)) - 1) * pieces;
        for (int32_t i = lane; i < pieces; i += 32) row[i] = make_uint4(0, 0, 0, 0);
    }
}

bool pdl_enabled()
{
    const char *v = std::getenv("CAKE_GG_PDL");
    return !(v && std::atoi(v) == 0);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename Kernel, typename... More>
cudaError_t launch(Kernel kernel, const CombineParams &p, int64_t blocks, int parts, int threads, cudaStream_t stream, More... more)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    if (pdl_enabled()) {
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    cfg.gridDim = dim3(unsigned(blocks), unsigned(parts), 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, p, more...);
}

int check(int64_t T, int64_t M, int32_t top_k, int32_t K, int rows_dtype, int out_dtype)
{
    if (T < 0 || T > INT32_MAX || M < 0 || M > INT32_MAX || top_k < 1 || top_k > kMaxTop || K < 1) return CAKE_GG_ERR_INVALID_ARG;
    if ((rows_dtype != CAKE_GG_BF16 && rows_dtype != CAKE_GG_FP32) || (out_dtype != CAKE_GG_BF16 && out_dtype != CAKE_GG_FP32))
        return CAKE_GG_ERR_UNSUPPORTED;
    if (K % 8 != 0) return CAKE_GG_ERR_ALIGNMENT;
    if (K > 1 << 20) return CAKE_GG_ERR_OVERFLOW;
    return CAKE_GG_OK;
}

// Threads for a token's row of K values, 8 a thread, up to 256: a power of two, whole warps.
int threads_for(int32_t K)
{
    int G = 32;
    while (G < 256 && G * 8 < K) G *= 2;
    return G;
}

}  // namespace

extern "C" {

int cake_gg_combine_rows(int64_t T, int64_t M, int32_t top_k, int32_t K, const void *rows, int rows_dtype, const int32_t *position,
                         const float *weight, void *out, int out_dtype, void *stream)
{
    int rc = check(T, M, top_k, K, rows_dtype, out_dtype);
    if (rc != CAKE_GG_OK) return rc;
    if (T == 0) return CAKE_GG_OK;
    if ((M > 0 && !rows) || !position || !out) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(position, 4) || !aligned(weight, 4)) return CAKE_GG_ERR_ALIGNMENT;
    int sms;
    if ((rc = device_sms(&sms)) != CAKE_GG_OK) return rc;
    CombineParams p{};
    p.rows = rows;
    p.position = position;
    p.weight = weight;
    p.out = out;
    p.T = T;
    p.M = M;
    p.top_k = top_k;
    p.K = K;
    const int warps = (K / 8 + 31) / 32, G = threads_for(K);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // (BF16 16384 tokens of 2 rows x 4096: 68 us with two tokens a block, 69 with one, 32768 of
    // 4 x 512 31 and 34, but 8192 of 4 x 6144 85 and 84)
    const bool two = T > 1 && (top_k <= 2 || K <= 1024), few = T > 1 && top_k * K <= 1024;
    const int threads = few || warps >= 8 ? 256 : warps * 32, parts = (warps * 32 + threads - 1) / threads;
    const int64_t tokens = (few ? 256 / G : 1) * (two ? 2 : 1), blocks = (T + tokens - 1) / tokens;
    auto run = [&](auto rows_of, auto out_of) {
        using RT = decltype(rows_of);
        using OT = decltype(out_of);
        return few   ? launch(combine_kernel<2, true, RT, OT>, p, blocks, parts, threads, s, G)
               : two ? launch(combine_kernel<2, false, RT, OT>, p, blocks, parts, threads, s, G)
                     : launch(combine_kernel<1, false, RT, OT>, p, blocks, parts, threads, s, G);
    };
    const bool r16 = rows_dtype == CAKE_GG_BF16, o16 = out_dtype == CAKE_GG_BF16;
    const cudaError_t err = r16 ? (o16 ? run(uint16_t(), uint16_t()) : run(uint16_t(), float())) : (o16 ? run(float(), uint16_t()) : run(float(), float()));
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

int cake_gg_combine_grad(int64_t T, int64_t M, int32_t top_k, int32_t K, const void *d_out, int out_dtype, const void *rows,
                         int rows_dtype, const int32_t *position, const float *weight, void *d_rows, float *d_weight, void *stream)
{
    int rc = check(T, M, top_k, K, rows_dtype, out_dtype);
    if (rc != CAKE_GG_OK) return rc;
    if (T == 0) return CAKE_GG_OK;
    if (!d_out || !position || (M > 0 && !d_rows) || (d_weight && M > 0 && !rows)) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(d_out, 16) || !aligned(rows, 16) || !aligned(d_rows, 16) || !aligned(position, 4) || !aligned(weight, 4) || !aligned(d_weight, 4))
        return CAKE_GG_ERR_ALIGNMENT;
    int sms;
    if ((rc = device_sms(&sms)) != CAKE_GG_OK) return rc;
    CombineParams p{};
    p.d_out = d_out;
    p.rows = rows;
    p.position = position;
    p.weight = weight;
    p.d_rows = d_rows;
    p.d_weight = d_weight;
    p.T = T;
    p.M = M;
    p.top_k = top_k;
    p.K = K;
    const int G = threads_for(K);
    const int vectors = (K / 8 + G - 1) / G;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t blocks = (T + 256 / G - 1) / (256 / G);
    using one = std::integral_constant<int, 1>;
    using two = std::integral_constant<int, 2>;
    using four = std::integral_constant<int, 4>;
    auto run = [&](auto rows_of, auto out_of) {
        using RT = decltype(rows_of);
        using OT = decltype(out_of);
        auto go = [&](auto c, auto u, auto dw) {
            return launch(combine_grad_kernel<decltype(c)::value, decltype(u)::value, decltype(dw)::value, RT, OT>, p, blocks, 1, 256, s, G);
        };
        // (8191 tokens to 2 rows x 4096: 31.5 us by one vector at a time, 30.6 by two; 16384 to
        // 2 x 2048, where the second is past the row, 31.9 and 33.0)
        if (!d_weight) return vectors == 1 ? go(one(), one(), std::false_type()) : go(two(), one(), std::false_type());
        // (16384 x 1 x 4096 72 us, two rows at a time 85; 42 tokens of 8 x 3128 FP32 6.1 us four at a time, 6.9 two)
        return top_k == 1       ? go(one(), one(), std::true_type())
               : blocks <= 152 ? go(one(), four(), std::true_type())
                               : go(one(), two(), std::true_type());
    };
    const bool r16 = rows_dtype == CAKE_GG_BF16, o16 = out_dtype == CAKE_GG_BF16;
    const cudaError_t err = r16 ? (o16 ? run(uint16_t(), uint16_t()) : run(uint16_t(), float())) : (o16 ? run(float(), uint16_t()) : run(float(), float()));
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

int cake_gg_zero_unnamed_rows(int64_t T, int64_t M, int32_t top_k, int32_t K, const int32_t *position, void *rows, int rows_dtype,
                              uint8_t *named, void *stream)
{
    int rc = check(T, M, top_k, K, rows_dtype, rows_dtype);
    if (rc != CAKE_GG_OK) return rc;
    if (M == 0) return CAKE_GG_OK;
    if ((T > 0 && !position) || !rows || !named) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(rows, 16) || !aligned(position, 4)) return CAKE_GG_ERR_ALIGNMENT;
    const int64_t n = T * top_k, blocks = (n + 255) / 256;
    if (blocks > INT32_MAX) return CAKE_GG_ERR_OVERFLOW;
    int sms;
    if ((rc = device_sms(&sms)) != CAKE_GG_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(named, 0, size_t(M), s) != cudaSuccess) return CAKE_GG_ERR_CUDA;
    if (n > 0) mark_kernel<<<unsigned(blocks), 256, 0, s>>>(position, n, M, named);
    clear_kernel<<<unsigned((M + 255) / 256), 256, 0, s>>>(named, M, K / (rows_dtype == CAKE_GG_BF16 ? 8 : 4), static_cast<uint4 *>(rows));
    return cudaGetLastError() == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

}  // extern "C"
