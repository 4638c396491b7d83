// cake_gg_int8_rows.cu -- the 8-bit integer products for few rows.
//
//   Y[m, n] = (sum_k q[r(m), k] W[e(m), n, k]) * ws[e(m), n] * xs[r(m)]
//
// With a handful of rows per expert every weight byte is used a handful of
// times, so the weights' bytes bound the time.  Each warp owns C channels of
// one expert and up to R of its rows; its lanes walk K in 16-byte vectors, so
// a warp load covers 512 contiguous bytes of a weight row, and U * C loads are
// in flight per lane before the first is used.  Products are summed four at a
// time in 32-bit integers (exact: K < 2^17 keeps |sum| below 2^31), so the
// order of the sums is free and a row's K can be divided over S warps of a
// block; the result is rounded once, at the end.  One token through 4 of 32
// experts 6144 -> 4096 takes 17.6 us with its token pass (5.7 TB/s over the call;
// two channels a warp with four loads each 18.9, one channel 19.3, K over two
// warps 21).
//
// Activations of one or two rows over few weights may be quantised by every
// block for itself, into shared memory, while its first weights are on the way
// (i8_rows_fused): called one by one, a launch less is worth more.
#include "cake_gg_int8.h"
#include "cake_gg_int8_quant.cuh"
#include "cake_gg_ptx.cuh"

namespace cakegg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kC = 4;              // channels of a warp
constexpr int kU = 2;              // vectors of each in flight per lane
constexpr int kFusedBytes = 32768; // rows quantised in shared memory at most
constexpr int64_t kFusedWeights = 32 << 20;
constexpr int64_t kFusedValues = 1 << 22, kFusedGated = 1 << 19;

// Blocks of a multiprocessor: the launch bounds below hold the registers to it.
// (Two rows at 66 registers had three: 2 x 4096 -> 4096 6.0 us, 4.5 with four.)
constexpr int blocks_of(int R) { return R == 4 ? 3 : 4; }

// K is divided over S warps while all warps still fit the multiprocessors at
// once and each has a vector of every lane (a wave and a bit: one token 4096 ->
// 6144 5.5 us, 4.7 with half the warps).
int k_warps(int R, int32_t E, int64_t M, int32_t N, int32_t K)
{
    const int64_t runs = E > 1 ? M : (M + R - 1) / R, warps = runs * (N / kC), most = 152ll * kWarps * blocks_of(R);
    int S = 1;
    while (S < kWarps && warps * S * 2 <= most && 512 * S < K) S *= 2;
    return S;
}
int channel_blocks(int S, int32_t N)
{
    const int per_block = kWarps / S * kC;
    return (N + per_block - 1) / per_block;
}

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

// The block's R rows of activations (null: none) as bytes in shared memory and
// their scales.  (The second reading comes from L1; held in registers between
// the two the values cost more in occupancy: 18.5 against 20.8 us for one token
// through 4 of 32 experts 6144 -> 4096.)
template <int R, typename XT, bool ACT>
__device__ __forceinline__ void quantise_rows(const XT *const (&x)[R], int32_t K, int8_t *q, float *scale, uint32_t (*top)[kWarps])
{
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint32_t m = 0;
        if (x[r])
            for (int k = int(threadIdx.x) * 8; k < K; k += kThreads * 8) {
                float v[8];
                row8<XT, ACT>(x[r], K, k, v);
                m = max_bits(v, m);
            }
        m = __reduce_max_sync(0xffffffffu, m);
        if (threadIdx.x % 32 == 0) top[r][threadIdx.x / 32] = m;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint32_t m = top[r][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = max(m, top[r][w]);
        const RowScale s(m);
        if (threadIdx.x == 0) scale[r] = s.scale;
        for (int k = int(threadIdx.x) * 8; k < K; k += kThreads * 8) {
            float v[8] = {};
            if (x[r]) row8<XT, ACT>(x[r], K, k, v);
            *reinterpret_cast<uint2 *>(q + int64_t(r) * K + k) = bytes8(v, s);
        }
    }
    __syncthreads();
}

// XT: int8_t (X holds the quantised tokens), uint16_t (BF16) or float.
// blockIdx.x = row * blocks_n + channel block.  The block whose row starts a
// run of R of its expert's rows computes the run; the others leave.
template <int R, typename XT, bool ACT>
__global__ void __launch_bounds__(kThreads, blocks_of(R))
    i8_rows_kernel(const I8Params p, const XT *__restrict__ X, int blocks_n, int S)
{
    constexpr bool kFused = sizeof(XT) > 1;
    extern __shared__ __align__(16) int8_t q_smem[];   // fused: [R][K]
    __shared__ int part[kWarps * R * kC];
    __shared__ uint32_t top[R][kWarps];
    __shared__ float scale[R];
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
    if (found[3] || e < 0 || (m - found[1]) % R != 0) {
        grid_dependency_wait();
        if (found[3] && threadIdx.x == 0) atomicCAS(p.status, 0, kI8StatusBadOffsets);
        return;
    }
    const int n_rows = int(found[2] - m < R ? found[2] - m : R);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ks = warp % S, groups = kWarps / S;
    const int n0 = (block_c * groups + warp / S) * kC;
    const int nv = p.K / 16;                 // 16-byte vectors of a row
    const int step = 32 * S;
    const bool live = n0 < p.N;              // N is a multiple of 8, so all C channels are
    const int8_t *w = p.W + (int64_t(e) * p.N + (live ? n0 : 0)) * p.K;
    uint4 wv[kU][kC];
    auto load = [&](int v0) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int v = v0 + u * step;
                wv[u][c] = live && v < nv ? ld_weights(w + int64_t(c) * p.K + int64_t(v) * 16) : make_uint4(0, 0, 0, 0);
            }
    };
    const int first = ks * 32 + lane;
    load(first);
    // while the token pass still runs the rest of the block's weights move to L2
    // (down one token, 4 x 2048 -> 6144: 11.2 us, 12.3 without)
    if (p.early && live && lane % 8 == 0)
        for (int v = first + kU * step; v < nv; v += step)
#pragma unroll
            for (int c = 0; c < kC; ++c) prefetch_l2(w + int64_t(c) * p.K + int64_t(v) * 16);

    // the tokens are complete once the grid before this one is
    grid_dependency_wait();
    const int8_t *x[R];
    const XT *row[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        int64_t t = m + (r < n_rows ? r : 0);
        if (p.rows) t = p.rows[t];
        const bool in = t >= 0 && t < p.T;                       // (others: reported where they are scaled)
        row[r] = r < n_rows && in ? X + t * (ACT ? 2 : 1) * int64_t(p.K) : kFused ? nullptr : X;
        x[r] = kFused ? q_smem + int64_t(r) * p.K : reinterpret_cast<const int8_t *>(row[r]);
    }
    if constexpr (kFused) quantise_rows<R, XT, ACT>(row, p.K, q_smem, scale, top);

    int acc[R][kC];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[r][c] = 0;
    for (int v0 = first; __any_sync(0xffffffffu, live && v0 < nv);) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int v = v0 + u * step < nv ? v0 + u * step : 0;   // past the end: weights are zero
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint4 xv = *reinterpret_cast<const uint4 *>(x[r] + int64_t(v) * 16);
#pragma unroll
                for (int c = 0; c < kC; ++c) acc[r][c] = dot16(wv[u][c], xv, acc[r][c]);
            }
        }
        v0 += kU * step;
        load(v0);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int s = __reduce_add_sync(0xffffffffu, acc[r][c]);
            if (lane == 0) part[warp * (R * kC) + r * kC + c] = s;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < groups * R * kC; i += kThreads) {
        const int g = i / (R * kC), r = i / kC % R, c = i % kC;
        const int n = (block_c * groups + g) * kC + c;
        if (r >= n_rows || n >= p.N) continue;
        int sum = 0;
        for (int k = 0; k < S; ++k) sum += part[(g * S + k) * (R * kC) + r * kC + c];
        int64_t t = m + r;
        if (p.rows) t = p.rows[t];
        if (t < 0 || t >= p.T) {
            atomicCAS(p.status, 0, kI8StatusBadRows);
            continue;
        }
        store_out(p, (m + r) * int64_t(p.N) + n, float(sum) * p.ws[int64_t(e) * p.N + n] * (kFused ? scale[r] : p.xs[t]));
    }
}

template <int R, typename XT, bool ACT>
cudaError_t launch(const I8Params &p, const void *X, bool pdl, cudaStream_t stream)
{
    const int S = k_warps(R, p.E, p.M, p.N, p.K), blocks_n = channel_blocks(S, p.N);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(unsigned(i8_rows_blocks(p)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = sizeof(XT) > 1 ? size_t(R) * size_t(p.K) : 0;
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, i8_rows_kernel<R, XT, ACT>, p, static_cast<const XT *>(X), blocks_n, S);
}

template <typename XT, bool ACT>
cudaError_t launch_fused(const I8Params &p, const void *X, bool pdl, cudaStream_t stream)
{
    return i8_run_rows(p.E, p.M, p.T) == 1 ? launch<1, XT, ACT>(p, X, pdl, stream) : launch<2, XT, ACT>(p, X, pdl, stream);
}

}  // namespace

// Rows of an expert that a block takes: all that there can be where rows are
// dense.  Where few rows meet many experts nearly every expert has one row (and
// a token does not meet an expert twice, unless there are more rows than tokens
// times experts), and the kernels for fewer rows hold more loads in flight; a
// second row of an expert is another block.
int i8_run_rows(int32_t E, int64_t M, int64_t T)
{
    const int64_t most = T < M && M <= E * T ? T : M;
    if (most <= 1 || (E > 1 && E >= 4 * M)) return 1;
    return most <= 2 || (E > 1 && E >= M) ? 2 : 4;
}

int64_t i8_rows_blocks(const I8Params &p)
{
    return p.M * channel_blocks(k_warps(i8_run_rows(p.E, p.M, p.T), p.E, p.M, p.N, p.K), p.N);
}

// Every block repeats the quantising of its rows, against one launch less: 2.1 us
// of the host where calls follow one another.  On the GPU the repeats cost 0.5 us
// a million values, gated ones 5 (two readings, each with an exponential and a
// division), and the limits leave them at most the launch's price.  Measured,
// graph replays, repeated and with a token pass (in brackets called one by one):
// one token 4096 -> 4096 5.0 (6.6), 3.8 (8.4) us; 8192 -> 2048, at the limit, 6.2
// (6.5), 4.0 (8.5); 8192 -> 4096 8.4 (8.7), 5.3 (8.5); gated 2048 -> 2048 4.1 (6.6),
// 3.5 (8.6); gated 4096 -> 4096 8.8 (9.1), 4.2 (8.5).
bool i8_rows_fused(const I8Params &p, int act)
{
    const int64_t bytes = (p.M < p.E ? p.M : p.E) * p.N * p.K;
    const int run = i8_run_rows(p.E, p.M, p.T);
    if (run > 2 || bytes * run > kFusedWeights || int64_t(run) * p.K > kFusedBytes) return false;
    const int64_t values = p.M * p.K * channel_blocks(k_warps(run, p.E, p.M, p.N, p.K), p.N);
    return values <= (act == CAKE_GG_ACT_NONE ? kFusedValues : kFusedGated);
}

cudaError_t launch_i8_rows(const I8Params &p, const void *X, int x_dtype, int act, bool pdl, cudaStream_t stream)
{
    const bool silu = act == CAKE_GG_ACT_SILU_MUL;
    if (x_dtype == CAKE_GG_BF16)
        return silu ? launch_fused<uint16_t, true>(p, X, pdl, stream) : launch_fused<uint16_t, false>(p, X, pdl, stream);
    if (x_dtype == CAKE_GG_FP32)
        return silu ? launch_fused<float, true>(p, X, pdl, stream) : launch_fused<float, false>(p, X, pdl, stream);
    switch (i8_run_rows(p.E, p.M, p.T)) {
    case 1: return launch<1, int8_t, false>(p, X, pdl, stream);
    case 2: return launch<2, int8_t, false>(p, X, pdl, stream);
    default: return launch<4, int8_t, false>(p, X, pdl, stream);
    }
}

}  // namespace cakegg
