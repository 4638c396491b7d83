// cake_gg_int8_warps.cu -- the 8-bit integer products for a few dozen rows.
//
//   Y[m, n] = (sum_k q[r(m), k] W[e(m), n, k]) * ws[e(m), n] * xs[r(m)]
//
// Between the few rows of 32-bit dot products and the tiles of the tensor-core
// path lies the decoding batch: the weights' bytes and the time until the first
// of them arrive bound it, and setting up tensor memory, copies and clusters
// costs more than the product.  Here warps multiply straight from registers.
// Every 8-bit integer is exact in FP16 and every sum below 2^24 in FP32, as in
// the tensor-core path.
//
// A block takes 32 channels of one expert and up to 8 * NT of its rows; its
// eight warps divide K in steps of 64.  In a step a lane loads 16 bytes of each
// of four weight rows (lane / 4 + 0, 8, 16, 24) and of NT token rows (lane / 4 +
// 8 i), all at offset 16 * (lane % 4), and widens them: since a sum over k may
// take k in any order that both operands share, the lane's 16 values are the
// A and B fragments of four m16n8k16 products without any exchange.  The warps'
// sums meet in shared memory and are added in warp order.
//
// Bound: small weights by the start of the kernel (16 x 1024 -> 2048: 4.4 us with
// the token pass), larger ones by the loads that the registers hold in flight (16 x
// 4096 -> 5120: 11.5 us, 1.9 TB/s), which is where the tensor-core path takes over.
#include "cake_gg_int8.h"
#include "cake_gg_int8_index.h"
#include "cake_gg_int8_widen.cuh"
#include "cake_gg_ptx.cuh"

namespace cakegg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChannels = 32;
constexpr int kPad = kChannels + 1;     // floats of a row's sums in shared memory

__device__ __forceinline__ uint4 ld_weights(const int8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 16 values: pairs 2 j and 2 j + 1 belong to the j-th product.
__device__ __forceinline__ void widen16(const uint4 &w, uint32_t (&f)[8])
{
    widen4(w.x, f[0], f[1]);
    widen4(w.y, f[2], f[3]);
    widen4(w.z, f[4], f[5]);
    widen4(w.w, f[6], f[7]);
}

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// blockIdx.x = row * blocks_n + channel block.  The block whose row starts a run
// of 8 * NT of its expert's rows computes the run; the others leave.
template <int NT>
__global__ void __launch_bounds__(kThreads)
    i8_warps_kernel(const I8Params p, const int8_t *__restrict__ q, int blocks_n)
{
    constexpr int R = 8 * NT;
    extern __shared__ float sums[];    // [warp][R][kPad]
    __shared__ int found[4];           // expert, its first row, its end, offsets invalid
    __shared__ float xs[R];
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();
    const int64_t m = blockIdx.x / unsigned(blocks_n);
    const int n0 = int(blockIdx.x % unsigned(blocks_n)) * kChannels;
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
    const int at = i8_warps_place(lane);
    const int steps = (p.K + 63) / 64;
    const int8_t *w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + (lane >> 2) + 8 * i;
        w[i] = p.W + (int64_t(e) * p.N + (n < p.N ? n : 0)) * p.K + at;    // (a channel past the end is not stored)
    }
    uint4 wv[4];
    auto load_w = [&](int s) {
        const bool in = i8_warps_in(s, lane, p.K);
#pragma unroll
        for (int i = 0; i < 4; ++i) wv[i] = in ? ld_weights(w[i] + s * 64) : make_uint4(0, 0, 0, 0);
    };
    load_w(warp);

    grid_dependency_wait();            // the tokens
    const int8_t *x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int r = (lane >> 2) + 8 * j;
        int64_t t = m + (r < n_rows ? r : 0);
        if (p.rows) t = p.rows[t];
        x[j] = q + (t >= 0 && t < p.T ? t : 0) * int64_t(p.K) + at;
    }
    if (threadIdx.x < n_rows) {
        int64_t t = m + threadIdx.x;
        if (p.rows) t = p.rows[t];
        const bool bad = t < 0 || t >= p.T;
        if (bad) atomicCAS(p.status, 0, kI8StatusBadRows);
        xs[threadIdx.x] = bad ? 0.0f : p.xs[t];
    }
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.0f;
    for (int s = warp; s < steps; s += kWarps) {
        const int k = i8_warps_token(s, lane, p.K) - at;
        uint4 xv[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            if (8 * j < n_rows) xv[j] = *reinterpret_cast<const uint4 *>(x[j] + k);
        uint32_t a[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) widen16(wv[i], a[i]);
        load_w(s + kWarps);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            if (8 * j < n_rows) {
                uint32_t b[8];
                widen16(xv[j], b);
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        mma_m16n8k16(acc[i][j], a[2 * i][2 * h], a[2 * i + 1][2 * h], a[2 * i][2 * h + 1],
                                     a[2 * i + 1][2 * h + 1], b[2 * h], b[2 * h + 1]);
            }
    }
    // lane: channels lane / 4 (+ 8) of each 16, rows 2 (lane % 4) + 0, 1 of each 8
    float *mine = sums + warp * (R * kPad);
#pragma unroll
    for (int j = 0; j < NT; ++j)
        if (8 * j < n_rows)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mine[(8 * j + 2 * (lane & 3) + (k & 1)) * kPad + 16 * i + (lane >> 2) + 8 * (k >> 1)] = acc[i][j][k];
    __syncthreads();
    const int c = threadIdx.x % kChannels, n = n0 + c;
    if (n >= p.N) return;
    const float ws = p.ws[int64_t(e) * p.N + n];
    for (int r = threadIdx.x / kChannels; r < n_rows; r += kThreads / kChannels) {
        float s = sums[r * kPad + c];
#pragma unroll
        for (int v = 1; v < kWarps; ++v) s += sums[v * (R * kPad) + r * kPad + c];
        const float y = s * ws * xs[r];
        const int64_t to = (m + r) * int64_t(p.N) + n;
        if (p.out_f32) static_cast<float *>(p.Y)[to] = y;
        else static_cast<uint16_t *>(p.Y)[to] = uint16_t(pack_bf16x2(y, 0.0f) & 0xffffu);
    }
}

int channel_blocks(int32_t N) { return (N + kChannels - 1) / kChannels; }

template <int NT>
cudaError_t launch(const I8Params &p, const int8_t *q, bool pdl, cudaStream_t stream)
{
    auto kern = i8_warps_kernel<NT>;
    constexpr size_t smem = size_t(kWarps) * 8 * NT * kPad * sizeof(float);
    static_assert(smem <= 48 * 1024, "no opt-in needed");
    const int blocks_n = channel_blocks(p.N);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(unsigned(i8_warps_blocks(p)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kern, p, q, blocks_n);
}

}  // namespace

int64_t i8_warps_blocks(const I8Params &p) { return p.M * channel_blocks(p.N); }

cudaError_t launch_i8_warps(const I8Params &p, const int8_t *q, int rows, bool pdl, cudaStream_t stream)
{
    return rows == 16 ? launch<2>(p, q, pdl, stream) : launch<4>(p, q, pdl, stream);
}

}  // namespace cakegg
