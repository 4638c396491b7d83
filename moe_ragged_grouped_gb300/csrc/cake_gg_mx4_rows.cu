// cake_gg_mx4_rows.cu -- the 4-bit products of a few rows: integer dot products.
//
//   Y[m, n] = sum_b 2^(sx - 127 - 1) 2^(sw - 127 - 1) sum_{k in block b} (2 x_k) (2 w_k)
//
// Twice a 4-bit value is a whole number up to 12, and the sum over a block of 32
// is exact in 32-bit integers (dp4a); the blocks' sums are added in FP32.  Eight
// codes become eight bytes of magnitudes by two byte permutes, whose selectors are
// the codes themselves; signs come the same way (a permute's selector has a bit
// that spreads a byte's sign), and with n the magnitudes of the negative ones the sum
// is m x - 2 n x: 13 instructions for 8 products.
//
// A block has up to R rows of one expert and 32 channels: a warp the channels c, c +
// 32, c + 64, c + 96 of a tile of 128, whose scales lie side by side.  A lane takes one
// block of 32 values at a time, 16 bytes of each channel, so a warp reads 512 bytes of
// each at once, the next while it multiplies.  The rows are bytes in shared memory,
// which the block makes of codes, or of activations that it quantises itself (gated ones
// come quantised: they are 64-bit work for some blocks).
//
// 4096 x 4096, one row: 4.9 us of codes, 5.3 of BF16 (1.7 TB/s; the tensor cores 7.6 and
// 8.0), of which a kernel that does nothing takes some 2; past that the instructions
// above bind, which run at half rate: 4 million weights a microsecond.  Runs of 1 row keep three
// blocks on a multiprocessor (4 of 32 experts 2880 -> 2880 8.9 us, with two 10.0).
#include "cake_gg_mx4.h"
#include "cake_gg_mx4_quant.cuh"
#include "cake_gg_ptx.cuh"
#include "cake_gg_shared_limit.h"

namespace cakegg {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kLow = 0x03020100u, kHigh = 0x0c080604u;   // twice the magnitudes of codes 0 .. 3, 4 .. 7
constexpr uint32_t kSigns = 0x80808080u;

// Magnitudes (doubled) of the low four codes of w, and 0xff or 0x80 for their signs.
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return __byte_perm(kLow, kHigh, w & 0x7777u); }
__device__ __forceinline__ uint32_t signs(uint32_t w)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(kSigns), "r"(w));
    return r;
}
// The low four codes of w as signed bytes.
__device__ __forceinline__ uint32_t signed_bytes(uint32_t w)
{
    const uint32_t m = magnitudes(w), s = __vcmpeq4(signs(w), 0xffffffffu);
    return __vsub4(m ^ s, s);
}

// A block's sum by its scales' bytes: of both exponents a half at a time, so that no
// product on the way leaves FP32's range unless the result does (four times the sum
// is given; two bytes whose sum is below 2 leave nothing that FP32 holds).
__device__ __forceinline__ float scaled_add(int32_t four, uint32_t sw, uint32_t sx, float to)
{
    const uint32_t both = max(sw + sx, 2u) - 2u, half = both >> 1;
    const float v = max(sw, sx) == 255u ? __uint_as_float(0x7fc00000u) : float(four);
    return fmaf(v * __uint_as_float(half << 23), __uint_as_float((both - half) << 23), to);
}

// XT: uint8_t for codes with scales in tiles, else activations.
template <int R, typename XT>
__global__ void __launch_bounds__(kThreads, R == 1 ? 3 : 2)
    mx4_rows_kernel(const Mx4Params p, const XT *__restrict__ X, const uint8_t *__restrict__ W, const uint8_t *__restrict__ ws)
{
    extern __shared__ __align__(16) uint8_t shared[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t K = p.K, blocks = K / 32, kt_all = (K + 127) / 128;
    uint8_t *bytes = shared;                                     // [R][K]
    uint8_t *sx = shared + size_t(R) * K;                        // [R][blocks]
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();
    // ---- the run of rows that is blockIdx.y's, the same in every warp ----
    int32_t e = -1, m0 = 0, rows = 0, before = 0;
    bool bad = false;
    const int32_t run = int32_t(blockIdx.y);
    for (int32_t base = 0; base < p.E; base += 32) {
        const int32_t i = base + lane;
        int32_t a = 0, b = 0;
        if (i < p.E) {
            a = p.offsets ? p.offsets[i] : 0;
            b = p.offsets ? p.offsets[i + 1] : int32_t(p.M);
            bad |= (i == 0 && a != 0) || b < a || int64_t(b) > p.M;
        }
        const int32_t n = (b - a + R - 1) / R;
        int32_t inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const int32_t first = before + inc - n;
        const unsigned has = __ballot_sync(0xffffffffu, n > 0 && run >= first && run < first + n);
        if (has) {
            const int at = __ffs(int(has)) - 1;
            e = base + at;
            m0 = __shfl_sync(0xffffffffu, a + (run - first) * R, at);
            rows = min(R, __shfl_sync(0xffffffffu, b, at) - m0);
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (__any_sync(0xffffffffu, bad)) {
        if (tid == 0) atomicCAS(p.status, 0, CAKE_GG_ERR_BAD_OFFSETS);
        e = -1;
    }
    if (e < 0) {
        grid_dependency_wait();
        return;
    }
    // ---- the first weights, while the rows are prepared ----
    const int32_t tile = int32_t(blockIdx.x) >> 2, c = (int32_t(blockIdx.x) & 3) * 8 + warp, n0 = tile * 128 + c;
    const int32_t tiles = (p.N + 127) / 128;
    const uint8_t *weights = W + (int64_t(e) * p.N + n0) * (K / 2) + lane * 16;
    const uint8_t *scales = ws + ((int64_t(e) * tiles + tile) * kt_all + (lane >> 2)) * kMx4Tile + c * 16;
    const int64_t apart = int64_t(32) * (K / 2);
    uint4 w[4], s;
    auto load = [&](int32_t b) {                                 // of block b of the reduction
        const bool in = b < blocks;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = in && n0 + 32 * i < p.N ? __ldcs(reinterpret_cast<const uint4 *>(weights + i * apart + int64_t(b - lane) * 16)) : make_uint4(0, 0, 0, 0);
        s = in ? __ldg(reinterpret_cast<const uint4 *>(scales + int64_t(b >> 5) * (8 * kMx4Tile))) : make_uint4(0, 0, 0, 0);
    };
    load(lane);
    // ---- the rows as bytes ----
    grid_dependency_wait();
    for (int r = 0; r < rows; ++r) {
        int64_t t = m0 + r;
        if (p.rows) t = p.rows[t];
        const bool lost = t < 0 || t >= p.T;
        if (lost && tid == 0) atomicCAS(p.status, 0, CAKE_GG_ERR_BAD_ROWS);
        if constexpr (sizeof(XT) == 1) {
            for (int32_t b = tid; b < blocks; b += kThreads) {
                const uint4 q = lost ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(X + t * (K / 2) + b * 16);
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
                uint4 *to = reinterpret_cast<uint4 *>(bytes + size_t(r) * K + b * 32);
                to[0] = make_uint4(signed_bytes(u[0]), signed_bytes(u[0] >> 16), signed_bytes(u[1]), signed_bytes(u[1] >> 16));
                to[1] = make_uint4(signed_bytes(u[2]), signed_bytes(u[2] >> 16), signed_bytes(u[3]), signed_bytes(u[3] >> 16));
                sx[r * blocks + b] = lost ? uint8_t(0) : p.xs[mx4_scale_at(t, b, kt_all)];
            }
        } else {
            // (every lane of a warp in each round: a block's four share its maximum)
            for (int32_t k0 = warp * 256; k0 < K; k0 += kThreads * 8) {
                const int32_t k = k0 + lane * 8;
                Raw<XT> raw;
                if (k < K && !lost) raw.load(X + t * K + k);
                else raw.zero();
                float v[8];
                raw.values(v);
                const uint32_t byte = scale_byte(block_max(largest8(v)));
                const uint32_t q = byte == 255 ? 0 : codes8(v, scale_inverse(byte));
                if (k < K) {
                    *reinterpret_cast<uint2 *>(bytes + size_t(r) * K + k) = make_uint2(signed_bytes(q), signed_bytes(q >> 16));
                    if ((lane & 3) == 0) sx[r * blocks + k / 32] = uint8_t(byte);
                }
            }
        }
    }
    __syncthreads();
    // ---- the products ----
    float sum[4][R] = {};
    for (int32_t b0 = 0; b0 < blocks; b0 += 32) {
        const int32_t b = b0 + lane;
        uint4 now[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) now[i] = w[i];
        const uint32_t sw[4] = {s.x, s.y, s.z, s.w};
        load(b + 32);
        if (b >= blocks) continue;
        uint32_t x[R][8];
        uint32_t f[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r < rows) {
                const uint4 *from = reinterpret_cast<const uint4 *>(bytes + size_t(r) * K + b * 32);
                const uint4 lo = from[0], hi = from[1];
                x[r][0] = lo.x, x[r][1] = lo.y, x[r][2] = lo.z, x[r][3] = lo.w;
                x[r][4] = hi.x, x[r][5] = hi.y, x[r][6] = hi.z, x[r][7] = hi.w;
                f[r] = sx[r * blocks + b];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[r][i] = 0;
                f[r] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
            int32_t all[R] = {}, negative[R] = {};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t code = h ? u[q] >> 16 : u[q], m = magnitudes(code), n = m & signs(code);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        all[r] = __dp4a(int32_t(m), int32_t(x[r][2 * q + h]), all[r]);
                        negative[r] = __dp4a(int32_t(n), int32_t(x[r][2 * q + h]), negative[r]);
                    }
                }
            const uint32_t by = sw[i] >> (8 * (b & 3)) & 255u;
#pragma unroll
            for (int r = 0; r < R; ++r) sum[i][r] = scaled_add(all[r] - 2 * negative[r], by, f[r], sum[i][r]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v = sum[i][r];
#pragma unroll
            for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            const int32_t n = n0 + 32 * i;
            if (lane == i && r < rows && n < p.N) {
                const int64_t at = (int64_t(m0) + r) * p.N + n;
                if (p.out_f32) static_cast<float *>(p.Y)[at] = v;
                else static_cast<uint16_t *>(p.Y)[at] = uint16_t(pack_bf16x2(v, 0.0f) & 0xffffu);
            }
        }
}

size_t rows_smem(int R, int32_t K) { return size_t(R) * K + size_t(R) * (K / 32); }

template <int R, typename XT>
cudaError_t launch(const Mx4Params &p, const void *X, const uint8_t *W, const uint8_t *ws, bool pdl, cudaStream_t stream)
{
    const cudaError_t err = raise_shared_limit<mx4_rows_kernel<R, XT>>(kMx4SmemLimit);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    if (pdl) {
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    cfg.gridDim = dim3(unsigned((p.N + 127) / 128 * 4), unsigned(mx4_runs(p.M, p.E)), 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = rows_smem(R, p.K);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, mx4_rows_kernel<R, XT>, p, static_cast<const XT *>(X), W, ws);
}

template <int R>
cudaError_t launch_as(const Mx4Params &p, const void *X, int x_dtype, const uint8_t *W, const uint8_t *ws, bool pdl, cudaStream_t stream)
{
    return x_dtype == CAKE_GG_MX4    ? launch<R, uint8_t>(p, X, W, ws, pdl, stream)
           : x_dtype == CAKE_GG_BF16 ? launch<R, uint16_t>(p, X, W, ws, pdl, stream)
                                     : launch<R, float>(p, X, W, ws, pdl, stream);
}

}  // namespace

bool mx4_rows_fit(int64_t M, int32_t E, int32_t K)
{
    return mx4_runs(M, E) <= 65535 && rows_smem(mx4_run_rows(M, E), K) <= kMx4SmemLimit;
}

cudaError_t launch_mx4_rows(const Mx4Params &p, const void *X, int x_dtype, const uint8_t *W, const uint8_t *ws, bool pdl,
                            cudaStream_t stream)
{
    return mx4_run_rows(p.M, p.E) == 1 ? launch_as<1>(p, X, x_dtype, W, ws, pdl, stream)
                                       : launch_as<2>(p, X, x_dtype, W, ws, pdl, stream);
}

}  // namespace cakegg
