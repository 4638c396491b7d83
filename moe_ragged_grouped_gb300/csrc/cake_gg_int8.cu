// cake_gg_int8.cu -- C entry points of the 8-bit integer products, and the
// kernel that quantises tokens row by row.
//
//   h[t, k] = x[t, k], or silu(g) * u of x[t] = [g | u]
//   a[t] = max_k |h[t, k]|     s[t] = a / 127     q[t, k] = rint(h[t, k] * (127 / a))
//   Y[m, n] = (sum_k q[r(m), k] W[e(m), n, k]) * ws[e(m), n] * s[r(m)]
//
// A call is one launch when its rows are few and X is 8-bit, or activations that
// the product's blocks quantise themselves.  Else it is two: the token pass below
// writes the integers of the tokens (for the tensor cores as FP16) and their
// scales to the workspace, and the product reads them.  A long call without
// routed rows may be two of each (choose_first).
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cake_gg_int8.h"
#include "cake_gg_int8_quant.cuh"
#include "cake_gg_int8_widen.cuh"
#include "cake_gg_ptx.cuh"

using namespace cakegg;

namespace {

constexpr uint64_t kHeader = 256;              // status word at byte 0
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kStagesMost = 12, kSlotsMost = 8;
constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxK = (1 << 17) - 16;      // |sum of K products| <= 2^14 K stays below 2^31
constexpr int32_t kMaxN = INT32_MAX - 511;     // channels of whole tiles (256) and storing warps stay below 2^31

uint64_t align_up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }

bool mul_ok(uint64_t a, uint64_t b, uint64_t *out)
{
    if (a != 0 && b > UINT64_MAX / a) return false;
    *out = a * b;
    return true;
}

bool pdl_enabled()
{
    const char *v = std::getenv("CAKE_GG_PDL");
    return !(v && std::atoi(v) == 0);
}

// Workspace: header | token scales [T] (activations only) | the tokens as the
// path reads them: FP16 integers [T, K] for the tensor cores, 8-bit ones for
// the few-row path (activations only).
struct Layout {
    uint64_t scales, tokens, total;
};

Layout layout(const cake_gg_i8_plan_t &pl)
{
    Layout L;
    const bool ready = pl.x_dtype == CAKE_GG_INT8;
    const uint64_t size = pl.path == CAKE_GG_I8_MMA ? 2 : ready ? 0 : 1;
    L.scales = kHeader;
    L.tokens = L.scales + (ready ? 0 : align_up(uint64_t(pl.T) * 4, 256));
    L.total = L.tokens + align_up(uint64_t(pl.T) * uint64_t(pl.K) * size, 256);
    return L;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------- token pass

__device__ __forceinline__ void store8(int8_t *out, const float (&v)[8], const RowScale &s)
{
    *reinterpret_cast<uint2 *>(out) = bytes8(v, s);
}
__device__ __forceinline__ void store8(__half *out, const float (&v)[8], const RowScale &s)
{
    *reinterpret_cast<uint4 *>(out) = halves8(v, s);
}

// Both kernels of the pass may run `beside` a product of other rows.  They then
// read what was there before the call and write rows that nobody else touches, so
// they wait for that product only at their end, in one block: their completion
// implies the product's, and with it everything before in the stream.

// blockDim.x threads per row.  The first kHeld vectors of 8 values that a thread owns
// stay in registers between the maximum and the rounding; longer rows read the
// rest again (from L2).  FP32 is bound by HBM (to bytes 16384 x 4096: 52 us, 6.5 TB/s
// read and written; to FP16 3001 x 5120: 16.5 us, 5.6), BF16 by its instructions and
// the latency of its loads (16384 x 4096: 41 us, 4.9 TB/s, 0.69 of the issue slots) and
// by how many rows are resident, so registers are held
// down as far as that pays (to bytes, BF16 16384 x 4096: 55 us with 50 registers, 41
// with 32; FP32 51, 49 with 48, 69 with 32, but to FP16 3001 x 5120 the 48 lose 1 us;
// gated BF16 92, 85 with 48); gated rows by the exponential and the division (some
// 30 instructions a value).  Two vectors a thread was best of 1, 2 and 4 (41 us; 58
// and 48).
constexpr int kHeld = 2;
constexpr int64_t kFewBlocks = 304;   // two rows a multiprocessor

template <typename XT, bool ACT, typename QT>
__global__ void __maxnreg__(ACT ? 48 : sizeof(XT) == 2 ? 32 : 64)
    i8_quant_kernel(const XT *__restrict__ X, int64_t T, int32_t K, QT *__restrict__ Q, float *__restrict__ S, bool beside)
{
    __shared__ uint32_t warp_max[32];
    if (!beside) grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const int n = t < T ? K : 0;                                 // values of this row
    const XT *row = X + t * (ACT ? 2 : 1) * int64_t(K);
    const int stride = int(blockDim.x) * 8;
    float held[kHeld][8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int k = int(threadIdx.x) * 8 + j * stride;
        if (k < n) {
            row8<XT, ACT>(row, K, k, held[j]);
            m = max_bits(held[j], m);
        }
    }
    for (int k = int(threadIdx.x) * 8 + kHeld * stride; k < n; k += stride) {
        float v[8];
        row8<XT, ACT>(row, K, k, v);
        m = max_bits(v, m);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const int warps = int(blockDim.x) / 32;
    if (warps > 1) {
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.y * warps + threadIdx.x / 32] = m;
        __syncthreads();
        m = int(threadIdx.x % 32) < warps ? warp_max[threadIdx.y * warps + threadIdx.x % 32] : 0;
        m = __reduce_max_sync(0xffffffffu, m);
    }
    const RowScale rs(m);
    if (threadIdx.x == 0 && n) S[t] = rs.scale;
    QT *out = Q + t * int64_t(K);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int k = int(threadIdx.x) * 8 + j * stride;
        if (k < n) store8(out + k, held[j], rs);
    }
    for (int k = int(threadIdx.x) * 8 + kHeld * stride; k < n; k += stride) {
        float v[8];
        row8<XT, ACT>(row, K, k, v);
        store8(out + k, v, rs);
    }
    if (beside && blockIdx.x == 0) grid_dependency_wait();
}

// 8-bit tokens as FP16 integers, 16 values a thread.
__global__ void __launch_bounds__(256) i8_expand_kernel(const int8_t *__restrict__ X, __half *__restrict__ Q, int64_t n16, bool beside)
{
    if (!beside) grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n16) return;
    const uint4 w = reinterpret_cast<const uint4 *>(X)[i];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint4 o;
        widen4(u[2 * h], o.x, o.y);
        widen4(u[2 * h + 1], o.z, o.w);
        *reinterpret_cast<uint4 *>(Q + i * 16 + h * 8) = o;
    }
    if (beside && blockIdx.x == 0) grid_dependency_wait();
}

// A kernel of the token pass: unless it runs beside a product, a programmatic dependent of the stream's
// previous kernel (it waits for it before it reads anything), and only then
// lets the product start, whose early reads of weights and offsets are thus
// ordered after everything before this call.
cudaLaunchConfig_t pass_config(int64_t blocks, int threads, cudaLaunchAttribute *attr, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.stream = stream;
    if (pdl_enabled()) {
        attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr->val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cfg;
}

template <typename XT, typename QT>
cudaError_t launch_quant_as(const void *X, int act, int64_t T, int32_t K, QT *Q, float *S, bool beside,
                            cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    // one vector a thread where rows are few and their latency counts, else kHeld
    const int held = T <= kFewBlocks ? 1 : kHeld;
    int threads = int(align_up((uint64_t(K) / 8 + held - 1) / held, 32));
    if (threads > 1024) threads = 1024;
    // many long rows: few threads each, so that several rows are resident and one's
    // loads run beside another's barrier (8192 x 16384 BF16: 92 us with 1024, 71 with
    // 256; but 4096 x 9216 FP32 31.7 with 576, 34.2)
    if (T > kFewBlocks && threads > 640) threads = 256;
    if (beside && threads > 256) threads = 256;   // (what fits beside the product)
    // short rows share a block of 256 threads: with a block of one or two warps each
    // the launching of blocks is the bound (12000 x 272: 13.0 us, 5.2; 12000 x 768: 12.9,
    // 9.0; 20000 x 1024: 21.4, 19.8, but gated 31.5, 33.6; gated 12000 x 512: 12.9, 10.0)
    const int rows = T > kFewBlocks && threads <= (act == CAKE_GG_ACT_NONE ? 64 : 32) ? 256 / threads : 1;
    cudaLaunchConfig_t cfg = pass_config((T + rows - 1) / rows, threads, &attr, stream);
    cfg.blockDim.y = unsigned(rows);
    const XT *x = static_cast<const XT *>(X);
    return act == CAKE_GG_ACT_SILU_MUL ? cudaLaunchKernelEx(&cfg, i8_quant_kernel<XT, true, QT>, x, T, K, Q, S, beside)
                                       : cudaLaunchKernelEx(&cfg, i8_quant_kernel<XT, false, QT>, x, T, K, Q, S, beside);
}

template <typename QT>
int launch_quant(const void *X, int x_dtype, int act, int64_t T, int32_t K, QT *Q, float *S, bool beside,
                 cudaStream_t stream)
{
    const cudaError_t err = x_dtype == CAKE_GG_BF16 ? launch_quant_as<uint16_t>(X, act, T, K, Q, S, beside, stream)
                                                    : launch_quant_as<float>(X, act, T, K, Q, S, beside, stream);
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

int64_t expand_blocks(int64_t T, int32_t K) { return (T * (K / 16) + 255) / 256; }

int launch_expand(const void *X, int64_t T, int32_t K, __half *Q, bool beside, cudaStream_t stream)
{
    const int64_t n16 = T * (K / 16);
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pass_config(expand_blocks(T, K), 256, &attr, stream);
    return cudaLaunchKernelEx(&cfg, i8_expand_kernel, static_cast<const int8_t *>(X), Q, n16, beside) == cudaSuccess
               ? CAKE_GG_OK
               : CAKE_GG_ERR_CUDA;
}

// The problem's own checks, shared by the plan and the call.
int check_problem(int32_t E, int64_t M_max, int64_t T, int32_t N, int32_t K, int x_dtype, int act, int out_dtype)
{
    if (E < 1 || E > kMaxExperts || M_max < 0 || M_max > INT32_MAX || T < 0 || T > INT32_MAX || N < 1 || K < 1 ||
        (M_max > 0 && T < 1))
        return CAKE_GG_ERR_INVALID_ARG;
    if (x_dtype != CAKE_GG_BF16 && x_dtype != CAKE_GG_FP32 && x_dtype != CAKE_GG_INT8) return CAKE_GG_ERR_UNSUPPORTED;
    if (out_dtype != CAKE_GG_BF16 && out_dtype != CAKE_GG_FP32) return CAKE_GG_ERR_UNSUPPORTED;
    if (act != CAKE_GG_ACT_NONE && act != CAKE_GG_ACT_SILU_MUL) return CAKE_GG_ERR_INVALID_ARG;
    if (act != CAKE_GG_ACT_NONE && x_dtype == CAKE_GG_INT8) return CAKE_GG_ERR_INVALID_ARG;
    if (N % 8 != 0 || K % 16 != 0) return CAKE_GG_ERR_ALIGNMENT;
    if (K > kMaxK || N > kMaxN) return CAKE_GG_ERR_OVERFLOW;
    uint64_t t;
    if (!mul_ok(uint64_t(T), uint64_t(K) * 8u, &t) || !mul_ok(uint64_t(E) * uint64_t(N), uint64_t(K), &t) ||
        !mul_ok(uint64_t(M_max), uint64_t(N) * 4u, &t))
        return CAKE_GG_ERR_OVERFLOW;
    return CAKE_GG_OK;
}

int env_int(const char *name, int dflt)
{
    const char *v = std::getenv(name);
    return v && *v ? std::atoi(v) : dflt;
}

// Tensor memory (512 columns of a CTA) left beside the two accumulators, in slots
// of 64 columns, and the ring depth that fits beside the rest of shared memory.
int slots_for(int nt)
{
    const int n = (512 - 2 * nt) / 64;
    return n > kSlotsMost ? kSlotsMost : n;
}

// Widened tiles that may be ahead of the MMAs.  The converter groups take alternate
// stages, so with an odd ring a group meets a stage's barrier every second round
// only and must not come there before the round between is over, or the
// barrier's parity would deceive it: it waits for the MMAs of the stage `slots`
// before its last, which have to be of that round or later.  (An even ring gives
// a group the same stages every round.)
int slots_most(int stages) { return stages % 2 == 0 ? stages : stages - 2; }

int stages_for(int pair, int nt, int splits, int E)
{
    int s = kStagesMost;
    while (s > 2 && i8_mma_smem(pair, nt, s, splits, E) > kI8SmemLimit) --s;
    return s;
}

// Which kernels: by the rows M and the weights that they meet.
//  - Rows that meet mostly experts of their own (at most two of an expert), up to
//    8 or up to 512 MB of weights: integer dot products (16 rows in 32 experts 4096 ->
//    1000: 12.3 us, 21.4 from warps' registers, 19.0 on the tensor cores; 64 rows
//    in 64, 3056 -> 2048: 51, 75, 54; 128 rows in 128, 562 MB: 74, 126, 75, 764 MB: 96,
//    145, 90).
//  - One or two rows, three or four of 2048 and longer, and up to 16 long ones
//    of few channels: the same (4 x 4096 -> 6144: 7.1, 10.6, 17.6; but 4 x 1024 ->
//    5120: 4.7, 4.0, 7.1; 6 x 8192 -> 256: 4.8, 11.3, 9.2; 12 x 4096 -> 256: 5.1, 7.7, 8.1).
//  - Up to 16 rows up to 4608 long over at most 16 MB, up to 32 up to 3200 long of
//    2048 channels: warps' registers, which start at once (16 x 2048 -> 4096: 6.6 us,
//    8.7 on the tensor cores; 32 x 2816 -> 1024: 8.0, 8.2; 24 x 1024 -> 2048: 4.7, 7.3;
//    but 16 x 8192 -> 1024: 15.8, 9.6; 32 x 1024 -> 4096: 9.5, 7.3).
//  - Else the tensor cores.
int choose_path(const cake_gg_i8_plan_t &pl)
{
    const int64_t M = pl.M_max, channels = (M < pl.E ? M : pl.E) * int64_t(pl.N), weights = channels * pl.K;
    const bool spread = i8_run_rows(pl.E, M, pl.T) <= 2;
    if ((spread && (M <= 8 || weights <= (512 << 20))) || (M <= 4 && (pl.K >= 2048 || weights > (16 << 20))) ||
        (pl.E == 1 && M <= 16 && pl.K > 2560 && M * pl.N <= 8192))
        return CAKE_GG_I8_ROWS;
    if ((M <= 16 && weights <= (16 << 20) && pl.K <= 4608) || (M <= 32 && channels <= 2048 && pl.K <= 3200))
        return CAKE_GG_I8_WARPS;
    return CAKE_GG_I8_MMA;
}

// Row tiles of nt rows that the call will have: exact for one expert; where E
// share the rows, whole tiles and half a tile more for each expert that can have
// rows, at least one each (the sizes are the device's).
int64_t row_tiles(const cake_gg_i8_plan_t &pl, int nt)
{
    const int64_t whole = (pl.M_max + nt - 1) / nt;
    if (pl.E == 1) return whole;
    const int64_t busy = pl.M_max < pl.E ? pl.M_max : pl.E;
    return whole + busy / 2 > busy ? whole + busy / 2 : busy;
}

constexpr int kSms = 152;
// Multiprocessors that clusters of `splits` CTAs can hold at once: a cluster lies
// within one of the GPU's groups of them, whose sizes differ from part to part.
// Here 152, 138, 144, 140, 138, 105, 120 for 2 .. 8; a call of one cluster more
// takes a second wave (374 x 3328 -> 1000 as 48 clusters of three 21.3 us, 15
// undivided).
int cluster_sms(int splits) { return splits <= 2 ? kSms : splits <= 6 ? 132 : 104; }
int64_t stage_ns(int pair, int nt) { return pair == 2 ? 250 + nt * 7 / 6 : 280 + nt * 11 / 10; }

// Rows of a first product, beside which the token pass prepares the others: its
// blocks live on the registers and threads that a product CTA leaves (a product
// is bound by the tensor cores, the pass by HBM and its arithmetic).  The pass
// runs there at some 0.4 of its own speed, so the first product should take 2.5
// times as long as the rest of the pass: that share f of the rows, for one
// expert cut where a wave of units ends.  Worth it where the pass hidden, of
// which about half is won (the power limit takes the rest), is more than a
// wave that the cut adds and the start of two more kernels.  Measured in turn, one
// call after another, so under the power limit: 16384 x 4096 -> 4096 from 8-bit
// tokens 333 us undivided, 317, 316, 329 with f = 0.12, 0.22, 0.28 (by itself, a few
// calls at a time, 315 and 297 with 0.22); gated 32768 x 2048 -> 6144 over 32
// experts 564, 567, 557, 551, 543 with f = 0, 0.12, 0.24, 0.37, 0.49.  8-bit tokens
// gain 4 to 9 % (32768 x 4096 -> 2048: 359 to 329; 16384 x 8192 -> 1024: 228 to 208),
// gated ones 2.5 % (16384 x 4096 -> 4096: 379 to 370).  BF16 that is not gated gains up
// to 2 % over long reductions (16384 x 8192 -> 8192: 1308 to 1280) and loses as much over
// short ones (16384 x 5120 -> 1000: 162 to 165), and FP32 loses 1 to 3 % (16384 x 4096 ->
// 4096: 334 to 341; 5 % into 1000 channels): there the pass takes from HBM and L2 what
// the product needs.
int choose_first(const cake_gg_i8_plan_t &pl)
{
    const int nt = pl.tile_rows;
    const int64_t workers = kSms / pl.pair, n_ct = (pl.N + 128 * pl.pair - 1) / (128 * pl.pair);
    const int64_t wave = (pl.K + 127) / 128 * stage_ns(pl.pair, nt), tiles = row_tiles(pl, nt);
    auto waves = [&](int64_t t) { return (t * n_ct + workers - 1) / workers; };
    // nanoseconds of the whole token pass: bytes at 5.8 TB/s, gated values 1.37 ps each
    const double values = double(pl.M_max) * pl.K;
    const double pass = pl.act != CAKE_GG_ACT_NONE ? values * 1.37e-3
                                                   : values * (pl.x_dtype == CAKE_GG_INT8 ? 3 : pl.x_dtype == CAKE_GG_BF16 ? 4 : 6) / 5800.0;
    const double product = double(waves(tiles) * wave), f = 2.5 * pass / (product + 2.5 * pass);
    int64_t t = int64_t(f * double(tiles)), extra = wave / 2;
    if (pl.E == 1) {
        t = (int64_t(f * double(tiles * n_ct)) / workers) * workers / n_ct;
        extra = (waves(t) + waves(tiles - t) - waves(tiles)) * wave;
    }
    const int64_t rows = pl.E == 1 ? t * nt : int64_t(f * double(pl.M_max));
    if (t < 1 || rows >= pl.M_max || pass * (1 - f) / 2 < double(extra) + 8000) return 0;
    return int(rows);
}

// Shape of the tensor-core path, from a model of its time in nanoseconds: waves
// of units over the multiprocessors (152, or 76 pairs), the stages of a unit,
// the storing of the last one, and the exchange between the CTAs that share a
// tile (33 x 4608 -> 496 over 1, 2, 3, 4, 6, 8 CTAs, 32 rows a tile: 16.3, 12.9, 11.4, 10.5,
// 10.2, 9.7 us; 247 x 4528 -> 304, 64 rows: 17.9, 15.1, 12.8, 12.0, 12.9, 12.6).  The
// times of a stage, with all multiprocessors at work (12288 x 4096 -> 4096), are for
// pairs 325, 362, 362, 419, 454 ns for 64, 96, 128, 160, 192 rows, for single CTAs
// 327, 348, 383, 435 ns for 32, 64, 96, 128; the lines that stand for them above are
// within 5 % of that but for pairs of 128 rows (10 % above).  What the model decides,
// measured with the neighbours: 3001 x 5120 -> 1000 takes 160 rows (40.4 us; 40.8 with
// 192, 50.6 with 128), 701 tokens through 2 of 8 experts 4096 -> 2048 take 96 (32.4;
// 34.1 with 128, 35.8 with 192), 200 x 4096 -> 4096 take 64 (17.7; 21.7 with pairs of
// 192), 33 x 4096 -> 5120 divide the reduction by 3 (12.2; 16.0 undivided).
void choose_mma(cake_gg_i8_plan_t *pl)
{
    const int64_t n_kb = (pl->K + 127) / 128;
    int64_t best = -1;
    auto consider = [&](int pair, int nt, int splits) {
        const int64_t units = row_tiles(*pl, nt) * ((pl->N + 128 * pair - 1) / (128 * pair));
        if (splits > 1 && (units * splits > cluster_sms(splits) || n_kb < 2 * splits)) return;
        const int64_t waves = (units * pair + kSms - 1) / kSms;
        const int64_t ns = waves * ((n_kb + splits - 1) / splits) * stage_ns(pair, nt) + 16 * nt + (splits > 1 ? 300 + nt * (45 + 4 * splits) : 0);
        if (best < 0 || ns < best) {
            best = ns;
            pl->pair = pair;
            pl->tile_rows = nt;
            pl->splits = splits;
        }
    };
    for (int nt = 192; nt >= 64; nt -= 32) consider(2, nt, 1);
    for (int nt = 128; nt >= 32; nt -= 32)
        for (int s = 1; s <= (nt <= 64 ? 8 : 1); ++s) consider(1, nt, s);
    pl->pair = env_int("CAKE_GG_I8_PAIR", pl->pair) == 2 ? 2 : 1;
    const int nt = env_int("CAKE_GG_I8_ROWS_PER_TILE", pl->tile_rows);
    if (nt >= 32 && nt <= 192 && nt % 32 == 0) pl->tile_rows = nt;
    const int sp = env_int("CAKE_GG_I8_SPLITS", pl->splits);
    pl->splits = sp >= 1 && sp <= 8 && pl->pair == 1 ? sp : 1;
    pl->stages = stages_for(pl->pair, pl->tile_rows, pl->splits, pl->E);
    if (pl->stages == 3) pl->stages = 2;
    pl->slots = slots_for(pl->tile_rows);
    const int most = slots_most(pl->stages);
    if (pl->slots > most) pl->slots = most;
    const int first = env_int("CAKE_GG_I8_FIRST_ROWS", -1);
    pl->first_rows = pl->splits > 1 ? 0 : first < 0 ? choose_first(*pl) : first < pl->M_max ? first : 0;
}

bool path_ok(int path) { return path == CAKE_GG_I8_ROWS || path == CAKE_GG_I8_MMA || path == CAKE_GG_I8_WARPS; }
bool warps_rows_ok(int rows) { return rows == 16 || rows == 32; }

// What the tensor-core kernel can run.
bool mma_plan_ok(const cake_gg_i8_plan_t &pl)
{
    return (pl.pair == 1 || pl.pair == 2) && pl.tile_rows >= 32 && pl.tile_rows <= (pl.pair == 2 ? 192 : 128) &&
           pl.tile_rows % 32 == 0 && pl.stages >= 2 && pl.stages <= kStagesMost && pl.slots >= 2 &&
           pl.slots <= slots_most(pl.stages) && pl.slots <= slots_for(pl.tile_rows) && pl.splits >= 1 && pl.splits <= 8 &&
           pl.first_rows >= 0 && (pl.first_rows == 0 || (pl.first_rows < pl.M_max && pl.splits == 1)) &&
           (pl.splits == 1 || pl.pair == 1) && pl.splits <= (pl.K + 127) / 128 &&   // (a stage for every CTA)
           i8_mma_smem(pl.pair, pl.tile_rows, pl.stages, pl.splits, pl.E) <= kI8SmemLimit;
}

}  // namespace

extern "C" {

int cake_gg_i8_plan(cake_gg_i8_plan_t *plan, int32_t E, int64_t M_max, int64_t T, int32_t N, int32_t K,
                    int x_dtype, int act, int out_dtype, int32_t max_sms)
{
    if (!plan) return CAKE_GG_ERR_INVALID_ARG;
    std::memset(plan, 0, sizeof(*plan));
    if (max_sms < 0) return CAKE_GG_ERR_INVALID_ARG;
    const int rc = check_problem(E, M_max, T, N, K, x_dtype, act, out_dtype);
    if (rc != CAKE_GG_OK) return rc;
    plan->abi_version = CAKE_GG_ABI_VERSION;
    plan->E = E;
    plan->M_max = M_max;
    plan->T = T;
    plan->N = N;
    plan->K = K;
    plan->x_dtype = x_dtype;
    plan->act = act;
    plan->out_dtype = out_dtype;
    plan->max_sms = max_sms;
    // (overrides that name no path, or no run of the path's, change nothing)
    const int path = env_int("CAKE_GG_I8_PATH", -1);
    plan->path = path_ok(path) ? path : choose_path(*plan);
    if (plan->path == CAKE_GG_I8_MMA) {
        choose_mma(plan);
        if (!mma_plan_ok(*plan)) return CAKE_GG_ERR_INVALID_ARG;   // (an override that does not fit)
    }
    if (plan->path == CAKE_GG_I8_WARPS) {
        const int rows = env_int("CAKE_GG_I8_ROWS_PER_TILE", 0);
        plan->tile_rows = warps_rows_ok(rows) ? rows : M_max <= 16 ? 16 : 32;
    }
    plan->timeout_ns = kTimeoutNs;
    plan->workspace_bytes = layout(*plan).total;
    return CAKE_GG_OK;
}

int cake_gg_i8_quant(const void *X, int x_dtype, int act, int64_t T, int32_t K, int8_t *Xq, float *xs, void *stream)
{
    if (x_dtype != CAKE_GG_BF16 && x_dtype != CAKE_GG_FP32) return CAKE_GG_ERR_UNSUPPORTED;
    const int rc = check_problem(1, 0, T, 8, K, x_dtype, act, CAKE_GG_BF16);
    if (rc != CAKE_GG_OK) return rc;
    if (T == 0) return CAKE_GG_OK;
    if (!X || !Xq || !xs) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(Xq, 16) || !aligned(xs, 4)) return CAKE_GG_ERR_ALIGNMENT;
    int sms;
    const int dev = device_sms(&sms);
    if (dev != CAKE_GG_OK) return dev;
    return launch_quant(X, x_dtype, act, T, K, Xq, xs, false, static_cast<cudaStream_t>(stream));
}

int cake_gg_i8_gemm(const cake_gg_i8_plan_t *plan, const void *X, const float *xs, const int32_t *rows,
                    const int8_t *W, const float *ws, void *Y, const int32_t *offsets, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    if (!plan || plan->abi_version != CAKE_GG_ABI_VERSION) return CAKE_GG_ERR_INVALID_ARG;
    const cake_gg_i8_plan_t &pl = *plan;
    int rc = check_problem(pl.E, pl.M_max, pl.T, pl.N, pl.K, pl.x_dtype, pl.act, pl.out_dtype);
    if (rc != CAKE_GG_OK) return rc;
    const bool warps = pl.path == CAKE_GG_I8_WARPS;
    if (pl.max_sms < 0 || !path_ok(pl.path) || (pl.path == CAKE_GG_I8_MMA && !mma_plan_ok(pl)) ||
        (warps && !warps_rows_ok(pl.tile_rows)))
        return CAKE_GG_ERR_INVALID_ARG;
    const bool ready = pl.x_dtype == CAKE_GG_INT8;   // tokens come quantised
    if (!workspace || !W || !ws || (pl.M_max > 0 && (!X || !Y || (ready && !xs))) || (!ready && xs))
        return CAKE_GG_ERR_INVALID_ARG;
    if ((!offsets && pl.E != 1) || (!rows && pl.T != pl.M_max)) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(workspace, 16) || !aligned(xs, 4) ||
        !aligned(ws, 4) || !aligned(rows, 4) || !aligned(offsets, 4))
        return CAKE_GG_ERR_ALIGNMENT;
    const Layout L = layout(pl);
    if (workspace_bytes < L.total || pl.workspace_bytes != L.total) return CAKE_GG_ERR_WORKSPACE;
    int sms;
    if ((rc = device_sms(&sms)) != CAKE_GG_OK) return rc;
    if (pl.M_max == 0) return CAKE_GG_OK;

    uint8_t *base = static_cast<uint8_t *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    I8Params p{};
    p.offsets = offsets;
    p.rows = rows;
    p.W = W;
    p.ws = ws;
    p.xs = xs;
    p.Y = Y;
    p.status = reinterpret_cast<int32_t *>(base);
    p.M = pl.M_max;
    p.T = pl.T;
    p.E = pl.E;
    p.N = pl.N;
    p.K = pl.K;
    p.out_f32 = pl.out_dtype == CAKE_GG_FP32;
    p.timeout_ns = pl.timeout_ns ? pl.timeout_ns : kTimeoutNs;
    const bool mma = pl.path == CAKE_GG_I8_MMA, pdl = pdl_enabled();
    auto status = [](cudaError_t err) { return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA; };
    // what cannot be launched is refused before anything is enqueued
    if ((warps ? i8_warps_blocks(p) : pl.path == CAKE_GG_I8_ROWS ? i8_rows_blocks(p) : ready ? expand_blocks(pl.T, pl.K) : 0) >
        INT32_MAX)
        return CAKE_GG_ERR_OVERFLOW;
    if (warps && ready)
        return status(launch_i8_warps(p, static_cast<const int8_t *>(X), pl.tile_rows, pdl, s));
    if (pl.path == CAKE_GG_I8_ROWS && (ready || i8_rows_fused(p, pl.act)))
        return status(launch_i8_rows(p, X, pl.x_dtype, pl.act, pdl, s));

    // the token pass, then the product
    void *tokens = base + L.tokens;
    float *scales = reinterpret_cast<float *>(base + L.scales);
    if (!ready) p.xs = scales;
    auto pass = [&](int64_t t0, int64_t n, bool beside) {
        __half *q = static_cast<__half *>(tokens) + t0 * pl.K;
        if (ready) return launch_expand(static_cast<const int8_t *>(X) + t0 * pl.K, n, pl.K, q, beside, s);
        const int64_t row = int64_t(pl.K) * (pl.act == CAKE_GG_ACT_NONE ? 1 : 2) * (pl.x_dtype == CAKE_GG_BF16 ? 2 : 4);
        const uint8_t *x = static_cast<const uint8_t *>(X) + t0 * row;
        return mma ? launch_quant(x, pl.x_dtype, pl.act, n, pl.K, q, scales + t0, beside, s)
                   : launch_quant(x, pl.x_dtype, pl.act, n, pl.K, static_cast<int8_t *>(tokens), scales, false, s);
    };
    p.early = 1;
    const int64_t first = mma && !rows && pdl ? pl.first_rows : 0;
    I8MmaLaunch products[2];
    if (mma) {
        I8MmaParams m{};
        m.b = p;
        m.nt = pl.tile_rows;
        m.stages = pl.stages;
        m.slots = pl.slots;
        m.splits = pl.splits;
        m.debug_flags = pl.debug_flags;
        const uint16_t *q = static_cast<const uint16_t *>(tokens);
        const int cap = pl.max_sms > 0 && pl.max_sms < sms ? pl.max_sms : sms;
        m.b.m_hi = first;
        if (first && (rc = prepare_i8_mma(&products[0], m, q, pl.pair, cap)) != CAKE_GG_OK) return rc;
        m.b.m_lo = first;
        m.b.m_hi = pl.M_max;
        if ((rc = prepare_i8_mma(&products[1], m, q, pl.pair, cap)) != CAKE_GG_OK) return rc;
    }
    if ((rc = pass(0, first ? first : pl.T, false)) != CAKE_GG_OK) return rc;
    if (warps) return status(launch_i8_warps(p, static_cast<const int8_t *>(tokens), pl.tile_rows, pdl, s));
    if (!mma) return status(launch_i8_rows(p, tokens, CAKE_GG_INT8, CAKE_GG_ACT_NONE, pdl, s));
    if (first) {
        if ((rc = launch_i8_mma(products[0], pdl, s)) != CAKE_GG_OK) return rc;
        if ((rc = pass(first, pl.T - first, true)) != CAKE_GG_OK) return rc;
    }
    return launch_i8_mma(products[1], pdl, s);
}

}  // extern "C"
