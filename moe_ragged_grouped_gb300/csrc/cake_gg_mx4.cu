// cake_gg_mx4.cu -- C entry points of the 4-bit products, and the kernel that
// quantises rows.
//
//   h = x, or silu(g) * u of x = [g | u];  a block is 32 values of a row
//   e = max(floor(log2(max |h|)) - 2, -127),  scale 2^e,  code = E2M1 nearest to h / 2^e
//   Y[m, n] = sum_k x[r(m), k] w[e(m), n, k]
//
// A call is one launch when X comes quantised; else the token pass below writes
// the tokens' codes and scales to the workspace and the product reads them.
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include <cuda_runtime.h>

#include "cake_gg_mx4.h"
#include "cake_gg_mx4_quant.cuh"
#include "cake_gg_ptx.cuh"

using namespace cakegg;

namespace {

constexpr uint64_t kHeader = 256;              // status word at byte 0
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxK = (1 << 17) - 32;
constexpr int32_t kMaxN = INT32_MAX - 511;     // channels of whole tiles (256) and storing warps stay below 2^31
constexpr int kSms = 152;
constexpr int kStagesLeast = 3;

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

int env_int(const char *name, int dflt)
{
    const char *v = std::getenv(name);
    return v && *v ? std::atoi(v) : dflt;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

uint64_t scale_bytes(uint64_t rows, int32_t K) { return (rows + 127) / 128 * uint64_t((K + 127) / 128) * kMx4Tile; }

// Workspace: header | the tokens' scales | their codes (activations only) | the
// rows' scales as a pair takes them | their codes, where they are routed.
struct Layout {
    uint64_t scales, tokens, arranged, rows, total;
};
Layout layout(const cake_gg_mx4_plan_t &pl)
{
    Layout L;
    const uint64_t T = pl.x_dtype == CAKE_GG_MX4 ? 0 : uint64_t(pl.T);
    L.scales = kHeader;
    L.tokens = L.scales + scale_bytes(T, pl.K);
    L.arranged = L.tokens + align_up(T * uint64_t(pl.K) / 2, 256);
    L.rows = L.arranged;
    L.total = L.arranged;
    if (pl.pair == 2 && pl.path == CAKE_GG_MX4_MMA) {
        L.rows += uint64_t(mx4_slots(pl.M_max, pl.E, pl.tile_rows)) * uint64_t((pl.K + 127) / 128 * mx4_row_atoms(pl.tile_rows)) * kMx4Tile;
        // (whether a call routes is known with the call: T other than M_max says that it
        // does, and it may all the same)
        L.total = L.rows + align_up(uint64_t(pl.M_max) * uint64_t(pl.K) / 2, 256);
    }
    return L;
}

// ---------------------------------------------------------------- token pass

// silu(g) * u, three ways.  By approximate instructions, for g > -32: the product g
// log2(e) rounds to 2^-24 of itself and its constant is off by 2^-26, of which the
// exponential makes |g| (2^-24 + 2^-26.2) <= 32 (7.3 x 10^-8) = 2.3 x 10^-6; the
// instructions are off by 2^-22 (ex2) and 2^-23 (rcp); the sum, the product of the two
// sums, g u, the quotient and the result round to 2^-24 each, and so does the result in
// units of its scale: 3.1 x 10^-6 in all, below 2^-18 = 3.8 x 10^-6.  (Two values share a
// reciprocal: 1 / a = b / (a b).)  In FP32: two units in the last place of the exponential
// (2^-22), 2^-24 each of the sum, the quotient, the product and its scaling: 2^-21, below
// 2^-20.  And in 64 bits.
constexpr float kFastError = 0x1p-18f, kSlowError = 0x1p-20f, kFastFrom = -32.0f, kSlowFrom = -80.0f;
// FP32's is of the normal range: half of a gate below kSlowGate may not be in it, whatever u
// makes of it, nor a value that a block of a scale below kSlowScale tells from its neighbours.
constexpr float kSlowGate = 0x1p-120f;
constexpr uint32_t kSlowScale = 8;

__device__ __forceinline__ void gate_fast(const float (&g)[8], const float (&u)[8], float (&h)[8])
{
    const uint64_t log2e = pair2(-1.44269504f, -1.44269504f), one = pair2(1.0f, 1.0f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float a, b, r;
        const uint64_t gg = pair2(g[j], g[j + 1]);
        unpair2(mul2(gg, log2e), a, b);
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
        unpair2(add2(pair2(a, b), one), a, b);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
        unpair2(mul2(mul2(gg, pair2(u[j], u[j + 1])), mul2(pair2(b, a), pair2(r, r))), h[j], h[j + 1]);
    }
}
__device__ __forceinline__ double gate_exact(float g, float u) { return double(g) / (1.0 + exp(-double(g))) * double(u); }

// The code of a magnitude in units of its scale.
__device__ __forceinline__ uint32_t code_of(double a)
{
    return uint32_t(a > 0.25) + uint32_t(a >= 0.75) + uint32_t(a > 1.25) + uint32_t(a >= 1.75) + uint32_t(a > 2.5) +
           uint32_t(a >= 3.5) + uint32_t(a > 5.0);
}

// Codes of h, known to a relative `error`, under the scale of the block, whose
// largest magnitude has the bits m: those that
// the error decides are marked in `unsure`, a bit in each's place (all of them: the
// scale is).
__device__ __forceinline__ uint32_t codes8_known(const float (&h)[8], uint32_t m, float error, uint32_t *byte, uint32_t *unsure)
{
    const float a = __uint_as_float(m);
    *byte = scale_byte(m);
    const float inv = scale_inverse(*byte);
    const uint32_t w = codes8(h, inv * (1.0f + error)), d = w ^ codes8(h, inv * (1.0f - error));
    *unsure = (d | d >> 1 | d >> 2) & 0x11111111u;
    if (scale_byte(__float_as_uint(a * (1.0f + error))) != scale_byte(__float_as_uint(a * (1.0f - error)))) *unsure = ~0u;
    if (*byte == 255) *unsure = 0;
    return w;
}

// What the approximate instructions leave open (one block of some thousand): FP32,
// and where that cannot tell either on which side of a border between two codes,
// or between two scales, a value lies, 64 bits; and where a negative g's exponential, or
// what FP32 makes of a small value, leaves its range.
__device__ __noinline__ uint32_t codes8_gated(const float (&g)[8], const float (&u)[8], uint32_t *byte)
{
    float h[8], least = 0.0f;
    bool tiny = false, some = false, over = false;               // (over: FP32 has no such product, 64 bits may)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        h[j] = g[j] / (1.0f + expf(-g[j])) * u[j];
        least = fminf(least, g[j]);
        const bool counts = g[j] != 0.0f && u[j] != 0.0f;
        some = some || counts;
        tiny = tiny || (counts && fabsf(g[j]) < kSlowGate);
        over = over || (isinf(h[j]) && isfinite(g[j]) && isfinite(u[j]));
    }
    uint32_t unsure, w = codes8_known(h, block_max(largest8(h)), kSlowError, byte, &unsure);
    const bool whole = unsure == ~0u || over || (*byte != 255 && (least < kSlowFrom || tiny || (some && *byte < kSlowScale)));
    if (__any_sync(0xffffffffu, whole)) {
        // (an infinity is what rounds to one in FP32)
        double m = 0.0;
        uint32_t lost = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double v = gate_exact(g[j], u[j]);
            m = fmax(m, fabs(v));
            lost |= !isfinite(float(v));
        }
        m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 2));
        lost = block_max(lost);
        *byte = lost ? 255u : m > 0.0 ? uint32_t(max(ilogb(m) + 125, 0)) : 0u;
        unsure = lost ? 0u : ~0u;
    }
    // (of a block that is unsure as a whole every value)
    if (unsure == ~0u) unsure = 0x11111111u;
    while (unsure) {
        const int at = __ffs(int(unsure)) - 1;
        unsure &= unsure - 1;
        float gj = g[0], uj = u[0];
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (at == 4 * j) gj = g[j], uj = u[j];
        const double v = gate_exact(gj, uj);
        const uint32_t c = code_of(fabs(v) * scalbn(1.0, 127 - int(*byte))) | (signbit(v) ? 8u : 0u);
        w = (w & ~(15u << at)) | c << at;
    }
    return w;
}

// E matrices of R rows.  A lane has 8 values of a row at a time, four lanes a block,
// a warp 256 values; it serves N such runs of one row, eight rows a block.  The runs
// go through each step together, so that their waits for shuffles and exponentials
// overlap: 32768 x 2048 gated takes 60 us (5.1 TB/s read and written), one run after
// the other 96, two together 67; BF16 16384 x 4096 28 us (6.1), FP32 44 (6.9).  Gated
// values are bound by their arithmetic, some 170 instructions for 8 of a lane, in
// registers held down to what keeps three blocks resident (with two 71 us).
template <typename XT, bool ACT, int N>
__global__ void __launch_bounds__(256, ACT ? 3 : 1)
    mx4_quant_kernel(const XT *__restrict__ X, int64_t rows, int64_t R, int32_t K, uint8_t *__restrict__ Q, uint8_t *__restrict__ S)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= rows) return;
    const int32_t kt = (K + 127) / 128;
    const XT *row = X + t * (ACT ? 2 : 1) * int64_t(K);
    const int k0 = int(blockIdx.y) * (256 * N) + lane * 8;
    Raw<XT> raw[N], raw_u[ACT ? N : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int k = k0 + i * 256;
        if (k < K) {
            raw[i].load(row + k);
            if (ACT) raw_u[ACT ? i : 0].load(row + K + k);
        } else {
            raw[i].zero();
            if (ACT) raw_u[ACT ? i : 0].zero();
        }
    }
    // (the scales of each matrix begin a tile of their own)
    const int64_t e = rows == R ? 0 : t / R;
    uint8_t *s = S + e * ((R + 127) / 128 * kt * kMx4Tile) + mx4_scale_at(t - e * R, 0, kt);
    uint8_t *q = Q + t * (int64_t(K) / 2);
    uint32_t byte[N], w[N];
    if constexpr (!ACT) {
        uint32_t m[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[8];
            raw[i].values(v);
            m[i] = largest8(v);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = block_max(m[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[8];
            raw[i].values(v);
            byte[i] = scale_byte(m[i]);
            w[i] = codes8(v, scale_inverse(byte[i]));
        }
    } else {
        float h[N][8], least[N];
        uint32_t m[N], open = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float g[8], u[8];
            raw[i].values(g);
            raw_u[ACT ? i : 0].values(u);
            gate_fast(g, u, h[i]);
            m[i] = largest8(h[i]);
            least[i] = least8(g);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = block_max(m[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t unsure;
            w[i] = codes8_known(h[i], m[i], kFastError, &byte[i], &unsure);
            // (a small block's g u may have left FP32's range before h does)
            if (unsure != 0 || !(least[i] > kFastFrom) || byte[i] < 32 || byte[i] == 255) open |= 1u << i;
        }
        if (__any_sync(0xffffffffu, open != 0)) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float g[8], u[8];
                raw[i].values(g);
                raw_u[ACT ? i : 0].values(u);
                // zeros are zeros, unless a far gate's exponential made a NaN of them
                bool zero = true;
#pragma unroll
                for (int j = 0; j < 8; ++j) zero = zero && (g[j] == 0.0f || u[j] == 0.0f);
                if (__any_sync(0xffffffffu, (open >> i & 1u) && (!zero || byte[i] == 255))) w[i] = codes8_gated(g, u, &byte[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int k = k0 + i * 256;
        if (byte[i] == 255) w[i] = 0;
        if (k < K) *reinterpret_cast<uint32_t *>(q + k / 2) = w[i];
        byte[i] <<= 8 * ((lane >> 2) & 3);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) byte[i] |= __shfl_xor_sync(0xffffffffu, byte[i], 4);
#pragma unroll
    for (int i = 0; i < N; ++i) byte[i] |= __shfl_xor_sync(0xffffffffu, byte[i], 8);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int k = k0 + i * 256;
        if ((lane & 15) == 0 && k < K) *reinterpret_cast<uint32_t *>(s + int64_t(k / 128) * kMx4Tile) = byte[i];
    }
}

// The token pass: a programmatic dependent of the stream's previous kernel (it
// waits for it before it reads anything), and only then lets the product start,
// whose early reads of weights and offsets are thus ordered after everything
// before this call.
template <typename XT>
cudaError_t launch_quant_as(const void *X, int act, int64_t E, int64_t R, int32_t K, uint8_t *Q, uint8_t *S, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = {};
    // (short rows: no runs past their end)
    const int runs = K <= 256 ? 1 : K <= 512 ? 2 : 4;
    cfg.gridDim = dim3(unsigned((E * R + 7) / 8), unsigned((K + 256 * runs - 1) / (256 * runs)), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    if (pdl_enabled()) {
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    const XT *x = static_cast<const XT *>(X);
    auto run = [&](auto act_of) {
        constexpr bool ACT = decltype(act_of)::value;
        return runs == 1   ? cudaLaunchKernelEx(&cfg, mx4_quant_kernel<XT, ACT, 1>, x, E * R, R, K, Q, S)
               : runs == 2 ? cudaLaunchKernelEx(&cfg, mx4_quant_kernel<XT, ACT, 2>, x, E * R, R, K, Q, S)
                           : cudaLaunchKernelEx(&cfg, mx4_quant_kernel<XT, ACT, 4>, x, E * R, R, K, Q, S);
    };
    return act == CAKE_GG_ACT_SILU_MUL ? run(std::true_type()) : run(std::false_type());
}

int launch_quant(const void *X, int x_dtype, int act, int64_t E, int64_t R, int32_t K, uint8_t *Q, uint8_t *S, cudaStream_t stream)
{
    const cudaError_t err = x_dtype == CAKE_GG_BF16 ? launch_quant_as<uint16_t>(X, act, E, R, K, Q, S, stream)
                                                    : launch_quant_as<float>(X, act, E, R, K, Q, S, stream);
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

// ---------------------------------------------------------------- scales of a pair's rows

// The scales of a slot's rows, put together from those of their tokens, and where
// rows are routed their codes.  A pair's even CTA issues for both, so what the odd
// one reads has to be ordered for the even one: copies by TMA are, by their barrier;
// stores of the odd CTA's warps are by a release at cluster scope, which takes some
// microseconds while outputs are stored (16384 x 4096 -> 4096: 117 us with one for each
// stage, 103 for every other, 87 so).  And gathered by TMA a row of 128 bytes takes
// some 8 clocks, for every channel tile again (32768 tokens through 2 of 8 experts
// 4096 -> 4096: 445 us).  A block serves 128 rows: one scale tile of every word, a thread
// four rows, 32 apart; then a warp a row's codes.
__global__ void __launch_bounds__(256)
    mx4_arrange_kernel(const int32_t *__restrict__ offsets, const int32_t *__restrict__ rows, const uint8_t *__restrict__ xs,
                       const uint8_t *__restrict__ x, uint8_t *__restrict__ out, uint8_t *__restrict__ out_x, int32_t *status, int64_t M,
                       int64_t T, int32_t E, int32_t K, int32_t nt, int32_t atoms)
{
    const int32_t n_kt = (K + 127) / 128;
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t slot = int32_t(blockIdx.x) / atoms, atom = int32_t(blockIdx.x) % atoms;
    // the last expert whose slots begin at or before this one; what the product would
    // refuse is left alone
    int32_t e = 0, first = 0, end = int32_t(M);
    if (offsets) {
        int32_t hi = E;
        while (hi - e > 1) {
            const int32_t mid = (e + hi) / 2;
            if (mx4_slot(offsets[mid], mid, 0, nt) <= slot) e = mid;
            else hi = mid;
        }
        first = offsets[e], end = offsets[e + 1];
    }
    if (first < 0 || end < first || end > M) return;
    const int64_t m0 = first + (int64_t(slot) - mx4_slot(first, e, 0, nt)) * nt + atom * 128;
    const int64_t m1 = min(int64_t(end), m0 - atom * 128 + nt);
    if (m0 < first || m0 >= m1) return;
    const int lane = threadIdx.x & 31;
    const uint8_t *src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int64_t r = m0 + i * 32 + lane;
        src[i] = nullptr;
        if (r < m1) {
            if (rows) r = rows[r];
            if (r >= 0 && r < T) src[i] = xs + mx4_scale_at(r, 0, n_kt);
            else atomicCAS(status, 0, CAKE_GG_ERR_BAD_ROWS);
        }
    }
    uint8_t *dst = out + (int64_t(slot) * n_kt * atoms + atom) * kMx4Tile + lane * 16;
    for (int kt = threadIdx.x >> 5; kt < n_kt; kt += 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = src[i] ? *reinterpret_cast<const uint32_t *>(src[i] + int64_t(kt) * kMx4Tile) : 0u;
        *reinterpret_cast<uint4 *>(dst + int64_t(kt) * atoms * kMx4Tile) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (!rows) return;
    const int32_t pieces = K / 32;                               // 16 bytes each
    const int64_t end_row = min(m1, m0 + 128);
    for (int64_t m = m0 + (threadIdx.x >> 5); m < end_row; m += 8) {
        const int64_t r = rows[m];
        if (r < 0 || r >= T) continue;
        const uint4 *from = reinterpret_cast<const uint4 *>(x + r * int64_t(K / 2));
        uint4 *to = reinterpret_cast<uint4 *>(out_x + m * int64_t(K / 2));
#pragma unroll 4
        for (int i = lane; i < pieces; i += 32) to[i] = from[i];
    }
}

cudaError_t launch_arrange(const Mx4Params &p, const int32_t *rows, int64_t T, const uint8_t *xs, const uint8_t *x, uint8_t *out,
                           uint8_t *out_x, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = {};
    const int32_t atoms = mx4_row_atoms(p.nt);
    cfg.gridDim = dim3(unsigned(mx4_slots(p.M, p.E, p.nt) * atoms), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    if (pdl_enabled()) {
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, mx4_arrange_kernel, p.offsets, rows, xs, x, out, out_x, p.status, p.M, T, p.E, p.K, p.nt, atoms);
}

// The problem's own checks, shared by the plan and the call.
int check_problem(int32_t E, int64_t M_max, int64_t T, int32_t N, int32_t K, int x_dtype, int act, int out_dtype)
{
    if (E < 1 || E > kMaxExperts || M_max < 0 || M_max > INT32_MAX || T < 0 || T > INT32_MAX || N < 1 || K < 1 ||
        (M_max > 0 && T < 1))
        return CAKE_GG_ERR_INVALID_ARG;
    if (x_dtype != CAKE_GG_BF16 && x_dtype != CAKE_GG_FP32 && x_dtype != CAKE_GG_MX4) return CAKE_GG_ERR_UNSUPPORTED;
    if (out_dtype != CAKE_GG_BF16 && out_dtype != CAKE_GG_FP32) return CAKE_GG_ERR_UNSUPPORTED;
    if (act != CAKE_GG_ACT_NONE && act != CAKE_GG_ACT_SILU_MUL) return CAKE_GG_ERR_INVALID_ARG;
    if (act != CAKE_GG_ACT_NONE && x_dtype == CAKE_GG_MX4) return CAKE_GG_ERR_INVALID_ARG;
    if (N % 8 != 0 || K % 32 != 0) return CAKE_GG_ERR_ALIGNMENT;
    if (K > kMaxK || N > kMaxN) return CAKE_GG_ERR_OVERFLOW;
    // (addresses of 64 bits, and scale tiles that a copy numbers in 31)
    uint64_t t;
    if (!mul_ok(uint64_t(E) * uint64_t(N), uint64_t(K), &t) || !mul_ok(uint64_t(M_max), uint64_t(N) * 4u, &t) ||
        uint64_t(E) * uint64_t((N + 127) / 128) > uint64_t(INT32_MAX) / uint64_t((K + 127) / 128))
        return CAKE_GG_ERR_OVERFLOW;
    return CAKE_GG_OK;
}

int stages_for(int pair, int nt, int splits, int E)
{
    int s = kMx4StagesMost;
    while (s > 0 && mx4_mma_smem(pair, nt, s, splits, E) > kMx4SmemLimit) --s;
    return s;
}

// Whether a call of few rows takes the dot products, in runs of up to two rows: they need some
// 2.5 us to begin with, and then their arithmetic, 4 million weights a microsecond; the
// tensor cores 5 to 8 us, and then what HBM gives.  By dot products and by tensor cores,
// BF16 rows: 1024 x 1024 2.7 and 5.9 us, 4096 x 4096 5.3 and 8.0, two rows of it 6.2 and
// 8.0, 6144 x 4096 7.8 and 8.9, one token through 8 of 128 experts 2048 -> 768 6.1 and
// 10.3; past the rule 4096 x 8192 10.0 and 8.4, 8192 x 8192 17 and 13.  Long rows leave few
// blocks much to do one after another (8192 x 512 7.9 and 7.7), and blocks that are not all
// resident begin anew: 9 rows of 256 x 4096 8.9 and 5.1, 64 of 256 x 1024 12.7 and 5.2.
bool few_rows(const cake_gg_mx4_plan_t &pl)
{
    const int R = mx4_run_rows(pl.M_max, pl.E);
    const int64_t runs = mx4_runs(pl.M_max, pl.E);
    return pl.K <= 8192 && runs <= 8 * int64_t(pl.E) && runs * pl.N <= int64_t(28) * 1000 * 1000 / pl.K &&
           runs * ((pl.N + 127) / 128 * 4) <= kSms * (R == 1 ? 3 : 2);
}

// Row tiles of nt rows that the call will have: exact for one expert; where E
// share the rows, whole tiles and half a tile more for each expert that can have
// rows, at least one each (the sizes are the device's).
int64_t row_tiles(const cake_gg_mx4_plan_t &pl, int nt)
{
    const int64_t whole = (pl.M_max + nt - 1) / nt;
    if (pl.E == 1) return whole;
    const int64_t busy = pl.M_max < pl.E ? pl.M_max : pl.E;
    return whole + busy / 2 > busy ? whole + busy / 2 : busy;
}

// Multiprocessors that clusters of `splits` CTAs can hold at once: a cluster lies
// within one of the GPU's groups of them, whose sizes differ from part to part.
int cluster_sms(int splits) { return splits <= 2 ? kSms : splits <= 6 ? 132 : 104; }

// Whether a copy can number the scale tiles of a pair's rows.
bool pair_fits(const cake_gg_mx4_plan_t &pl, int nt)
{
    return mx4_slots(pl.M_max, pl.E, nt) * ((pl.K + 127) / 128) * mx4_row_atoms(nt) <= INT32_MAX;
}

// The shape, from a model of its time in nanoseconds: waves of units over the
// multiprocessors (152, or 76 pairs), the stages of a unit, or the reading of the
// weights where that is longer; the storing of the last unit, the laying out of a
// pair's rows, and the exchange between the CTAs that share a tile.  The times of a stage, with all multiprocessors at work (16384 x
// 4096 -> 4096), are for single CTAs 260, 272, 307, 337 ns for 96, 128, 160, 192 rows,
// for pairs 245, 238, 275, 276; the lines below are within 7 % of that.  What the model
// decides, measured with the neighbours: 33 x 8192 -> 512 divides the reduction by 8
// (8.2 us; 8.0 by 6, 10.9 undivided), 701 tokens through 2 of 8 experts 4096 -> 2048 take
// tiles of 96 rows (16.4; 18.9 with 128, 18.5 with 64), 300 through 4 of 32 6144 -> 4096
// take 64 (70.9; 78 with 32), 1024 x 4096 -> 4096 single CTAs of 128 (14.6; 15.3 with pairs of
// 160), 3001 x 5120 -> 1000 of 160 (12.7; 12.5 with pairs of 192, 16.9 with 128).
void choose(cake_gg_mx4_plan_t *pl)
{
    const int64_t n_kb = (pl->K + 255) / 256;
    // the weights of the experts that can have rows, at what HBM gives
    const int64_t weights = (pl->M_max < pl->E ? pl->M_max : pl->E) * pl->N * pl->K / 2 / 6000;
    int64_t best = -1;
    auto consider = [&](int pair, int nt, int splits) {
        const int64_t units = row_tiles(*pl, nt) * ((pl->N + 128 * pair - 1) / (128 * pair));
        if (splits > 1 && (units * splits > cluster_sms(splits) || n_kb < 2 * splits)) return;
        if (pair == 2 && !pair_fits(*pl, nt)) return;
        const int64_t waves = (units * pair + kSms - 1) / kSms;
        int64_t ns = waves * ((n_kb + splits - 1) / splits) * (200 + nt * (pair == 2 ? 4 : 7) / 10);
        ns = (ns > weights ? ns : weights) + 12 * nt;
        if (splits > 1) ns += 300 + nt * (45 + 4 * splits);
        if (pair == 2) ns += 1800 + (pl->T != pl->M_max ? pl->M_max * pl->K / 12000 : 0);   // (routed: rows copied)
        if (best < 0 || ns < best) {
            best = ns;
            pl->pair = pair;
            pl->tile_rows = nt;
            pl->splits = splits;
        }
    };
    for (int nt = kMx4RowsMost; nt >= 64; nt -= 32) consider(2, nt, 1);
    for (int nt = kMx4RowsMost; nt >= 32; nt -= 32)
        for (int sp = 1; sp <= (nt <= 64 ? 8 : 1); ++sp) consider(1, nt, sp);
    const int path = env_int("CAKE_GG_MX4_PATH", few_rows(*pl) ? CAKE_GG_MX4_ROWS : CAKE_GG_MX4_MMA);
    pl->path = path == CAKE_GG_MX4_ROWS && mx4_rows_fit(pl->M_max, pl->E, pl->K) ? CAKE_GG_MX4_ROWS : CAKE_GG_MX4_MMA;
    pl->pair = env_int("CAKE_GG_MX4_PAIR", pl->pair) == 2 ? 2 : 1;
    const int nt = env_int("CAKE_GG_MX4_ROWS_PER_TILE", pl->tile_rows);
    if (nt >= 32 && nt <= kMx4RowsMost && nt % 32 == 0) pl->tile_rows = nt;
    const int sp = env_int("CAKE_GG_MX4_SPLITS", pl->splits);
    pl->splits = sp >= 1 && sp <= 8 && pl->pair == 1 ? sp : 1;
    pl->stages = stages_for(pl->pair, pl->tile_rows, pl->splits, pl->E);
}

// What the kernel can run.
bool plan_ok(const cake_gg_mx4_plan_t &pl)
{
    if (pl.path != CAKE_GG_MX4_MMA && !(pl.path == CAKE_GG_MX4_ROWS && mx4_rows_fit(pl.M_max, pl.E, pl.K))) return false;
    return (pl.pair == 1 || pl.pair == 2) && pl.tile_rows >= 32 && pl.tile_rows <= kMx4RowsMost && pl.tile_rows % 32 == 0 &&
           pl.stages >= kStagesLeast && pl.stages <= kMx4StagesMost && pl.splits >= 1 && pl.splits <= 8 &&
           (pl.splits == 1 || pl.pair == 1) && pl.splits <= (pl.K + 255) / 256 &&   // (a stage for every CTA)
           (pl.pair == 1 || pair_fits(pl, pl.tile_rows)) &&
           mx4_mma_smem(pl.pair, pl.tile_rows, pl.stages, pl.splits, pl.E) <= kMx4SmemLimit;
}

}  // namespace

extern "C" {

int cake_gg_mx4_plan(cake_gg_mx4_plan_t *plan, int32_t E, int64_t M_max, int64_t T, int32_t N, int32_t K, int x_dtype, int act,
                     int out_dtype, int32_t max_sms)
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
    choose(plan);
    if (!plan_ok(*plan)) return CAKE_GG_ERR_INVALID_ARG;   // (an override that does not fit)
    plan->timeout_ns = kTimeoutNs;
    plan->workspace_bytes = layout(*plan).total;
    return CAKE_GG_OK;
}

int cake_gg_mx4_quant(const void *X, int x_dtype, int act, int32_t E, int64_t R, int32_t K, uint8_t *Xq, uint8_t *xs, void *stream)
{
    if (x_dtype != CAKE_GG_BF16 && x_dtype != CAKE_GG_FP32) return CAKE_GG_ERR_UNSUPPORTED;
    if (E < 1 || E > kMaxExperts) return CAKE_GG_ERR_INVALID_ARG;
    const int rc = check_problem(1, 0, R, 8, K, x_dtype, act, CAKE_GG_BF16);
    if (rc != CAKE_GG_OK) return rc;
    if (R == 0) return CAKE_GG_OK;
    if ((int64_t(E) * R + 7) / 8 > INT32_MAX) return CAKE_GG_ERR_OVERFLOW;
    if (!X || !Xq || !xs) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(Xq, 16) || !aligned(xs, 16)) return CAKE_GG_ERR_ALIGNMENT;
    int sms;
    const int dev = device_sms(&sms);
    if (dev != CAKE_GG_OK) return dev;
    return launch_quant(X, x_dtype, act, E, R, K, Xq, xs, static_cast<cudaStream_t>(stream));
}

int cake_gg_mx4_gemm(const cake_gg_mx4_plan_t *plan, const void *X, const uint8_t *xs, const int32_t *rows, const uint8_t *W,
                     const uint8_t *ws, void *Y, const int32_t *offsets, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!plan || plan->abi_version != CAKE_GG_ABI_VERSION) return CAKE_GG_ERR_INVALID_ARG;
    const cake_gg_mx4_plan_t &pl = *plan;
    int rc = check_problem(pl.E, pl.M_max, pl.T, pl.N, pl.K, pl.x_dtype, pl.act, pl.out_dtype);
    if (rc != CAKE_GG_OK) return rc;
    if (pl.max_sms < 0 || !plan_ok(pl)) return CAKE_GG_ERR_INVALID_ARG;
    const bool ready = pl.x_dtype == CAKE_GG_MX4;   // tokens come quantised
    if (!workspace || !W || !ws || (pl.M_max > 0 && (!X || !Y || (ready && !xs))) || (!ready && xs))
        return CAKE_GG_ERR_INVALID_ARG;
    if ((!offsets && pl.E != 1) || (!rows && pl.M_max > 0 && pl.T != pl.M_max)) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(workspace, 16) || !aligned(xs, 16) ||
        !aligned(ws, 16) || !aligned(rows, 4) || !aligned(offsets, 4))
        return CAKE_GG_ERR_ALIGNMENT;
    const Layout L = layout(pl);
    if (workspace_bytes < L.total || pl.workspace_bytes != L.total) return CAKE_GG_ERR_WORKSPACE;
    int sms;
    if ((rc = device_sms(&sms)) != CAKE_GG_OK) return rc;
    if (pl.M_max == 0) return CAKE_GG_OK;

    uint8_t *base = static_cast<uint8_t *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Mx4Params p{};
    p.offsets = offsets;
    // (a pair's rows are laid out before: for it row m is token m)
    const bool few = pl.path == CAKE_GG_MX4_ROWS, pair = pl.pair == 2 && !few;
    const bool pass = !ready && (!few || pl.act != CAKE_GG_ACT_NONE);   // (a few rows are quantised by the blocks)
    const uint8_t *scales = ready ? xs : base + L.scales, *x = ready ? static_cast<const uint8_t *>(X) : base + L.tokens;
    const uint8_t *x_rows = pair && rows ? base + L.rows : x;
    p.rows = pair ? nullptr : rows;
    p.xs = pair ? base + L.arranged : scales;
    p.Y = Y;
    p.status = reinterpret_cast<int32_t *>(base);
    p.M = pl.M_max;
    p.T = pair ? pl.M_max : pl.T;
    p.E = pl.E;
    p.N = pl.N;
    p.K = pl.K;
    p.out_f32 = pl.out_dtype == CAKE_GG_FP32;
    p.early = pass || pair;
    p.nt = pl.tile_rows;
    p.stages = pl.stages;
    p.splits = pl.splits;
    p.debug_flags = pl.debug_flags;
    p.timeout_ns = pl.timeout_ns ? pl.timeout_ns : kTimeoutNs;
    const int cap = pl.max_sms > 0 && pl.max_sms < sms ? pl.max_sms : sms;
    // what cannot be launched is refused before anything is enqueued
    Mx4Launch product;
    if (!few && (rc = prepare_mx4_mma(&product, p, W, ws, x_rows, pl.pair, cap)) != CAKE_GG_OK) return rc;
    if (pass && (rc = launch_quant(X, pl.x_dtype, pl.act, 1, pl.T, pl.K, base + L.tokens, base + L.scales, s)) != CAKE_GG_OK)
        return rc;
    if (few) {
        const bool codes = ready || pass;
        return launch_mx4_rows(p, codes ? x : static_cast<const uint8_t *>(X), codes ? int(CAKE_GG_MX4) : pl.x_dtype, W, ws,
                               pdl_enabled(), s) == cudaSuccess
                   ? CAKE_GG_OK
                   : CAKE_GG_ERR_CUDA;
    }
    if (pair && launch_arrange(p, rows, pl.T, scales, x, base + L.arranged, base + L.rows, s) != cudaSuccess) return CAKE_GG_ERR_CUDA;
    return launch_mx4_mma(product, pdl_enabled(), s);
}

}  // extern "C"
