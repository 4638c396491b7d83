// cake_gg_int8.cu -- C entry points of the 8-bit integer products, and the
// kernel that quantises tokens row by row.
//
//   h[t, k] = x[t, k], or silu(g) * u of x[t] = [g | u]
//   a[t] = max_k |h[t, k]|     s[t] = a / 127     q[t, k] = rint(h[t, k] * (127 / a))
//   Y[m, n] = (sum_k q[r(m), k] W[e(m), n, k]) * ws[e(m), n] * s[r(m)]
//
// A call is one launch when X is already 8-bit and its rows are few, else two:
// the token pass below writes 8-bit rows and their scales to the workspace,
// and the product reads them.
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cake_gg_int8.h"
#include "cake_gg_ptx.cuh"

using namespace cakegg;

namespace {

constexpr uint64_t kHeader = 256;              // status word at byte 0
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxK = (1 << 17) - 16;      // |sum of K products| <= 2^14 K stays below 2^31

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

// Workspace: header | token scales [T] | 8-bit tokens [T, K].
struct Layout {
    uint64_t scales, tokens, total;
};

Layout layout(const cake_gg_i8_plan_t &pl)
{
    Layout L;
    const bool pass = pl.x_dtype != CAKE_GG_INT8;
    L.scales = kHeader;
    L.tokens = L.scales + (pass ? align_up(uint64_t(pl.T) * 4, 256) : 0);
    L.total = L.tokens + (pass ? align_up(uint64_t(pl.T) * uint64_t(pl.K), 256) : 0);
    return L;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------- token pass

template <typename XT>
__device__ __forceinline__ void load8(const XT *p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t *p, float (&v)[8])
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Eight values of a row, the gate applied: silu(g) * u = g / (1 + e^-g) * u.
// (g = -inf gives NaN, as the formula does; a large negative g gives 0.)
template <typename XT, bool ACT>
__device__ __forceinline__ void row8(const XT *row, int32_t K, int k, float (&v)[8])
{
    load8(row + k, v);
    if (ACT) {
        float u[8];
        load8(row + K + k, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * u[i];
    }
}

// One block per row.  The first kHeld vectors of 8 values that a thread owns
// stay in registers between the maximum and the rounding; longer rows read the
// rest again (from L2).  |h| is compared by its bit pattern, so a NaN or an
// infinity wins the maximum: such a row gets the scale NaN and zero integers
// (its products are NaN).  A row whose largest value is below 2^-120 counts as
// zero (127 / a would not be finite).
constexpr int kHeld = 2;

template <typename XT, bool ACT>
__global__ void __launch_bounds__(1024)
    i8_quant_kernel(const XT *__restrict__ X, int32_t K, int8_t *__restrict__ Q, float *__restrict__ S)
{
    __shared__ uint32_t warp_max[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x;
    const XT *row = X + t * (ACT ? 2 : 1) * int64_t(K);
    const int stride = int(blockDim.x) * 8;
    float held[kHeld][8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int k = int(threadIdx.x) * 8 + j * stride;
        if (k < K) {
            row8<XT, ACT>(row, K, k, held[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(held[j][i]) & 0x7fffffffu);
        }
    }
    for (int k = int(threadIdx.x) * 8 + kHeld * stride; k < K; k += stride) {
        float v[8];
        row8<XT, ACT>(row, K, k, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
    m = threadIdx.x % 32 < blockDim.x / 32 ? warp_max[threadIdx.x % 32] : 0;
    m = __reduce_max_sync(0xffffffffu, m);
    const float a = __uint_as_float(m);
    const bool finite = m < 0x7f800000u, tiny = a < 0x1p-120f;
    const float inv = finite && !tiny ? 127.0f / a : 0.0f;
    if (threadIdx.x == 0) S[t] = !finite ? __uint_as_float(0x7fc00000u) : tiny ? 0.0f : a / 127.0f;
    int8_t *out = Q + t * int64_t(K);
    auto emit = [&](const float (&v)[8], int k) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int q = finite ? __float2int_rn(v[i] * inv) : 0;
            w[i / 4] |= uint32_t(q & 0xff) << (8 * (i % 4));
        }
        *reinterpret_cast<uint2 *>(out + k) = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int k = int(threadIdx.x) * 8 + j * stride;
        if (k < K) emit(held[j], k);
    }
    for (int k = int(threadIdx.x) * 8 + kHeld * stride; k < K; k += stride) {
        float v[8];
        row8<XT, ACT>(row, K, k, v);
        emit(v, k);
    }
}

int launch_quant(const void *X, int x_dtype, int act, int64_t T, int32_t K, int8_t *Q, float *S, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int threads = int(align_up((uint64_t(K) / 8 + kHeld - 1) / kHeld, 32));
    if (threads > 1024) threads = 1024;
    cfg.gridDim = dim3(unsigned(T), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.stream = stream;
    if (pdl_enabled()) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const bool silu = act == CAKE_GG_ACT_SILU_MUL;
    cudaError_t err;
    if (x_dtype == CAKE_GG_BF16) {
        const uint16_t *x = static_cast<const uint16_t *>(X);
        err = silu ? cudaLaunchKernelEx(&cfg, i8_quant_kernel<uint16_t, true>, x, K, Q, S)
                   : cudaLaunchKernelEx(&cfg, i8_quant_kernel<uint16_t, false>, x, K, Q, S);
    } else {
        const float *x = static_cast<const float *>(X);
        err = silu ? cudaLaunchKernelEx(&cfg, i8_quant_kernel<float, true>, x, K, Q, S)
                   : cudaLaunchKernelEx(&cfg, i8_quant_kernel<float, false>, x, K, Q, S);
    }
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
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
    if (K > kMaxK) return CAKE_GG_ERR_OVERFLOW;
    uint64_t t;
    if (!mul_ok(uint64_t(T), uint64_t(K) * 8u, &t) || !mul_ok(uint64_t(E) * uint64_t(N), uint64_t(K), &t) ||
        !mul_ok(uint64_t(M_max), uint64_t(N) * 4u, &t))
        return CAKE_GG_ERR_OVERFLOW;
    return CAKE_GG_OK;
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
    plan->path = CAKE_GG_I8_ROWS;
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
    return launch_quant(X, x_dtype, act, T, K, Xq, xs, static_cast<cudaStream_t>(stream));
}

int cake_gg_i8_gemm(const cake_gg_i8_plan_t *plan, const void *X, const float *xs, const int32_t *rows,
                    const int8_t *W, const float *ws, void *Y, const int32_t *offsets, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    if (!plan || plan->abi_version != CAKE_GG_ABI_VERSION) return CAKE_GG_ERR_INVALID_ARG;
    const cake_gg_i8_plan_t &pl = *plan;
    int rc = check_problem(pl.E, pl.M_max, pl.T, pl.N, pl.K, pl.x_dtype, pl.act, pl.out_dtype);
    if (rc != CAKE_GG_OK) return rc;
    if (pl.path != CAKE_GG_I8_ROWS || pl.max_sms < 0) return CAKE_GG_ERR_INVALID_ARG;
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
    const int8_t *q = static_cast<const int8_t *>(X);
    if (!ready) {
        int8_t *Xq = reinterpret_cast<int8_t *>(base + L.tokens);
        float *scales = reinterpret_cast<float *>(base + L.scales);
        if ((rc = launch_quant(X, pl.x_dtype, pl.act, pl.T, pl.K, Xq, scales, s)) != CAKE_GG_OK) return rc;
        q = Xq;
        xs = scales;
    }
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
    p.early = ready ? 0 : 1;
    p.timeout_ns = pl.timeout_ns ? pl.timeout_ns : kTimeoutNs;
    return launch_i8_rows(p, q, pdl_enabled(), s) == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

}  // extern "C"
