// cake_gg_route.cu -- C entry points of the routing, and the kernel that numbers
// rows across blocks; the others are in cake_gg_route.cuh.
#include <cstring>

#include "cake_gg_ptx.cuh"
#include "cake_gg_route.h"

using namespace cakegg;

namespace {

constexpr int kThreads = kRouteThreads;
constexpr int32_t kMaxExperts = kRouteMaxExperts, kMaxTop = kRouteMaxTop, kMaxGroups = 32;
constexpr int64_t kMaxTokens = 1 << 23;        // (a block's tokens are below 2^16)
constexpr int kClusterBlocks = 8;
constexpr int kSms = 152;
constexpr uint64_t kHeader = 256;              // (as in the products' workspaces; its status word stays 0)

// Places within a block to rows: each block sums the counts of all blocks and of
// those before it (at most 152 of them), eight experts a load, all threads.  (One
// block that does it for all while the others wait took 6 us for 256 experts; all of
// them, an expert a load, 7.)
__global__ void __launch_bounds__(kThreads)
    route_number_kernel(const RouteParams p)
{
    __shared__ int32_t sums[kMaxExperts], before[kMaxExperts];   // of expert 8 v + i at i * (vectors) + v
    grid_dependency_wait();
    grid_launch_dependents();
    const int blocks = int(gridDim.x), me = int(blockIdx.x), vectors = count_pitch(p.E) / 8;
    const int64_t t0 = int64_t(me) * p.block_tokens, n = min(int64_t(p.block_tokens), p.T - t0) * p.top_k, at0 = t0 * p.top_k;
    // (the first of the thread's choices, while the counts come)
    int32_t position = 0, expert = 0;
    if (threadIdx.x < n) position = p.position[at0 + threadIdx.x], expert = p.expert[at0 + threadIdx.x];
    for (int e = threadIdx.x; e < vectors * 8; e += kThreads) sums[e] = before[e] = 0;
    __syncthreads();
    const int v = int(threadIdx.x) % vectors, part = int(threadIdx.x) / vectors, parts = kThreads / vectors;
    if (part < parts) {
        int32_t all[8] = {}, mine[8] = {};
#pragma unroll 5
        for (int b = part; b < blocks; b += parts) {
            const uint4 c = *reinterpret_cast<const uint4 *>(p.counts + int64_t(b) * (vectors * 8) + v * 8);
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t lo = int32_t(w[i] & 0xffffu), hi = int32_t(w[i] >> 16);
                all[2 * i] += lo, all[2 * i + 1] += hi;
                if (b < me) mine[2 * i] += lo, mine[2 * i + 1] += hi;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            atomicAdd(&sums[i * vectors + v], all[i]);           // (whole numbers: their order changes nothing)
            atomicAdd(&before[i * vectors + v], mine[i]);
        }
    }
    __syncthreads();
    const int e = int(threadIdx.x), at = e % 8 * vectors + e / 8;
    const int32_t all = e < p.E ? sums[at] : 0, mine = e < p.E ? before[at] : 0;
    int32_t total;
    const int32_t first = block_scan(all, &total);               // (a barrier inside)
    if (e < p.E) {
        before[at] = first + mine;
        if (me == 0) p.offsets[e] = first;
    }
    if (me == 0 && e == 0) p.offsets[p.E] = total;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        if (i >= kThreads) position = p.position[at0 + i], expert = p.expert[at0 + i];
        const int32_t row = position + before[expert % 8 * vectors + expert / 8];
        p.position[at0 + i] = row;
        p.rows[row] = int32_t(t0) + int32_t(p.top_k == 1 ? i : i / p.top_k);
    }
}

// ---------------------------------------------------------------- host

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_sizes(int64_t T, int32_t E, int32_t top_k)
{
    if (T < 0 || E < 1 || E > kMaxExperts || top_k < 1 || top_k > kMaxTop || top_k > E) return CAKE_GG_ERR_INVALID_ARG;
    if (T > kMaxTokens || T * top_k > INT32_MAX) return CAKE_GG_ERR_OVERFLOW;
    return CAKE_GG_OK;
}
int check_scores(int logits_dtype, int64_t stride, int32_t E, int score)
{
    if (logits_dtype != CAKE_GG_BF16 && logits_dtype != CAKE_GG_FP32) return CAKE_GG_ERR_UNSUPPORTED;
    if (score != CAKE_GG_SCORE_SOFTMAX && score != CAKE_GG_SCORE_SIGMOID) return CAKE_GG_ERR_INVALID_ARG;
    if (stride < E || stride > INT64_MAX / kMaxTokens / 4) return CAKE_GG_ERR_INVALID_ARG;
    return CAKE_GG_OK;
}

// Blocks and their tokens: as few blocks of one cluster as have a warp for a token
// (of 256 experts 256 tokens 12 us, 260 by two kernels 12; of 512 experts 128 10.3, and 256,
// two for each warp, 15.1, by two kernels 10.6), or blocks of eight tokens (257 in groups 13.3
// us, in blocks of two 14.0, of thirty-two 15.6) or of more, one for each multiprocessor,
// which holds the bits of a chunk of its tokens.
void choose_blocks(cake_gg_route_plan_t *pl)
{
    const int64_t T = pl->T;
    pl->cluster = T <= kClusterBlocks * (pl->E <= kRouteNarrow ? kRouteThreads : kRouteThreads / 2) / 32;
    int64_t blocks = pl->cluster ? (T + 3) / 4 : T < 8 * kSms ? (T + 7) / 8 : kSms;
    if (pl->cluster && blocks > kClusterBlocks) blocks = kClusterBlocks;
    if (blocks < 1) blocks = 1;
    const int64_t per = T == 0 ? 1 : (T + blocks - 1) / blocks;
    pl->block_tokens = int32_t(per);
    pl->blocks = int32_t(T == 0 ? 1 : (T + per - 1) / per);
}

uint64_t workspace_of(const cake_gg_route_plan_t &pl) { return kHeader + (pl.cluster ? 0 : uint64_t(pl.blocks) * uint64_t(count_pitch(pl.E)) * 2); }

}  // namespace

extern "C" {

int cake_gg_route_plan(cake_gg_route_plan_t *plan, int64_t T, int32_t E, int32_t top_k)
{
    if (!plan) return CAKE_GG_ERR_INVALID_ARG;
    std::memset(plan, 0, sizeof(*plan));
    const int rc = check_sizes(T, E, top_k);
    if (rc != CAKE_GG_OK) return rc;
    plan->abi_version = CAKE_GG_ABI_VERSION;
    plan->T = T;
    plan->E = E;
    plan->top_k = top_k;
    choose_blocks(plan);
    plan->workspace_bytes = workspace_of(*plan);
    return CAKE_GG_OK;
}

int cake_gg_route(const cake_gg_route_plan_t *plan, const cake_gg_route_options_t *options, const void *logits, int logits_dtype,
                  int64_t row_stride, const float *bias, int32_t *expert, float *weight, int32_t *offsets, int32_t *rows,
                  int32_t *position, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!plan || plan->abi_version != CAKE_GG_ABI_VERSION || !options) return CAKE_GG_ERR_INVALID_ARG;
    const cake_gg_route_plan_t &pl = *plan;
    const cake_gg_route_options_t &op = *options;
    int rc = check_sizes(pl.T, pl.E, pl.top_k);
    if (rc == CAKE_GG_OK) rc = check_scores(logits_dtype, row_stride, pl.E, op.score);
    if (rc != CAKE_GG_OK) return rc;
    cake_gg_route_plan_t own = pl;
    choose_blocks(&own);
    if (own.cluster != pl.cluster || own.blocks != pl.blocks || own.block_tokens != pl.block_tokens) return CAKE_GG_ERR_INVALID_ARG;
    if (op.groups < 1 || op.groups > kMaxGroups || pl.E % op.groups != 0 || op.top_groups < 1 || op.top_groups > op.groups ||
        pl.top_k > pl.E / op.groups * op.top_groups)
        return CAKE_GG_ERR_INVALID_ARG;
    if (op.group_score != CAKE_GG_GROUP_MAX && op.group_score != CAKE_GG_GROUP_TOP2) return CAKE_GG_ERR_INVALID_ARG;
    if (op.group_score == CAKE_GG_GROUP_TOP2 && pl.E / op.groups < 2) return CAKE_GG_ERR_INVALID_ARG;
    if (!offsets || !workspace || (pl.T > 0 && (!logits || !expert || !weight || !rows || !position))) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(logits, logits_dtype == CAKE_GG_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(expert, 4) || !aligned(weight, 4) ||
        !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(position, 4) || !aligned(workspace, 16))
        return CAKE_GG_ERR_ALIGNMENT;
    if (pl.workspace_bytes != workspace_of(pl) || workspace_bytes < pl.workspace_bytes) return CAKE_GG_ERR_WORKSPACE;
    int sms;
    if ((rc = device_sms(&sms)) != CAKE_GG_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RouteParams p{};
    p.logits = logits;
    p.bias = bias;
    p.expert = expert;
    p.offsets = offsets;
    p.rows = rows;
    p.position = position;
    p.weight = weight;
    p.counts = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(workspace) + kHeader);
    p.T = pl.T;
    p.stride = row_stride;
    p.E = pl.E;
    p.top_k = pl.top_k;
    p.bf16 = logits_dtype == CAKE_GG_BF16;
    p.score = op.score;
    p.groups = op.groups;
    p.top_groups = op.top_groups;
    p.pair = op.group_score == CAKE_GG_GROUP_TOP2;
    p.renormalize = op.renormalize != 0;
    p.scale = op.scale;
    p.block_tokens = pl.block_tokens;
    p.chunk = pl.block_tokens < kRouteChunk ? pl.block_tokens : kRouteChunk;
    p.div_top = uint32_t((uint64_t(1) << 32) / uint32_t(pl.top_k) + ((uint64_t(1) << 32) % uint32_t(pl.top_k) != 0));
    const int32_t size = pl.E / op.groups;
    p.div_group = uint32_t(((1 << 20) + size - 1) / size);
    const size_t shared = route_shared_bytes(pl.E, pl.top_k, p.chunk);
    cudaError_t err = with_experts(pl.E, [&](auto vpl) {
        return launch_route<decltype(vpl)::value>(p, pl.blocks, pl.cluster != 0, shared, s);
    });
    if (err == cudaSuccess && !pl.cluster) err = route_launch(route_number_kernel, p, pl.blocks, kThreads, 0, 1, s);
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

int cake_gg_route_grad(int64_t T, int32_t E, int32_t top_k, int score, int renormalize, float scale, const void *logits,
                       int logits_dtype, int64_t row_stride, const int32_t *expert, const float *d_weight, void *d_logits,
                       void *stream)
{
    int rc = check_sizes(T, E, top_k);
    if (rc == CAKE_GG_OK) rc = check_scores(logits_dtype, row_stride, E, score);
    if (rc != CAKE_GG_OK) return rc;
    if (T == 0) return CAKE_GG_OK;
    if (!logits || !expert || !d_weight || !d_logits) return CAKE_GG_ERR_INVALID_ARG;
    if (!aligned(logits, logits_dtype == CAKE_GG_BF16 ? 2 : 4) || !aligned(d_logits, logits_dtype == CAKE_GG_BF16 ? 2 : 4) ||
        !aligned(expert, 4) || !aligned(d_weight, 4))
        return CAKE_GG_ERR_ALIGNMENT;
    int sms;
    if ((rc = device_sms(&sms)) != CAKE_GG_OK) return rc;
    RouteGradParams p{};
    p.logits = logits;
    p.expert = expert;
    p.d_weight = d_weight;
    p.d_logits = d_logits;
    p.T = T;
    p.stride = row_stride;
    p.E = E;
    p.top_k = top_k;
    p.bf16 = logits_dtype == CAKE_GG_BF16;
    p.score = score;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool whole = score == CAKE_GG_SCORE_SOFTMAX && !p.renormalize;
    const cudaError_t err = !whole ? launch_route_grad(p, s)
                                   : with_experts(E, [&](auto vpl) { return launch_route_grad_whole<decltype(vpl)::value>(p, s); });
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

}  // extern "C"
