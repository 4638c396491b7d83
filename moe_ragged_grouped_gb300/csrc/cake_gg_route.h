// cake_gg_route.h -- internal interface of the routing: parameters, sizes and
// launches shared by the C entry points (cake_gg_route.cu) and the translation
// units that hold the kernels of some experts a lane (a power of two).
#pragma once

#include <cstdint>
#include <cstdlib>
#include <type_traits>

#include <cuda_runtime.h>

#include "../../include/cake_gg.h"

namespace cakegg {

int device_sms(int *sms);   // (cake_gg_capi.cu)

constexpr int kRouteThreads = 1024;            // of a block that routes up to kRouteNarrow experts, half beyond
constexpr int32_t kRouteNarrow = 256;
constexpr int32_t kRouteMaxExperts = 1024;
constexpr int32_t kRouteMaxTop = 32;
constexpr int kRouteChunk = 1024;              // tokens that a block numbers at a time, at most
constexpr size_t kRouteSharedDefault = 48 << 10;   // what a launch may take without asking

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *expert, *offsets, *rows, *position;
    float *weight;
    uint16_t *counts;         // [block][E rounded up to 8]
    int64_t T, stride;
    int32_t E, top_k, bf16, score, groups, top_groups, pair, renormalize, block_tokens, chunk;
    uint32_t div_top;         // 2^32 / top_k, rounded up
    uint32_t div_group;       // 2^20 / (E / groups), rounded up: e / (E / groups) for e < 1024
    float scale;
};

struct RouteGradParams {
    const void *logits;
    const int32_t *expert;
    const float *d_weight;
    void *d_logits;
    int64_t T, stride;
    int32_t E, top_k, bf16, score, renormalize;
    float scale;
};


// Words of a block's bits of an expert, one more than tokens / 32 where that is even:
// experts' first words then lie in different banks.
__host__ __device__ constexpr int bit_words(int tokens) { return ((tokens + 31) / 32) | 1; }
// Shared memory of a block: bits, counts, where rows begin, what was chosen.
constexpr size_t route_shared_bytes(int32_t E, int32_t top_k, int chunk)
{
    return size_t(E) * bit_words(chunk) * 4 + size_t(E) * 8 + (size_t(chunk) * top_k * 2 + 15) / 16 * 16;
}

__host__ __device__ constexpr int32_t count_pitch(int32_t E) { return (E + 7) / 8 * 8; }

// Exclusive sums over the threads' v (kRouteThreads of them at most), and the total to all.
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t *total)
{
    __shared__ int32_t sums[kRouteThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int32_t w = lane < int(blockDim.x >> 5) ? sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += o;
    }
    const int32_t before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    *total = __shfl_sync(0xffffffffu, w, 31);
    return before + inc - v;
}

inline bool pdl_enabled()
{
    const char *v = std::getenv("CAKE_GG_PDL");
    return !(v && std::atoi(v) == 0);
}

template <typename Kernel, typename Params>
cudaError_t route_launch(Kernel kernel, const Params &p, int64_t blocks, int threads, size_t shared, int cluster, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = unsigned(cluster);
        attr[na].val.clusterDim.y = 1;
        attr[na++].val.clusterDim.z = 1;
    }
    if (pdl_enabled()) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = unsigned(na);
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The kernels of VPL experts a lane.
template <int VPL>
cudaError_t launch_route(const RouteParams &p, int blocks, bool cluster, size_t shared, cudaStream_t stream);
template <int VPL>
cudaError_t launch_route_grad_whole(const RouteGradParams &p, cudaStream_t stream);   // softmax, not renormalised
cudaError_t launch_route_grad(const RouteGradParams &p, cudaStream_t stream);         // the others: the chosen alone

// Calls f with a constant: the experts of a lane.
template <typename F>
auto with_experts(int32_t E, F f)
{
    if (E <= 32) return f(std::integral_constant<int, 1>());
    if (E <= 64) return f(std::integral_constant<int, 2>());
    if (E <= 128) return f(std::integral_constant<int, 4>());
    if (E <= 256) return f(std::integral_constant<int, 8>());
    if (E <= 512) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace cakegg
