// cake_gg_route.cu -- routing to experts: from router logits to each token's
// experts and weights and to the rows in expert order that the grouped products
// take; and the logits' gradient from the weights'.
//
//   s = softmax(l) or sigmoid(l) of a token's E logits
//   experts: the top_k largest by s + bias (by l, which orders as s, without a
//   bias), ties to the lowest index; where experts come in groups only from the
//   top_groups of the largest group scores (a group's largest, or the sum of its
//   two largest)
//   w = s of the chosen, / their sum if asked, * scale
//   rows by expert, then by token
//
// A warp has a token, a lane every 32nd expert; each round takes the largest key
// and the lowest index among its equals by two warp reductions.  A choice by s + bias
// is made in FP32 where that decides it; where two keys lie closer than FP32's error the
// candidates are compared in 64 bits.
//
// Rows are numbered by counting: for each expert a bit per token of the block says
// who chose it, so a token's place among them is a population count, in the
// order of the tokens and the same on every run.  Up to kClusterTokens one cluster of
// blocks does it all, counts read from one another's shared memory; more tokens
// take a kernel that counts (its last block sums over the blocks) and one that
// numbers.
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include <cuda_runtime.h>

#include "../../include/cake_gg.h"
#include "cake_gg_ptx.cuh"

namespace cakegg {
int device_sms(int *sms);   // (cake_gg_capi.cu)
}
using namespace cakegg;

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int32_t kMaxExperts = 1024, kMaxTop = 32, kMaxGroups = 32;
constexpr int64_t kMaxTokens = 1 << 24;
constexpr int64_t kClusterTokens = 1024;       // what one cluster serves
constexpr int kClusterBlocks = 8;
constexpr int kBlockTokens = 1024;             // tokens of a block at most
constexpr int kSms = 152;
constexpr uint64_t kHeader = 256;              // the ticket at byte 4 (byte 0: the status word)
constexpr unsigned kFull = 0xffffffffu;

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *expert, *offsets, *rows, *position;
    float *weight;
    uint32_t *ticket;
    int32_t *counts;          // [block][E]
    int64_t T, stride;
    int32_t E, top_k, bf16, score, groups, top_groups, pair, renormalize, block_tokens;
    uint32_t div_group;       // 2^20 / (E / groups), rounded up: e / (E / groups) for e < 1024
    float scale;
};

__device__ __forceinline__ float load_logit(const RouteParams &p, int64_t t, int32_t e)
{
    const int64_t at = t * p.stride + e;
    return p.bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t *>(p.logits)[at]) << 16) : static_cast<const float *>(p.logits)[at];
}

// Whole numbers that order as the values do, a NaN below all others; 0 is nobody.
__device__ __forceinline__ uint32_t order(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);               // (-0 as 0)
    return v != v ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key <= 1u ? 0x7fc00000u : key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint64_t order(double v)
{
    const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));
    return v != v ? 1ull : b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }
__device__ __forceinline__ double sigmoid(double l) { return 1.0 / (1.0 + exp(-l)); }

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kFull, uint32_t(v >> 32));
    return uint64_t(hi) << 32 | __reduce_max_sync(kFull, uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
}

// A lane's N values, summed as a tree (with the warp's five levels at most ten
// roundings on the way of any of them).
template <int N, typename F>
__device__ __forceinline__ F tree_sum(F (&v)[N])
{
#pragma unroll
    for (int d = N / 2; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < d; ++i) v[i] += v[i + d];
    return v[0];
}

// Scores in F of the lane's experts from its logits; and the softmax's maximum and sum.
template <int VPL, typename F>
__device__ __forceinline__ void scores(const RouteParams &p, const float (&l)[VPL], F (&s)[VPL], int lane, float *most, F *sum)
{
    if (p.score == CAKE_GG_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = sigmoid(F(l[i]));
        return;
    }
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    F e[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = e[i] = i * 32 + lane < p.E ? exp(F(l[i]) - F(m)) : F(0);
    const F total = warp_sum(tree_sum(e));
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = s[i] / total;
    *most = m, *sum = total;
}

// The lane's experts that stay where only the groups of the largest scores do, by
// keys of the experts (0: nobody) and the values that they stand for.  *close: FP32
// cannot tell the last group that stays from the first that does not (`error`:
// relative, of a score, which is one at most; 0 where keys are exact).
template <int VPL, typename K, typename V>
__device__ __forceinline__ void keep_groups(const RouteParams &p, K (&key)[VPL], const V (&value)[VPL], int lane, float error, bool *close)
{
    const int32_t size = p.E / p.groups;
    K mine = 0;                                                  // lane g: the score of group g
    float mine_v = 0.0f, mine_m = 0.0f;                          // (and what it was added up from)
    for (int32_t g = 0; g < p.groups; ++g) {
        K best = 0;
        int at = -1;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = i * 32 + lane;
            if (e >= g * size && e < (g + 1) * size && key[i] > best) best = key[i], at = i;
        }
        K most;
        if constexpr (sizeof(K) == 4) most = __reduce_max_sync(kFull, best);
        else most = warp_max(best);
        if (!p.pair) {
            if (lane == g) {
                mine = most;
                if constexpr (sizeof(K) == 4) mine_v = value_of(most), mine_m = fabsf(mine_v);
            }
            continue;
        }
        // the largest two: the first lane that has the largest puts in its next
        const int owner = __ffs(int(__ballot_sync(kFull, best == most))) - 1;
        V v0 = 0, v1 = 0;
        K next = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = i * 32 + lane;
            if (i == at) v0 = value[i];
            if (e >= g * size && e < (g + 1) * size && !(lane == owner && i == at) && key[i] > next) next = key[i], v1 = value[i];
        }
        K second;
        if constexpr (sizeof(K) == 4) second = __reduce_max_sync(kFull, next);
        else second = warp_max(next);
        const int other = __ffs(int(__ballot_sync(kFull, next == second))) - 1;
        v0 = __shfl_sync(kFull, v0, owner);
        v1 = __shfl_sync(kFull, v1, other);
        if (lane == g) mine = order(v0 + v1), mine_v = float(v0 + v1), mine_m = fabsf(float(v0)) + fabsf(float(v1));
    }
    // a group's rank: how many are larger, or as large and before it
    int rank = 0;
    for (int32_t g = 0; g < p.groups; ++g) {
        const K o = __shfl_sync(kFull, mine, g);
        rank += o > mine || (o == mine && g < lane);
    }
    const unsigned kept = __ballot_sync(kFull, lane < p.groups && rank < p.top_groups);
    if (error > 0.0f && p.top_groups < p.groups) {
        // the last that is in and the first that is out
        const int in = __ffs(int(__ballot_sync(kFull, lane < p.groups && rank == p.top_groups - 1))) - 1;
        const int out = __ffs(int(__ballot_sync(kFull, lane < p.groups && rank == p.top_groups))) - 1;
        const float a = __shfl_sync(kFull, mine_v, in), b = __shfl_sync(kFull, mine_v, out);
        const float m = __shfl_sync(kFull, mine_m, in) + __shfl_sync(kFull, mine_m, out);
        // (two scores on either side at most)
        *close = !(a - b > error * 4.0f + m * 0x1p-22f);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const uint32_t e = uint32_t(i * 32 + lane);
        if (!(kept >> (e * p.div_group >> 20) & 1u)) key[i] = 0;
    }
}

// The next largest key of the warp and its expert, taken out of `key`.
template <int VPL, typename K>
__device__ __forceinline__ int32_t take(K (&key)[VPL], int lane, K *most)
{
    K best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = key[i] > best ? key[i] : best;
    if constexpr (sizeof(K) == 4) *most = __reduce_max_sync(kFull, best);
    else *most = warp_max(best);
    uint32_t at = 0x7fffffffu;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == *most) at = uint32_t(i * 32 + lane);
    at = __reduce_min_sync(kFull, at);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (i * 32 + lane == int(at)) key[i] = 0;
    return int32_t(at);
}

// Everything in 64 bits, for a token whose FP32 keys leave the choice open: lane
// j gets the j-th expert.
template <int VPL>
__device__ __noinline__ int32_t choose_in_64_bits(const RouteParams &p, int64_t t, int lane)
{
    float l[VPL];
    double s[VPL], by[VPL], sum;
    uint64_t key[VPL];
    float most;
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = i * 32 + lane < p.E ? load_logit(p, t, i * 32 + lane) : __uint_as_float(0xff800000u);
    scores(p, l, s, lane, &most, &sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t e = i * 32 + lane;
        by[i] = p.bias && e < p.E ? s[i] + double(p.bias[e]) : s[i];
        key[i] = e < p.E ? order(by[i]) : 0;
    }
    if (p.groups > 1) {
        bool close = false;
        keep_groups(p, key, by, lane, 0.0f, &close);
    }
    if (!p.bias) {
        // (within the groups that stay by the logits)
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = key[i] ? uint64_t(order(l[i])) << 32 : 0;
    }
    int32_t mine = 0;
    for (int j = 0; j < p.top_k; ++j) {
        uint64_t best;
        const int32_t e = take(key, lane, &best);
        if (lane == j) mine = e;
    }
    return mine;
}

// FP32's error of a score, relative to it: the exponential is off by two units in
// its last place (2^-22), a sum or a quotient by 2^-24; the softmax's argument l - max
// rounds to 2^-24 of itself (x e^-x <= 0.37 bounds what that is of the largest
// score), its sum has ten roundings and its terms' 2^-22.  s + bias rounds by 2^-24 of
// itself.
constexpr float kSigmoidError = 0x1p-21f, kSoftmaxError = 0x1p-19f;

// The experts of token t: lane j < top_k gets the j-th, and of it the logit, or
// where the softmax is not renormalised the score.
template <int VPL>
__device__ __forceinline__ int32_t choose(const RouteParams &p, int64_t t, int lane, float *of_it)
{
    float l[VPL];
    uint32_t key[VPL];
    float most = 0.0f, sum = 1.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = i * 32 + lane < p.E ? load_logit(p, t, i * 32 + lane) : __uint_as_float(0xff800000u);
    const bool softmax = p.score == CAKE_GG_SCORE_SOFTMAX;
    const bool by_score = p.bias || (p.pair && p.groups > 1);
    const float error = softmax ? kSoftmaxError : kSigmoidError;
    bool open = false;
    if (by_score || (softmax && !p.renormalize)) {
        float s[VPL];
        scores(p, l, s, lane, &most, &sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = i * 32 + lane;
            if (p.bias && e < p.E) s[i] += p.bias[e];
            key[i] = e < p.E ? order(s[i]) : 0;
        }
        if (by_score && p.groups > 1) keep_groups(p, key, s, lane, error, &open);
    }
    if (!p.bias) {
        const bool grouped = by_score;                           // (what is out has the key 0)
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = i * 32 + lane < p.E && !(grouped && key[i] == 0) ? order(l[i]) : 0;
        if (p.groups > 1 && !grouped) keep_groups(p, key, l, lane, 0.0f, &open);
    }
    int32_t mine = 0;
    uint32_t mine_key = 0;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best;
        const int32_t e = take(key, lane, &best);
        if (lane == j) mine = e, mine_key = best;
    }
    if (p.bias && !open) {
        // Is each of the chosen, and the first that is not, further from the one before
        // than FP32's error?  Equal logits with equal biases are equal, whatever it is.
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
        const uint32_t after_key = __reduce_max_sync(kFull, best);
        const float k = value_of(mine_key), b = p.bias[mine], ml = load_logit(p, t, mine), s = k - b;
        const float far = error * (softmax ? 0.37f * 0x1p-4f : 0.0f);
        float k1 = __shfl_down_sync(kFull, k, 1);
        const float s1 = __shfl_down_sync(kFull, s, 1), l1 = __shfl_down_sync(kFull, ml, 1), b1 = __shfl_down_sync(kFull, b, 1);
        const bool apart = k - k1 > error * (fabsf(s) + fabsf(s1)) + far + 0x1p-22f * (fabsf(k) + fabsf(b));
        open = __any_sync(kFull, lane + 1 < p.top_k && !apart && !(ml == l1 && b == b1));
        // (the one after may have any score up to one)
        k1 = value_of(after_key);
        const float line = k - (2.0f * error + 0x1p-22f * (fabsf(k) + fabsf(b) + 1.0f));
        const bool near = lane == p.top_k - 1 && after_key != 0 && !(k1 < line);
        if (__any_sync(kFull, near)) {
            // all that come near the last chosen have to be its equals
            const float line_all = __shfl_sync(kFull, line, p.top_k - 1), l_all = __shfl_sync(kFull, ml, p.top_k - 1),
                        b_all = __shfl_sync(kFull, b, p.top_k - 1);
            bool other = false;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (key[i] != 0 && !(value_of(key[i]) < line_all)) other |= !(l[i] == l_all && p.bias[i * 32 + lane] == b_all);
            open = open || __any_sync(kFull, other);
        }
    }
    if (open) mine = choose_in_64_bits<VPL>(p, t, lane);
    *of_it = 0.0f;
    if (lane < p.top_k) {
        const float ml = load_logit(p, t, mine);
        *of_it = softmax && !p.renormalize ? expf(ml - most) / sum : ml;
    }
    return mine;
}

// The weights of a token's chosen experts from what choose() gave each lane: the
// score itself where the softmax is not renormalised, else the logit.
__device__ __forceinline__ float finish(const RouteParams &p, float v, int lane)
{
    const bool in = lane < p.top_k;
    if (p.score == CAKE_GG_SCORE_SOFTMAX) {
        if (!p.renormalize) return v * p.scale;
        // the softmax over the chosen; where all of them are -inf, nothing
        const float m = warp_max(in ? v : __uint_as_float(0xff800000u));
        const float e = in && m > __uint_as_float(0xff800000u) ? expf(v - m) : in && v != v ? v : 0.0f;
        const float sum = warp_sum(e);
        return sum == 0.0f ? 0.0f : e / sum * p.scale;
    }
    if (!p.renormalize) return in ? sigmoid(v) * p.scale : 0.0f;
    // where all chosen logits are far below zero their sigmoids vanish, not their
    // ratios: e^(l - m) / (1 + e^l) with m the largest of them, if below zero
    const float m = fminf(warp_max(in ? v : __uint_as_float(0xff800000u)), 0.0f);
    float s = 0.0f;
    if (in) s = v > 0.0f || v != v ? sigmoid(v) : m > __uint_as_float(0xff800000u) ? expf(v - m) / (1.0f + expf(v)) : 0.0f;
    const float sum = warp_sum(s);
    return sum == 0.0f ? 0.0f : s / sum * p.scale;
}

// Words of a block's bits of an expert, one more than tokens / 32 where that is even:
// experts' first words then lie in different banks.
__host__ __device__ constexpr int bit_words(int tokens) { return ((tokens + 31) / 32) | 1; }

struct Shared {
    uint32_t *bits;       // [E][words] tokens of the block that chose the expert
    int32_t *counts;      // [E]
    int32_t *base;        // [E]
    uint16_t *chosen;     // [token][top_k]
};
__device__ __forceinline__ Shared shared_of(uint8_t *raw, const RouteParams &p)
{
    Shared s;
    s.bits = reinterpret_cast<uint32_t *>(raw);
    s.counts = reinterpret_cast<int32_t *>(s.bits + p.E * bit_words(p.block_tokens));
    s.base = s.counts + p.E;
    s.chosen = reinterpret_cast<uint16_t *>(s.base + p.E);
    return s;
}
__host__ __device__ size_t shared_bytes(int32_t E, int32_t top_k, int block_tokens)
{
    return size_t(E) * bit_words(block_tokens) * 4 + size_t(E) * 8 + (size_t(block_tokens) * top_k * 2 + 15) / 16 * 16;
}

// The block's tokens [t0, t0 + n): their experts and weights, and who chose whom.
template <int VPL>
__device__ __forceinline__ void choose_all(const RouteParams &p, const Shared &s, int64_t t0, int n)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, words = bit_words(p.block_tokens);
    for (int i = threadIdx.x; i < p.E * words; i += kThreads) s.bits[i] = 0;
    __syncthreads();
    for (int i = warp; i < n; i += kWarps) {
        float v;
        const int32_t e = choose<VPL>(p, t0 + i, lane, &v);
        const float w = finish(p, v, lane);
        if (lane < p.top_k) {
            const int64_t at = (t0 + i) * p.top_k + lane;
            p.expert[at] = e;
            p.weight[at] = w;
            s.chosen[i * p.top_k + lane] = uint16_t(e);
            atomicOr(&s.bits[e * words + (i >> 5)], 1u << (i & 31));
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        int32_t c = 0;
        for (int w = 0; w < words; ++w) c += __popc(s.bits[e * words + w]);
        s.counts[e] = c;
    }
}

// A token's place among those of the block that chose the same expert.
__device__ __forceinline__ int32_t place(const Shared &s, int words, int32_t e, int i)
{
    const uint32_t *b = s.bits + e * words;
    int32_t r = __popc(b[i >> 5] & ((1u << (i & 31)) - 1u));
    for (int w = 0; w < i >> 5; ++w) r += __popc(b[w]);
    return r;
}

// Exclusive sums over v of thread e (E <= kThreads), in place of each; the total to all.
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t *total)
{
    __shared__ int32_t sums[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(kFull, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int32_t w = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(kFull, w, d);
        if (lane >= d) w += o;
    }
    const int32_t before = warp ? __shfl_sync(kFull, w, warp - 1) : 0;
    *total = __shfl_sync(kFull, w, 31);
    return before + inc - v;
}

template <int VPL>
__global__ void __launch_bounds__(kThreads)
    route_cluster_kernel(const RouteParams p)
{
    extern __shared__ __align__(16) uint8_t raw[];
    const Shared s = shared_of(raw, p);
    grid_dependency_wait();
    grid_launch_dependents();
    const int rank = int(blockIdx.x), blocks = int(gridDim.x), e = threadIdx.x, words = bit_words(p.block_tokens);
    const int64_t t0 = int64_t(rank) * p.block_tokens;
    const int n = int(t0 >= p.T ? 0 : p.T - t0 < p.block_tokens ? p.T - t0 : p.block_tokens);
    choose_all<VPL>(p, s, t0, n);
    if (blocks > 1) cluster_sync_all();
    else __syncthreads();
    int32_t all = 0, before = 0;
    if (e < p.E) {
        const uint32_t mine = smem_u32(&s.counts[e]);
        for (int b = 0; b < blocks; ++b) {
            int32_t c;
            if (b == rank) c = s.counts[e];
            else asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(map_to_cta(mine, uint32_t(b))) : "memory");
            if (b < rank) before += c;
            all += c;
        }
    }
    int32_t total;
    const int32_t first = block_scan(all, &total);
    if (e < p.E) {
        s.base[e] = first + before;
        if (rank == 0) p.offsets[e] = first;
    }
    if (rank == 0 && e == 0) p.offsets[p.E] = total;
    __syncthreads();
    for (int i = threadIdx.x; i < n * p.top_k; i += kThreads) {
        const int32_t x = s.chosen[i], token = i / p.top_k, row = s.base[x] + place(s, words, x, token);
        p.position[t0 * p.top_k + i] = row;
        p.rows[row] = int32_t(t0) + token;
    }
    if (blocks > 1) cluster_sync_all();                          // the others may still read this one's counts
}

// Experts, weights and places within the block (to `position`); the last block
// turns the blocks' counts into where their rows of an expert begin.
template <int VPL>
__global__ void __launch_bounds__(kThreads)
    route_count_kernel(const RouteParams p)
{
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ bool last;
    const Shared s = shared_of(raw, p);
    grid_dependency_wait();
    grid_launch_dependents();
    const int words = bit_words(p.block_tokens), blocks = int(gridDim.x);
    const int64_t t0 = int64_t(blockIdx.x) * p.block_tokens;
    const int n = int(p.T - t0 < p.block_tokens ? p.T - t0 : p.block_tokens);
    choose_all<VPL>(p, s, t0, n);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kThreads) p.counts[int64_t(blockIdx.x) * p.E + e] = s.counts[e];
    for (int i = threadIdx.x; i < n * p.top_k; i += kThreads)
        p.position[t0 * p.top_k + i] = place(s, words, s.chosen[i], i / p.top_k);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.ticket, 1u) + 1u == gridDim.x;
    __syncthreads();
    if (!last) return;
    __threadfence();
    // `parts` threads an expert, each a run of blocks: their sums, then the runs of
    // each expert and the experts before it
    int parts = 1;
    while (parts * 2 * p.E <= kThreads) parts *= 2;
    const int e = int(threadIdx.x) % p.E, part = int(threadIdx.x) / p.E, run = (blocks + parts - 1) / parts;
    const int b0 = part * run, b1 = min(b0 + run, blocks);
    const bool mine = part < parts;
    int32_t sum = 0;
    if (mine) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += __ldcg(&p.counts[int64_t(b) * p.E + e]);
    }
    int32_t *sums = reinterpret_cast<int32_t *>(raw + shared_bytes(p.E, p.top_k, p.block_tokens));   // [part][expert]
    if (mine) sums[part * p.E + e] = sum;
    __syncthreads();
    int32_t all = 0, before = 0;
    if (mine)
        for (int q = 0; q < parts; ++q) {
            const int32_t c = sums[q * p.E + e];
            if (q < part) before += c;
            all += c;
        }
    int32_t total;
    const int32_t first = block_scan(part == 0 ? all : 0, &total);
    if (part == 0) {
        s.base[e] = first;
        p.offsets[e] = first;
    }
    if (threadIdx.x == 0) p.offsets[p.E] = total, *p.ticket = 0;
    __syncthreads();
    if (mine) {
        int32_t at = s.base[e] + before;
#pragma unroll 8
        for (int b = b0; b < b1; ++b) {
            int32_t *c = &p.counts[int64_t(b) * p.E + e];
            const int32_t v = __ldcg(c);
            __stcg(c, at);
            at += v;
        }
    }
}

__global__ void __launch_bounds__(256)
    route_number_kernel(const RouteParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.T * p.top_k) return;
    const int32_t t = int32_t(i / p.top_k);
    const int32_t row = p.position[i] + p.counts[int64_t(t / p.block_tokens) * p.E + p.expert[i]];
    p.position[i] = row;
    p.rows[row] = t;
}

// ---------------------------------------------------------------- backward

struct GradParams {
    const void *logits;
    const int32_t *expert;
    const float *d_weight;
    void *d_logits;
    int64_t T, stride;
    int32_t E, top_k, bf16, score, renormalize;
    float scale;
};

// A warp a token.  With g the weights' gradient times the scale:
//   softmax, renormalised: w = softmax over the chosen, dl_j = w_j (g_j - sum g w)
//   softmax:               dl_e = p_e ([e chosen] g_e - sum g p), over all experts
//   sigmoid, renormalised: r = s / S of the chosen, dl_j = r_j (1 - s_j) (g_j - sum g r)
//   sigmoid:               dl_j = g_j s_j (1 - s_j)
// and zeros elsewhere.  1 - s is computed as the sigmoid of -l.
template <int VPL>
__global__ void __launch_bounds__(256)
    route_grad_kernel(const GradParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const bool in = lane < p.top_k;
    RouteParams r{};
    r.logits = p.logits, r.stride = p.stride, r.bf16 = p.bf16, r.E = p.E, r.score = p.score;
    const bool whole = p.score == CAKE_GG_SCORE_SOFTMAX && !p.renormalize;
    const float ninf = __uint_as_float(0xff800000u);
    int32_t e = in ? p.expert[t * p.top_k + lane] : -1;
    if (e < 0 || e >= p.E) e = -1;                               // (nobody: nothing is read or written for it)
    const float g = e >= 0 ? p.d_weight[t * p.top_k + lane] * p.scale : 0.0f;
    float s[VPL], most = 0.0f, sum = 1.0f;
    if (whole) {
        float l[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = i * 32 + lane < p.E ? load_logit(r, t, i * 32 + lane) : ninf;
        scores(r, l, s, lane, &most, &sum);
    }
    const float ml = e >= 0 ? load_logit(r, t, e) : ninf;
    float d = 0.0f, inner = 0.0f;
    if (whole) {
        d = e >= 0 ? g * (expf(ml - most) / sum) : 0.0f;
        inner = warp_sum(d);
    } else if (p.score == CAKE_GG_SCORE_SOFTMAX) {
        const float m = warp_max(ml);
        const float x = e >= 0 && m > ninf ? expf(ml - m) : 0.0f;
        const float total = warp_sum(x), w = total == 0.0f ? 0.0f : x / total;
        inner = warp_sum(g * w);
        d = w * (g - inner);
    } else if (p.renormalize) {
        const float m = fminf(warp_max(ml), 0.0f);
        float x = 0.0f;
        if (e >= 0) x = ml > 0.0f || ml != ml ? sigmoid(ml) : m > ninf ? expf(ml - m) / (1.0f + expf(ml)) : 0.0f;
        const float total = warp_sum(x), w = total == 0.0f ? 0.0f : x / total;
        inner = warp_sum(g * w);
        d = w * sigmoid(-ml) * (g - inner);
    } else if (e >= 0) d = g * sigmoid(ml) * sigmoid(-ml);
    // the lane's experts of the row, and what the lanes of the chosen have for them
    float out[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) out[i] = whole ? -s[i] * inner : 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
        const int32_t x = __shfl_sync(kFull, e, j);
        const float v = __shfl_sync(kFull, d, j);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (x == i * 32 + lane) out[i] += v;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t x = i * 32 + lane;
        if (x < p.E) {
            if (p.bf16) static_cast<uint16_t *>(p.d_logits)[t * p.E + x] = uint16_t(pack_bf16x2(out[i], 0.0f) & 0xffffu);
            else static_cast<float *>(p.d_logits)[t * p.E + x] = out[i];
        }
    }
}

// ---------------------------------------------------------------- host

bool pdl_enabled()
{
    const char *v = std::getenv("CAKE_GG_PDL");
    return !(v && std::atoi(v) == 0);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Calls f with a constant: the experts of a lane, a power of two.
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

template <typename Kernel, typename Params>
cudaError_t launch(Kernel kernel, const Params &p, int64_t blocks, int threads, size_t shared, int cluster, cudaStream_t stream)
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
    if (shared > 48 << 10) {
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shared));
        if (err != cudaSuccess) return err;
    }
    cfg.gridDim = dim3(unsigned(blocks), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = unsigned(na);
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

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

// Blocks and their tokens: as few blocks of one cluster as have a warp for a token,
// or one for each multiprocessor.
void choose_blocks(cake_gg_route_plan_t *pl)
{
    const int64_t T = pl->T;
    pl->cluster = T <= kClusterTokens;
    int64_t blocks = pl->cluster ? (T + kWarps - 1) / kWarps : kSms;
    if (pl->cluster && blocks > kClusterBlocks) blocks = kClusterBlocks;
    if (blocks < 1) blocks = 1;
    int64_t per = (T + blocks - 1) / blocks;
    if (per > kBlockTokens) per = kBlockTokens;
    if (per < 1) per = 1;
    pl->block_tokens = int32_t(per);
    pl->blocks = int32_t(T == 0 ? 1 : (T + per - 1) / per);
}

uint64_t workspace_of(const cake_gg_route_plan_t &pl) { return kHeader + (pl.cluster ? 0 : uint64_t(pl.blocks) * uint64_t(pl.E) * 4); }

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
    p.ticket = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + 4);
    p.counts = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + kHeader);
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
    const int32_t size = pl.E / op.groups;
    p.div_group = uint32_t(((1 << 20) + size - 1) / size);
    const size_t shared = shared_bytes(pl.E, pl.top_k, pl.block_tokens);
    cudaError_t err = with_experts(pl.E, [&](auto vpl) {
        constexpr int VPL = decltype(vpl)::value;
        return pl.cluster ? launch(route_cluster_kernel<VPL>, p, pl.blocks, kThreads, shared, pl.blocks, s)
                          : launch(route_count_kernel<VPL>, p, pl.blocks, kThreads, shared + kThreads * 4, 1, s);
    });
    if (err == cudaSuccess && !pl.cluster) err = launch(route_number_kernel, p, (pl.T * pl.top_k + 255) / 256, 256, 0, 1, s);
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
    GradParams p{};
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
    const cudaError_t err = with_experts(E, [&](auto vpl) {
        return launch(route_grad_kernel<decltype(vpl)::value>, p, (T + 7) / 8, 256, 0, 1, static_cast<cudaStream_t>(stream));
    });
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

}  // extern "C"
