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
// take a kernel that counts and one that numbers.
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
constexpr int64_t kMaxTokens = 1 << 23;        // (a block's tokens are below 2^16)
constexpr int64_t kClusterTokens = 256;        // what one cluster serves
constexpr int kClusterBlocks = 8;
constexpr int kChunk = 1024;                   // tokens that a block numbers at a time, at most
constexpr int kSms = 152;
constexpr uint64_t kHeader = 256;              // (as in the products' workspaces; its status word stays 0)
constexpr unsigned kFull = 0xffffffffu;

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

// The experts of token t by whole FP32 keys: lane j < top_k gets the j-th.
template <int VPL>
__device__ __noinline__ int32_t choose_by_keys(const RouteParams &p, int64_t t, int lane)
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
    if (by_score) {
        float s[VPL];
        scores(p, l, s, lane, &most, &sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = i * 32 + lane;
            if (p.bias && e < p.E) s[i] += p.bias[e];
            key[i] = e < p.E ? order(s[i]) : 0;
        }
        if (p.groups > 1) keep_groups(p, key, s, lane, error, &open);
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
    return open ? choose_in_64_bits<VPL>(p, t, lane) : mine;
}

// A lane's keys in descending order (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&k)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j <= N - 1 - q; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (p * 2) == (i + j + q) / (p * 2)) {
                        const uint32_t a = max(k[i + j], k[i + j + q]), b = min(k[i + j], k[i + j + q]);
                        k[i + j] = a, k[i + j + q] = b;
                    }
}

// Packed keys of up to N experts: the upper bits of a key, which order as values
// do, and below them the expert, counted down, so that one maximum gives both and
// equals go to the lowest.  Experts beyond E are 0.
template <int N>
struct Packed {
    static constexpr uint32_t kMask = uint32_t(N) - 1;           // (N a power of two)
    // (a NaN without a sign above infinity, one with below: the caller looks at the largest)
    static __device__ __forceinline__ uint32_t of(float v, int32_t e)
    {
        const uint32_t b = __float_as_uint(v + 0.0f);           // (-0 as 0)
        return ((b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u)) & ~kMask) | (kMask - uint32_t(e));
    }
    static __device__ __forceinline__ int32_t expert(uint32_t key) { return int32_t(kMask - (key & kMask)); }
    // the largest value that a key may stand for
    static __device__ __forceinline__ float most(uint32_t key) { return value_of(key | kMask); }
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504f;
// How far scores by approximate instructions may be off, of the value: the argument
// of the exponential rounds twice to 2^-24 of itself, which is 88 log2(e) at most
// before it vanishes and counts e^-x x <= 0.37 times of the largest value, the
// rest is 2^-21.
constexpr float kFastError = 0x1p-19f;

// Steps of a sum or maximum over the lanes below top_k (the others hold nothing).
template <typename Op>
__device__ __forceinline__ float over_chosen(const RouteParams &p, float v, Op op)
{
    for (int d = 16; d; d >>= 1)
        if (d < p.top_k) v = op(v, __shfl_xor_sync(kFull, v, d));
    return __shfl_sync(kFull, v, 0);
}

template <int VPL>
__device__ __forceinline__ void load_logits(const RouteParams &p, int64_t t, int lane, float (&l)[VPL])
{
    const float ninf = __uint_as_float(0xff800000u);
    if (p.bf16) {
        const uint16_t *row = static_cast<const uint16_t *>(p.logits) + t * p.stride + lane;
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = i * 32 + lane < p.E ? __uint_as_float(uint32_t(row[i * 32]) << 16) : ninf;
    } else {
        const float *row = static_cast<const float *>(p.logits) + t * p.stride + lane;
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = i * 32 + lane < p.E ? row[i * 32] : ninf;
    }
}

// The experts of token t: lane j < top_k gets the j-th, and of it the logit, or
// where the softmax is not renormalised the score.
//
// A first pass finds candidates by packed keys of scores from approximate
// instructions; then the scores of the candidates alone are computed in FP32, one
// a lane.  Where those are further apart than FP32's error, and the last chosen
// from all that the candidate after it may stand for, the choice is certain; else
// all that may be among the chosen are compared in 64 bits, one a lane, and where
// these are more than a warp has lanes, or groups are as near, or NaNs are among
// them, it is made again by whole keys.  (All scores in FP32 and whole keys, of which each
// round takes a maximum and a minimum of indices, took 50 us for 16384 x 256.)
template <int VPL>
__device__ __forceinline__ int32_t choose(const RouteParams &p, int64_t t, int lane, const float (&l)[VPL], float *of_it)
{
    using Keys = Packed<VPL * 32>;
    const bool softmax = p.score == CAKE_GG_SCORE_SOFTMAX, by_score = p.bias || (p.pair && p.groups > 1);
    const float ninf = __uint_as_float(0xff800000u);
    uint32_t key[VPL];
    float most = 0.0f, sum = 1.0f;
    if (softmax && (by_score || !p.renormalize)) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
        most = warp_max(m);
        float e[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) e[i] = exp2_fast((l[i] - most) * kLog2e);
        sum = warp_sum(tree_sum(e));
    }
    // the score of a logit in FP32, of a candidate
    auto score_of = [&](float v) { return softmax ? expf(v - most) / sum : sigmoid(v); };
    const float error = softmax ? kSoftmaxError : kSigmoidError;
    bool open = false;
    if (by_score) {
        const float over = softmax ? rcp_fast(sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = i * 32 + lane;
            const float s = softmax ? exp2_fast((l[i] - most) * kLog2e) * over : rcp_fast(1.0f + exp2_fast(l[i] * -kLog2e));
            key[i] = e < p.E ? Keys::of(p.bias ? s + p.bias[e] : s, e) : 0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = i * 32 + lane < p.E ? Keys::of(l[i], i * 32 + lane) : 0;
    }
    unsigned kept = kFull;
    if (p.groups > 1) {
        // each group's largest two
        const int32_t size = p.E / p.groups;
        uint32_t first = 0, second = 0;                          // lane g: those of group g
        auto group = [&](int g, uint32_t a, uint32_t b) {        // from each lane's largest two
            const uint32_t m1 = __reduce_max_sync(kFull, a);
            if (lane == g) first = m1;
            if (p.pair) {
                const uint32_t m2 = __reduce_max_sync(kFull, a == m1 ? b : a);
                if (lane == g) second = m2;
            }
        };
        if (size % 32 == 0) {                                    // whole registers
            const int per = size / 32;
            uint32_t a = 0, b = 0;
            int in = 0, g = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                b = max(b, min(a, key[i]));
                a = max(a, key[i]);
                if (++in == per && g < p.groups) {
                    group(g++, a, b);
                    a = b = 0, in = 0;
                }
            }
        } else {
            for (int g = 0; g < p.groups; ++g) {
                uint32_t a = 0, b = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    const int32_t e = i * 32 + lane;
                    const uint32_t k = e >= g * size && e < (g + 1) * size ? key[i] : 0;
                    b = max(b, min(a, k));
                    a = max(a, k);
                }
                group(g, a, b);
            }
        }
        // a group's score: of the experts found, in FP32 (which are its largest for certain
        // unless another comes as near as the line below allows)
        float v = ninf, m = 0.0f, slack = 0.0f;
        if (lane < p.groups) {
            const int32_t e1 = Keys::expert(first), e2 = Keys::expert(second);
            const float l1 = load_logit(p, t, e1);
            float k1 = by_score ? score_of(l1) : l1;
            if (p.bias) k1 += p.bias[e1];
            v = k1, m = fabsf(k1), slack = Keys::most(first) - k1;
            if (p.pair) {
                float k2 = score_of(load_logit(p, t, e2));
                if (p.bias) k2 += p.bias[e2];
                v += k2, m += fabsf(k2), slack += Keys::most(second) - k2;
            }
            // (how much more than v the group's score may be: a packed key's lower bits)
            slack = fmaxf(slack, 0.0f);
        }
        // a group's rank: how many are larger, or as large and before it
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float o = __shfl_sync(kFull, v, g);
            rank += o > v || (o == v && g < lane);
        }
        kept = __ballot_sync(kFull, lane < p.groups && rank < p.top_groups);
        // certain where every group that stays is above every one that does not
        const bool in = kept >> lane & 1u, out = lane < p.groups && !in;
        const float worst = __uint_as_float(0x7f800000u);
        float low = in ? v : worst, high = out ? v + slack : ninf, size_of = m;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            low = fminf(low, __shfl_xor_sync(kFull, low, d));
            high = fmaxf(high, __shfl_xor_sync(kFull, high, d));
            size_of = fmaxf(size_of, __shfl_xor_sync(kFull, size_of, d));
        }
        const bool nan = __any_sync(kFull, lane < p.groups && !(v - v == 0.0f));   // (NaNs and infinities go the long way)
        open = nan || (p.top_groups < p.groups && !(low - high > (by_score ? 4.0f * (error + kFastError) : 0.0f) + size_of * 0x1p-21f));
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const uint32_t e = uint32_t(i * 32 + lane);
            if (!(kept >> (e * p.div_group >> 20) & 1u)) key[i] = 0;
        }
        if (by_score && !p.bias) {
            // (within the groups that stay by the logits)
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (key[i]) key[i] = Keys::of(l[i], i * 32 + lane);
        }
    }
    // the chosen, and the one after them: the largest of the lanes' first, whose lane
    // goes on to its next
    sort_down(key);
    auto next = [&] {
        const uint32_t m = __reduce_max_sync(kFull, key[0]);
        const bool own = key[0] == m;
#pragma unroll
        for (int i = 0; i + 1 < VPL; ++i) key[i] = own ? key[i + 1] : key[i];
        if (own) key[VPL - 1] = 0;
        return m;
    };
    uint32_t mine_key = 0, after = 0;
    for (int j = 0; j <= p.top_k; ++j) {
        after = next();
        if (lane == j && j < p.top_k) mine_key = after;
    }
    const bool in = lane < p.top_k;
    int32_t mine = Keys::expert(in ? mine_key : Keys::kMask);
    float ml = in ? load_logit(p, t, mine) : ninf, k = ml, past = 0.0f;
    // certain?
    bool sure = true;
    {
        float tol = 0.0f;
        if (p.bias) {
            const float b = in ? p.bias[mine] : 0.0f, s = score_of(ml);
            k = s + b;
            tol = error * s + 0x1p-22f * (fabsf(k) + fabsf(b)) + (softmax ? error * 0.03f : 0.0f);
            past = 2.0f * (error + kFastError) + 0x1p-21f * (fabsf(k) + fabsf(b) + 1.0f);
        }
        const float k1 = __shfl_down_sync(kFull, k, 1), tol1 = __shfl_down_sync(kFull, tol, 1);
        const int32_t e1 = __shfl_down_sync(kFull, mine, 1);
        if (lane + 1 < p.top_k) sure = k - k1 > tol + tol1 || (!p.bias && k == k1 && mine < e1);
        else if (lane + 1 == p.top_k) sure = after == 0 ? k == k : k - Keys::most(after) > past;
        // (a NaN comes first, or the sum is one; then nothing is certain)
        if (lane == 0 && !(k == k && sum == sum && mine_key <= (0xff800000u | Keys::kMask))) open = true;
        open = __any_sync(kFull, open);
    }
    if (!open && !__all_sync(kFull, sure)) {
        // All that may be among the chosen, one a lane, compared in 64 bits.
        float line = in ? k - past : __uint_as_float(0x7f800000u);
#pragma unroll
        for (int d = 16; d; d >>= 1) line = fminf(line, __shfl_xor_sync(kFull, line, d));
        int n = p.top_k;
        while (n < 32 && after != 0 && !(Keys::most(after) < line)) {
            if (lane == n) mine_key = after;
            ++n;
            after = next();
        }
        // (a softmax needs its sum in 64 bits, and NaNs and infinities their order)
        open = (p.bias && softmax) || (after != 0 && !(Keys::most(after) < line)) || !(line - line == 0.0f);
        if (!open) {
            const int32_t e = Keys::expert(lane < n ? mine_key : Keys::kMask);
            double by = double(load_logit(p, t, e));
            if (p.bias) by = sigmoid(by) + double(p.bias[e]);
            int rank = 0;
            for (int i = 0; i < n; ++i) {
                const double o = __shfl_sync(kFull, by, i);
                const int32_t oe = __shfl_sync(kFull, e, i);
                rank += o > by || (o == by && oe < e);
            }
            for (int i = 0; i < n; ++i) {
                const int to = __shfl_sync(kFull, rank, i);
                const int32_t oe = __shfl_sync(kFull, e, i);
                if (lane == to) mine = oe;
            }
            ml = in ? load_logit(p, t, mine) : ninf;
        }
    }
    if (open) {
        mine = choose_by_keys<VPL>(p, t, lane);
        ml = in ? load_logit(p, t, mine) : ninf;
    }
    *of_it = !in ? 0.0f : softmax && !p.renormalize ? expf(ml - most) / sum : ml;
    return mine;
}

// The weights of a token's chosen experts from what choose() gave each lane: the
// score itself where the softmax is not renormalised, else the logit.
__device__ __forceinline__ float finish(const RouteParams &p, float v, int lane)
{
    const bool in = lane < p.top_k;
    const float ninf = __uint_as_float(0xff800000u);
    auto largest = [](float a, float b) { return fmaxf(a, b); };
    auto plus = [](float a, float b) { return a + b; };
    if (!p.renormalize) {
        if (p.score == CAKE_GG_SCORE_SOFTMAX) return v * p.scale;
        return in ? sigmoid(v) * p.scale : 0.0f;
    }
    // (by the logits the first is the largest; a NaN is the last, and found by the sum)
    const float most = p.bias ? over_chosen(p, in ? v : ninf, largest) : fmaxf(__shfl_sync(kFull, v, 0), ninf);
    float s = 0.0f;
    if (p.score == CAKE_GG_SCORE_SOFTMAX) {
        // the softmax over the chosen; where all of them are -inf, nothing
        s = in && most > ninf ? expf(v - most) : in && v != v ? v : 0.0f;
    } else {
        // where all chosen logits are far below zero their sigmoids vanish, not their
        // ratios: e^(l - m) / (1 + e^l) with m the largest of them, if below zero
        const float m = fminf(most, 0.0f);
        if (in) s = v > 0.0f || v != v ? sigmoid(v) : m > ninf ? expf(v - m) / (1.0f + expf(v)) : 0.0f;
    }
    const float sum = over_chosen(p, s, plus);
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
    s.counts = reinterpret_cast<int32_t *>(s.bits + p.E * bit_words(p.chunk));
    s.base = s.counts + p.E;
    s.chosen = reinterpret_cast<uint16_t *>(s.base + p.E);
    return s;
}
size_t shared_bytes(int32_t E, int32_t top_k, int chunk)
{
    return size_t(E) * bit_words(chunk) * 4 + size_t(E) * 8 + (size_t(chunk) * top_k * 2 + 15) / 16 * 16;
}

// The block's tokens [t0, t0 + n): their experts and weights, and who chose whom.
template <int VPL>
__device__ __forceinline__ void choose_all(const RouteParams &p, const Shared &s, int64_t t0, int n)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, words = bit_words(p.chunk);
    float l[VPL];
    if (warp < n) load_logits(p, t0 + warp, lane, l);
    for (int i = threadIdx.x; i < p.E * words; i += kThreads) s.bits[i] = 0;
    __syncthreads();
    for (int i = warp; i < n; i += kWarps) {
        float v;
        const int32_t e = choose<VPL>(p, t0 + i, lane, l, &v);
        if (i + kWarps < n) load_logits(p, t0 + i + kWarps, lane, l);   // (while this token's is finished)
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

// The token of the i-th choice of a chunk.
__device__ __forceinline__ int token_of(const RouteParams &p, int i) { return p.top_k == 1 ? i : int(__umulhi(uint32_t(i), p.div_top)); }

// A token's place among those of the chunk that chose the same expert.
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
    const int rank = int(blockIdx.x), blocks = int(gridDim.x), e = threadIdx.x, words = bit_words(p.chunk);
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
        const int32_t x = s.chosen[i], token = token_of(p, i), row = s.base[x] + place(s, words, x, token);
        p.position[t0 * p.top_k + i] = row;
        p.rows[row] = int32_t(t0) + token;
    }
    if (blocks > 1) cluster_sync_all();                          // the others may still read this one's counts
}

__host__ __device__ constexpr int32_t count_pitch(int32_t E) { return (E + 7) / 8 * 8; }

// Experts, weights and places within the block (to `position`), a chunk of its
// tokens after the other, and its counts.
template <int VPL>
__global__ void __launch_bounds__(kThreads)
    route_count_kernel(const RouteParams p)
{
    extern __shared__ __align__(16) uint8_t raw[];
    const Shared s = shared_of(raw, p);
    grid_dependency_wait();
    grid_launch_dependents();
    const int words = bit_words(p.chunk);
    const int64_t begin = int64_t(blockIdx.x) * p.block_tokens, end = min(p.T, begin + p.block_tokens);
    for (int e = threadIdx.x; e < p.E; e += kThreads) s.base[e] = 0;
    for (int64_t t0 = begin; t0 < end; t0 += p.chunk) {
        const int n = int(min(int64_t(p.chunk), end - t0));
        choose_all<VPL>(p, s, t0, n);
        for (int i = threadIdx.x; i < n * p.top_k; i += kThreads) {
            const int32_t x = s.chosen[i];
            p.position[t0 * p.top_k + i] = s.base[x] + place(s, words, x, token_of(p, i));
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kThreads) s.base[e] += s.counts[e];
        __syncthreads();
    }
    uint16_t *counts = p.counts + int64_t(blockIdx.x) * count_pitch(p.E);
    for (int e = threadIdx.x; e < count_pitch(p.E); e += kThreads) counts[e] = e < p.E ? uint16_t(s.base[e]) : 0;
}

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
        float m = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
        most = warp_max(m);
        float x[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = x[i] = i * 32 + lane < p.E ? expf(l[i] - most) : 0.0f;
        sum = warp_sum(tree_sum(x));
        const float over = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] *= over;
    }
    const float ml = e >= 0 ? load_logit(r, t, e) : ninf;
    float d = 0.0f, inner = 0.0f;
    if (whole) {
        const float q = e >= 0 ? expf(ml - most) / sum : 0.0f;
        inner = warp_sum(g * q);
        d = q * (g - inner);
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
    // the row, then over it the chosen
    auto put = [&](int32_t x, float v) {
        if (p.bf16) static_cast<uint16_t *>(p.d_logits)[t * p.E + x] = uint16_t(pack_bf16x2(v, 0.0f) & 0xffffu);
        else static_cast<float *>(p.d_logits)[t * p.E + x] = v;
    };
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (i * 32 + lane < p.E) put(i * 32 + lane, whole ? -s[i] * inner : 0.0f);
    __syncwarp();
    if (e >= 0) put(e, d);
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
// or one for each multiprocessor, which holds the bits of a chunk of its tokens.
void choose_blocks(cake_gg_route_plan_t *pl)
{
    const int64_t T = pl->T;
    pl->cluster = T <= kClusterTokens;
    int64_t blocks = pl->cluster ? (T + 3) / 4 : kSms;
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
    p.chunk = pl.block_tokens < kChunk ? pl.block_tokens : kChunk;
    p.div_top = uint32_t((uint64_t(1) << 32) / uint32_t(pl.top_k) + ((uint64_t(1) << 32) % uint32_t(pl.top_k) != 0));
    const int32_t size = pl.E / op.groups;
    p.div_group = uint32_t(((1 << 20) + size - 1) / size);
    const size_t shared = shared_bytes(pl.E, pl.top_k, p.chunk);
    cudaError_t err = with_experts(pl.E, [&](auto vpl) {
        constexpr int VPL = decltype(vpl)::value;
        return pl.cluster ? launch(route_cluster_kernel<VPL>, p, pl.blocks, kThreads, shared, pl.blocks, s)
                          : launch(route_count_kernel<VPL>, p, pl.blocks, kThreads, shared, 1, s);
    });
    if (err == cudaSuccess && !pl.cluster) err = launch(route_number_kernel, p, pl.blocks, kThreads, 0, 1, s);
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
