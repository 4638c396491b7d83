// cake_gg_route.cuh -- routing to experts: from router logits to each token's
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
// A warp has a token, a lane every 32nd expert.  A key packs the upper bits of a score
// and the expert into one word, so that each round finds the largest and the lowest
// index among its equals by one warp reduction over the lanes' sorted keys.  Scores of
// the keys are approximate; those of the chosen, and of all that come near them, are
// computed in FP32, and in 64 bits where two lie closer than FP32's error.
//
// Rows are numbered by counting: for each expert a bit per token of the block says
// who chose it, so a token's place among them is a population count, in the
// order of the tokens and the same on every run.  As many tokens as a cluster of blocks
// has warps are that cluster's, counts read from one another's shared memory; more
// tokens take a kernel that counts and one that numbers.
//
// Included by the translation units that hold the kernels of some experts a lane.
#pragma once

#include "cake_gg_ptx.cuh"
#include "cake_gg_route.h"
#include "cake_gg_shared_limit.h"

namespace cakegg {
namespace {

// Threads of a block.  The keys and logits of a token of more than 256 experts do not
// stay in the 64 registers that 1024 threads have each (8 of 384, 64 tokens 12.5 us, 8192
// tokens 38; with 512 threads 10.5 and 34); of 256 either does (21 us for 16384 tokens).
template <int VPL> constexpr int kThreadsOf = VPL * 32 <= kRouteNarrow ? kRouteThreads : kRouteThreads / 2;
constexpr unsigned kFull = 0xffffffffu;

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

// 1 / x to a unit in the last place, without the branches of a division.
__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid(float l) { return reciprocal(1.0f + expf(-l)); }
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
        if (!(kept >> min(e * p.div_group >> 20, 31u) & 1u)) key[i] = 0;
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

// FP32's error of a score, relative to it.  A sigmoid: the exponential is off by two
// units in its last place (2^-22), the sum rounds to 2^-24, its reciprocal is off by
// 2^-23: below 2^-21.  A softmax, in units of 2^-24: its sum of up to 1024 terms rounds
// ten times (10), each term is off by 4 (exponential), and of its argument x = l - max,
// which rounds to |x| and, where the exponential is approximate, is multiplied by a
// rounded constant (1.2 |x| more), the terms' mean counts, at most 4.5 (of n terms e^-x
// beside the largest, n x e^-x / (1 + n e^-x)): 24 of the sum; the numerator 4, reciprocal
// and product 3: 31, below 2^-19.  (A sum by exponentials in FP32 would be off by 19 in
// place of 24, measured by the same 3 x 10^-7 of logits of deviation 1, and costs 0.5 us
// of 21 for 16384 x 256.)  The numerator's own argument: x e^-x <= 0.37 bounds what it
// is of the largest score.  s + bias rounds by 2^-24 of itself.
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

// A token's logits of the lane's experts, -inf beyond E.
template <typename LT>
__device__ __forceinline__ float as_float(LT v)
{
    if constexpr (sizeof(LT) == 2) return __uint_as_float(uint32_t(v) << 16);
    else return v;
}
template <int VPL, typename LT>
__device__ __forceinline__ void load_row(const LT *row, int32_t E, int lane, float (&l)[VPL])
{
    // (the last expert's in place of those beyond: no branches)
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = as_float(row[min(i * 32 + lane, E - 1)]);
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = i * 32 + lane < E ? l[i] : __uint_as_float(0xff800000u);
}
template <int VPL>
__device__ __forceinline__ void load_logits(const RouteParams &p, int64_t t, int lane, float (&l)[VPL])
{
    if (p.bf16) load_row(static_cast<const uint16_t *>(p.logits) + t * p.stride, p.E, lane, l);
    else load_row(static_cast<const float *>(p.logits) + t * p.stride, p.E, lane, l);
}

// Each lane's expert's score with its bias in 64 bits (all lanes of the warp; `most`: the token's largest logit).
template <bool SOFTMAX>
__device__ __noinline__ double score_in_64_bits(const RouteParams &p, int64_t t, int32_t e, float most, int lane)
{
    double s = double(load_logit(p, t, e));
    if (SOFTMAX) {
        double all = 0.0;
        for (int32_t i = lane; i < p.E; i += 32) all += exp(double(load_logit(p, t, i)) - double(most));
        s = exp(s - double(most)) / warp_sum(all);
    } else {
        s = sigmoid(s);
    }
    return p.bias ? s + double(p.bias[e]) : s;
}

// What experts are chosen by: logits, or scores of one kind (with a bias, or because
// groups compete by sums).
enum Mode { kByLogits, kBySoftmax, kBySigmoid };

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
// (bias: the lane's experts'.)
template <int VPL, Mode MODE>
__device__ __forceinline__ int32_t choose(const RouteParams &p, int64_t t, int lane, const float (&l)[VPL], const float (&bias)[VPL],
                                          float *of_it)
{
    using Keys = Packed<VPL * 32>;
    constexpr bool by_score = MODE != kByLogits;
    const bool softmax = MODE == kBySoftmax || (MODE == kByLogits && p.score == CAKE_GG_SCORE_SOFTMAX);
    const float ninf = __uint_as_float(0xff800000u);
    uint32_t key[VPL];
    float most = 0.0f, sum = 1.0f;
    if (softmax && (by_score || !p.renormalize)) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
        most = m == ninf ? 0.0f : m;                             // (nothing left: all exponentials are 0)
        float e[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) e[i] = exp2_fast((l[i] - most) * kLog2e);
        sum = warp_sum(tree_sum(e));
    }
    // the score of a logit in FP32, of a candidate
    auto score_of = [&](float v) { return softmax ? expf(v - most) * reciprocal(sum) : sigmoid(v); };
    const float error = softmax ? kSoftmaxError : kSigmoidError;
    // no score is larger: errors are of it (with one in its place, 16384 tokens, 8 of 256 by a softmax with a
    // bias, took 39 to 53 us, of the few tokens that go the long way)
    const float top = MODE == kBySoftmax ? reciprocal(sum) * 1.001f : 1.0f;
    bool open = false;
    if constexpr (by_score) {
        const float over = MODE == kBySoftmax ? rcp_fast(sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = i * 32 + lane;
            const float s = MODE == kBySoftmax ? exp2_fast((l[i] - most) * kLog2e) * over : rcp_fast(1.0f + exp2_fast(l[i] * -kLog2e));
            key[i] = e < p.E ? Keys::of(s + bias[i], e) : 0;
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
        float v = ninf, m = 0.0f, slack = 0.0f, line = 0.0f;
        int32_t e1 = 0, e2 = 0;
        if (lane < p.groups) {
            e1 = Keys::expert(first), e2 = Keys::expert(second);
            const float l1 = load_logit(p, t, e1);
            float k1 = by_score ? score_of(l1) : l1;
            if (p.bias) k1 += p.bias[e1];
            v = line = k1, m = fabsf(k1), slack = Keys::most(first) - k1;
            if (p.pair) {
                float k2 = score_of(load_logit(p, t, e2));
                if (p.bias) k2 += p.bias[e2];
                v += k2, line = k2, m += fabsf(k2), slack += Keys::most(second) - k2;
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
        open = nan || (p.top_groups < p.groups && !(low - high > (by_score ? 4.0f * (error + kFastError) * top : 0.0f) + size_of * 0x1p-21f));
        if (by_score && open && !nan) {
            // where what was found is larger for certain than the rest of its group, the
            // groups' scores in 64 bits (16384 tokens, 4 of 8 groups by their two largest:
            // 50 us where these went the long way)
            line -= 2.0f * (error + kFastError) * top + 0x1p-20f * (m + top);
            uint32_t near = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float line_of = __shfl_sync(kFull, line, min(uint32_t(i * 32 + lane) * p.div_group >> 20, 31u));
                near += key[i] != 0 && !(Keys::most(key[i]) < line_of);
            }
            if (__reduce_add_sync(kFull, near) == uint32_t(p.pair ? 2 * p.groups : p.groups)) {
                double by = score_in_64_bits<MODE == kBySoftmax>(p, t, e1, most, lane);
                if (p.pair) by += score_in_64_bits<MODE == kBySoftmax>(p, t, e2, most, lane);
                rank = 0;
                for (int g = 0; g < p.groups; ++g) {
                    const double o = __shfl_sync(kFull, by, g);
                    rank += o > by || (o == by && g < lane);
                }
                kept = __ballot_sync(kFull, lane < p.groups && rank < p.top_groups);
                open = false;
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const uint32_t e = uint32_t(i * 32 + lane);
            if (!(kept >> min(e * p.div_group >> 20, 31u) & 1u)) key[i] = 0;
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
            tol = error * s + 0x1p-22f * (fabsf(k) + fabsf(b)) + (softmax ? error * 0.03f * top : 0.0f);
            past = 2.0f * (error + kFastError) * top + 0x1p-21f * (fabsf(k) + fabsf(b) + top);
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
        // (NaNs and infinities need their order)
        open = (after != 0 && !(Keys::most(after) < line)) || !(line - line == 0.0f);
        if (!open) {
            const int32_t e = Keys::expert(lane < n ? mine_key : Keys::kMask);
            const double by = p.bias ? score_in_64_bits<MODE == kBySoftmax>(p, t, e, most, lane) : double(load_logit(p, t, e));
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
    *of_it = !in ? 0.0f : !softmax || p.renormalize ? ml : sum == 0.0f ? 0.0f : expf(ml - most) * reciprocal(sum);
    return mine;
}

// A chosen score up to a factor that all of a token's have, of logit v, the largest
// of them `most`: e^(v - most) of a softmax; of a sigmoid e^(v - m) / (1 + e^v), m the
// largest if that is below zero (where all sigmoids vanish their ratios do not), or 1 /
// (1 + e^-v).  Where all are -inf, nothing.
__device__ __forceinline__ float share(float v, float most, bool in, int32_t score)
{
    const bool softmax = score == CAKE_GG_SCORE_SOFTMAX;
    const float e = expf(!softmax && v > 0.0f ? 0.0f : v - (softmax ? most : fminf(most, 0.0f)));
    const float s = softmax ? e : e * reciprocal(1.0f + expf(-fabsf(v)));
    return !in ? 0.0f : most > __uint_as_float(0xff800000u) || v != v ? s : 0.0f;
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
    const float s = share(v, most, in, p.score), sum = over_chosen(p, s, plus);
    return sum == 0.0f ? 0.0f : s * (reciprocal(sum) * p.scale);
}

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
// The block's tokens [t0, t0 + n): their experts and weights, and who chose whom.
template <int VPL, Mode MODE>
__device__ __forceinline__ void choose_all(const RouteParams &p, const Shared &s, int64_t t0, int n)
{
    constexpr int kThreads = kThreadsOf<VPL>, kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, words = bit_words(p.chunk);
    float l[VPL], bias[VPL];
    if (MODE != kByLogits && p.bias) load_row(p.bias, p.E, lane, bias);
    else
#pragma unroll
        for (int i = 0; i < VPL; ++i) bias[i] = 0.0f;
    if (warp < n) load_logits(p, t0 + warp, lane, l);
    for (int i = threadIdx.x; i < p.E * words; i += kThreads) s.bits[i] = 0;
    __syncthreads();
    for (int i = warp; i < n; i += kWarps) {
        float v;
        const int32_t e = choose<VPL, MODE>(p, t0 + i, lane, l, bias, &v);
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

template <int VPL, Mode MODE>
__global__ void __launch_bounds__(kThreadsOf<VPL>, 1)
    route_cluster_kernel(const RouteParams p)
{
    extern __shared__ __align__(16) uint8_t raw[];
    const Shared s = shared_of(raw, p);
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kThreads = kThreadsOf<VPL>;
    const int rank = int(blockIdx.x), blocks = int(gridDim.x), words = bit_words(p.chunk);
    const int64_t t0 = int64_t(rank) * p.block_tokens;
    const int n = int(t0 >= p.T ? 0 : p.T - t0 < p.block_tokens ? p.T - t0 : p.block_tokens);
    choose_all<VPL, MODE>(p, s, t0, n);
    if (blocks > 1) cluster_sync_all();
    else __syncthreads();
    int32_t total = 0;
    for (int e0 = 0; e0 < p.E; e0 += kThreads) {
        const int e = e0 + int(threadIdx.x);
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
        int32_t sum;
        if (e0) __syncthreads();
        const int32_t first = total + block_scan(all, &sum);
        total += sum;
        if (e < p.E) {
            s.base[e] = first + before;
            if (rank == 0) p.offsets[e] = first;
        }
    }
    if (rank == 0 && threadIdx.x == 0) p.offsets[p.E] = total;
    __syncthreads();
    for (int i = threadIdx.x; i < n * p.top_k; i += kThreads) {
        const int32_t x = s.chosen[i], token = token_of(p, i), row = s.base[x] + place(s, words, x, token);
        p.position[t0 * p.top_k + i] = row;
        p.rows[row] = int32_t(t0) + token;
    }
    if (blocks > 1) cluster_sync_all();                          // the others may still read this one's counts
}

// Experts, weights and places within the block (to `position`), a chunk of its
// tokens after the other, and its counts.
template <int VPL, Mode MODE>
__global__ void __launch_bounds__(kThreadsOf<VPL>, 1)
    route_count_kernel(const RouteParams p)
{
    extern __shared__ __align__(16) uint8_t raw[];
    const Shared s = shared_of(raw, p);
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kThreads = kThreadsOf<VPL>;
    const int words = bit_words(p.chunk);
    const int64_t begin = int64_t(blockIdx.x) * p.block_tokens, end = min(p.T, begin + p.block_tokens);
    for (int e = threadIdx.x; e < p.E; e += kThreads) s.base[e] = 0;
    for (int64_t t0 = begin; t0 < end; t0 += p.chunk) {
        const int n = int(min(int64_t(p.chunk), end - t0));
        choose_all<VPL, MODE>(p, s, t0, n);
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

// ---------------------------------------------------------------- backward

// With g the weights' gradient times the scale:
//   softmax, renormalised: w = softmax over the chosen, dl_j = w_j (g_j - sum g w)
//   softmax:               dl_e = p_e ([e chosen] g_e - sum g p), over all experts
//   sigmoid, renormalised: r = s / S of the chosen, dl_j = r_j (1 - s_j) (g_j - sum g r)
//   sigmoid:               dl_j = g_j s_j (1 - s_j)
// and zeros elsewhere.  1 - s is computed as the sigmoid of -l.
template <typename LT>
__device__ __forceinline__ LT rounded(float v)
{
    if constexpr (sizeof(LT) == 2) return LT(pack_bf16x2(v, 0.0f) & 0xffffu);
    else return v;
}

// The softmax over all experts: a warp a token, a lane every 32nd expert.  (16384 x 256
// FP32: 7.0 us, 4.9 TB/s read and written.)
template <int VPL, typename LT>
__global__ void __launch_bounds__(256)
    route_grad_whole_kernel(const RouteGradParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const LT *row = static_cast<const LT *>(p.logits) + t * p.stride;
    float s[VPL], x[VPL];
    load_row(row, p.E, lane, s);
    int32_t e = lane < p.top_k ? p.expert[t * p.top_k + lane] : -1;
    if (uint32_t(e) >= uint32_t(p.E)) e = -1;                    // (nobody: nothing is read or written for it)
    const float g = e >= 0 ? p.d_weight[t * p.top_k + lane] * p.scale : 0.0f, l = as_float(row[max(e, 0)]);
    float m = s[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, s[i]);
    m = warp_max(m);
    if (m == __uint_as_float(0xff800000u)) m = 0.0f;             // (nothing left: all exponentials are 0)
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = x[i] = expf(s[i] - m);
    const float q = e >= 0 ? expf(l - m) : 0.0f;
    // (both sums at once)
    float sum = tree_sum(x), inner = g * q;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        sum += __shfl_xor_sync(kFull, sum, d);
        inner += __shfl_xor_sync(kFull, inner, d);
    }
    const float over = sum == 0.0f ? 0.0f : reciprocal(sum);
    inner *= over;
    const float by = -inner * over;
    LT *out = static_cast<LT *>(p.d_logits) + t * p.E;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (i * 32 + lane < p.E) out[i * 32 + lane] = rounded<LT>(s[i] * by);
    __syncwarp();
    if (e >= 0) out[e] = rounded<LT>(q * over * (g - inner));    // (over what the row has there)
}

// The chosen alone: G lanes a token, the power of two that holds them; a warp
// zeroes its tokens' rows and puts them in.
template <typename LT>
__global__ void __launch_bounds__(256)
    route_grad_kernel(const RouteGradParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    int G = 1;
    while (G < p.top_k) G *= 2;
    const int lane = threadIdx.x & 31, many = 32 / G, mine = lane / G, j = lane & (G - 1);
    const int64_t t0 = (int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5)) * many, t = t0 + mine;
    if (t0 >= p.T) return;
    const float ninf = __uint_as_float(0xff800000u);
    int32_t e = t < p.T && j < p.top_k ? p.expert[t * p.top_k + j] : -1;
    if (uint32_t(e) >= uint32_t(p.E)) e = -1;                    // (nobody: nothing is read or written for it)
    const float g = e >= 0 ? p.d_weight[t * p.top_k + j] * p.scale : 0.0f;
    const float l = e >= 0 ? as_float(static_cast<const LT *>(p.logits)[t * p.stride + e]) : ninf;
    // the rows, while these come
    const int64_t count = min(int64_t(many), p.T - t0) * p.E;
    LT *out = static_cast<LT *>(p.d_logits) + t0 * p.E;
    if (((reinterpret_cast<uintptr_t>(out) | uintptr_t(count * sizeof(LT))) & 15) == 0)
        for (int64_t i = lane; i < count * int64_t(sizeof(LT)) / 16; i += 32) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
    else
        for (int64_t i = lane; i < count; i += 32) out[i] = LT(0);
    float d;
    if (p.score == CAKE_GG_SCORE_SIGMOID && !p.renormalize) {
        d = g * sigmoid(l) * sigmoid(-l);
    } else {
        float most = l;
        for (int s = 1; s < G; s *= 2) most = fmaxf(most, __shfl_xor_sync(kFull, most, s));
        const float x = share(l, most, e >= 0, p.score);
        float sum = x, inner = g * x;
        for (int s = 1; s < G; s *= 2) {
            sum += __shfl_xor_sync(kFull, sum, s);
            inner += __shfl_xor_sync(kFull, inner, s);
        }
        const float over = sum == 0.0f ? 0.0f : reciprocal(sum);
        // (a weight on its own is a constant, also where its reciprocal rounds)
        d = p.top_k == 1 ? 0.0f : x * over * (g - inner * over);
        if (p.score == CAKE_GG_SCORE_SIGMOID) d *= sigmoid(-l);
    }
    __syncwarp();
    if (e >= 0) out[int64_t(mine) * p.E + e] = rounded<LT>(d);
}

// ---------------------------------------------------------------- launches

}  // namespace

template <int VPL>
cudaError_t launch_route(const RouteParams &p, int blocks, bool cluster, size_t shared, cudaStream_t stream)
{
    auto with_mode = [&](auto mode) {
        constexpr Mode MODE = decltype(mode)::value;
        // (a cluster's blocks have a few tokens each)
        if (!cluster && shared > kRouteSharedDefault) {
            const cudaError_t err = raise_shared_limit<route_count_kernel<VPL, MODE>>(route_shared_bytes(VPL * 32, kRouteMaxTop, kRouteChunk));
            if (err != cudaSuccess) return err;
        }
        return cluster ? route_launch(route_cluster_kernel<VPL, MODE>, p, blocks, kThreadsOf<VPL>, shared, blocks, stream)
                       : route_launch(route_count_kernel<VPL, MODE>, p, blocks, kThreadsOf<VPL>, shared, 1, stream);
    };
    if (!p.bias && !(p.pair && p.groups > 1)) return with_mode(std::integral_constant<Mode, kByLogits>());
    return p.score == CAKE_GG_SCORE_SOFTMAX ? with_mode(std::integral_constant<Mode, kBySoftmax>())
                                            : with_mode(std::integral_constant<Mode, kBySigmoid>());
}

template <int VPL>
cudaError_t launch_route_grad_whole(const RouteGradParams &p, cudaStream_t stream)
{
    return p.bf16 ? route_launch(route_grad_whole_kernel<VPL, uint16_t>, p, (p.T + 7) / 8, 256, 0, 1, stream)
                  : route_launch(route_grad_whole_kernel<VPL, float>, p, (p.T + 7) / 8, 256, 0, 1, stream);
}

}  // namespace cakegg
