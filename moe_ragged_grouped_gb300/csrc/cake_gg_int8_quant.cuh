// cake_gg_int8_quant.cuh -- how a row of activations becomes 8-bit integers and
// a scale; shared by the token pass and the few-row product that quantises on
// the way.
//
//   h = x, or silu(g) * u of x = [g | u];  a = max |h|
//   scale = a / 127,  q = round(h * (127 / a)), ties to even, all in FP32
//
// |h| is compared by its bit pattern, so a NaN or an infinity wins the maximum:
// such a row gets the scale NaN and zero integers (its products are NaN).  A
// row whose a is below 2^-120 counts as zero (127 / a would not be finite).
#pragma once

#include <cstdint>

namespace cakegg {

template <typename XT>
__device__ __forceinline__ void load8(const XT *p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t *p, float (&v)[8])   // BF16
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

// Eight values h of a row.  (g = -inf gives NaN, as the formula does; a large
// negative g gives 0.)
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

__device__ __forceinline__ uint32_t max_bits(const float (&v)[8], uint32_t m)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// From the largest bit pattern of a row: its scale, and what its values are
// multiplied by.
struct RowScale {
    float scale, inv;
    bool finite;
    __device__ __forceinline__ explicit RowScale(uint32_t m)
    {
        const float a = __uint_as_float(m);
        finite = m < 0x7f800000u;
        const bool tiny = a < 0x1p-120f;
        inv = finite && !tiny ? 127.0f / a : 0.0f;
        scale = !finite ? __uint_as_float(0x7fc00000u) : tiny ? 0.0f : a / 127.0f;
    }
    // The integer q of h in the low 16 bits, above 0x6600: floats from 2^23 to 2^24
    // are integers one apart, so adding 1.5 * 2^23 + 0x6600 rounds h * inv (at most
    // 127 in magnitude) to an integer, ties to even, by an ordinary addition.  (The
    // rounding and conversion instructions run at an eighth of its rate.)
    __device__ __forceinline__ uint32_t biased(float h) const
    {
        return __float_as_uint(__fadd_rn(__fmul_rn(h, inv), 12582912.0f + float(0x6600)));
    }
};

// Eight integers of a row as bytes.
__device__ __forceinline__ uint2 bytes8(const float (&v)[8], const RowScale &s)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = __byte_perm(s.biased(v[4 * i]), s.biased(v[4 * i + 1]), 0x0040);
        const uint32_t b = __byte_perm(s.biased(v[4 * i + 2]), s.biased(v[4 * i + 3]), 0x0040);
        w[i] = s.finite ? __byte_perm(a, b, 0x5410) : 0;
    }
    return make_uint2(w[0], w[1]);
}

// Eight integers of a row as FP16: the pattern 0x6600 + q is 1536 + q.
__device__ __forceinline__ uint4 halves8(const float (&v)[8], const RowScale &s)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = __byte_perm(s.biased(v[2 * i]), s.biased(v[2 * i + 1]), 0x5410);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(a), "r"(0x66006600u));
        if (!s.finite) w[i] = 0;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace cakegg
