// cake_gg_mx4_quant.cuh -- how blocks of 32 values become 4-bit codes and a scale;
// shared by the token pass and the few-row product that quantises on the way.
//
//   e = max(floor(log2(max |h|)) - 2, -127),  scale 2^e,  code = E2M1 nearest to h / 2^e
#pragma once

#include <cstdint>

namespace cakegg {

// Two FP32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Four pairs of values as E2M1 codes, to nearest, ties to even, held at 6; the
// first of a pair in the low half of its byte.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float inv)
{
    float w[8];
    const uint64_t by = pair2(inv, inv);
#pragma unroll
    for (int i = 0; i < 8; i += 2) unpair2(mul2(pair2(v[i], v[i + 1]), by), w[i], w[i + 1]);
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]), "f"(w[4]), "f"(w[5]), "f"(w[6]), "f"(w[7]));
    return r;
}

// The scale's byte (exponent + 127; 255: a NaN) of a block's largest magnitude,
// by its bits, and the reciprocal of the scale.  (Powers of two: exact.)
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits)
{
    const int e = int(max_bits >> 23);
    return e == 255 ? 255u : uint32_t(max(e - 2, 0));
}
__device__ __forceinline__ float scale_inverse(uint32_t byte)
{
    return byte == 255 ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// The bits of the largest magnitude of eight values; a NaN's if there is one.
__device__ __forceinline__ uint32_t largest8(const float (&v)[8])
{
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(v[0]), "f"(v[1]), "f"(v[2]));
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[3]), "f"(v[4]));
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[5]), "f"(v[6]));
    asm("max.NaN.abs.f32 %0, %0, %1, %1;" : "+f"(m) : "f"(v[7]));
    return __float_as_uint(m);
}
__device__ __forceinline__ float least8(const float (&v)[8])
{
    float m;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(v[0]), "f"(v[1]), "f"(v[2]));
    asm("min.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[3]), "f"(v[4]));
    asm("min.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[5]), "f"(v[6]));
    return fminf(m, v[7]);
}

__device__ __forceinline__ uint32_t block_max(uint32_t m)    // over the four lanes of a block
{
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Eight values of a row as they are in memory, read once.
template <typename XT> struct Raw;
template <> struct Raw<uint16_t> {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};

}  // namespace cakegg
