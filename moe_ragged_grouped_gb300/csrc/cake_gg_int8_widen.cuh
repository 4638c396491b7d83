// cake_gg_int8_widen.cuh -- 8-bit integers as FP16 ones, exactly.
#pragma once

#include <cstdint>

namespace cakegg {

// Four 8-bit integers (a 32-bit word) as two packed pairs of FP16: with its
// sign bit flipped a byte is b + 128, and as the low byte of the FP16 pattern
// 0x6400 (1024, one unit in the last place) it reads 1024 + 128 + b.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));   // 1152 each
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

}  // namespace cakegg
