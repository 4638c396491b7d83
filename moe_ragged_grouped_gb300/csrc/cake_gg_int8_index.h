// cake_gg_int8_index.h -- where lanes of the 8-bit products read, as plain
// arithmetic that a host program can check over every length.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define CAKE_GG_INDEX __host__ __device__ __forceinline__
#else
#define CAKE_GG_INDEX inline
#endif

namespace cakegg {

// A lane's place in a step of 64 values of a row: 16 bytes.
CAKE_GG_INDEX int32_t i8_warps_place(int32_t lane) { return (lane & 3) * 16; }

// Whether that place of step s lies in a row of K values (a multiple of 16).
CAKE_GG_INDEX bool i8_warps_in(int32_t s, int32_t lane, int32_t K) { return s * 64 + i8_warps_place(lane) < K; }

// Where the lane reads the token's row, from its start: its place, or, past the
// row's end, the row's first 16 bytes, which are always there (the weights are
// zero then).  (The lane's place in the first step would be past the end of rows
// shorter than 64.)
CAKE_GG_INDEX int32_t i8_warps_token(int32_t s, int32_t lane, int32_t K)
{
    return i8_warps_in(s, lane, K) ? s * 64 + i8_warps_place(lane) : 0;
}

}  // namespace cakegg
