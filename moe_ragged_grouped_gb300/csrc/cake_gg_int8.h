// cake_gg_int8.h -- internal interface of the 8-bit integer products: kernel
// parameters and launchers shared by the C entry points (cake_gg_int8.cu) and
// the kernel translation units.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/cake_gg.h"

namespace cakegg {

// (cake_gg_capi.cu) checks that the current device is sm_103 and gives its SM count
int device_sms(int *sms);

// One call of the products, as every kernel sees it.
//   Y[m, n] = (sum_k q[r(m), k] W[e(m), n, k]) * ws[e(m), n] * xs[r(m)]
struct I8Params {
    const int32_t *offsets;   // [E + 1], or null: one expert owning rows [0, M)
    const int32_t *rows;      // [M] token of each row, or null: the row itself
    const int8_t *W;          // [E, N, K]
    const float *ws;          // [E, N]
    const float *xs;          // [T]
    void *Y;                  // [M, N]
    int32_t *status;          // sticky status word (workspace byte 0)
    int64_t M, T;
    int32_t E, N, K;
    int32_t out_f32;
    int32_t early;            // the grid before this one is this call's own token pass, so
                              // weights and offsets may be read before it has completed
    uint64_t timeout_ns;
};

constexpr int32_t kI8StatusBadOffsets = CAKE_GG_ERR_BAD_OFFSETS;
constexpr int32_t kI8StatusBadRows = CAKE_GG_ERR_BAD_ROWS;
constexpr int32_t kI8StatusTimeout = CAKE_GG_ERR_TIMEOUT;

constexpr int kI8RowChunk = 8;   // rows of one expert that the row kernel computes together

// Few-row path: 32-bit integer dot products, weights streamed once per row chunk.
cudaError_t launch_i8_rows(const I8Params &p, const int8_t *q, bool pdl, cudaStream_t stream);

}  // namespace cakegg
