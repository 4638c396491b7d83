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
// (cake_gg_capi.cu) tensor map of a dense tensor, dims[0] contiguous, byte strides of
// dims 1 .. given, zero fill outside the tensor, 128-byte swizzled boxes unless told
int encode_tiled(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dims,
                 const uint64_t *strides, const uint32_t *box, bool swizzled = true);

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
    int64_t M, T;             // rows of all experts (offsets' bound), tokens
    int64_t m_lo, m_hi;       // rows of this launch (tensor-core path)
    int32_t E, N, K;
    int32_t out_f32;
    int32_t early;            // the grid before this one is this call's own token pass, so
                              // weights and offsets may be read before it has completed
    uint64_t timeout_ns;
};

constexpr int32_t kI8StatusBadOffsets = CAKE_GG_ERR_BAD_OFFSETS;
constexpr int32_t kI8StatusBadRows = CAKE_GG_ERR_BAD_ROWS;
constexpr int32_t kI8StatusTimeout = CAKE_GG_ERR_TIMEOUT;

// The tensor-core path's own numbers.
struct I8MmaParams {
    I8Params b;
    int32_t nt;               // rows of a tile at most (a multiple of 32)
    int32_t stages;           // shared-memory ring depth
    int32_t slots;            // widened weight tiles in tensor memory
    int32_t splits;           // CTAs that share a tile's reduction (one cluster; 1 = none)
    int32_t debug_flags;
    // (set by the launch) channel tiles, stages of a tile, rows of a copy, 2^32 / (nt / 16) rounded up
    int32_t n_ct, n_kb, box;
    uint32_t div_nt;
};

constexpr size_t kI8SmemLimit = 232448;   // opt-in dynamic shared memory per CTA (227 KB)

// Dynamic shared memory of a CTA.
size_t i8_mma_smem(int pair, int nt, int stages, int splits, int E);

// Tensor-core path: q [T, K] as FP16 integers.  Everything that can be refused
// is refused by the preparation, which enqueues nothing.  Both return a
// cake_gg_status_t.
struct I8MmaLaunch {
    CUtensorMap mw, mx;
    I8MmaParams p;
    int32_t pair, grid;
};
int prepare_i8_mma(I8MmaLaunch *l, const I8MmaParams &p, const uint16_t *q, int pair, int sms);
int launch_i8_mma(const I8MmaLaunch &l, bool pdl, cudaStream_t stream);

// Few-row path: 32-bit integer dot products, weights streamed once per run of
// an expert's rows.  X: the quantised tokens [T, K] (x_dtype CAKE_GG_INT8), or
// activations where i8_rows_fused() says that the blocks quantise their rows
// themselves.
bool i8_rows_fused(const I8Params &p, int act);
int i8_run_rows(int32_t E, int64_t M, int64_t T);   // rows of a run: 1, 2 or 4
int64_t i8_rows_blocks(const I8Params &p);          // blocks of the launch, at most INT32_MAX of which there can be
cudaError_t launch_i8_rows(const I8Params &p, const void *X, int x_dtype, int act, bool pdl, cudaStream_t stream);

// A few dozen rows: warp-level products from registers, runs of 16 or 32 of an
// expert's rows; q [T, K].
int64_t i8_warps_blocks(const I8Params &p);
cudaError_t launch_i8_warps(const I8Params &p, const int8_t *q, int rows, bool pdl, cudaStream_t stream);

}  // namespace cakegg
