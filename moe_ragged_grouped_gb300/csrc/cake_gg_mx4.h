// cake_gg_mx4.h -- internal interface of the 4-bit products: kernel parameters
// and launchers shared by the C entry points (cake_gg_mx4.cu) and the kernel
// translation units.
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

// Scales lie in tiles of 128 rows x 4 blocks (512 bytes), which is how the tensor
// cores take them: byte of row r and block b of 32 values, of a matrix whose rows
// have `kt` such tiles.
__host__ __device__ __forceinline__ int64_t mx4_scale_at(int64_t r, int32_t b, int32_t kt)
{
    return ((r >> 7) * kt + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}
constexpr int32_t kMx4Tile = 512;

// Rows of a tile at most: two accumulators of 192 columns leave room in tensor
// memory for the scales of five stages (beside two of 224 there are two, and each
// stage waits for the one before last: 16384 x 4096 -> 4096 106 us, 87).
constexpr int kMx4RowsMost = 192;

// Scale tiles of a word (128 values) of the reduction for a tile of nt rows.
__host__ __device__ constexpr int mx4_row_atoms(int nt) { return nt > 128 ? 2 : 1; }

// A pair of CTAs takes the scales of its rows as a row tile has them: for each
// slot and each word of the reduction the scale tiles of nt rows.  The slot of
// an expert's tile j needs the expert's offset only: nothing is summed, and since
// floor((a + n) / nt) + 1 >= floor(a / nt) + ceil(n / nt), no two tiles share one.
__host__ __device__ __forceinline__ int32_t mx4_slot(int32_t offset, int32_t e, int32_t j, int32_t nt) { return offset / nt + e + j; }
__host__ __device__ __forceinline__ int64_t mx4_slots(int64_t M, int32_t E, int32_t nt) { return M / nt + E; }

// One call of the products.
//   Y[m, n] = sum_k x[r(m), k] w[e(m), n, k]
struct Mx4Params {
    const int32_t *offsets;   // [E + 1], or null: one expert owning rows [0, M)
    const int32_t *rows;      // [M] token of each row, or null: the row itself (for a pair: laid out so)
    const uint8_t *xs;        // token scales, in tiles (for a pair: of its rows, by slot)
    void *Y;                  // [M, N]
    int32_t *status;          // sticky status word (workspace byte 0)
    int64_t M, T;             // rows of all experts (offsets' bound), tokens
    int32_t E, N, K;
    int32_t out_f32;
    int32_t early;            // the grid before this one is this call's own token pass, so
                              // weights and offsets may be read before it has completed
    int32_t nt;               // rows of a tile at most (a multiple of 32)
    int32_t stages;           // shared-memory ring depth
    int32_t splits;           // CTAs that share a tile's reduction (one cluster; 1 = none)
    int32_t debug_flags;
    uint64_t timeout_ns;
    // (set by the preparation) channel tiles, stages and scale tiles of the
    // reduction, scale tiles of an expert's channels, rows of a copy, 2^32 / (nt / 16) rounded up
    int32_t n_ct, n_kb, n_kt, n_nt, box;
    uint32_t div_nt;
};

// Few rows are taken in runs of an expert's: of one where there are no more rows than
// experts, else of up to two; and as many runs as a call can have.
__host__ __device__ __forceinline__ int mx4_run_rows(int64_t M, int32_t E) { return M > E ? 2 : 1; }
__host__ __device__ __forceinline__ int64_t mx4_runs(int64_t M, int32_t E) { return M <= E ? M : E == 1 ? (M + 1) / 2 : (M + E) / 2; }

constexpr size_t kMx4SmemLimit = 232448;   // opt-in dynamic shared memory per CTA (227 KB)
constexpr int kMx4StagesMost = 12;

// Dynamic shared memory of a CTA.
size_t mx4_mma_smem(int pair, int nt, int stages, int splits, int E);

// Everything that can be refused is refused by the preparation, which enqueues
// nothing.  Both return a cake_gg_status_t.
struct Mx4Launch {
    CUtensorMap mw, ms, mx, mr;
    Mx4Params p;
    int32_t pair, grid;
};
int prepare_mx4_mma(Mx4Launch *l, const Mx4Params &p, const uint8_t *W, const uint8_t *ws, const uint8_t *x, int pair, int sms);
int launch_mx4_mma(const Mx4Launch &l, bool pdl, cudaStream_t stream);

// Few rows: integer dot products.  X: codes (x_dtype CAKE_GG_MX4, scales in p.xs), or
// activations that the blocks quantise themselves.
bool mx4_rows_fit(int64_t M, int32_t E, int32_t K);
cudaError_t launch_mx4_rows(const Mx4Params &p, const void *X, int x_dtype, const uint8_t *W, const uint8_t *ws, bool pdl,
                            cudaStream_t stream);

}  // namespace cakegg
