// cake_gg_mx4_mma.cu -- the 4-bit products on the tensor cores.
//
//   Y[m, n] = sum_k x[r(m), k] w[e(m), n, k]
//
// Both operands are E2M1 with a power of two for each block of 32 along k, which
// tcgen05.mma.kind::mxf4 multiplies as they lie in memory: two values a byte in
// shared memory, the scales in tensor memory, sums in FP32.
//
// A tile is 128 channels (256 for a pair of CTAs) x up to nt rows of one
// expert, computed transposed: D[channel, row] += W x^T, so the width of B
// follows the rows that the tile really has and a ragged end or a decoding
// batch costs its own size only.  A stage is 256 values of the reduction: 128
// bytes of every channel and row, two scale tiles of 128 channels x 4 blocks, and
// the same of the rows.  The scales of the channels lie in memory as the tensor
// cores take them and come by TMA; those of the rows, which begin anywhere in a
// scale tile, or are routed, are put together by warps of a single CTA, two stages at a
// time; a pair has them (and routed rows' codes) laid out before it starts, so that all
// that its MMAs read comes by TMA.  Both go from shared to tensor memory by tcgen05.cp,
// which the MMAs of the stage follow in the pipe.
//
// Roles of a CTA: warp 0 copies weights and their scales, warp 1 issues MMAs, warps
// 2-9 store (two groups on alternate 32 rows of a tile), warps 10-13 put the rows' scales
// together where they do not come by TMA, warp 14 copies scales to tensor memory, warp 15
// copies rows, or, where they are routed, warps 15-18 gather them, two on every other stage.
//
// Bound: long calls by the MMA loop (16384 x 4096 -> 4096 86 us, 6.3 PFLOP/s: a stage takes
// 490 to 600 clocks with its hand-over, of which the tensor pipe is active some 410, at four
// times BF16's rate; with rows in 192 and pairs, since a wider B takes the same hand-over), decoding by HBM (64 tokens through 4 of
// 32 experts 6144 -> 4096: 70 us, 6.1 TB/s), a single token by what 128 units draw on 152
// multiprocessors (15.2 us).
#include <type_traits>

#include "cake_gg_mx4.h"
#include "cake_gg_ptx.cuh"
#include "cake_gg_roles.cuh"
#include "cake_gg_shared_limit.h"

namespace cakegg {
namespace {

constexpr int kThreads = 512, kThreadsRouted = 608;
constexpr int kStoreWarp0 = 2, kStoreWarps = 8;
constexpr int kScaleWarp0 = 10, kScaleWarps = 4;
constexpr int kCopyWarp = 14;
constexpr int kRowsWarp0 = 15, kGatherWarps = 4;
constexpr int kKB = 256;                      // reduction length of a stage
constexpr uint32_t kWBytes = 128 * kKB / 2;   // weight tile of a stage
constexpr int kRowWords = kMx4RowsMost / 32;  // words of scales that a lane puts together
constexpr int kChunk = 2;                     // stages whose scales come together
constexpr int kWords = 2 * kChunk;            // words (128 values) of the reduction in them
constexpr uint32_t kOutTile = 2048;           // 32 BF16 or 16 FP32 rows x 32 channels of output, per storing warp
constexpr int kGatherRows = kMx4RowsMost / 2;  // rows that a gathering warp serves at most: half a tile's

// Stages whose scales tensor memory holds beside the two accumulators.
__host__ __device__ constexpr int scale_slots(int nt) { return (512 - 2 * nt) / (8 + 8 * mx4_row_atoms(nt)); }
// Shared memory of scales, the channels' and the rows', of some words; of a stage:
// weights, rows, and for a pair the scales; of a chunk (not for a pair).
__host__ __device__ constexpr uint32_t scale_bytes_of(int words, int nt) { return uint32_t(words * kMx4Tile) * uint32_t(1 + mx4_row_atoms(nt)); }
__host__ __device__ constexpr uint32_t stage_bytes_of(int pair, int nt)
{
    return kWBytes + uint32_t(nt / pair) * 128u + (pair == 2 ? scale_bytes_of(2, nt) : 0u);
}
__host__ __device__ constexpr uint32_t chunk_bytes_of(int nt) { return scale_bytes_of(kWords, nt); }

struct __align__(16) Ctrl {
    uint64_t full[kMx4StagesMost], empty[kMx4StagesMost];   // stage: copies landed, scales in tensor memory / MMAs done
    uint64_t scales[kMx4StagesMost], sfree[kScaleWarps];    // chunk (pair: stage): scales in shared memory / copied from there
    uint64_t tfull[2], tempty[2];                           // accumulator: complete / stored
    uint64_t drain, drain_copies;
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t total;                                          // row tiles of all experts
};

// E2M1 operands (format 1), both K-major, E8M0 scales (bit 23), FP32 accumulators;
// an MMA of 64 values takes two bytes of a scale word, from byte 0 or (kSecondHalf) 2.
__device__ __forceinline__ uint32_t idesc_mxf4(uint32_t M, uint32_t N)
{
    return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24);
}

constexpr uint32_t kSecondHalf = (2u << 4) | (2u << 29);

// Descriptor of a scale tile for tcgen05.cp: no swizzle, 32 rows of 16 bytes, eight
// to a core matrix of 128.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr)
{
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}

// A scale tile to four columns of tensor memory, lane r % 32 of every quarter,
// column r / 32 (of both CTAs of a pair, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc)
{
    if constexpr (CG == 2) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T over 64 values, each block of 32 scaled.
template <int CG>
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sa,
                                          uint32_t sb, uint32_t accumulate)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// A stage's copies of scales to tensor memory, and its MMAs.  WHOLE: all four
// MMAs; else `steps` of them, at the end of the reduction.  (ATOMS: scale tiles of
// the rows in a word.)
template <int PAIR, int ATOMS, bool WHOLE>
__device__ __forceinline__ void issue_copies(uint32_t from_a, uint32_t from_b, uint32_t to, int steps)
{
    constexpr uint64_t kStep = kMx4Tile >> 4;
    const uint64_t a = scale_desc(from_a), b = scale_desc(from_b);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!WHOLE && 2 * h >= steps) break;
        copy_scales<PAIR>(to + uint32_t(h) * 4u, a + uint64_t(h) * kStep);
#pragma unroll
        for (int i = 0; i < ATOMS; ++i)
            copy_scales<PAIR>(to + 8u + uint32_t(h * ATOMS + i) * 4u, b + uint64_t(h * ATOMS + i) * kStep);
    }
}
template <int PAIR, int ATOMS, bool WHOLE>
__device__ __forceinline__ void issue_mmas(uint32_t d, uint32_t at, uint32_t sa, uint32_t idesc, bool more, int steps)
{
    const uint64_t a = smem_desc_sw128(at, 16, 1024), b = smem_desc_sw128(at + kWBytes, 16, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!WHOLE && k >= steps) break;
        umma_mxf4<PAIR>(d, a + uint64_t(k * 2), b + uint64_t(k * 2), k & 1 ? idesc | kSecondHalf : idesc, sa + uint32_t(k >> 1) * 4u,
                        sa + 8u + uint32_t((k >> 1) * ATOMS) * 4u, k > 0 || more ? 1u : 0u);
    }
}

template <int PAIR, bool OUT_F32>
__global__ void __maxnreg__(96)
    mx4_mma_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapS,
                   const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapR,
                   const Mx4Params p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const uint32_t stage_bytes = stage_bytes_of(PAIR, p.nt);
    const int atoms = mx4_row_atoms(p.nt);
    uint8_t *after = ring_ptr + size_t(p.stages) * stage_bytes;
    const uint32_t chunks = ring + uint32_t(p.stages) * stage_bytes, chunk_bytes = chunk_bytes_of(p.nt);
    constexpr uint32_t kRowScales = kWords * kMx4Tile;           // the rows' in a chunk
    if (PAIR == 1) after += kScaleWarps * chunk_bytes;
    const uint32_t scales_at = stage_bytes - scale_bytes_of(2, p.nt);   // (pair) in a stage
    float *recv = reinterpret_cast<float *>(after);              // split: [split][channel][columns + 4]
    after += p.splits > 1 ? split_bytes(p.nt, p.splits) : 0;
    uint8_t *out_tile = after;                                   // [warp][row][32 channels]
    after += kStoreWarps * kOutTile;
    Ctrl *c = reinterpret_cast<Ctrl *>(after);
    int32_t *row_ids = reinterpret_cast<int32_t *>(c + 1);       // [gathering warp][row]
    int32_t *off = row_ids + kGatherWarps * kGatherRows;
    int32_t *pref = off + p.E + 1;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // (uniform to the compiler)
    const int E = p.E;
    const int rank = PAIR == 2 || p.splits > 1 ? int(cluster_ctarank()) : 0;
    const int half = PAIR == 2 ? rank : 0;
    const bool leader = half == 0;

    // ---- set-up: TMEM, barriers, offsets and the prefix of their row tiles ----
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) {
        for (int i = lane; i <= E; i += 32) off[i] = p.offsets ? p.offsets[i] : (i ? int32_t(p.M) : 0);
        __syncwarp();
        // lane l sums the row tiles of its run of experts, then the runs are scanned
        const int per = (E + 31) / 32, e0 = min(lane * per, E), e1 = min(e0 + per, E);
        int32_t sum = 0;
        bool bad = lane == 0 && off[0] != 0;
        for (int e = e0; e < e1; ++e) {
            bad |= off[e + 1] < off[e] || int64_t(off[e + 1]) > p.M;
            sum += row_tiles(off[e + 1] - off[e], p);
        }
        int32_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        int32_t at = inc - sum;
        for (int e = e0; e < e1; ++e) {
            pref[e] = at;
            at += row_tiles(off[e + 1] - off[e], p);
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 31) {
            pref[E] = inc;
            c->total = bad ? 0 : inc;
            if (bad) atomicCAS(p.status, 0, CAKE_GG_ERR_BAD_OFFSETS);
        }
    } else if (warp == 1) {
        tmem_alloc<PAIR>(smem_u32(&c->tmem_base), 512u);
        tmem_relinquish<PAIR>();
    } else if (tid == 64) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(smem_u32(&c->full[s]), PAIR == 1 && p.rows ? 4 : 3);    // the weights' arming, the rows', the copies of scales
            mbar_init(smem_u32(&c->empty[s]), 1);
            mbar_init(smem_u32(&c->scales[s]), 1);               // the warp that puts them together; its arming
        }
        for (int v = 0; v < kScaleWarps; ++v) mbar_init(smem_u32(&c->sfree[v]), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&c->tfull[b]), 1);
            mbar_init(smem_u32(&c->tempty[b]), uint32_t(kStoreWarps) * PAIR);       // storing warps, of both CTAs
        }
        mbar_init(smem_u32(&c->drain), 1);
        mbar_init(smem_u32(&c->drain_copies), 1);
        fence_barrier_init();
    } else if (tid == 96) {
        c->abort_flag = 0;
        tma_prefetch_desc(&mapW);
        tma_prefetch_desc(&mapS);
        tma_prefetch_desc(&mapX);
        if (PAIR == 2) tma_prefetch_desc(&mapR);
    }
    if (PAIR == 2 || p.splits > 1) cluster_sync_all();           // peers' barriers are ready
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, c->tmem_base, 0);
    const uint32_t d_stride = uint32_t(p.nt);                    // two accumulators, then some stages' scales
    const uint32_t scales0 = tmem + 2u * d_stride, scales_step = 8u + 8u * uint32_t(atoms);
    const int slots = min(scale_slots(p.nt), p.stages);

    // A split cluster takes one unit, each of its CTAs a part of the reduction.
    const uint32_t unit0 = blockIdx.x / uint32_t(PAIR * p.splits);
    const uint32_t step = p.splits > 1 ? uint32_t(p.n_ct) : gridDim.x / PAIR;
    const int32_t total = __shfl_sync(0xffffffffu, c->total, 0);
    const int32_t tiles = p.splits > 1 ? min(total, int32_t(unit0 / uint32_t(p.n_ct)) + 1) : total;
    const int kb0 = p.splits > 1 ? p.n_kb * rank / p.splits : 0;
    const int kb1 = p.splits > 1 ? p.n_kb * (rank + 1) / p.splits : p.n_kb;
    constexpr int kNAlign = 16 * PAIR;
    const uint16_t pair_mask = 3;
    // The MMAs of a pair read the operands and scales of both CTAs, so everything
    // counts on the even one's barrier, which it arms for both.  (A stage's copies
    // follow its `empty`, so that barrier is in the same round; the bytes may come
    // before the arming.)
    auto full_bar = [&](int s) { return PAIR == 2 ? map_to_cta(smem_u32(&c->full[s]), 0) : smem_u32(&c->full[s]); };

    if (warp == 0) {
        // ======================= weight copies =======================
        // The first ring of them does not wait for the token pass.  (Every role waits
        // for the pass before its first wait with a limit, so that the limit does
        // not count the pass.)
        Turn st;
        int issued = 0;       // stages filled, up to the ring's depth
        bool ok = true, passed = false;
        for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next()) {
            const Tile t = w.tile(p.nt, off, pref);
            // (the odd CTA's channels of a pair's last tile may be past the last: their
            // weights come as zeros, for which any scales do)
            const int ct = t.ct * PAIR + half;
            const int32_t scale_w = (t.e * p.n_nt + min(ct, p.n_nt - 1)) * p.n_kt;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (issued == p.stages && !passed) {
                    grid_dependency_wait();
                    passed = true;
                }
                ok = warp_wait(smem_u32(&c->empty[st.at]), st.parity ^ 1u, c, p);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = full_bar(st.at), dst = ring + uint32_t(st.at) * stage_bytes;
                    if (leader) mbar_arrive_expect_tx(smem_u32(&c->full[st.at]), PAIR * kWBytes);
                    if (!((p.debug_flags & CAKE_GG_DEBUG_DROP_FIRST_LOAD) && blockIdx.x == 0 && issued == 0)) {
                        if (PAIR == 2) tma_load_3d_pair(dst, &mapW, bar, kb * (kKB / 2), ct * 128, t.e);
                        else tma_load_3d(dst, &mapW, bar, kb * (kKB / 2), ct * 128, t.e);
                    }
                    if (PAIR == 2) {
                        // (the second words of an odd last stage are another row's: nobody uses them)
                        const uint32_t bar_s = map_to_cta(smem_u32(&c->scales[st.at]), 0);
                        if (leader) mbar_arrive_expect_tx(smem_u32(&c->scales[st.at]), 2u * scale_bytes_of(2, p.nt));
                        tma_load_2d_pair(dst + scales_at, &mapS, bar_s, 0, scale_w + 2 * kb);
                    }
                }
                __syncwarp();
                st.next(p.stages);
                if (issued < p.stages) ++issued;
            }
        }
        grid_dependency_wait();
        if (!ok || aborted(c)) {
            if (leader) {
                drain_stages(st, issued, 1, lane, p.stages, c);
                drain_blind();                                   // (the scales)
            } else drain_blind();
        }
        __syncwarp();
    } else if (warp == 1) {
        // ======================= MMAs (the even CTA of a pair) =======================
        grid_dependency_wait();
        bool ok = true, any = false;
        if (leader) {
            // (with the number of scale tiles a constant each issue is a few instructions)
            auto run = [&](auto n_atoms) {
                constexpr int ATOMS = decltype(n_atoms)::value;
                Turn st, acc, sl;
                for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next()) {
                    const Tile t = w.tile(p.nt, off, pref);
                    const uint32_t n = __shfl_sync(0xffffffffu, uint32_t((t.rows + kNAlign - 1) / kNAlign * kNAlign), 0);
                    const uint32_t idesc = idesc_mxf4(128u * PAIR, n);
                    const int buf = acc.at;
                    if (!warp_wait<PAIR == 2>(smem_u32(&c->tempty[buf]), acc.parity ^ 1u, c, p)) {
                        ok = false;
                        break;
                    }
                    const uint32_t d = tmem + uint32_t(buf) * d_stride;
                    for (int kb = kb0; kb < kb1; ++kb) {
                        ok = warp_wait(smem_u32(&c->full[st.at]), st.parity, c, p);
                        if (!ok) break;
                        if (elect_one()) {
                            tc_fence_after_sync();
                            const uint32_t at = ring + uint32_t(st.at) * stage_bytes, sa = scales0 + uint32_t(sl.at) * scales_step;
                            const int steps = (p.K - kb * kKB + 63) / 64;
                            if (steps >= 4) issue_mmas<PAIR, ATOMS, true>(d, at, sa, idesc, kb > kb0, 4);
                            else issue_mmas<PAIR, ATOMS, false>(d, at, sa, idesc, kb > kb0, steps);
                            if (PAIR == 2) umma_commit_mc<2>(smem_u32(&c->empty[st.at]), pair_mask);
                            else umma_commit<1>(smem_u32(&c->empty[st.at]));
                            if (kb + 1 == kb1) {
                                if (PAIR == 2) umma_commit_mc<2>(smem_u32(&c->tfull[buf]), pair_mask);
                                else umma_commit<1>(smem_u32(&c->tfull[buf]));
                            }
                        }
                        any = true;
                        __syncwarp();
                        st.next(p.stages);
                        sl.next(slots);
                    }
                    acc.next(2);
                }
            };
            if (atoms == 2) run(std::integral_constant<int, 2>());
            else run(std::integral_constant<int, 1>());
            if (!ok && any && elect_one()) {                     // (the lane that issued them)
                umma_commit<PAIR>(smem_u32(&c->drain));
                drain_wait(smem_u32(&c->drain), 0);
            }
        }
        __syncwarp();
    } else if (warp < kScaleWarp0) {
        // ======================= stores =======================
        grid_dependency_wait();                                  // (Y may still be read by the grid before the pass)
        const int q = warp & 3;                                  // tensor memory lanes 32 q ..
        const int side = (warp - kStoreWarp0) >> 2;              // which 32 rows of 64
        Turn acc;
        for (Walk w(unit0, step, p.n_ct); w.g < tiles; w.next()) {
            const Tile t = w.tile(p.nt, off, pref);
            const int n = (t.ct * PAIR + half) * 128 + q * 32 + lane;
            const int buf = acc.at;
            if (!warp_wait(smem_u32(&c->tfull[buf]), acc.parity, c, p)) break;
            tc_fence_after_sync();
            const uint32_t d = tmem + uint32_t(buf) * d_stride + (uint32_t(q * 32) << 16);
            const int per = split_columns(t.rows, p.splits);
            uint8_t *tile = out_tile + (warp - kStoreWarp0) * kOutTile;
            for (int c0 = 32 * side; c0 < t.rows; c0 += 64) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(d + uint32_t(c0), r);
                tmem_ld_wait();
                if (p.splits > 1) {
                    // four columns at a time to the CTA that sums them
                    const uint32_t mine = smem_u32(recv + (size_t(rank) * 128 + q * 32 + lane) * (per + 4));
                    int owner = c0 / per, col = c0 - owner * per;
                    uint32_t to = map_to_cta(mine, uint32_t(owner));
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        if (c0 + j < t.rows) {
                            if (col == per) {
                                col = 0;
                                to = map_to_cta(mine, uint32_t(++owner));
                            }
                            st_cluster_v4(to + uint32_t(col) * 4u,
                                          make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]),
                                                      __uint_as_float(r[j + 3])));
                            col += 4;
                        }
                    continue;
                }
                // through shared memory, transposed: a lane writes its channel of kRows
                // rows, then stores 16 bytes of a row's channels at a time
                constexpr int kSize = OUT_F32 ? 4 : 2, kRows = int(kOutTile) / (32 * kSize);
                constexpr int kPieces = 2 * kSize, kPer = 16 / kSize;   // 16-byte pieces of a row
                const int piece = lane % kPieces, nv = n - lane + piece * kPer;
#pragma unroll
                for (int h = 0; h < 32; h += kRows) {
#pragma unroll
                    for (int j = 0; j < kRows; j += 4) {
                        if (OUT_F32) {
                            uint32_t *dst = reinterpret_cast<uint32_t *>(tile) + j * 32 + lane;
                            dst[0] = r[h + j], dst[32] = r[h + j + 1], dst[64] = r[h + j + 2], dst[96] = r[h + j + 3];
                        } else {
                            const uint32_t a = pack_bf16x2(__uint_as_float(r[h + j]), __uint_as_float(r[h + j + 1]));
                            const uint32_t b = pack_bf16x2(__uint_as_float(r[h + j + 2]), __uint_as_float(r[h + j + 3]));
                            uint16_t *dst = reinterpret_cast<uint16_t *>(tile) + j * 32 + lane;
                            dst[0] = uint16_t(a & 0xffffu), dst[32] = uint16_t(a >> 16);
                            dst[64] = uint16_t(b & 0xffffu), dst[96] = uint16_t(b >> 16);
                        }
                    }
                    __syncwarp();
                    uint8_t *y = static_cast<uint8_t *>(p.Y) + ((int64_t(t.m0) + c0 + h) * p.N + nv) * kSize;
#pragma unroll
                    for (int i = 0; i < kRows * kPieces / 32; ++i) {
                        const int row = lane / kPieces + i * (32 / kPieces);
                        const uint4 v = *reinterpret_cast<const uint4 *>(tile + row * (32 * kSize) + piece * 16);
                        if (c0 + h + row < t.rows && nv < p.N)
                            *reinterpret_cast<uint4 *>(y + int64_t(row) * p.N * kSize) = v;
                    }
                    __syncwarp();
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(smem_u32(&c->tempty[buf]));
                else mbar_arrive_relaxed_cluster(map_to_cta(smem_u32(&c->tempty[buf]), 0));
            }
            acc.next(2);
        }
    } else if (warp < kCopyWarp) {
        // ======================= the rows' scales =======================
        // (A pair's are laid out before, see mx4_arrange_kernel.)  A chunk of stages at a
        // time, each warp with a buffer of its own: the channels' by TMA, the rows' put
        // together, lane l those of the rows l, l + 32, .. of the tile (a word of theirs is
        // 16 bytes of a scale tile's lane).
        grid_dependency_wait();                                  // the tokens
        if constexpr (PAIR == 1) {
            const int v = warp - kScaleWarp0, n_kb = kb1 - kb0;
            const uint32_t dst = chunks + uint32_t(v) * chunk_bytes, bar_free = smem_u32(&c->sfree[v]);
            const uint32_t bar = smem_u32(&c->scales[v]);
            Walk w(unit0, step, p.n_ct);
            const uint8_t *src[kRowWords];
            int kb = v * kChunk;
            bool fresh = true;
            Tile t = {};
            // the warp's next chunk: on to a unit that has one, whose rows are looked up
            auto find = [&] {
                while (kb >= n_kb) {
                    kb -= (n_kb + kChunk - 1) / kChunk * kChunk;     // (a unit's last chunk may be short)
                    w.next();
                    fresh = true;
                }
                if (w.g >= tiles) return false;
                if (fresh) {
                    t = w.tile(p.nt, off, pref);
#pragma unroll
                    for (int i = 0; i < kRowWords; ++i) {
                        const int32_t m = i * 32 + lane;
                        src[i] = nullptr;
                        if (m < t.rows) {
                            int64_t r = int64_t(t.m0) + m;
                            if (p.rows) r = p.rows[r];
                            if (r >= 0 && r < p.T) src[i] = p.xs + mx4_scale_at(r, 0, p.n_kt);
                            else atomicCAS(p.status, 0, CAKE_GG_ERR_BAD_ROWS);
                        }
                    }
                    fresh = false;
                }
                return true;
            };
            uint32_t s[kWords][8] = {};
            auto load = [&] {
#pragma unroll
                for (int h = 0; h < kWords; ++h) {
                    const int kt = 2 * (kb0 + kb) + h;
#pragma unroll
                    for (int i = 0; i < kRowWords; ++i)
                        s[h][i] = src[i] && kt < p.n_kt ? __ldg(reinterpret_cast<const uint32_t *>(src[i] + int64_t(kt) * kMx4Tile)) : 0u;
                }
            };
            uint32_t round = 0;
            bool more = find(), ok = true;
            if (more) load();
            while (more) {
                ok = warp_wait(bar_free, round ^ 1u, c, p);
                if (!ok) break;
                // (a copy may go on into the next row's words, which nobody uses)
                if (elect_one()) tma_load_2d(dst, &mapS, bar, 0, (t.e * p.n_nt + t.ct) * p.n_kt + 2 * (kb0 + kb));
                __syncwarp();
#pragma unroll
                for (int h = 0; h < kWords; ++h) {
                    const uint32_t to = dst + kRowScales + uint32_t(h * atoms) * kMx4Tile + uint32_t(lane) * 16u;
                    sts_v4(to, s[h][0], s[h][1], s[h][2], s[h][3]);
                    if (atoms == 2) sts_v4(to + kMx4Tile, s[h][4], s[h][5], s[h][6], s[h][7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(bar, kRowScales);
                round ^= 1u;
                kb += kScaleWarps * kChunk;
                // (loaded while the buffer is waited for)
                if ((more = find())) load();
            }
            if ((!ok || aborted(c)) && lane == 0) drain_wait(bar, round ^ 1u);
        }
        __syncwarp();
    } else if (warp == kCopyWarp) {
        // ======================= scales to tensor memory (the even CTA of a pair) =======================
        grid_dependency_wait();
        bool ok = true, any = false;
        if (leader) {
            auto run = [&](auto n_atoms) {
                constexpr int ATOMS = decltype(n_atoms)::value;
                Turn st, sl, old, ch;
                int count = 0;                                   // stages so far, up to the slots
                for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next())
                    for (int kb = kb0; kb < kb1; ++kb) {
                        const int i = PAIR == 2 ? 0 : (kb - kb0) % kChunk;
                        if (i == 0) ok = warp_wait(smem_u32(&c->scales[PAIR == 2 ? st.at : ch.at]), PAIR == 2 ? st.parity : ch.parity, c, p);
                        // the stage that had these columns is done (and with it all of this
                        // stage's barrier that came before)
                        if (ok && count == slots) {
                            ok = warp_wait(smem_u32(&c->empty[old.at]), old.parity, c, p);
                            old.next(p.stages);
                        } else ++count;
                        if (!ok) break;
                        const bool last = PAIR == 1 && (i + 1 == kChunk || kb + 1 == kb1);   // of a chunk
                        if (elect_one()) {
                            tc_fence_after_sync();
                            const int steps = (p.K - kb * kKB + 63) / 64;
                            const uint32_t to = scales0 + uint32_t(sl.at) * scales_step;
                            const uint32_t from = PAIR == 2 ? ring + uint32_t(st.at) * stage_bytes + scales_at : chunks + uint32_t(ch.at) * chunk_bytes;
                            const uint32_t fa = from + uint32_t(2 * i) * kMx4Tile;
                            const uint32_t fb = from + (PAIR == 2 ? 2u * kMx4Tile : kRowScales) + uint32_t(2 * i * ATOMS) * kMx4Tile;
                            if (steps >= 4) issue_copies<PAIR, ATOMS, true>(fa, fb, to, 4);
                            else issue_copies<PAIR, ATOMS, false>(fa, fb, to, steps);
                            umma_commit<PAIR>(smem_u32(&c->full[st.at]));
                            if (last) umma_commit<1>(smem_u32(&c->sfree[ch.at]));
                        }
                        any = true;
                        __syncwarp();
                        st.next(p.stages);
                        sl.next(slots);
                        if (last) ch.next(kScaleWarps);
                    }
            };
            if (atoms == 2) run(std::integral_constant<int, 2>());
            else run(std::integral_constant<int, 1>());
            if ((!ok || aborted(c)) && any && elect_one()) {     // (the lane that issued them)
                umma_commit<PAIR>(smem_u32(&c->drain_copies));
                drain_wait(smem_u32(&c->drain_copies), 0);
            }
        }
        __syncwarp();
    } else {
        // ======================= rows =======================
        const int v = warp - kRowsWarp0, n_kb = kb1 - kb0;
        Turn st;
        int issued = 0;
        bool ok = true;
        // a pair's scales of a tile's rows, as they were laid out
        auto scales_of = [&](const Tile &t) { return mx4_slot(off[t.e], t.e, (t.m0 - off[t.e]) / p.nt, p.nt) * int64_t(p.n_kt * atoms); };
        auto load_scales = [&](int s, int64_t at, int kb) {
            tma_load_2d_pair(ring + uint32_t(s) * stage_bytes + scales_at + 2u * kMx4Tile, &mapR, map_to_cta(smem_u32(&c->scales[s]), 0), 0,
                             int32_t(at) + 2 * kb * atoms);
        };
        if (PAIR == 2 || p.rows == nullptr) {                    // (a pair's rows are laid out before)
            grid_dependency_wait();                              // the tokens
            for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next()) {
                const Tile t = w.tile(p.nt, off, pref);
                const int n_half = (t.rows + kNAlign - 1) / kNAlign * 16;   // rows of B in this CTA
                const int n_box = (n_half + p.box - 1) / p.box;
                const uint32_t mb = uint32_t(t.m0 + half * n_half);         // (a box past 2^31 is past the tokens)
                const uint32_t bytes = 128u * uint32_t(n_box * p.box);
                const int64_t scales = scales_of(t);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = warp_wait(smem_u32(&c->empty[st.at]), st.parity ^ 1u, c, p);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t bar = full_bar(st.at), dst = ring + uint32_t(st.at) * stage_bytes + kWBytes;
                        if (leader) mbar_arrive_expect_tx(smem_u32(&c->full[st.at]), PAIR * bytes);
                        if (PAIR == 2) load_scales(st.at, scales, kb);
                        for (int b = 0; b < n_box; ++b)
                            tma_rows<PAIR>(dst + uint32_t(b * p.box) * 128u, &mapX, bar, kb * (kKB / 2), int32_t(mb + uint32_t(b * p.box)));
                    }
                    __syncwarp();
                    st.next(p.stages);
                    if (issued < p.stages) ++issued;
                }
            }
            if (!ok || aborted(c)) {
                if (leader) drain_stages(st, issued, 1, lane, p.stages, c);
                else drain_blind();
            }
        } else {
            // warps 0, 1 and 2, 3 gather alternate stages, each every other four rows
            const int group = v >> 1, side = v & 1;
            int32_t *mine = row_ids + v * kGatherRows;           // tokens of this warp's rows
            const uint32_t ids = smem_u32(mine);
            if (group) st.next(p.stages);
            int kb = group;
            for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next()) {
                const Tile t = w.tile(p.nt, off, pref);
                const int n = (t.rows + 15) / 16 * 16;
                __syncwarp();
                for (int i = lane; i < n / 2; i += 32) {
                    // (counted from the tile's first row: past its last one the sum may pass 2^31)
                    const int32_t m = (i >> 2) * 8 + side * 4 + (i & 3);
                    const int32_t id = m < t.rows ? p.rows[t.m0 + m] : 0;
                    mine[i] = id >= 0 && id < p.T ? id : 0;      // (reported where its scales are read)
                }
                grid_dependency_wait();                          // the tokens (the caller's row numbers were there)
                __syncwarp();
                for (; kb < n_kb; kb += 2) {
                    ok = warp_wait(smem_u32(&c->empty[st.at]), st.parity ^ 1u, c, p);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t bar = smem_u32(&c->full[st.at]);
                        const uint32_t dst = ring + uint32_t(st.at) * stage_bytes + kWBytes + uint32_t(side) * 512u;
                        const int32_t k = (kb0 + kb) * (kKB / 2);
                        mbar_arrive_expect_tx(bar, uint32_t(n) * 64u);
#pragma unroll 4
                        for (int i = 0; i < n / 2; i += 4) {
                            const int4 id = lds_i4(ids + uint32_t(i) * 4u);
                            tma_gather4<1>(dst + uint32_t(i) * 256u, &mapX, bar, k, id.x, id.y, id.z, id.w);
                        }
                    }
                    __syncwarp();
                    st.next(p.stages), st.next(p.stages);
                    if (issued < p.stages) ++issued;
                }
                kb -= n_kb;
            }
            grid_dependency_wait();
            if (!ok || aborted(c)) drain_stages(st, issued, 2, lane, p.stages, c);
        }
        __syncwarp();
    }

    if (PAIR == 1 && p.splits > 1) {
        // every part of this CTA's columns has arrived: sum them in split order
        __syncwarp();
        cluster_sync_all();
        Walk w(unit0, step, p.n_ct);
        if (warp >= kStoreWarp0 && warp < kScaleWarp0 && w.g < tiles && !aborted(c)) {
            const Tile t = w.tile(p.nt, off, pref);
            const int per = split_columns(t.rows, p.splits);
            const int row = (warp & 3) * 32 + lane, n = t.ct * 128 + row;
            const int m0 = rank * per;
            for (int j0 = 16 * ((warp - kStoreWarp0) >> 2); j0 < per && m0 + j0 < t.rows; j0 += 32) {
                // up to 16 rows at a time: their loads do not wait for each other's sums
                float4 sum[4];
                for (int v = 0; v < p.splits; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j0 + 4 * i < per) {
                            const float4 o = *reinterpret_cast<const float4 *>(recv + (size_t(v) * 128 + row) * (per + 4) + j0 + 4 * i);
                            if (v == 0) sum[i] = o;
                            else sum[i].x += o.x, sum[i].y += o.y, sum[i].z += o.z, sum[i].w += o.w;
                        }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y[4] = {sum[i].x, sum[i].y, sum[i].z, sum[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int m = m0 + j0 + 4 * i + k;
                        if (j0 + 4 * i < per && m < t.rows && n < p.N) {
                            const int64_t at = (int64_t(t.m0) + m) * p.N + n;
                            if (OUT_F32) static_cast<float *>(p.Y)[at] = y[k];
                            else static_cast<uint16_t *>(p.Y)[at] = uint16_t(pack_bf16x2(y[k], 0.0f) & 0xffffu);
                        }
                    }
                }
            }
        }
    }

    // ---- teardown ----
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1 && PAIR == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, 512u);
    }
    if (PAIR == 2) {
        // no CTA leaves while its peer may still use its memory or barriers
        cluster_sync_all();
        if (warp == 1) {
            tc_fence_after_sync();
            tmem_dealloc<2>(tmem, 512u);
        }
    }
}

template <int PAIR, bool OUT_F32>
cudaError_t launch(const Mx4Launch &l, bool pdl, cudaStream_t stream)
{
    const Mx4Params &p = l.p;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int na = 0;
    const int cluster = PAIR * p.splits;
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = unsigned(cluster);
        attr[na].val.clusterDim.y = 1;
        attr[na++].val.clusterDim.z = 1;
    }
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3(unsigned(l.grid), 1, 1);
    cfg.blockDim = dim3(PAIR == 1 && p.rows ? kThreadsRouted : kThreads, 1, 1);
    cfg.dynamicSmemBytes = mx4_mma_smem(PAIR, p.nt, p.stages, p.splits, p.E);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = unsigned(na);
    return cudaLaunchKernelEx(&cfg, mx4_mma_kernel<PAIR, OUT_F32>, l.mw, l.ms, l.mx, l.mr, p);
}

}  // namespace

size_t mx4_mma_smem(int pair, int nt, int stages, int splits, int E)
{
    return 1024 + size_t(stages) * stage_bytes_of(pair, nt) + (pair == 2 ? 0 : size_t(kScaleWarps) * chunk_bytes_of(nt)) + (splits > 1 ? split_bytes(nt, splits) : 0) +
           kStoreWarps * kOutTile + sizeof(Ctrl) + size_t(kGatherWarps * kGatherRows) * 4 + size_t(2 * (E + 1)) * 4;
}

int prepare_mx4_mma(Mx4Launch *l, const Mx4Params &p0, const uint8_t *W, const uint8_t *ws, const uint8_t *x, int pair, int sms)
{
    Mx4Params &p = l->p;
    p = p0;
    p.n_ct = (p.N + 128 * pair - 1) / (128 * pair);
    p.n_nt = (p.N + 127) / 128;
    p.n_kb = (p.K + kKB - 1) / kKB;
    p.n_kt = (p.K + 127) / 128;
    p.div_nt = uint32_t((uint64_t(1) << 32) / uint32_t(p.nt / 16) + ((uint64_t(1) << 32) % uint32_t(p.nt / 16) != 0));
    p.box = p.nt / pair % 32 == 0 ? 32 : 16;
    const uint64_t row = uint64_t(p.K) / 2;
    const uint64_t dw[3] = {row, uint64_t(p.N), uint64_t(p.E)};
    const uint64_t sw[2] = {row, uint64_t(p.N) * row};
    const uint32_t bw[3] = {uint32_t(kKB) / 2, 128, 1};
    int rc = encode_tiled(&l->mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, W, dw, sw, bw);
    if (rc != CAKE_GG_OK) return rc;
    const uint64_t ds[2] = {uint64_t(kMx4Tile) / 4, uint64_t(p.E) * uint64_t(p.n_nt) * uint64_t(p.n_kt)};
    const uint64_t ss[1] = {uint64_t(kMx4Tile)};
    const uint32_t bs[2] = {uint32_t(kMx4Tile) / 4, pair == 2 ? 2u : uint32_t(kWords)};
    if (ds[1] > INT32_MAX) return CAKE_GG_ERR_OVERFLOW;
    rc = encode_tiled(&l->ms, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, ws, ds, ss, bs, false);
    if (rc != CAKE_GG_OK) return rc;
    const uint64_t dx[2] = {row, uint64_t(p.T)};
    const uint64_t sx[1] = {row};
    const uint32_t bx[2] = {uint32_t(kKB) / 2, p.rows ? 1u : uint32_t(p.box)};   // (gathered four rows at a time)
    rc = encode_tiled(&l->mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x, dx, sx, bx);
    if (rc != CAKE_GG_OK) return rc;

    if (pair == 2) {
        const int atoms = mx4_row_atoms(p.nt);
        const uint64_t dr[2] = {uint64_t(kMx4Tile) / 4, uint64_t(mx4_slots(p.M, p.E, p.nt)) * uint64_t(p.n_kt * atoms)};
        const uint32_t br[2] = {uint32_t(kMx4Tile) / 4, 2u * uint32_t(atoms)};
        if (dr[1] > INT32_MAX) return CAKE_GG_ERR_OVERFLOW;
        rc = encode_tiled(&l->mr, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, p.xs, dr, ss, br, false);
        if (rc != CAKE_GG_OK) return rc;
    } else l->mr = l->ms;

    // row tiles at most: a whole one per nt rows and a last one per expert with rows
    const int64_t tiles = p.E == 1 ? (p.M + p.nt - 1) / p.nt : p.M / p.nt + (p.M < p.E ? p.M : p.E);
    const int64_t bound = tiles * p.n_ct;
    int64_t grid;
    if (p.splits > 1) {
        grid = bound * p.splits;                       // one cluster per unit
        if (grid > INT32_MAX) return CAKE_GG_ERR_OVERFLOW;
    } else {
        grid = sms / pair < bound ? sms / pair : bound;
        grid = (grid < 1 ? 1 : grid) * pair;
    }
    l->pair = pair;
    l->grid = int32_t(grid);
    auto raise = [&](auto f32) {
        return pair == 2 ? raise_shared_limit<mx4_mma_kernel<2, decltype(f32)::value>>(kMx4SmemLimit)
                         : raise_shared_limit<mx4_mma_kernel<1, decltype(f32)::value>>(kMx4SmemLimit);
    };
    const cudaError_t err = p.out_f32 ? raise(std::true_type()) : raise(std::false_type());
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

int launch_mx4_mma(const Mx4Launch &l, bool pdl, cudaStream_t stream)
{
    cudaError_t err;
    if (l.pair == 2) err = l.p.out_f32 ? launch<2, true>(l, pdl, stream) : launch<2, false>(l, pdl, stream);
    else err = l.p.out_f32 ? launch<1, true>(l, pdl, stream) : launch<1, false>(l, pdl, stream);
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

}  // namespace cakegg
