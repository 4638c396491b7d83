// cake_gg_int8_mma.cu -- the 8-bit integer products on the tensor cores.
//
//   Y[m, n] = (sum_k q[r(m), k] W[e(m), n, k]) * ws[e(m), n] * xs[r(m)]
//
// sm_103a multiplies 8-bit integers slowly, but every 8-bit integer is exact in
// FP16, every product of two exact in FP32 and so is every sum below 2^24: the
// products run at the FP16 tensor rate and the weights stay 8-bit in memory.
//
// A tile is 128 channels (256 for a pair of CTAs) x up to nt rows of one
// expert, computed transposed: D[channel, row] += W q^T.  The weights are the
// MMA's A operand, which may come from tensor memory: 8-bit tiles arrive in
// shared memory by TMA, converter warps widen them to FP16 and write them to
// tensor memory, so the widened weights cost no shared memory bandwidth.  The
// rows are the B operand, FP16 integers that the token pass wrote: TMA copies
// them, or, where they are routed, gather warps do, row by row through `rows`.
// (Widened here as well, from 8-bit ones, by eight more warps, they made 16384 x
// 4096 -> 4096 take 370 us instead of 302 with the token pass that writes them.)
// B's width follows the rows the tile really has, so a ragged end costs its own
// size only.
//
// Bound: long inputs by the tensor cores and the power limit (12288 x 4096 -> 4096 a
// few calls at a time 204 us, 2.02 PFLOP/s; one after another 16384 x 4096 -> 4096 290
// us, 1.89, and 32768 tokens through 2 of 8 experts 4096 -> 4096 1.24 ms, 1.77),
// decoding batches by the weights' bytes (64 tokens through 4 of 32 experts 6144 ->
// 4096: 6.2 TB/s over the call).
//
// Roles of a CTA: warp 0 copies weights, warp 1 issues MMAs, warps 2-9 scale and
// store (two groups on alternate 32 rows of a tile; with one group short
// reductions wait for it: 20000 x 512 -> 4096 104 us, 88 with two and a tile's scales
// loaded during the one before, long ones 0.5 % less), warps 10-17 convert (two
// groups on alternate stages), warp 18 copies rows, or, where they are routed,
// warps 18-21 gather them, two on every other stage (the first issue of a batch
// of copies takes a few hundred clocks: all four on every stage were late).
#include "cake_gg_int8.h"
#include "cake_gg_int8_widen.cuh"
#include "cake_gg_ptx.cuh"

namespace cakegg {
namespace {

constexpr int kThreads = 608, kThreadsRouted = 704;
constexpr int kStoreWarp0 = 2, kStoreWarps = 8, kStoreThreads = kStoreWarps * 32;
constexpr int kConvWarp0 = 10;
constexpr int kKB = 128;                     // reduction length of a stage
constexpr uint32_t kWBytes = 128 * kKB;      // 8-bit weight tile of a stage
constexpr int kStagesMax = 12;
constexpr int kSlotsMax = 8;
constexpr int kRowsWarp0 = 18;
constexpr int kGatherWarps = 4;
constexpr int kRowsPerCta = 128;             // B rows of a CTA at most
constexpr uint32_t kOutTile = 2048;           // 32 BF16 or 16 FP32 rows x 32 channels of output, per storing warp
constexpr uint32_t kSlotCols = kKB / 2;      // tensor memory columns of a widened weight tile
constexpr uint64_t kDrainNs = 20000000ull;

struct __align__(16) Ctrl {
    uint64_t full[kStagesMax], empty[kStagesMax];     // stage: copies landed / MMAs done
    uint64_t conv[kSlotsMax];                         // slot: weights widened
    uint64_t tfull[2], tempty[2];                     // accumulator: complete / stored
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t total;                                    // row tiles of all experts
};

__device__ __forceinline__ bool aborted(Ctrl *c) { return *reinterpret_cast<volatile int32_t *>(&c->abort_flag) != 0; }

// Bounded wait on one mbarrier phase by every lane of a warp; warp-uniform
// verdict (false: it ran out, or another role gave up).  PEERS: a barrier on
// which the other CTA of a pair arrives too.
template <bool PEERS = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, Ctrl *c, const I8Params &p)
{
    auto poll = [&] { return PEERS ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    bool ok = poll();
    // (the global timer is slow to read: a wait that is soon over never asks it)
    for (int i = 0; i < 256 && !ok; ++i) ok = poll();
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        while (true) {
            for (int i = 0; i < 256 && !ok; ++i) ok = poll();
            if (ok || aborted(c)) break;
            if (global_timer_ns() - t0 > p.timeout_ns) {
                *reinterpret_cast<volatile int32_t *>(&c->abort_flag) = 1;
                atomicCAS(p.status, 0, kI8StatusTimeout);
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// A copy phase in flight lands before the CTA leaves (bounded).
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > kDrainNs) return;
}

// After an abort, copies whose barrier is another CTA's: they land in a time that
// drain_wait would give up after.
__device__ __forceinline__ void drain_blind()
{
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kDrainNs) {}
}

// One lane of a converged warp.  (The MMA's descriptors then stay in uniform
// registers: under a test of the lane number each of the eight issues of a
// stage took 70 clocks, a stage 960; elected, 281.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Four rows of a tensor (its box one row high) to consecutive 128-byte rows (of a
// CTA of a pair: counted on the mbarrier of either of the two, by cluster address).
template <int PAIR>
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t r0,
                                            int32_t r1, int32_t r2, int32_t r3)
{
    if constexpr (PAIR == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
            : "memory");
}
template <int PAIR>
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t row)
{
    if constexpr (PAIR == 2) tma_load_2d_pair(dst, map, bar, x, row);
    else tma_load_2d(dst, map, bar, x, row);
}

// FP32 accumulators, FP16 operands (A and B format fields 0), both K-major.
__device__ __forceinline__ uint32_t idesc_f16(uint32_t M, uint32_t N)
{
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// A place in a ring and the parity of its current round.  A wait for the
// opposite parity passes at once in the first round: the ring starts free.
struct Turn {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++at == n) {
            at = 0;
            parity ^= 1u;
        }
    }
    __device__ __forceinline__ void back(int n)
    {
        if (at-- == 0) {
            at = n - 1;
            parity ^= 1u;
        }
    }
};

// After an abort: the copies into this warp's last `issued` stages, `every` apart
// before `st`, land before the CTA leaves.  (A phase that lacks the other
// warp's part runs into the limit, by when the copies have long landed.)
__device__ __forceinline__ void drain_stages(Turn st, int issued, int every, int lane, int stages, Ctrl *c)
{
    if (lane != 0) return;
    for (int i = 0; i < issued; ++i) {
        for (int k = 0; k < every; ++k) st.back(stages);
        drain_wait(smem_u32(&c->full[st.at]), st.parity);
    }
}

__device__ __forceinline__ int32_t within(int32_t v, int32_t lo, int32_t hi) { return min(max(v, lo), hi); }

// Row tiles of n rows: n / nt rounded up, by a multiplication (nt = 16 k, 2 <= k <=
// 12; exact for n < 2^31).
__device__ __forceinline__ int32_t row_tiles(int32_t n, const I8MmaParams &p)
{
    if (n <= 0) return 0;
    const uint32_t t = (uint32_t(n) + 15u) >> 4;                 // (n + nt - 1) / nt = (t + k - 1) / k
    return int32_t(__umulhi(t + uint32_t(p.nt >> 4) - 1u, p.div_nt));
}

__device__ __forceinline__ int4 lds_i4(uint32_t addr)
{
    int4 v;
    asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// A split tile's rows are summed by the CTAs of its cluster, each its share, in
// whole fours; what a CTA receives (a row of it padded by 16 bytes: no bank
// conflicts).
__host__ __device__ constexpr int split_columns(int rows, int splits)
{
    return ((rows + 3) / 4 + splits - 1) / splits * 4;
}
__host__ __device__ constexpr size_t split_bytes(int nt, int splits)
{
    return size_t(splits) * 128 * size_t(split_columns(nt, splits) + 4) * sizeof(float);
}

struct Tile {
    int e, ct;                // expert, channel tile
    int32_t m0, rows;         // first row, rows in the tile
};

// The units of a CTA (pair), a fixed stride over (row tile, channel tile) with
// the channel tile fastest: concurrent CTAs share an expert's rows, and its
// weights stay in L2 between its row tiles.
struct Walk {
    int32_t g, ct, e, dg, dct, n_ct;
    __device__ __forceinline__ Walk(uint32_t first, uint32_t step, int32_t n) : e(0), n_ct(n)
    {
        g = int32_t(first / uint32_t(n));
        ct = int32_t(first % uint32_t(n));
        dg = int32_t(step / uint32_t(n));
        dct = int32_t(step % uint32_t(n));
    }
    __device__ __forceinline__ void next()
    {
        g += dg;
        ct += dct;
        if (ct >= n_ct) {
            ct -= n_ct;
            ++g;
        }
    }
    __device__ __forceinline__ Tile tile(int nt, const int32_t *off, const int32_t *pref)
    {
        while (pref[e + 1] <= g) ++e;
        Tile t;
        t.ct = ct;
        t.e = e;
        t.m0 = off[e] + (g - pref[e]) * nt;
        t.rows = min(nt, off[e + 1] - t.m0);
        return t;
    }
};

template <int PAIR, bool OUT_F32>
__global__ void __maxnreg__(80)
    i8_mma_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
                  const I8MmaParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const uint32_t x_rows = uint32_t(p.nt / PAIR);               // B rows of this CTA in a stage
    const uint32_t stage_bytes = kWBytes + x_rows * 256u;
    uint8_t *after = ring_ptr + size_t(p.stages) * stage_bytes;
    float *recv = reinterpret_cast<float *>(after);              // split: [split][channel][columns + 4]
    after += p.splits > 1 ? split_bytes(p.nt, p.splits) : 0;
    uint8_t *out_tile = after;                                   // [warp][row][32 channels]
    after += kStoreWarps * kOutTile;
    Ctrl *c = reinterpret_cast<Ctrl *>(after);
    float *xs_tile = reinterpret_cast<float *>(c + 1);           // [2][nt]
    int32_t *row_ids = reinterpret_cast<int32_t *>(xs_tile + 2 * p.nt);   // [gathering warp][row]
    int32_t *off = row_ids + kGatherWarps * kRowsPerCta / 2;
    int32_t *pref = off + p.b.E + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = p.b.E;
    const int rank = PAIR == 2 || p.splits > 1 ? int(cluster_ctarank()) : 0;
    const int half = PAIR == 2 ? rank : 0;
    const bool leader = half == 0;

    // ---- set-up: TMEM, barriers, offsets and the prefix of their row tiles ----
    if (!p.b.early) grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) {
        for (int i = lane; i <= E; i += 32) off[i] = p.b.offsets ? p.b.offsets[i] : (i ? int32_t(p.b.M) : 0);
        __syncwarp();
        // lane l sums the row tiles of its run of experts, then the runs are scanned
        const int per = (E + 31) / 32, e0 = min(lane * per, E), e1 = min(e0 + per, E);
        const int32_t lo = int32_t(p.b.m_lo), hi = int32_t(p.b.m_hi);
        int32_t sum = 0;
        bool bad = lane == 0 && off[0] != 0;
        for (int e = e0; e < e1; ++e) {
            bad |= off[e + 1] < off[e] || int64_t(off[e + 1]) > p.b.M;
            sum += row_tiles(within(off[e + 1], lo, hi) - within(off[e], lo, hi), p);
        }
        __syncwarp();
        if (lo > 0 || hi < p.b.M)                                // each expert's rows of this launch
            for (int i = lane; i <= E; i += 32) off[i] = within(off[i], lo, hi);
        __syncwarp();
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
            if (bad) atomicCAS(p.b.status, 0, kI8StatusBadOffsets);
        }
    } else if (warp == 1) {
        tmem_alloc<PAIR>(smem_u32(&c->tmem_base), 512u);
        tmem_relinquish<PAIR>();
    } else if (tid == 64) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(smem_u32(&c->full[s]), !leader ? 1 : p.b.rows ? 3 : 2);   // the weights' arming and the rows'
            mbar_init(smem_u32(&c->empty[s]), 1);
        }
        for (int a = 0; a < p.slots; ++a) mbar_init(smem_u32(&c->conv[a]), 4u * PAIR);   // the group's warps, of both CTAs
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&c->tfull[b]), 1);
            mbar_init(smem_u32(&c->tempty[b]), uint32_t(kStoreWarps) * PAIR);       // storing warps, of both CTAs
        }
        mbar_init(smem_u32(&c->drain), 1);
        fence_barrier_init();
    } else if (tid == 96) {
        c->abort_flag = 0;
        tma_prefetch_desc(&mapW);
        tma_prefetch_desc(&mapX);
    }
    if (PAIR == 2 || p.splits > 1) cluster_sync_all();           // peers' barriers are ready
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = c->tmem_base;
    const uint32_t d_stride = uint32_t(p.nt);                    // two accumulators, then the widened weights
    const uint32_t slots0 = tmem + 2u * d_stride;

    // A split cluster takes one unit, each of its CTAs a part of the reduction.
    const uint32_t unit0 = blockIdx.x / uint32_t(PAIR * p.splits);
    const uint32_t step = p.splits > 1 ? uint32_t(p.n_ct) : gridDim.x / PAIR;
    const int32_t tiles = p.splits > 1 ? min(c->total, int32_t(unit0 / uint32_t(p.n_ct)) + 1) : c->total;
    const int kb0 = p.splits > 1 ? p.n_kb * rank / p.splits : 0;
    const int kb1 = p.splits > 1 ? p.n_kb * (rank + 1) / p.splits : p.n_kb;
    constexpr int kNAlign = 16 * PAIR;
    float ws_split = 0.0f;                                       // a storing thread's channel scale, for the split sum
    const uint16_t pair_mask = 3;

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
            for (int kb = kb0; kb < kb1; ++kb) {
                if (issued == p.stages && !passed) {
                    grid_dependency_wait();
                    passed = true;
                }
                ok = warp_wait(smem_u32(&c->empty[st.at]), st.parity ^ 1u, c, p.b);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = smem_u32(&c->full[st.at]);
                    mbar_arrive_expect_tx(bar, kWBytes);
                    if (!((p.debug_flags & CAKE_GG_DEBUG_DROP_FIRST_LOAD) && blockIdx.x == 0 && issued == 0))
                        tma_load_3d(ring + uint32_t(st.at) * stage_bytes, &mapW, bar, kb * kKB, (t.ct * PAIR + half) * 128, t.e);
                }
                __syncwarp();
                st.next(p.stages);
                if (issued < p.stages) ++issued;
            }
        }
        grid_dependency_wait();
        if (!ok || aborted(c)) drain_stages(st, issued, 1, lane, p.stages, c);
        __syncwarp();
    } else if (warp == 1) {
        // ======================= MMAs (the even CTA of a pair) =======================
        grid_dependency_wait();
        Turn st, sl, acc;
        bool ok = true, any = false;
        if (leader) {
            for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next()) {
                const Tile t = w.tile(p.nt, off, pref);
                const uint32_t n = uint32_t((t.rows + kNAlign - 1) / kNAlign * kNAlign);
                const uint32_t idesc = idesc_f16(128u * PAIR, n);
                const int buf = acc.at;
                if (!warp_wait<PAIR == 2>(smem_u32(&c->tempty[buf]), acc.parity ^ 1u, c, p.b)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem + uint32_t(buf) * d_stride;
                for (int kb = kb0; kb < kb1; ++kb) {
                    // the converters of both CTAs saw their weights land, and this
                    // CTA's the rows of both
                    ok = warp_wait<PAIR == 2>(smem_u32(&c->conv[sl.at]), sl.parity, c, p.b);
                    if (!ok) break;
                    if (elect_one()) {
                        tc_fence_after_sync();
                        const uint32_t xb = ring + uint32_t(st.at) * stage_bytes + kWBytes;
                        const uint64_t b0 = smem_desc_sw128(xb, 16, 1024), b1 = smem_desc_sw128(xb + x_rows * 128u, 16, 1024);
                        const uint32_t at = slots0 + uint32_t(sl.at) * kSlotCols;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            umma_bf16_ta<PAIR>(d, at + uint32_t(k) * 8u, (k < 4 ? b0 : b1) + uint64_t(k & 3) * 2u, idesc,
                                               kb > kb0 || k > 0 ? 1u : 0u);
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
                    sl.next(p.slots);
                }
                acc.next(2);
            }
            if (!ok && any && elect_one()) {                     // (the lane that issued them)
                umma_commit<PAIR>(smem_u32(&c->drain));
                drain_wait(smem_u32(&c->drain), 0);
            }
        }
        __syncwarp();
    } else if (warp < kConvWarp0) {
        // ======================= scales and stores =======================
        grid_dependency_wait();                                  // the token scales
        const int q = warp & 3;                                  // tensor memory lanes 32 q ..
        const int side = (warp - kStoreWarp0) >> 2;              // which 32 rows of 64
        Turn acc, xb;
        // A tile's scales (a row and a channel of each thread) are loaded while the
        // tile before it is stored.
        static_assert(kStoreThreads >= 192, "a row a thread");
        const int mine = tid - 32 * kStoreWarp0;
        float x_next = 0.0f, ws_next = 0.0f;
        auto scales = [&](const Tile &t) {
            if (mine < t.rows) {
                int64_t r = t.m0 + mine;
                if (p.b.rows) r = p.b.rows[r];
                const bool bad = r < 0 || r >= p.b.T;
                if (bad) atomicCAS(p.b.status, 0, kI8StatusBadRows);
                x_next = bad ? 0.0f : p.b.xs[r];
            }
            const int n = (t.ct * PAIR + half) * 128 + q * 32 + lane;
            ws_next = n < p.b.N ? p.b.ws[int64_t(t.e) * p.b.N + n] : 0.0f;
        };
        Walk w(unit0, step, p.n_ct);
        Tile t = {}, t_next = {};
        if (w.g < tiles) scales(t_next = w.tile(p.nt, off, pref));
        while (w.g < tiles) {
            t = t_next;
            float *xs = xs_tile + xb.at * p.nt;
            if (mine < t.rows) xs[mine] = x_next;
            const float ws = ws_next;
            const int n = (t.ct * PAIR + half) * 128 + q * 32 + lane;
            const int buf = acc.at;
            const bool ok = warp_wait(smem_u32(&c->tfull[buf]), acc.parity, c, p.b);
            // the scales are in (their buffer is rewritten two tiles on, after the
            // barrier between), and the warps go on or give up together
            if (!named_bar_and(1, kStoreThreads, ok)) break;
            tc_fence_after_sync();
            w.next();
            if (w.g < tiles) scales(t_next = w.tile(p.nt, off, pref));
            const uint32_t d = tmem + uint32_t(buf) * d_stride + (uint32_t(q * 32) << 16);
            const int per = split_columns(t.rows, p.splits);
            uint8_t *tile = out_tile + (warp - kStoreWarp0) * kOutTile;
            ws_split = ws;
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
                        const float4 x4 = *reinterpret_cast<const float4 *>(xs + c0 + h + j);
                        const float v[4] = {__uint_as_float(r[h + j]) * ws * x4.x, __uint_as_float(r[h + j + 1]) * ws * x4.y,
                                            __uint_as_float(r[h + j + 2]) * ws * x4.z, __uint_as_float(r[h + j + 3]) * ws * x4.w};
                        if (OUT_F32) {
                            float *dst = reinterpret_cast<float *>(tile) + j * 32 + lane;
                            dst[0] = v[0], dst[32] = v[1], dst[64] = v[2], dst[96] = v[3];
                        } else {
                            const uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
                            uint16_t *dst = reinterpret_cast<uint16_t *>(tile) + j * 32 + lane;
                            dst[0] = uint16_t(a & 0xffffu), dst[32] = uint16_t(a >> 16);
                            dst[64] = uint16_t(b & 0xffffu), dst[96] = uint16_t(b >> 16);
                        }
                    }
                    __syncwarp();
                    uint8_t *y = static_cast<uint8_t *>(p.b.Y) + ((int64_t(t.m0) + c0 + h) * p.b.N + nv) * kSize;
#pragma unroll
                    for (int i = 0; i < kRows * kPieces / 32; ++i) {
                        const int row = lane / kPieces + i * (32 / kPieces);
                        const uint4 v = *reinterpret_cast<const uint4 *>(tile + row * (32 * kSize) + piece * 16);
                        if (c0 + h + row < t.rows && nv < p.b.N)
                            *reinterpret_cast<uint4 *>(y + int64_t(row) * p.b.N * kSize) = v;
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
            xb.next(2);
        }
    } else if (warp < kRowsWarp0) {
        // ======================= weights to FP16 =======================
        const int q = warp & 3, group = (warp - kConvWarp0) >> 2;
        const int row = q * 32 + lane;                           // weight row = tensor memory lane
        const int n_kb = kb1 - kb0;
        grid_dependency_wait();
        // A slot is free once the MMAs of the stage that last used it, `slots` before
        // this one, are done: that stage's `empty` says so.  (slots <= stages, and <=
        // stages - 2 in an odd ring: a group then meets a barrier every second round,
        // and this wait at its last stage has to cover the round between.)
        Turn st, sl, last;
        if (group) st.next(p.stages), sl.next(p.slots);
        int it = group, kb = group;
        Walk w(unit0, step, p.n_ct);
        auto widen = [&](const uint8_t *src, int h, uint32_t (&f)[32]) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src + (((h * 4 + v) ^ (row & 7)) << 4));
                widen4(x.x, f[v * 8], f[v * 8 + 1]);
                widen4(x.y, f[v * 8 + 2], f[v * 8 + 3]);
                widen4(x.z, f[v * 8 + 4], f[v * 8 + 5]);
                widen4(x.w, f[v * 8 + 6], f[v * 8 + 7]);
            }
        };
        while (true) {
            while (kb >= n_kb) {
                kb -= n_kb;
                w.next();
            }
            if (w.g >= tiles) break;
            if (!warp_wait(smem_u32(&c->full[st.at]), st.parity, c, p.b)) break;
            const uint8_t *src = ring_ptr + size_t(st.at) * stage_bytes + row * 128;
            const uint32_t dst = slots0 + uint32_t(sl.at) * kSlotCols + (uint32_t(q * 32) << 16);
            uint32_t f[32];
            widen(src, 0, f);
            if (it >= p.slots) {
                if (it > p.slots) last.next(p.stages);
                if (it > p.slots + 1) last.next(p.stages);
                if (!warp_wait(smem_u32(&c->empty[last.at]), last.parity, c, p.b)) break;
                tc_fence_after_sync();
            }
            tmem_st_32x32b_x32(dst, f);
            uint32_t g[32];
            widen(src, 1, g);
            tmem_st_32x32b_x32(dst + 32u, g);
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                // What the other CTA's MMAs read of this one: tensor memory, complete
                // and ordered by the fence above and the one after their wait, for which
                // an arrival at cluster scope is enough (as a release there it takes 557 us
                // for 319, 16384 x 4096 -> 4096); and rows, whose copies count on that
                // CTA's own barrier.
                if (leader) mbar_arrive(smem_u32(&c->conv[sl.at]));
                else mbar_arrive_relaxed_cluster(map_to_cta(smem_u32(&c->conv[sl.at]), 0));
            }
            st.next(p.stages), st.next(p.stages);
            sl.next(p.slots), sl.next(p.slots);
            it += 2;
            kb += 2;
        }
        __syncwarp();
    } else {
        // ======================= rows =======================
        // The MMAs of a pair read the rows of both CTAs, so both count on the even
        // one's barrier, which it arms for both; the odd one's holds its weights only.
        // (A stage's copies follow its `empty`, so the even one's barrier is in the
        // same round; the bytes may come before the arming.)
        const int v = warp - kRowsWarp0, n_kb = kb1 - kb0;
        auto full_bar = [&](int s) { return PAIR == 2 ? map_to_cta(smem_u32(&c->full[s]), 0) : smem_u32(&c->full[s]); };
        Turn st;
        int issued = 0;
        bool ok = true;
        if (p.b.rows == nullptr) {
            grid_dependency_wait();                              // the tokens
            for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next()) {
                const Tile t = w.tile(p.nt, off, pref);
                const int n_half = (t.rows + kNAlign - 1) / kNAlign * 16;   // rows of B in this CTA
                const int n_box = (n_half + p.box - 1) / p.box;
                const uint32_t mb = uint32_t(t.m0 + half * n_half);         // (a box past 2^31 is past the tokens)
                const uint32_t bytes = 256u * uint32_t(n_box * p.box);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = warp_wait(smem_u32(&c->empty[st.at]), st.parity ^ 1u, c, p.b);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t bar = full_bar(st.at), dst = ring + uint32_t(st.at) * stage_bytes + kWBytes;
                        if (leader) mbar_arrive_expect_tx(smem_u32(&c->full[st.at]), PAIR * bytes);
                        for (int b = 0; b < n_box; ++b) {
                            tma_rows<PAIR>(dst + uint32_t(b * p.box) * 128u, &mapX, bar, kb * kKB, int32_t(mb + uint32_t(b * p.box)));
                            tma_rows<PAIR>(dst + (x_rows + uint32_t(b * p.box)) * 128u, &mapX, bar, kb * kKB + 64, int32_t(mb + uint32_t(b * p.box)));
                        }
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
            int32_t *mine = row_ids + v * (kRowsPerCta / 2);     // tokens of this warp's rows
            const uint32_t ids = smem_u32(mine);
            if (group) st.next(p.stages);
            int kb = group;
            for (Walk w(unit0, step, p.n_ct); ok && w.g < tiles; w.next()) {
                const Tile t = w.tile(p.nt, off, pref);
                const int n_half = (t.rows + kNAlign - 1) / kNAlign * 16;
                __syncwarp();
                for (int i = lane; i < n_half / 2; i += 32) {
                    // (counted from the tile's first row: past its last one the sum may pass 2^31)
                    const int32_t m = half * n_half + (i >> 2) * 8 + side * 4 + (i & 3);
                    const int32_t id = m < t.rows ? p.b.rows[t.m0 + m] : 0;
                    mine[i] = id >= 0 && id < p.b.T ? id : 0;    // (reported where it is scaled)
                }
                grid_dependency_wait();                          // the tokens (the caller's row numbers were there)
                __syncwarp();
                for (; kb < n_kb; kb += 2) {
                    ok = warp_wait(smem_u32(&c->empty[st.at]), st.parity ^ 1u, c, p.b);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t bar = full_bar(st.at);
                        const uint32_t dst = ring + uint32_t(st.at) * stage_bytes + kWBytes + uint32_t(side) * 512u;
                        const int32_t k = (kb0 + kb) * kKB;
                        if (leader) mbar_arrive_expect_tx(smem_u32(&c->full[st.at]), PAIR * uint32_t(n_half) * 128u);
#pragma unroll 4
                        for (int i = 0; i < n_half / 2; i += 4) {
                            const int4 id = lds_i4(ids + uint32_t(i) * 4u);
                            tma_gather4<PAIR>(dst + uint32_t(i) * 256u, &mapX, bar, k, id.x, id.y, id.z, id.w);
                            tma_gather4<PAIR>(dst + x_rows * 128u + uint32_t(i) * 256u, &mapX, bar, k + 64, id.x, id.y, id.z, id.w);
                        }
                    }
                    __syncwarp();
                    st.next(p.stages), st.next(p.stages);
                    if (issued < p.stages) ++issued;
                }
                kb -= n_kb;
            }
            grid_dependency_wait();
            if (!ok || aborted(c)) {
                if (leader) drain_stages(st, issued, 2, lane, p.stages, c);
                else drain_blind();
            }
        }
        __syncwarp();
    }

    if (PAIR == 1 && p.splits > 1) {
        // every part of this CTA's columns has arrived: sum them in split order
        __syncwarp();
        cluster_sync_all();
        Walk w(unit0, step, p.n_ct);
        if (warp >= kStoreWarp0 && warp < kConvWarp0 && w.g < tiles && !aborted(c)) {
            const Tile t = w.tile(p.nt, off, pref);
            const int per = split_columns(t.rows, p.splits);
            const int row = (warp & 3) * 32 + lane, n = t.ct * 128 + row;
            const float ws = ws_split;
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
                    const float v[4] = {sum[i].x, sum[i].y, sum[i].z, sum[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int m = m0 + j0 + 4 * i + k;
                        if (j0 + 4 * i < per && m < t.rows && n < p.b.N) {
                            const float y = v[k] * ws * xs_tile[m];
                            const int64_t at = (int64_t(t.m0) + m) * p.b.N + n;
                            if (OUT_F32) static_cast<float *>(p.b.Y)[at] = y;
                            else static_cast<uint16_t *>(p.b.Y)[at] = uint16_t(pack_bf16x2(y, 0.0f) & 0xffffu);
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

// The opt-in limit of shared memory, raised once per device.
template <int PAIR, bool OUT_F32>
cudaError_t raise_limit()
{
    static bool raised[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!raised[dev]) {
        err = cudaFuncSetAttribute(i8_mma_kernel<PAIR, OUT_F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kI8SmemLimit));
        if (err != cudaSuccess) return err;
        raised[dev] = true;
    }
    return cudaSuccess;
}

template <int PAIR, bool OUT_F32>
cudaError_t launch(const I8MmaLaunch &l, bool pdl, cudaStream_t stream)
{
    const I8MmaParams &p = l.p;
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
    cfg.blockDim = dim3(p.b.rows ? kThreadsRouted : kThreads, 1, 1);
    cfg.dynamicSmemBytes = i8_mma_smem(PAIR, p.nt, p.stages, p.splits, p.b.E);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = unsigned(na);
    return cudaLaunchKernelEx(&cfg, i8_mma_kernel<PAIR, OUT_F32>, l.mw, l.mx, p);
}

}  // namespace

size_t i8_mma_smem(int pair, int nt, int stages, int splits, int E)
{
    return 1024 + size_t(stages) * (kWBytes + size_t(nt / pair) * 256) +
           (splits > 1 ? split_bytes(nt, splits) : 0) + kStoreWarps * kOutTile + sizeof(Ctrl) + size_t(2 * nt) * 4 +
           size_t(kGatherWarps * kRowsPerCta / 2) * 4 + size_t(2 * (E + 1)) * 4;
}

int prepare_i8_mma(I8MmaLaunch *l, const I8MmaParams &p0, const uint16_t *q, int pair, int sms)
{
    I8MmaParams &p = l->p;
    p = p0;
    p.n_ct = (p.b.N + 128 * pair - 1) / (128 * pair);
    p.n_kb = (p.b.K + kKB - 1) / kKB;
    p.div_nt = uint32_t((uint64_t(1) << 32) / uint32_t(p.nt / 16) + ((uint64_t(1) << 32) % uint32_t(p.nt / 16) != 0));
    p.box = p.nt / pair % 32 == 0 ? 32 : 16;
    const uint64_t dw[3] = {uint64_t(p.b.K), uint64_t(p.b.N), uint64_t(p.b.E)};
    const uint64_t sw[2] = {uint64_t(p.b.K), uint64_t(p.b.N) * uint64_t(p.b.K)};
    const uint32_t bw[3] = {uint32_t(kKB), 128, 1};
    int rc = encode_tiled(&l->mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.b.W, dw, sw, bw);
    if (rc != CAKE_GG_OK) return rc;

    const uint64_t dx[2] = {uint64_t(p.b.K), uint64_t(p.b.T)};
    const uint64_t sx[1] = {uint64_t(p.b.K) * 2};
    const uint32_t bx[2] = {64, p.b.rows ? 1u : uint32_t(p.box)};   // (gathered four rows at a time)
    rc = encode_tiled(&l->mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, q, dx, sx, bx);
    if (rc != CAKE_GG_OK) return rc;

    // row tiles at most: a whole one per nt rows and a last one per expert with rows
    const int64_t m = p.b.m_hi - p.b.m_lo;
    const int64_t tiles = p.b.E == 1 ? (m + p.nt - 1) / p.nt : m / p.nt + (m < p.b.E ? m : p.b.E);
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
    const cudaError_t err = pair == 2 ? (p.b.out_f32 ? raise_limit<2, true>() : raise_limit<2, false>())
                                      : (p.b.out_f32 ? raise_limit<1, true>() : raise_limit<1, false>());
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

int launch_i8_mma(const I8MmaLaunch &l, bool pdl, cudaStream_t stream)
{
    cudaError_t err;
    if (l.pair == 2) err = l.p.b.out_f32 ? launch<2, true>(l, pdl, stream) : launch<2, false>(l, pdl, stream);
    else err = l.p.b.out_f32 ? launch<1, true>(l, pdl, stream) : launch<1, false>(l, pdl, stream);
    return err == cudaSuccess ? CAKE_GG_OK : CAKE_GG_ERR_CUDA;
}

}  // namespace cakegg
