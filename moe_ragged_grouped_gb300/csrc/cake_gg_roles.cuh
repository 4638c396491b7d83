// cake_gg_roles.cuh -- what the warp-specialised product kernels share: bounded
// waits, the walk over an expert list's row tiles, places in a ring of stages,
// and what a CTA that gives up waits for before it leaves.
//
// Ctrl is a kernel's block of barriers in shared memory (full[], abort_flag),
// Params its parameters (status, timeout_ns; nt, div_nt).
#pragma once

#include <cstdint>

#include "../../include/cake_gg.h"
#include "cake_gg_ptx.cuh"

namespace cakegg {

constexpr uint64_t kDrainNs = 20000000ull;

template <class Ctrl>
__device__ __forceinline__ bool aborted(Ctrl *c) { return *reinterpret_cast<volatile int32_t *>(&c->abort_flag) != 0; }

// Bounded wait on one mbarrier phase by every lane of a warp; warp-uniform
// verdict (false: it ran out, or another role gave up).  PEERS: a barrier on
// which the other CTA of a pair arrives too.
template <bool PEERS = false, class Ctrl, class Params>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, Ctrl *c, const Params &p)
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
                atomicCAS(p.status, 0, CAKE_GG_ERR_TIMEOUT);
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
template <class Ctrl>
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
// 16; exact for n < 2^31).
template <class Params>
__device__ __forceinline__ int32_t row_tiles(int32_t n, const Params &p)
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

}  // namespace cakegg
