// What the kernels of the expanded form of latent attention and of its
// gradients share on the device: units of packed sequences, bounded waits,
// rows of a tile past a sequence's end.
#pragma once

#include "latent.h"
#include "rows.cuh"
#include "stream_order.cuh"

namespace attn {

// A block of rows (of queries, or of keys) of one head of one sequence.
struct LatentUnit {
    int head, row0;   // the block's first row, within its sequence
    int q0, sq;       // the sequence's first query token, its queries
    int k0, sk;       // its first key token, its keys
};

// Unit u of sequences x groups of heads x blocks of rows x heads of a group:
// the blocks of some heads together, so that the L2 holds what they share; of
// queries (`last_first`) the later blocks, which see more keys, first.  A
// sequence whose offsets fall outside the totals is empty.
struct LatentWork {
    int head, row0, q0, q1, k0, k1;
};

// (What the answer takes from memory is on its way when this returns, and
// looked at by latent_unit.)
__device__ __forceinline__ LatentWork latent_work(const LatentSeqs &s, unsigned u, int blocks, int group, int rows, bool last_first)
{
    const unsigned per_seq = static_cast<unsigned>(blocks) * s.h, seq = u / per_seq;
    LatentWork w;
    w.q0 = s.cu_q[seq], w.q1 = s.cu_q[seq + 1], w.k0 = s.cu_k[seq], w.k1 = s.cu_k[seq + 1];
    u -= seq * per_seq;
    const unsigned hg = u / (blocks * group);
    u -= hg * blocks * group;
    const int heads = min(group, s.h - static_cast<int>(hg) * group);
    const int blk = u / heads;
    w.head = hg * group + u - blk * heads;
    w.row0 = (last_first ? blocks - 1 - blk : blk) * rows;
    return w;
}

__device__ __forceinline__ LatentUnit latent_unit(const LatentSeqs &s, const LatentWork &w)
{
    LatentUnit un{w.head, w.row0, w.q0, w.q1 - w.q0, w.k0, w.k1 - w.k0};
    if (un.q0 < 0 || un.sq < 0 || un.q0 > s.total_q - un.sq || un.k0 < 0 || un.sk < 0 || un.k0 > s.total_k - un.sk)
        un.q0 = un.sq = un.k0 = un.sk = 0;
    return un;
}

// Waits of a CTA that give up together: one that runs out records where in
// the status word and raises the flag that ends the others.
struct BoundedWaits {
    uint32_t *abort;
    uint32_t *status;
    uint64_t timeout_ns;

    __device__ __forceinline__ bool one(uint32_t bar, uint32_t parity, uint32_t site) const
    {
        if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
        volatile uint32_t *flag = abort;
        const uint64_t t0 = global_timer_ns();
        while (true) {
            for (int i = 0; i < 64; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*flag) return false;
            if (global_timer_ns() - t0 > timeout_ns) {
                *flag = 1u;
                record_status(status, STATUS_TIMEOUT, site);
                return false;
            }
        }
    }
    // two of them: the second is looked at while the first's answer is on its way
    __device__ __forceinline__ bool warp(uint32_t bar_a, uint32_t parity_a, uint32_t bar_b, uint32_t parity_b, uint32_t site) const
    {
        bool a = mbar_try_wait(bar_a, parity_a), b = mbar_try_wait(bar_b, parity_b);
        if (!(a && b)) a = one(bar_a, parity_a, site), b = one(bar_b, parity_b, site);
        return static_cast<bool>(__all_sync(0xffffffffu, a && b));
    }
    // by every lane of a warp, with a warp-uniform result
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity, uint32_t site) const
    {
        return static_cast<bool>(__all_sync(0xffffffffu, one(bar, parity, site)));
    }
};

// Rows [valid, rows) of a panel of 128-byte rows, zeroed by a whole warp and
// visible to the products that it issues afterwards.  (0 times what is not
// finite would not be 0.)
__device__ __forceinline__ void zero_panel_rows(uint32_t panel, int valid, int rows)
{
    const int lane = threadIdx.x & 31;
    for (int c = max(valid, 0) * 8 + lane; c < rows * 8; c += 32) st_shared_v4(panel + c * 16, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncwarp();
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

}  // namespace attn
