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

// The offsets of the sequence of this lane's number, of 32 from `first` on.
struct LatentCu {
    int first;
    int q0, q1, k0, k1;
};

__device__ __forceinline__ LatentCu latent_cu(const LatentSeqs &s, int first = 0)
{
    const int i = first + (threadIdx.x & 31);
    if (i >= s.batch) return {first, -1, -1, -1, -1};
    return {first, s.cu_q[i], s.cu_q[i + 1], s.cu_k[i], s.cu_k[i + 1]};
}

// The sequence and first row of a slot, by all lanes of a warp (`cu`: of the
// first 32 sequences).  The blocks of ROWS rows of a sequence that begins at
// token t and is the i-th stand in the slots from t / ROWS + i on: none meets
// the next one's, and of total / ROWS + batch slots no more than one a
// sequence is empty, however their lengths differ.  (A grid of batch times
// the longest one's blocks, most of them empty: 115 us, not 103, for the
// outputs of 6001 tokens in four sequences of 1 to 3107, 16 heads.)  An empty
// slot's unit has no rows; of a sequence whose offsets fall outside the totals
// all slots are empty.
template <int ROWS, bool OF_KEYS>
__device__ __forceinline__ LatentUnit latent_slot(const LatentSeqs &s, LatentCu cu, int slot)
{
    const int lane = threadIdx.x & 31;
    if (s.batch > 32) {  // 32 sequences among which it is, if the offsets do not decrease
        const int32_t *starts = OF_KEYS ? s.cu_k : s.cu_q;
        int lo = 0, n = s.batch;
        while (n > 32) {
            const int step = (n + 31) / 32, i = lane * step;
            const uint32_t before = __ballot_sync(0xffffffffu, i < n && starts[lo + i] / ROWS + lo + i <= slot);
            const int at = before ? (31 - __clz(before)) * step : 0;
            lo += at;
            n = min(step, n - at);
        }
        cu = latent_cu(s, lo);
    }
    const int t0 = OF_KEYS ? cu.k0 : cu.q0, t1 = OF_KEYS ? cu.k1 : cu.q1;
    const int blk = slot - t0 / ROWS - cu.first - lane;
    const bool in = 0 <= cu.q0 && cu.q0 <= cu.q1 && cu.q1 <= s.total_q && 0 <= cu.k0 && cu.k0 <= cu.k1 && cu.k1 <= s.total_k && t0 < t1 &&
                    0 <= blk && blk <= (t1 - t0 - 1) / ROWS;
    const uint32_t found = __ballot_sync(0xffffffffu, in);
    if (found == 0u) return {0, 0, 0, 0, 0, 0};
    const int src = __ffs(found) - 1;
    auto from = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
    return {0, from(blk) * ROWS, from(cu.q0), from(cu.q1 - cu.q0), from(cu.k0), from(cu.k1 - cu.k0)};
}

// Unit u of groups of heads x slots x heads of a group: the blocks of some
// heads together, so that the L2 holds what they share; of queries the later
// blocks, which see more keys, first.
template <int ROWS, bool OF_KEYS>
__device__ __forceinline__ LatentUnit latent_unit(const LatentSeqs &s, const LatentCu &cu, unsigned u, int slots, int group)
{
    const unsigned hg = u / (static_cast<unsigned>(slots) * group);
    u -= hg * slots * group;
    const int heads = min(group, s.h - static_cast<int>(hg) * group), slot = u / heads;
    LatentUnit un = latent_slot<ROWS, OF_KEYS>(s, cu, OF_KEYS ? slot : slots - 1 - slot);
    un.head = hg * group + u - slot * heads;
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
        bool late = false;
#pragma unroll 1
        while (!late) {
#pragma unroll 1
            for (int i = 0; i < 64; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*flag) return false;
            late = global_timer_ns() - t0 > timeout_ns;
        }
        *flag = 1u;
        record_status(status, STATUS_TIMEOUT, site);
        return false;
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
