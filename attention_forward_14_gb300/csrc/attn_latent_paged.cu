// Attention over the paged cache of latent attention (absorbed form):
//   s = scale q . c   (576 values: latent and rotated key part)
//   O = softmax(s [+ mask]) latent   (512 values)
// for queries that have been multiplied by the keys' projection.  All heads
// share a token's vector c, so a request's keys meet rows = h * sq query rows
// (row i * h + head: the heads of one query stand together).
//
// Work.  An item is 16, 32 or 64 rows of one request, a unit 128 of the keys
// that some of its rows see.  A team of up to twelve CTAs takes the same units
// for neighbouring items of a request, so that the cache leaves memory once
// for all of them.  The units of all items, in order, are dealt to the teams
// in equal contiguous shares, from the lengths that the device holds; an item
// that several teams share is written as partial results, which a second
// kernel joins.
//
// A CTA, 12 warps.  Keys, and values of the latent, are the 128 rows of the
// tensor cores' products and the query rows their columns, so that few query
// rows waste little and O^T of 64 rows (4 x 128 lanes x 64 columns of fp32)
// leaves tensor memory room for the scores:
//   S^T = C Q^T      [128 keys x rows], contraction over 576
//   O^T += L^T P^T   [4 x 128 values x rows], contraction over 128 keys
// A tile of the cache lies in shared memory once and serves both: [64-value
// panel][key], which is K-major for the first product and MN-major for the
// second.
//   warps 0-3, 4-7  softmax of half of the rows each, one thread to a key;
//                   bring Q and store O
//   warp  8         issues the products
//   warp  9         copies the cache's tiles (TMA), two panels (or the key
//                   parts' one) at a time
//   warps 10, 11    make a tile's values harmless where some row does not see
//                   them (zeros behind the length; NaN and infinities of keys
//                   that a mask hides from some rows)
// P^T takes the place of the tile's key parts once the scores are there.
//
// What bounds it.  16 rows: memory (32 requests of up to 16383 tokens, fp16:
// 66 us, of which the join 5 and some 10 the ramp; between them the cache at
// 6.2 TB/s).  64 rows: a tile of 128 keys takes 2.6 us, of which the tensor
// cores work 1.7 (their N of 64 takes 3/4 of the rate of 128: keys as the
// rows of A let 64 query rows keep O and S in tensor memory), the rest is the
// softmax between the two products.  Shared memory has no room for a second
// tile beside Q (72 KB) and this one (144 KB) that the tensor cores could work
// on meanwhile.  64 requests of 1000 to 8191 tokens, 128 heads: 107 us, 0.72
// PFLOP/s; 512 queries of 128 heads on 8192 tokens: 1.10 ms, 1.03 PFLOP/s.
// The code is kept short (waits, copies and first weights in rolled loops):
// what is executed once in a call comes from memory at its first use.
//
// Softmax, in log2.  A thread has one key of every row, so the rows' maxima
// are maxima over threads: the reference m of a row is raised, and O and the
// sums rescaled, only when some score exceeds it by more than 8 (a vote of the
// 128 threads a tile), and the threads' own sums meet at an item's end.  Two
// sums are kept, as in the other kernels: of the weights (LSE) and of the
// weights as rounded for the product (O is divided by it).
#include "latent.h"

#include "attn_kv8_common.cuh"
#include "latent_seq.cuh"
#include "mma_issue.cuh"
#include "tmem_cols.cuh"

namespace attn {

namespace {

constexpr int kTileKeys = 128;
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // 256 * 216 + 128 * 72 = 384 * 168
constexpr int kPanels = kLatentToken / 64, kPairs = kLatent / 128;
constexpr float kSlackLog2 = 8.f;

enum : uint32_t { SITE_LAT_EMPTY = 80, SITE_LAT_FULL = 81, SITE_LAT_Q = 82, SITE_LAT_S = 83, SITE_LAT_P = 84, SITE_LAT_O = 85,
                  SITE_LAT_CLEAN = 86 };

template <int N>
struct LatentCfg {
    static constexpr int PANEL = kTileKeys * 128;        // 128 keys of 64 values, 128-byte swizzle
    static constexpr int PAIR = 2 * PANEL;
    static constexpr int Q_PANEL = N * 128;
    static constexpr int COLS = N / 2;                   // rows (columns of S^T) of a softmax thread
    static constexpr int PAIR_SLOTS = N == 64 ? 4 : 5, KEY_SLOTS = N == 16 ? 2 : 1;
    static constexpr int CTL = 9216;
    static constexpr int Q_OFF = CTL;
    static constexpr int PAIR_OFF = Q_OFF + kPanels * Q_PANEL;
    static constexpr int KEY_OFF = PAIR_OFF + PAIR_SLOTS * PAIR;
    static constexpr int SMEM = KEY_OFF + KEY_SLOTS * PANEL + 1024;  // +1 KiB for alignment
    static constexpr int TM_O = 0, TM_S = kPairs * N;    // O^T block j at TM_O + j * N
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(Q_OFF % 1024 == 0 && PAIR_OFF % 1024 == 0 && Q_PANEL % 1024 == 0, "swizzle atoms");
    static_assert(TM_S + N <= 512, "tensor memory budget");
};

struct LatentCtl {
    uint64_t pair_full[6], pair_empty[6], key_full[2], key_empty[2];
    uint64_t q_full, s_full, p_full, pv_done, dirty, clean, mma_done;
    uint32_t tmem_base, abort;
    int32_t query[64];       // the query of each row
    float ref[64];           // the reference of each row, which its scores are less in the exponent
    float inv[64];
    float red[2][4][32];     // of a softmax group's warps: a value for each of its rows
    float red2[2][4][32];
    float shrink[2][4][32];
    int64_t o_at[64];        // where each row of o begins (elements)
    uint32_t lost[2][kLatent];  // of a softmax group's rows, a bit each: those in which a value of O is 0 times infinity
    uint32_t any_lost[2];
};
static_assert(sizeof(LatentCtl) <= LatentCfg<16>::CTL, "control block");

// ---------------------------------------------------------------- work

// Keys that some row of a team's tiles sees.
__device__ __forceinline__ int group_end(const LatentPagedParams &p, int len, int group, int tile_rows)
{
    if (p.mask != LATENT_MASK_CAUSAL) return len;
    const int64_t past = static_cast<int64_t>(group + 1) * p.team * tile_rows;
    const int last = static_cast<int>(min(past, static_cast<int64_t>(p.rows))) - 1;
    return min(max(len - p.sq + last / p.h + 1, 0), len);
}

struct LatentPlace {
    int entry;         // b * groups + group
    int b, group;
    int j, n;          // unit of the item (negative: of its cost), units of the item
    int len, end;      // cached keys; those that some row sees
};

__device__ __forceinline__ int latent_len(const LatentPagedParams &p, int b) { return min(max(p.seqlens[b], 0), p.cap); }

// One unit at least, which writes the rows of an item that sees no key.
__device__ __forceinline__ int units_for(int end) { return max((end + kTileKeys - 1) / kTileKeys, 1); }

// An item's units and, before them, as many as its beginning and end cost.
__device__ __forceinline__ int entry_units(const LatentPagedParams &p, int entry, int tile_rows)
{
    if (entry >= p.b * p.groups) return 0;
    const int b = entry / p.groups;
    return latent_item_cost(tile_rows) + units_for(group_end(p, latent_len(p, b), entry - b * p.groups, tile_rows));
}

// Where the units of the entries stand, held by a warp: a lane has as many
// neighbouring entries as the others, and the number of units up to its last.
struct LatentIndex {
    int64_t upto;
    int each;
};

__device__ __forceinline__ LatentIndex latent_index(const LatentPagedParams &p, int tile_rows)
{
    const int lane = threadIdx.x & 31, each = (p.b * p.groups + 31) / 32;
    int64_t t = 0;
#pragma unroll 2
    for (int i = 0; i < each; ++i) t += entry_units(p, lane * each + i, tile_rows);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, t, off);
        if (lane >= off) t += o;
    }
    return {t, each};
}

__device__ __forceinline__ void set_entry(const LatentPagedParams &p, LatentPlace &c, int entry, int tile_rows)
{
    c.entry = entry;
    c.b = entry / p.groups;
    c.group = entry - c.b * p.groups;
    c.j = -latent_item_cost(tile_rows);
    if (c.b >= p.b) return;
    c.len = latent_len(p, c.b);
    c.end = group_end(p, c.len, c.group, tile_rows);
    c.n = units_for(c.end);
}

// The place of unit u (< total), by every lane of a warp.
__device__ __forceinline__ LatentPlace latent_place(const LatentPagedParams &p, const LatentIndex &x, int64_t u, int tile_rows)
{
    const int lane = threadIdx.x & 31;
    const int at = __popc(__ballot_sync(0xffffffffu, x.upto <= u));  // the lane that has it
    const int64_t before = __shfl_sync(0xffffffffu, x.upto, max(at - 1, 0));
    if (at > 0) u -= before;
    LatentPlace c{};
    const int end = (at + 1) * x.each;
#pragma unroll 1
    for (int e0 = at * x.each; e0 < end; e0 += 32) {
        int inc = x.each > 1 && e0 + lane < end ? entry_units(p, e0 + lane, tile_rows) : 0;
        int src = 0;
        if (x.each > 1) {  // (32 entries have less than 2^24 units each)
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += o;
            }
            src = __popc(__ballot_sync(0xffffffffu, inc <= u));
            const int past = __shfl_sync(0xffffffffu, inc, min(max(src - 1, 0), 31));
            if (src > 0) u -= past;
            if (src == 32) continue;
        }
        set_entry(p, c, e0 + src, tile_rows);
        c.j += static_cast<int>(u);
        break;
    }
    return c;
}

// ---------------------------------------------------------------- pieces

// Whether any of a warpgroup's 128 threads says so.
__device__ __forceinline__ bool group_any(int barrier, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(v ? 1u : 0u), "r"(barrier)
                 : "memory");
    return r != 0u;
}

// The largest of a warp's values (NaN only if all are).
__device__ __forceinline__ float warp_top(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Brings `bytes` (a multiple of 16) from `src` on into the L2.
__device__ __forceinline__ void l2_prefetch(const uint8_t *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// v[c] over the warp's lanes (their sum, or largest): lane l has it for
// column l % C.  A step halves the columns that a lane looks after.
template <int C, typename F>
__device__ __forceinline__ float reduce_columns(float (&v)[C], F f)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 16; off >= C; off >>= 1)
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = f(v[c], __shfl_xor_sync(0xffffffffu, v[c], off));
#pragma unroll
    for (int off = C / 2; off > 0; off >>= 1)
#pragma unroll
        for (int c = 0; c < off; ++c) {
            const bool up = (lane & off) != 0;
            const float keep = up ? v[c + off] : v[c], give = up ? v[c] : v[c + off];
            v[c] = f(keep, __shfl_xor_sync(0xffffffffu, give, off));
        }
    return v[0];
}

// Natural log-sum-exp of a row from its reference and sum.
__device__ __forceinline__ float latent_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f; }

// Instruction descriptor of O^T: both operands MN-major.
__host__ __device__ constexpr uint32_t idesc_mn(int M, int N, bool bf16) { return idesc_f16(M, N, bf16, true) | (1u << 15); }

// The non-finite 16-bit values of a word, zeroed.
template <bool BF16>
__device__ __forceinline__ uint32_t finite_halves(uint32_t w)
{
    constexpr uint32_t EXP = BF16 ? 0x7F80u : 0x7C00u;
    if ((w & EXP) == EXP) w &= 0xFFFF0000u;
    if ((w >> 16 & EXP) == EXP) w &= 0x0000FFFFu;
    return w;
}

// A bit for each of a query's h rows from r on that is one of 32: none where
// the 32 lie past a request's last row, which counts as the last query's.
__host__ __device__ constexpr uint32_t rows_of_query(int r, int h)
{
    const int lo = r > 0 ? r : 0, end = r + h < 32 ? r + h : 32, n = end > lo ? end - lo : 0;
    return (n < 32 ? (1u << n) - 1u : ~0u) << lo;
}
// (an undefined shift is no constant)
static_assert(rows_of_query(-8, 4) == 0u && rows_of_query(-4, 4) == 0u && rows_of_query(31, 4) == 0x80000000u && rows_of_query(-1, 4) == 7u &&
              rows_of_query(28, 8) == 0xF0000000u && rows_of_query(0, 32) == ~0u && rows_of_query(-40, 100) == ~0u);

template <int N, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    attn_latent_paged_kernel(const __grid_constant__ CUtensorMap tmPool, const __grid_constant__ LatentPagedParams p)
{
    using C = LatentCfg<N>;
    constexpr int COLS = C::COLS;
    constexpr bool BF16 = Elem<T>::BF16;
    constexpr uint32_t IDESC_S = idesc_f16(kTileKeys, N, BF16, false);
    constexpr uint32_t IDESC_O = idesc_mn(128, N, BF16);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    LatentCtl *ctl = reinterpret_cast<LatentCtl *>(smem);
    const uint32_t sQ = base + C::Q_OFF, sPair = base + C::PAIR_OFF, sKey = base + C::KEY_OFF;
    auto B = [&](const uint64_t &bar) { return smem_addr(&bar); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t *abort_flag = &ctl->abort;
    const BoundedWaits waits{&ctl->abort, p.status, p.timeout_ns};
    auto warp_waits = [&](uint32_t bar, uint32_t parity, uint32_t site) { return waits.warp(bar, parity, site); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::PAIR_SLOTS; ++i) {
            mbar_init(B(ctl->pair_full[i]), 1);
            mbar_init(B(ctl->pair_empty[i]), 1);
        }
        for (int i = 0; i < C::KEY_SLOTS; ++i) {
            mbar_init(B(ctl->key_full[i]), 1);
            mbar_init(B(ctl->key_empty[i]), 1);
        }
        mbar_init(B(ctl->q_full), 8);
        mbar_init(B(ctl->s_full), 1);
        mbar_init(B(ctl->p_full), 8);
        mbar_init(B(ctl->pv_done), 1);
        mbar_init(B(ctl->dirty), 1);
        mbar_init(B(ctl->clean), 2);
        mbar_init(B(ctl->mma_done), 1);
        ctl->abort = 0u;
        ctl->any_lost[0] = ctl->any_lost[1] = 0u;
        fence_barrier_init();
    }
    for (int i = threadIdx.x; i < 2 * kLatent; i += kThreads) ctl->lost[0][i] = 0u;
    if (warp == 8) {
        tmem_alloc(smem_addr(&ctl->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == 9 && lane == 0) tma_prefetch_desc(&tmPool);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    await_previous();

    const int team = blockIdx.x / p.team, rank = blockIdx.x - team * p.team;
    const LatentIndex index = latent_index(p, N);
    const Shares shared_out(__shfl_sync(0xffffffffu, index.upto, 31), static_cast<int>(gridDim.x) / p.team, 1);
    const bool works = team < shared_out.ctas;
    // (a team that gives up on a wait leaves it so: the join must not meet what was in the workspace)
    if (threadIdx.x == 0 && rank == 0) p.cut[team] = LatentCut{0, 0, {0, 0}};
    const int64_t u0 = works ? shared_out.start(team) : 0;
    const int n_units = works ? static_cast<int>(shared_out.start(team + 1) - u0) : 0;
    LatentPlace at = latent_place(p, index, u0, N);
    auto place_in_bounds = [&]() {
        const bool ok = ATTN_OPS_IN_BOUNDS(at.b >= 0 && at.b < p.b && at.group >= 0 && at.group < p.groups && at.j >= 0 && at.j < at.n,
                                           p, SITE_OPS_UNIT);
        if (!ok) *abort_flag = 1u;
        return ok;
    };
    // Of an item: the CTA's first row, its tiles within the share, and the keys that all of its rows see.
    auto first_row = [&](const LatentPlace &c) { return static_cast<int64_t>(c.group * p.team + rank) * N; };
    auto has_tiles = [&](const LatentPlace &c) { return c.end > 0 && first_row(c) < p.rows; };
    auto item_tiles = [&](int j_end) { return has_tiles(at) ? j_end - at.j : 0; };
    // To the item's first unit in the share; false if there is none.
    auto enter = [&](int &it) {
        const int skip = min(max(-at.j, 0), n_units - it);
        at.j += skip, it += skip;
        return it < n_units && place_in_bounds();
    };
    auto all_see = [&]() {
        if (p.mask == LATENT_MASK_NONE) return at.len;
        const int i0 = p.mask == LATENT_MASK_TREE ? -1 : static_cast<int>(first_row(at)) / p.h;
        return min(max(at.len - p.sq + i0 + 1, 0), at.len);
    };

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9) {
            // -------------------------------------------------------- copies
            // Lane 8 s + i looks after keys 16 i .. 16 i + 15 of panel s of a pair (s = 0, 1).
            const int nowhere = p.num_pages * p.page_size;  // the token past the pool's end: the copy fills zeros
            const uint64_t pol = l2_evict_normal();
            const int group = lane & 7, side = (lane >> 3) & 1;
            uint32_t np = 0u, nk = 0u;  // pairs and key parts copied
            bool ok = true;
            for (int it = 0; ok && it < n_units;) {
                if (!enter(it)) break;
                const int j_end = min(at.n, at.j + n_units - it);
                const int tiles = item_tiles(j_end);
                const int32_t *table = p.block_table + static_cast<int64_t>(at.b) * p.pages_per_seq;
                // where the lane's keys of a tile lie: a copy begins there, or none (-1)
                auto token_of = [&](int t) {
                    const int k = (at.j + t) * kTileKeys + 16 * group;
                    if (t >= tiles || lane >= 16 || k >= at.len || (16 * group) % p.box != 0) return -1;
                    const int pg = k / p.page_size, page = table[pg];
                    return page >= 0 && page < p.num_pages ? page * p.page_size + (k - pg * p.page_size) : nowhere;
                };
                int next = token_of(0);
                for (int t = 0; ok && t < tiles; ++t) {
                    const int token = next;
                    const bool there = token >= 0;
                    next = token_of(t + 1);
                    // The next tile is on its way to the L2 meanwhile: a slot that is let go waits for that only.  The
                    // tokens of a page lie one after another; half of a copy's to a lane.
                    if (next >= 0 && next != nowhere && rank == (at.j + t) % p.team)
                        l2_prefetch(p.pool + (static_cast<int64_t>(next) * 2 + side * p.box) * kLatentToken, p.box * kLatentToken);
                    const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, there) & 0xFFu);
#pragma unroll 1
                    for (int pr = 0; ok && pr < kPairs; ++pr, ++np) {
                        const uint32_t st = np % C::PAIR_SLOTS, bar = B(ctl->pair_full[st]);
                        ok = warp_waits(B(ctl->pair_empty[st]), ((np / C::PAIR_SLOTS) & 1u) ^ 1u, SITE_LAT_EMPTY);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(bar, 2 * boxes * p.box * 128);
                        __syncwarp();
                        if (there)
                            tma_load_3d(sPair + st * C::PAIR + side * C::PANEL + 16 * group * 128, &tmPool, bar,
                                        pr * 128 + side * 64, token, 0, pol);
                    }
                    if (!ok) break;
                    const uint32_t st = nk % C::KEY_SLOTS, bar = B(ctl->key_full[st]);
                    ok = warp_waits(B(ctl->key_empty[st]), ((nk / C::KEY_SLOTS) & 1u) ^ 1u, SITE_LAT_EMPTY);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar, boxes * p.box * 128);
                    __syncwarp();
                    if (there && lane < 8)
                        tma_load_3d(sKey + st * C::PANEL + 16 * group * 128, &tmPool, bar, kLatent, token, 0, pol);
                    ++nk;
                }
                it += j_end - at.j;
                set_entry(p, at, at.entry + 1, N);
            }
            // wait (bounded) for the last copies, so that none lands after the CTA
#pragma unroll 1
            for (uint32_t i = np > C::PAIR_SLOTS ? np - C::PAIR_SLOTS : 0u; i < np; ++i)
                drain_wait(B(ctl->pair_full[i % C::PAIR_SLOTS]), (i / C::PAIR_SLOTS) & 1u, p.timeout_ns);
#pragma unroll 1
            for (uint32_t i = nk > C::KEY_SLOTS ? nk - C::KEY_SLOTS : 0u; i < nk; ++i)
                drain_wait(B(ctl->key_full[i % C::KEY_SLOTS]), (i / C::KEY_SLOTS) & 1u, p.timeout_ns);
        } else if (warp >= 10) {
            // -------------------------------------------------------- cleaning
            // The scores of keys that a row does not see are replaced, but 0 times a value is 0 for finite values
            // only.  Behind the length: zeros.  Of keys that some rows see: NaN and infinities become zeros.  A row
            // that sees such a key has a score of NaN or infinity, and with NaN and +infinity it has NaN everywhere;
            // with -infinity the weight is 0, and the softmax warps keep account of what the zeros replaced.  The tile
            // is touched when its scores are complete, not only issued: they are formed from what was there.
            uint32_t np = 0u, n_dirty = 0u;
            bool ok = true;
            for (int it = 0; ok && it < n_units;) {
                if (!enter(it)) break;
                const int j_end = min(at.n, at.j + n_units - it);
                const int tiles = item_tiles(j_end);
                const int all = all_see();
                for (int t = 0; ok && t < tiles; ++t, np += kPairs) {
                    const int k0 = (at.j + t) * kTileKeys;
                    if (k0 + kTileKeys <= all) continue;
                    ok = warp_waits(B(ctl->dirty), n_dirty & 1u, SITE_LAT_CLEAN);
                    if (!ok) break;
                    ++n_dirty;
                    const int left = min(at.len - k0, kTileKeys), whole = max(all - k0, 0);
#pragma unroll 1
                    for (int pr = warp - 10; ok && pr < kPairs; pr += 2) {
                        const uint32_t n = np + pr, st = n % C::PAIR_SLOTS;
                        // (the issuing warp has seen it; this orders the copies before what follows)
                        ok = warp_waits(B(ctl->pair_full[st]), (n / C::PAIR_SLOTS) & 1u, SITE_LAT_FULL);
                        if (!ok) break;
#pragma unroll 1
                        for (int side = 0; side < 2; ++side) {
                            uint8_t *panel = smem + C::PAIR_OFF + st * C::PAIR + side * C::PANEL;
#pragma unroll 1
                            for (int c = whole * 8 + lane; c < left * 8; c += 32) {
                                uint4 *v = reinterpret_cast<uint4 *>(panel) + c;
                                const uint4 a = *v;
                                const uint4 f = make_uint4(finite_halves<BF16>(a.x), finite_halves<BF16>(a.y),
                                                           finite_halves<BF16>(a.z), finite_halves<BF16>(a.w));
                                if (f.x != a.x || f.y != a.y || f.z != a.z || f.w != a.w) *v = f;
                            }
#pragma unroll 1
                            for (int c = left * 8 + lane; c < kTileKeys * 8; c += 32)
                                reinterpret_cast<uint4 *>(panel)[c] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B(ctl->clean));
                }
                it += j_end - at.j;
                set_entry(p, at, at.entry + 1, N);
            }
        } else if (warp == 8) {
            const uint32_t leader = issuing_lane();
            // -------------------------------------------------------- products
            uint32_t np = 0u, nk = 0u, n_dirty = 0u, q_it = 0u, tile_it = 0u;
            bool ok = true;
            const uint32_t dq = desc_lo(sQ, 16), dk_pair = desc_lo(sPair, 16), dk_key = desc_lo(sKey, 16);
            const uint32_t dv = desc_lo(sPair, C::PANEL), dp = desc_lo(sKey, 16);
            for (int it = 0; ok && it < n_units;) {
                if (!enter(it)) break;
                const int j_end = min(at.n, at.j + n_units - it);
                const int tiles = item_tiles(j_end);
                const int all = all_see();
                if (tiles > 0) ok = warp_waits(B(ctl->q_full), q_it++ & 1u, SITE_LAT_Q);
                for (int t = 0; ok && t < tiles; ++t, np += kPairs, ++nk, ++tile_it) {
                    const bool dirty = (at.j + t + 1) * kTileKeys > all;
                    // S^T
#pragma unroll 1
                    for (int pr = 0; pr < kPairs; ++pr) {
                        const uint32_t st = (np + pr) % C::PAIR_SLOTS;
                        if (!(ok = warp_waits(B(ctl->pair_full[st]), ((np + pr) / C::PAIR_SLOTS) & 1u, SITE_LAT_FULL))) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)  // 16 values a step
                            mma_ss_by(leader, tmem + C::TM_S, dk_pair + ((st * C::PAIR + (kk / 4) * C::PANEL + (kk % 4) * 32) >> 4),
                                   dq + (((2 * pr + kk / 4) * C::Q_PANEL + (kk % 4) * 32) >> 4), IDESC_S, (pr > 0 || kk > 0) ? 1u : 0u);
                    }
                    if (!ok) break;
                    const uint32_t ks = nk % C::KEY_SLOTS;
                    if (!(ok = warp_waits(B(ctl->key_full[ks]), (nk / C::KEY_SLOTS) & 1u, SITE_LAT_FULL))) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss_by(leader, tmem + C::TM_S, dk_key + ((ks * C::PANEL + kk * 32) >> 4), dq + ((8 * C::Q_PANEL + kk * 32) >> 4),
                               IDESC_S, 1u);
                    tc_commit_by(leader, B(ctl->s_full));
                    if (dirty) tc_commit_by(leader, B(ctl->dirty));  // the scores are of the values as they were
                    // O^T
                    if (dirty && !(ok = warp_waits(B(ctl->clean), n_dirty++ & 1u, SITE_LAT_CLEAN))) break;
                    if (!(ok = warp_waits(B(ctl->p_full), tile_it & 1u, SITE_LAT_P))) break;
                    tc_fence_after();
                    {
#pragma unroll 1
                        for (int pr = 0; pr < kPairs; ++pr) {
                            const uint32_t st = (np + pr) % C::PAIR_SLOTS;
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)  // 16 keys a step
                                mma_ss_by(leader, tmem + C::TM_O + pr * N, dv + ((st * C::PAIR + kk * 2048) >> 4),
                                       dp + ((ks * C::PANEL + kk * 2048) >> 4), IDESC_O, (t > 0 || kk > 0) ? 1u : 0u);
                            tc_commit_by(leader, B(ctl->pair_empty[st]));
                        }
                        tc_commit_by(leader, B(ctl->key_empty[ks]));
                        tc_commit_by(leader, B(ctl->pv_done));
                    }
                }
                it += j_end - at.j;
                set_entry(p, at, at.entry + 1, N);
            }
            // every product completes before tensor memory is freed
            tc_commit_by(leader, B(ctl->mma_done));
            __syncwarp();
            drain_wait(B(ctl->mma_done), 0u, p.timeout_ns);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax
        // A wait that ran out does not leave the loops: the barriers of the group's warps stay in step.
        regs_inc<kSoftmaxRegs>();
        const int w = warp >> 2, in_group = warp & 3, key = in_group * 32 + lane, bar_id = 1 + w;
        const uint32_t lane_off = static_cast<uint32_t>(in_group * 32) << 16;
        const uint32_t tS = tmem + lane_off + C::TM_S + w * COLS, tO = tmem + lane_off + C::TM_O + w * COLS;
        auto group_sync = [&]() { named_barrier(bar_id, 128); };
        uint32_t tile_it = 0u, nk = 0u;
        bool ok = true, asked = false;
        // An item's rows of Q: 72 pieces of 16 bytes a row, all of them on their way at once; eight lanes to a panel's row.
        auto ask_q = [&](const LatentPlace &c) {
            const int64_t row0 = first_row(c);
            const int nr = static_cast<int>(min(static_cast<int64_t>(N), p.rows - row0)), sub = lane & 7;
            const T *q = static_cast<const T *>(p.q) + c.b * p.qb;
#pragma unroll 1
            for (int r = warp * 4 + (lane >> 3); r < N; r += 32) {
                const int row = static_cast<int>(row0) + min(r, nr - 1), i = row / p.h, head = row - i * p.h;
                const uint4 *src = reinterpret_cast<const uint4 *>(q + head * p.qh + i * p.qs) + sub;
                const uint32_t to = sQ + r * 128 + ((sub ^ (r & 7)) << 4);
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn) cp_async16(to + pn * C::Q_PANEL, src + pn * 8, r < nr);
            }
        };
        auto give_q = [&]() {
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(B(ctl->q_full));
        };
        for (int it = 0; it < n_units;) {
            if (!enter(it)) break;
            const int j_end = min(at.n, at.j + n_units - it);
            const int tiles = item_tiles(j_end);
            const int64_t row0 = first_row(at);
            const int nr = static_cast<int>(min(static_cast<int64_t>(N), max(p.rows - row0, int64_t(0))));
            const int all = all_see(), before = at.len - p.sq;
            // The rows of the group's half that see key k: query by query, since a query's heads stand together.
            auto rows_that_see = [&](int k) {
                uint32_t sees = 0u;
                if (k >= at.len) return sees;
                const int drafted = k - before;
                const int32_t *tree = p.tree + static_cast<int64_t>(at.b) * p.sq * p.tree_words + (drafted >> 5);
                const int first = ctl->query[w * COLS], last = ctl->query[w * COLS + COLS - 1];
                int r = static_cast<int>(first * static_cast<int64_t>(p.h) - row0) - w * COLS;  // the query's first row
#pragma unroll 1
                for (int i = first; i <= last; ++i, r += p.h) {
                    bool one = true;
                    if (p.mask == LATENT_MASK_CAUSAL) one = drafted <= i;
                    if (p.mask == LATENT_MASK_TREE && drafted >= 0)
                        one = (tree[static_cast<int64_t>(i) * p.tree_words] >> (drafted & 31) & 1) != 0;
                    if (one) sees |= rows_of_query(r, p.h);
                }
                return sees;
            };
            // Key k, whose score is -infinity for `rows` of the group's half, which see it: 0 times its infinite values
            // is NaN.  (In a tile that all rows see whole, the product itself comes to that.)
            auto lose = [&](int k, uint32_t rows) {
                const int pg = k / p.page_size, page = p.block_table[static_cast<int64_t>(at.b) * p.pages_per_seq + pg];
                if (page < 0 || page >= p.num_pages) return;
                const uint16_t *c = reinterpret_cast<const uint16_t *>(p.pool) +
                                    (static_cast<int64_t>(page) * p.page_size + (k - pg * p.page_size)) * kLatentToken;
#pragma unroll 1
                for (int i = 0; i < kLatent; ++i) {
                    if (finite_halves<BF16>(c[i]) == c[i]) continue;
                    atomicOr(&ctl->lost[w][i], rows);
                    ctl->any_lost[w] = 1u;
                }
            };
            // what is needed of each row of the group's half
            if (key < COLS) {
                const int r = w * COLS + key;
                const int64_t row = min(row0 + r, static_cast<int64_t>(p.rows) - 1);
                const int i = static_cast<int>(row / p.h), head = static_cast<int>(row - static_cast<int64_t>(i) * p.h);
                ctl->query[r] = i;
                ctl->o_at[r] = at.b * p.ob + head * p.oh + i * p.os;
            }
            if (tiles > 0 && !asked) {
                ask_q(at);
                give_q();
            }
            if (key < COLS) ctl->ref[w * COLS + key] = 0.f;
            float2 l[COLS / 2], lr[COLS / 2];
#pragma unroll
            for (int c = 0; c < COLS / 2; ++c) l[c] = lr[c] = make_float2(0.f, 0.f);
            uint32_t unset = COLS == 32 ? ~0u : (1u << COLS) - 1u;  // rows without a reference: they have seen no key yet
            group_sync();
            for (int t = 0; t < tiles; ++t, ++tile_it, ++nk) {
                if (ok) ok = warp_waits(B(ctl->s_full), tile_it & 1u, SITE_LAT_S);
                tc_fence_after();
                const int k0 = (at.j + t) * kTileKeys;
                float2 x[COLS / 2];  // the scores less their rows' references
                {
                    uint32_t s[COLS];
                    tmem_load(tS, s);
                    const float2 scale2 = make_float2(p.sl2e, p.sl2e);
                    const float2 *ref = reinterpret_cast<const float2 *>(ctl->ref + w * COLS);
#pragma unroll
                    for (int c = 0; c < COLS / 2; ++c) {
                        const float2 m = ref[c];
                        x[c] = __ffma2_rn(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2,
                                          make_float2(-m.x, -m.y));
                    }
                }
                if (k0 + kTileKeys > all) {
                    const uint32_t sees = rows_that_see(k0 + key);
                    float low = x[0].x;
#pragma unroll
                    for (int c = 0; c < COLS / 2; ++c) low = min3f(low, x[c].x, x[c].y);
                    if (low == -INFINITY) {
                        uint32_t rows = 0u;
#pragma unroll
                        for (int c = 0; c < COLS / 2; ++c)
                            rows |= (x[c].x == -INFINITY ? 1u : 0u) << (2 * c) | (x[c].y == -INFINITY ? 2u : 0u) << (2 * c);
                        if ((rows & sees) != 0u) lose(k0 + key, rows & sees);
                    }
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < COLS / 2; ++c) {
                        x[c].x = sees >> (2 * c) & 1 ? x[c].x : -INFINITY;
                        x[c].y = sees >> (2 * c + 1) & 1 ? x[c].y : -INFINITY;
                    }
                }
                float top = x[0].x;
#pragma unroll
                for (int c = 0; c < COLS / 2; ++c) top = max3f(top, x[c].x, x[c].y);
                if (group_any(bar_id, top > kSlackLog2 || unset != 0u)) {
                    float up = 0.f;  // lane c: of column c
#pragma unroll
                    for (int c = 0; c < COLS / 2; ++c) {
                        const float a = warp_top(x[c].x), b = warp_top(x[c].y);
                        up = lane == 2 * c ? a : (lane == 2 * c + 1 ? b : up);
                    }
                    if (lane < COLS) ctl->red[w][in_group][lane] = up;
                    if (t > 0) {  // O^T has the tiles before: let the last one's products end
                        if (ok) ok = warp_waits(B(ctl->pv_done), (tile_it - 1) & 1u, SITE_LAT_O);
                        tc_fence_after();
                    }
                    group_sync();
                    // by how much each row's reference rises (is set): a column's by its lane of every warp, for itself
                    float *rise = ctl->red2[w][in_group], *shrink = ctl->shrink[w][in_group];
                    if (lane < COLS) {
                        const float mx = fmaxf(fmaxf(ctl->red[w][0][lane], ctl->red[w][1][lane]), fmaxf(ctl->red[w][2][lane], ctl->red[w][3][lane]));
                        const bool first = unset >> lane & 1;
                        const float by = first ? (mx > -INFINITY ? mx : 0.f) : fmaxf(mx, 0.f);
                        up = mx;
                        rise[lane] = by;
                        shrink[lane] = first ? 1.f : ex2_approx(-by);
                        if (in_group == 0) ctl->ref[w * COLS + lane] += by;
                    }
                    unset &= ~__ballot_sync(0xffffffffu, lane < COLS && up > -INFINITY);
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < COLS / 2; ++c) {
                        const float2 by = reinterpret_cast<const float2 *>(rise)[c];
                        x[c] = __fadd2_rn(x[c], make_float2(-by.x, -by.y));
                    }
                    if (t > 0) {
                        const float2 *f = reinterpret_cast<const float2 *>(shrink);
#pragma unroll
                        for (int c = 0; c < COLS / 2; ++c) l[c] = __fmul2_rn(l[c], f[c]), lr[c] = __fmul2_rn(lr[c], f[c]);
#pragma unroll 1
                        for (int j = 0; j < kPairs; ++j) {
                            uint32_t o[COLS];
                            tmem_load(tO + j * N, o);
#pragma unroll
                            for (int c = 0; c < COLS / 2; ++c) {
                                const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[2 * c]), __uint_as_float(o[2 * c + 1])), f[c]);
                                o[2 * c] = __float_as_uint(v.x), o[2 * c + 1] = __float_as_uint(v.y);
                            }
                            tmem_store(tO + j * N, o);
                        }
                        tmem_wait_st();
                    }
                    group_sync();  // the references, before they are read again
                }
                // this key's weights, into its row of P^T
                const uint32_t row = sKey + (nk % C::KEY_SLOTS) * C::PANEL + key * 128;
#pragma unroll
                for (int c = 0; c < COLS / 8; ++c) {
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = make_float2(ex2_approx(x[4 * c + e].x), ex2_approx(x[4 * c + e].y));
                        l[4 * c + e] = __fadd2_rn(l[4 * c + e], v);
                        pk[e] = Pair<T>::put(v.x, v.y);
                        lr[4 * c + e] = __fadd2_rn(lr[4 * c + e], Pair<T>::get(pk[e]));
                    }
                    st_shared_v4(row + (((w * (COLS / 8) + c) ^ (key & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B(ctl->p_full));
            }
            // The next item's Q, as soon as the last scores are there: its first products run while this one is stored.
            LatentPlace next = at;
            set_entry(p, next, at.entry + 1, N);
            const bool goes_on = n_units - it - (j_end - at.j) > latent_item_cost(N) && has_tiles(next);
            if (goes_on) ask_q(next);
            asked = goes_on;
            // the item ends, or goes on in the next team
            const bool item_ends = j_end == at.n;
            const int64_t first_unit = u0 + it - at.j;  // of the item
            const bool whole = first_unit >= u0 && item_ends;
            const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + (first_unit > u0 ? 1 : 0)) * N;
            {
                float v[COLS];
#pragma unroll
                for (int c = 0; c < COLS / 2; ++c) v[2 * c] = l[c].x, v[2 * c + 1] = l[c].y;
                const float ls = reduce_columns<COLS>(v, [](float a, float b) { return a + b; });
#pragma unroll
                for (int c = 0; c < COLS / 2; ++c) v[2 * c] = lr[c].x, v[2 * c + 1] = lr[c].y;
                const float lrs = reduce_columns<COLS>(v, [](float a, float b) { return a + b; });
                if (lane < COLS) {
                    ctl->red[w][in_group][lane] = ls;
                    ctl->red2[w][in_group][lane] = lrs;
                }
            }
            group_sync();
            if (key < COLS) {
                const int r = w * COLS + key;
                const float ls = (ctl->red[w][0][key] + ctl->red[w][1][key]) + (ctl->red[w][2][key] + ctl->red[w][3][key]);
                const float lrs = (ctl->red2[w][0][key] + ctl->red2[w][1][key]) + (ctl->red2[w][2][key] + ctl->red2[w][3][key]);
                ctl->inv[r] = !whole ? 1.f : (ls == 0.f ? 0.f : 1.f / lrs);
                if (r < nr) {
                    if (!whole) {
                        p.ml_part[part0 + r] = make_float4(ls == 0.f ? -INFINITY : ctl->ref[r], ls, lrs, 0.f);
                    } else if (p.lse) {
                        const int64_t row = row0 + r;
                        const int i = ctl->query[r], head = static_cast<int>(row - static_cast<int64_t>(i) * p.h);
                        p.lse[(static_cast<int64_t>(at.b) * p.h + head) * p.sq + i] = latent_lse(ctl->ref[r], ls);
                    }
                }
            }
            group_sync();
            if (tiles > 0) {
                if (ok) ok = warp_waits(B(ctl->pv_done), (tile_it - 1) & 1u, SITE_LAT_O);
                tc_fence_after();
            }
            if (goes_on) give_q();
            const bool lost = ctl->any_lost[w] != 0u;
#pragma unroll 1
            for (int j = 0; j < kPairs; ++j) {
                uint32_t o[COLS];
                if (tiles > 0) {
                    tmem_load(tO + j * N, o);
                } else {
#pragma unroll
                    for (int c = 0; c < COLS; ++c) o[c] = 0u;
                }
                const int col = j * 128 + key;
                if (lost) {
                    const uint32_t rows = ctl->lost[w][col];
                    ctl->lost[w][col] = 0u;
#pragma unroll
                    for (int c = 0; c < COLS; ++c) o[c] = rows >> c & 1 ? 0x7FFFFFFFu : o[c];
                }
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < COLS; ++c)
                        if (w * COLS + c < nr) p.o_part[(part0 + w * COLS + c) * kLatent + col] = __uint_as_float(o[c]);
                } else {
                    // two neighbouring columns of a row to a lane: even lanes take the even row of a pair, odd the odd one
#pragma unroll
                    for (int c = 0; c < COLS; c += 2) {
                        const int r = w * COLS + c, mine = lane & 1;
                        const float a = ctl->inv[r] == 0.f ? 0.f : __uint_as_float(o[c]) * ctl->inv[r];
                        const float b = ctl->inv[r + 1] == 0.f ? 0.f : __uint_as_float(o[c + 1]) * ctl->inv[r + 1];
                        const float got = __shfl_xor_sync(0xffffffffu, mine ? a : b, 1);
                        const uint32_t v = mine ? Pair<T>::put(got, b) : Pair<T>::put(a, got);
                        if (r + mine < nr)
                            *reinterpret_cast<uint32_t *>(static_cast<T *>(p.o) + ctl->o_at[r + mine] + (col - mine)) = v;
                    }
                }
            }
            tc_fence_before();
            group_sync();  // before the rows' values are written again
            if (key == 0) ctl->any_lost[w] = 0u;
            it += j_end - at.j;
            if (it == n_units && threadIdx.x == 0 && rank == 0) {
                // the item that this team begins and others go on with, if there is one
                if (!item_ends && first_unit >= u0) {
                    const int parts = static_cast<int>(shared_out.owner(first_unit + at.n - 1) - team) + 1;
                    p.cut[team] = LatentCut{first_unit > u0 ? -parts : parts, at.entry, {0, 0}};
                }
            }
            at = next;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- join

// Joins the parts of an item that several teams share: the blockIdx.x-th of
// such items, blockIdx.y which `rows` of its rows (of all its tiles).  The
// parts are added up in a fixed order: a row's parts by one warp, or by all
// eight, each a share of them.
constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_latent_join_kernel(const __grid_constant__ LatentPagedParams p, int tile_rows,
                                                                          int teams, int rows)
{
    constexpr int LOADS = kLatentMaxCtas / 32, VEC = kLatent / 32;
    __shared__ float red[kJoinWarps][kLatent];
    __shared__ float weight[kJoinWarps][kLatentMaxCtas];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    await_previous();
    int team = -1, parts = 0, entry = 0;
    int before = 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int4 c = lane + 32 * i < teams ? __ldcg(reinterpret_cast<const int4 *>(p.cut + lane + 32 * i)) : make_int4(0, 0, 0, 0);
        const uint32_t cuts = __ballot_sync(0xffffffffu, c.x != 0);
        const bool it_is = c.x != 0 && before + __popc(cuts & ((1u << lane) - 1u)) == static_cast<int>(blockIdx.x);
        const uint32_t found = __ballot_sync(0xffffffffu, it_is);
        if (found != 0u) {
            const int src = __ffs(found) - 1;
            team = 32 * i + src;
            parts = __shfl_sync(0xffffffffu, c.x, src);
            entry = __shfl_sync(0xffffffffu, c.y, src);
        }
        before += __popc(cuts);
    }
    if (team < 0) return;
    const int n = abs(parts);
    if (!ATTN_OPS_IN_BOUNDS(team + n <= teams && entry >= 0 && entry < p.b * p.groups, p, SITE_OPS_PART)) return;
    const int b = entry / p.groups, group = entry - b * p.groups;
    const int64_t row0 = static_cast<int64_t>(group) * p.team * tile_rows;
    const bool alone = rows > 1;  // a row to a warp
    for (int k = alone ? warp : 0; k < rows; k += alone ? kJoinWarps : 1) {
        const int r = blockIdx.y * rows + k;  // of the team's rows
        const int64_t row = row0 + r;
        const bool have = r < p.team * tile_rows && row < p.rows;
        if (!have && alone) break;
        const int rank = r / tile_rows, in_tile = r - rank * tile_rows;
        auto part_of = [&](int q) {
            return (2 * (static_cast<int64_t>(team + q) * p.team + rank) + (q == 0 && parts < 0 ? 1 : 0)) * tile_rows + in_tile;
        };
        float4 a[LOADS];
        float m = -INFINITY, l = 0.f, lr = 0.f;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int q = lane + 32 * i;
            a[i] = have && q < n ? __ldcg(p.ml_part + part_of(q)) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            m = fmaxf(m, a[i].x);
        }
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const float f = a[i].x == m ? 1.f : ex2_approx(a[i].x - m);
            if (32 * i < n) weight[warp][lane + 32 * i] = f;
            l = fmaf(a[i].y, f, l);
            lr = fmaf(a[i].z, f, lr);
        }
        l = row_sum<32>(l);
        lr = row_sum<32>(lr);
        __syncwarp();
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = 0.f;
        const int step = alone ? 1 : kJoinWarps;
#pragma unroll 2
        for (int q = alone ? 0 : warp; have && q < n; q += step) {
            const float4 *src = reinterpret_cast<const float4 *>(p.o_part + part_of(q) * kLatent) + lane;
            const float f = weight[warp][q];
#pragma unroll
            for (int e = 0; e < VEC / 4; ++e) {
                const float4 v = __ldcg(src + 32 * e);
                o[4 * e] = fmaf(v.x, f, o[4 * e]);
                o[4 * e + 1] = fmaf(v.y, f, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(v.z, f, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(v.w, f, o[4 * e + 3]);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / lr;
        const int i = have ? static_cast<int>(row / p.h) : 0;
        const int head = have ? static_cast<int>(row - static_cast<int64_t>(i) * p.h) : 0;
        T *dst = static_cast<T *>(p.o) + b * p.ob + head * p.oh + i * p.os;
        if (alone) {
#pragma unroll
            for (int e = 0; e < VEC / 4; ++e)
                reinterpret_cast<uint2 *>(dst)[lane + 32 * e] =
                    inv == 0.f ? make_uint2(0u, 0u)
                               : make_uint2(Pair<T>::put(o[4 * e] * inv, o[4 * e + 1] * inv), Pair<T>::put(o[4 * e + 2] * inv, o[4 * e + 3] * inv));
        } else {
#pragma unroll
            for (int e = 0; e < VEC / 4; ++e)
                *reinterpret_cast<float4 *>(&red[warp][(lane + 32 * e) * 4]) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            __syncthreads();
            const int c = 2 * threadIdx.x;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < kJoinWarps; ++q) {
                sum.x += red[q][c];
                sum.y += red[q][c + 1];
            }
            if (have) reinterpret_cast<uint32_t *>(dst)[threadIdx.x] = inv == 0.f ? 0u : Pair<T>::put(sum.x * inv, sum.y * inv);
            __syncthreads();
        }
        if (have && lane == 0 && (alone || warp == 0) && p.lse)
            p.lse[(static_cast<int64_t>(b) * p.h + head) * p.sq + i] = latent_lse(m, l);
        __syncwarp();
    }
}

template <int N, typename T>
cudaError_t launch_paged_t(const LatentPagedArgs &a)
{
    auto kern = attn_latent_paged_kernel<N, T>;
    std::atomic<int> &ready = a.attr_ready[(N == 16 ? 0 : (N == 32 ? 2 : 4)) + (Elem<T>::BF16 ? 1 : 0)];
    cudaError_t e;
    if (ready.load(std::memory_order_acquire) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LatentCfg<N>::SMEM);
        if (e != cudaSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    e = launch_overlapped(kern, dim3(a.grid), kThreads, LatentCfg<N>::SMEM, a.stream, a.pool, a.p);
    const int teams = a.grid / a.p.team;
    if (e != cudaSuccess || teams < 2) return e;
    // no more items are cut than there are items, or cuts between teams
    const int64_t items = static_cast<int64_t>(a.p.b) * a.p.groups;
    const int64_t cuts = items < teams - 1 ? items : teams - 1;
    const int used = a.p.rows < a.p.team * N ? a.p.rows : a.p.team * N;  // rows of an item, of all its tiles
    const int rows = teams / items + 2 > 4 ? 1 : kJoinWarps;
    const dim3 blocks(static_cast<unsigned>(cuts), static_cast<unsigned>((used + rows - 1) / rows));
    return launch_overlapped(attn_latent_join_kernel<T>, blocks, kJoinWarps * 32, 0, a.stream, a.p, N, teams, rows);
}

template <typename T>
cudaError_t launch_paged_rows(const LatentPagedArgs &a)
{
    switch (a.tile_rows) {
    case 16: return launch_paged_t<16, T>(a);
    case 32: return launch_paged_t<32, T>(a);
    default: return launch_paged_t<64, T>(a);
    }
}

}  // namespace

cudaError_t launch_latent_paged(const LatentPagedArgs &a, bool bf16)
{
    return bf16 ? launch_paged_rows<__nv_bfloat16>(a) : launch_paged_rows<__half>(a);
}

}  // namespace attn
