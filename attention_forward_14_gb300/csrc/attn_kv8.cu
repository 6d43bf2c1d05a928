// Attention of new queries over an e4m3 paged cache:
//   O = softmax(scale Q K^T [+ causal mask]) V,  K = ks k8,  V = vs v8,
// with one scale ks, vs for each block of tokens (16, 32, 64 or 128) and key
// head.  A key head serves `group` query heads, so its keys meet
// rows = group * sq query rows.
//
// Work.  Eight consumer warps of a CTA work on 32 keys each at a time: on
// `heads` (8, 4, 2 or 1) consecutive key heads, 8 / heads warps to a head.  A
// cached token's heads lie side by side, so this is what makes a CTA's reads
// contiguous (8 heads of 128 values: 1 KB; one head's 128 bytes at that
// stride reached 2.2 of 6.8 TB/s).  An item is 16 query rows of such a group
// of heads of one batch element; a unit is the 32 * 8 / heads keys that the
// warps take together.  The units of all items, in order, are dealt to the
// CTAs in equal contiguous shares, from the lengths that the device holds:
// ragged batches need no split count and leave no CTA behind.  An item that
// several CTAs share is written as partial results, which a second kernel
// joins.
//
// A CTA.  A producer warp copies a unit's K and V rows of all the heads with
// one TMA copy each ([head][key][d] in shared memory, swizzled) and the
// blocks' scales, a few units ahead and across items.  The consumers of one
// head meet at an item's end only.  Per 32 keys a warp computes S = Q K^T
// (16 x 32) and O += P V with fp16 matrix instructions on e4m3 values
// converted to fp16 (exact) in registers.  The order of the head's values in a
// dot product is free, so a lane takes 32 contiguous ones (d = 128) of its
// key's row in two 16-byte loads; the columns of O are dealt likewise.
//
// Types.  Q enters the product as fp16: fp16 inputs as they are, bf16 inputs
// times a power of two for each row that puts the row's largest value at
// 2^14, which keeps all 8 significant bits of every value down to 2^-29 of
// the largest.  P is rounded to fp16 (2^-11 relative) between 2^-24 and
// 2^14.  Sums and statistics are fp32.
//
// Softmax, in log2: x = ks scale log2(e) (q . k8) + log2(vs).  P = 2^(x - m +
// 10) carries the value scale, so O needs no product with it, and the sum of
// the weights is sum(P) / vs, in fp32.  m follows the maximum of x lazily: it
// is raised (and O and the sum rescaled) only when some x exceeds it by more
// than 4, so P <= 2^14.
#include "attn_kv8.h"

#include "attn_fwd_kernel.cuh"
#include "rows.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;                         // consumers
constexpr int kThreads = (kWarps + 4) * 32;       // and a warpgroup of which one warp copies
constexpr int kConsumerRegs = 232, kProducerRegs = 40;  // 256 * 232 + 128 * 40 = 384 * 168
constexpr int kStepKeys = 32;                     // keys of a warp's step
constexpr float kOffset = 10.f, kSlack = 4.f;
enum : uint32_t { SITE_KV8_FULL = 40, SITE_KV8_EMPTY = 41 };

template <int D>
struct Kv8Cfg {
    static constexpr int KBYTES = kStepKeys * D;           // a warp's K (or V) rows of a step
    static constexpr int STAGE = 2 * kWarps * KBYTES;      // K of all warps, then V
    static constexpr int STAGES = D == 128 ? 2 : 4;        // 128 KB in flight
    static constexpr int O_OFF = STAGES * STAGE;           // where the warps of one head meet [warps][8 rows][D]
    static constexpr int ML_OFF = O_OFF + kWarps * 8 * D * 4;     // [warps][16] float2
    static constexpr int SC_OFF = ML_OFF + kWarps * 16 * 8;       // [STAGES][warps] scales: K, K, V, V
    static constexpr int BAR_OFF = SC_OFF + kWarps * STAGES * 16; // [STAGES] full, then empty
    static constexpr int CTL_OFF = BAR_OFF + 2 * STAGES * 8;
    static constexpr int SMEM = CTL_OFF + 16 + 1024;       // +1 KiB for alignment
    static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Arrives on `bar` when this thread's earlier cp.async have landed (the
// barrier's count includes it).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float lg2_approx(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int cached_len(const Kv8Params &p, int b) { return min(max(p.seqlens[b], 0), p.cap); }

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The top bit of every byte that is an e4m3 NaN (0x7F, 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Units of one item of a batch element with n keys: an item that sees no
// key still has one, which writes its rows.
__device__ __forceinline__ int units_of(const Kv8Params &p, int n) { return max((n + p.unit_keys - 1) / p.unit_keys, 1); }

// Where in the work a unit lies.
struct Place {
    int b, hg, tile;
    int j, n;    // unit of the item, units of the item
    int len;     // cached keys of the batch element
};

__device__ __forceinline__ int64_t total_units(const Kv8Params &p)
{
    const int lane = threadIdx.x & 31;
    int64_t t = 0;
    for (int i = lane; i < p.b; i += 32) t += units_of(p, cached_len(p, i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t * p.head_groups * p.tiles;
}

// a / b of non-negative numbers that mostly fit 32 bits (a 64-bit division
// is a hundred instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The units dealt to the CTAs: the first `rem` get one more than `per`.  No
// more CTAs than there are units, and none with fewer than kMinUnits of them
// when that leaves a CTA.
constexpr int kMinUnits = 2;
struct Shares {
    int64_t per, rem;
    int ctas;
    __device__ __forceinline__ Shares(int64_t total, int grid)
    {
        ctas = static_cast<int>(min(static_cast<int64_t>(grid), max(total / kMinUnits, int64_t(1))));
        per = quotient(total, ctas);
        rem = total - per * ctas;
    }
    __device__ __forceinline__ int64_t start(int64_t c) const { return c * per + min(c, rem); }
    // the CTA that has unit u
    __device__ __forceinline__ int64_t owner(int64_t u) const
    {
        const int64_t big = rem * (per + 1);
        return u < big ? quotient(u, per + 1) : rem + quotient(u - big, per);
    }
};

// The place of unit u (< total), by every lane of a warp.
__device__ __forceinline__ Place place_of(const Kv8Params &p, int64_t u)
{
    const int lane = threadIdx.x & 31;
    const int64_t per = static_cast<int64_t>(p.head_groups) * p.tiles;
    Place c;
    for (int b0 = 0;; b0 += 32) {
        const int len = b0 + lane < p.b ? cached_len(p, b0 + lane) : 0;
        int64_t inc = b0 + lane < p.b ? units_of(p, len) * per : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, inc > u);
        if (past != 0u || b0 + 32 >= p.b) {
            const int src = past != 0u ? __ffs(past) - 1 : 31;
            const int64_t before = __shfl_sync(0xffffffffu, inc, src > 0 ? src - 1 : 0);
            if (src > 0) u -= before;
            c.b = b0 + src;
            c.len = __shfl_sync(0xffffffffu, len, src);
            break;
        }
        u -= __shfl_sync(0xffffffffu, inc, 31);
    }
    c.n = units_of(p, c.len);
    const int64_t item = quotient(u, c.n);
    c.j = static_cast<int>(u - item * c.n);
    c.hg = static_cast<int>(quotient(item, p.tiles));
    c.tile = static_cast<int>(item - static_cast<int64_t>(c.hg) * p.tiles);
    return c;
}

__device__ __forceinline__ void next_unit(const Kv8Params &p, Place &c)
{
    if (++c.j < c.n) return;
    c.j = 0;
    if (++c.tile < p.tiles) return;
    c.tile = 0;
    if (++c.hg < p.head_groups) return;
    c.hg = 0;
    if (++c.b >= p.b) return;
    c.len = cached_len(p, c.b);
    c.n = units_of(p, c.len);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Keys [0, end) are seen by some row of the tile, keys [0, all) by every one.
struct Seen {
    int end, all;
};

__device__ __forceinline__ Seen seen_keys(const Kv8Params &p, const Place &c)
{
    if (!p.causal) return {c.len, c.len};
    const int r0 = c.tile * kKv8Tile, r1 = min(r0 + kKv8Tile, p.rows) - 1;
    const bool wraps = r0 / p.sq != r1 / p.sq;  // the rows of one query head are consecutive
    const int i0 = wraps ? 0 : r0 % p.sq, i1 = wraps ? p.sq - 1 : r1 % p.sq;
    return {max(c.len - p.sq + i1 + 1, 0), max(c.len - p.sq + i0 + 1, 0)};
}

// Row r of key head kvh's query rows, among the rows of q and o.
__device__ __forceinline__ int64_t row_at(const Kv8Params &p, int b, int kvh, int r)
{
    return (static_cast<int64_t>(b) * p.h_kv + kvh) * p.rows + r;
}

// Partial results: slot 2 c for CTA c's first item, 2 c + 1 for its last, and
// `hw` the head of the item's group.
__device__ __forceinline__ int64_t part_at(int64_t slot, int hw) { return (slot * kWarps + hw) * kKv8Tile; }

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? -INFINITY : (m - kOffset + log2f(l)) * 0.69314718055994531f;
}

template <int D, typename T>
__device__ __forceinline__ void store4(T *o, float4 v)
{
    *reinterpret_cast<uint2 *>(o) = make_uint2(Pair<T>::put(v.x, v.y), Pair<T>::put(v.z, v.w));
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kv8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ Kv8Params p)
{
    using C = Kv8Cfg<D>;
    constexpr int STAGES = C::STAGES;
    constexpr int KS = D / 16;      // k-steps of S, and words of a lane's share of a K row
    constexpr int VW = D / 32;      // words of a lane's share of a V row
    constexpr int NO = D / 8;       // column tiles of O
    constexpr bool BF16 = Elem<T>::BF16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + C::CTL_OFF);
    auto full_bar = [&](uint32_t st) { return base + C::BAR_OFF + st * 8; };
    auto empty_bar = [&](uint32_t st) { return base + C::BAR_OFF + (STAGES + st) * 8; };

    if (threadIdx.x == 0) {
        *abort_flag = 0u;
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1 && lane < STAGES) {
        mbar_init(full_bar(lane), 33);        // the bytes' announcement and a scale of every producer lane
        mbar_init(empty_bar(lane), kWarps);
        fence_barrier_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const Shares shared_out(total_units(p), static_cast<int>(gridDim.x));
    if (blockIdx.x >= shared_out.ctas) {
        if (threadIdx.x == 0) p.cut[blockIdx.x].parts = 0;
        return;
    }
    const int64_t u0 = shared_out.start(blockIdx.x);
    const int n_units = static_cast<int>(shared_out.start(blockIdx.x + 1) - u0);
    Place cur = place_of(p, u0);

    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = global_timer_ns();
        while (true) {
            for (int i = 0; i < 64; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > p.timeout_ns) {
                *abort_flag = 1u;
                record_status(p.status, STATUS_TIMEOUT, site);
                return false;
            }
        }
    };

    const int head_shift = 31 - __clz(p.heads);
    const bool wide = p.page_size % kStepKeys == 0;  // a step of 32 keys lies in one page
    if (warp >= kWarps) {
        // ------------------------------------------------------------ producer
        // Lane 4 w + 2 kv + half fetches the scale of consumer w's 16 keys
        // `half`, of K or V; the lanes of each share's first head copy.
        regs_dec<kProducerRegs>();
        if (warp != kWarps) return;
        const int half = lane & 1, kv = (lane >> 1) & 1, w = lane >> 2;
        const int hw = w & (p.heads - 1), kshare = w >> head_shift;
        const float *scales = kv ? p.v_scale : p.k_scale;
        const CUtensorMap *map = kv ? &tmV : &tmK;
        const int blocks_per_page = p.page_size >> p.block_shift;
        const int page_shift = (p.page_size & (p.page_size - 1)) == 0 ? 31 - __clz(p.page_size) : -1;
        const int nowhere = p.num_pages * p.page_size;   // the token past the pool's end
        const bool copies = hw == 0 && (half == 0 || !wide);
        // [K | V][share][head][32 keys][D], or, copied 16 keys at a time, [K | V][share][half][head][16 keys][D]
        const uint32_t to = kv * (kWarps * C::KBYTES) + kshare * p.heads * C::KBYTES + half * p.heads * (C::KBYTES / 2);
        const uint64_t pol = l2_evict_normal();
        uint32_t issued = 0u;
        int end = 0;
        const int32_t *table = nullptr;
        const float *head_scales = nullptr;
        for (int it = 0; it < n_units; ++it) {
            if (it == 0 || cur.j == 0) {
                end = seen_keys(p, cur).end;
                table = p.block_table + static_cast<int64_t>(cur.b) * p.pages_per_seq;
                head_scales = scales + static_cast<int64_t>(cur.hg * p.heads + hw) * blocks_per_page;
            }
            const int u_key = cur.j * p.unit_keys;
            if (u_key < end) {
                const int shares = min((end - u_key + kStepKeys - 1) / kStepKeys, kWarps >> head_shift);
                const int k = u_key + kshare * kStepKeys + 16 * half;
                const int pg = page_shift >= 0 ? k >> page_shift : k / p.page_size, off = k - pg * p.page_size;
                const int page = k < end ? __ldg(table + pg) : -1;
                const bool in = page >= 0 && page < p.num_pages;
                const uint32_t st = issued % STAGES, bar = full_bar(st);
                if (!__all_sync(0xffffffffu, wait(empty_bar(st), ((issued / STAGES) & 1u) ^ 1u, SITE_KV8_EMPTY))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar, shares * p.heads * (2 * C::KBYTES));
                if (copies && kshare < shares)
                    // a page outside the pool is read at the token past its end: the copy fills zeros
                    tma_load_3d(base + st * C::STAGE + to, map, bar, 0, in ? page * p.page_size + off : nowhere,
                                cur.hg * p.heads, pol);
                const uint32_t sc = base + C::SC_OFF + st * (kWarps * 16) + (w * 4 + kv * 2 + half) * 4;
                if (in) {
                    cp_async4(sc, head_scales + static_cast<int64_t>(page) * p.h_kv * blocks_per_page + (off >> p.block_shift));
                    cp_async_arrive(bar);
                } else {
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc), "f"(1.f) : "memory");
                    mbar_arrive(bar);
                }
                ++issued;
                __syncwarp();
            }
            next_unit(p, cur);
        }
        // wait (bounded) for the last copies, so that none lands after the CTA
        for (uint32_t n = issued > STAGES ? issued - STAGES : 0u; n < issued; ++n)
            drain_wait(full_bar(n % STAGES), (n / STAGES) & 1u, p.timeout_ns);
        return;
    }
    regs_inc<kConsumerRegs>();

    // ---------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    const int hw = warp & (p.heads - 1), kshare = warp >> head_shift, shares = kWarps >> head_shift;
    // this warp's rows of a stage: keys 0..15 and, `second` bytes on, 16..31
    const uint8_t *mine = smem + kshare * p.heads * C::KBYTES + hw * (wide ? C::KBYTES : C::KBYTES / 2);
    const uint32_t second = (wide ? 1 : p.heads) * (C::KBYTES / 2);
    const float4 *sc_ptr = reinterpret_cast<const float4 *>(smem + C::SC_OFF + warp * 16);
    uint32_t used = 0u;
    bool ok = true;
    uint32_t qa[KS][4];
    float acc[NO][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, c0 = 0.f, c1 = 0.f;
    int lim0 = 0, lim1 = 0;
    Seen seen{0, 0};
    for (int it = 0; it < n_units; ++it) {
        if (it == 0 || cur.j == 0) {  // an item begins
            seen = seen_keys(p, cur);
            const int r = cur.tile * kKv8Tile + g;
            float f[2] = {1.f, 1.f};
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int rr = r + 8 * hh;
                uint32_t w[KS * 2];
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) +
                                                                   row_at(p, cur.b, cur.hg * p.heads + hw, rr < p.rows ? rr : 0) * D +
                                                                   t * (D / 4));
#pragma unroll
                for (int i = 0; i < KS / 2; ++i) {
                    const uint4 v = rr < p.rows ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
                    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
                }
                if constexpr (BF16) {
                    uint32_t mx = 0u;  // largest magnitude of the row, as the bits of a non-negative float
#pragma unroll
                    for (int i = 0; i < KS * 2; ++i) mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const int e = max(static_cast<int>(mx >> 7) - 127, -100);
                    const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
                    f[hh] = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
                    for (int i = 0; i < KS * 2; ++i) {
                        const float2 v = Pair<T>::get(w[i]);
                        w[i] = Pair<__half>::put(v.x * up, v.y * up);
                    }
                }
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qa[s][hh] = w[2 * s];
                    qa[s][2 + hh] = w[2 * s + 1];
                }
            }
            c0 = p.sl2e * f[0];
            c1 = p.sl2e * f[1];
            lim0 = lim1 = cur.len;
            if (p.causal) {
                lim0 = cur.len - p.sq + r % p.sq + 1;
                lim1 = cur.len - p.sq + (r + 8) % p.sq + 1;
            }
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
#pragma unroll
            for (int i = 0; i < NO; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        }
        const int k0 = cur.j * p.unit_keys + kshare * kStepKeys;
        const uint32_t st = used % STAGES;
        const bool loaded = cur.j * p.unit_keys < seen.end;  // the unit has a stage
        if (ok && loaded) ok = __all_sync(0xffffffffu, wait(full_bar(st), (used / STAGES) & 1u, SITE_KV8_FULL));
        if (ok && k0 < seen.end) {
            const uint8_t *ks_at = mine + st * C::STAGE, *vs_at = ks_at + kWarps * C::KBYTES;
            const float4 sc = sc_ptr[st * kWarps];
            // S: four tiles of eight keys
            float s[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int c = 0; c < KS / 4; ++c) {  // 16 bytes of the lane's share of each key's row
                uint32_t w[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int row = (n & 1) * 8 + g;
                    const uint4 a = *reinterpret_cast<const uint4 *>(
                        ks_at + (n >= 2 ? second : 0u) + (D == 128 ? row * 128 + (((2 * t + c) ^ g) << 4) : row * 64 + ((t ^ ((row >> 1) & 3)) << 4)));
                    w[n][0] = a.x, w[n][1] = a.y, w[n][2] = a.z, w[n][3] = a.w;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        mma16816(s[n], qa[4 * c + k][0], qa[4 * c + k][1], qa[4 * c + k][2], qa[4 * c + k][3],
                                 e4m3x2_to_f16x2(w[n][k]), e4m3x2_to_f16x2(w[n][k] >> 16));
            }
            // the scales of the two halves; a V scale of 0 is a block of zeros
            float lv[2], ivs[2];
            bool vzero[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float vs = h ? sc.w : sc.z;
                vzero[h] = vs < 1.1754944e-38f;
                vs = vzero[h] ? 1.f : vs;
                lv[h] = lg2_approx(vs);
                ivs[h] = rcp_approx(vs);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float ks = n < 2 ? sc.x : sc.y, a0 = c0 * ks, a1 = c1 * ks;
                s[n][0] = fmaf(s[n][0], a0, lv[n >> 1]);
                s[n][1] = fmaf(s[n][1], a0, lv[n >> 1]);
                s[n][2] = fmaf(s[n][2], a1, lv[n >> 1]);
                s[n][3] = fmaf(s[n][3], a1, lv[n >> 1]);
            }
            const bool partly = k0 + kStepKeys > seen.all;  // some row does not see some of these keys
            if (partly) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int k = k0 + n * 8 + 2 * t;
                    s[n][0] = k < lim0 ? s[n][0] : -INFINITY;
                    s[n][1] = k + 1 < lim0 ? s[n][1] : -INFINITY;
                    s[n][2] = k < lim1 ? s[n][2] : -INFINITY;
                    s[n][3] = k + 1 < lim1 ? s[n][3] : -INFINITY;
                }
            }
            const float t0 = max3f(max3f(s[0][0], s[0][1], s[1][0]), max3f(s[1][1], s[2][0], s[2][1]), fmaxf(s[3][0], s[3][1]));
            const float t1 = max3f(max3f(s[0][2], s[0][3], s[1][2]), max3f(s[1][3], s[2][2], s[2][3]), fmaxf(s[3][2], s[3][3]));
            if (__any_sync(0xffffffffu, t0 > m0 + kSlack || t1 > m1 + kSlack)) {
                float n0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
                float n1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
                n0 = fmaxf(m0, fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 2)));
                n1 = fmaxf(m1, fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 2)));
                const float f0 = n0 == m0 ? 1.f : ex2_approx(m0 - n0);
                const float f1 = n1 == m1 ? 1.f : ex2_approx(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    acc[i][0] *= f0;
                    acc[i][1] *= f0;
                    acc[i][2] *= f1;
                    acc[i][3] *= f1;
                }
            }
            const float b0 = m0 == -INFINITY ? 0.f : m0 - kOffset, b1 = m1 == -INFINITY ? 0.f : m1 - kOffset;
            uint32_t pa[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2_approx(s[2 * h + n][0] - b0), p1 = ex2_approx(s[2 * h + n][1] - b0);
                    const float p2 = ex2_approx(s[2 * h + n][2] - b1), p3 = ex2_approx(s[2 * h + n][3] - b1);
                    sum0 += p0 + p1;
                    sum1 += p2 + p3;
                    pa[h][2 * n] = vzero[h] ? 0u : Pair<__half>::put(p0, p1);
                    pa[h][2 * n + 1] = vzero[h] ? 0u : Pair<__half>::put(p2, p3);
                }
                l0 = fmaf(sum0, ivs[h], l0);
                l1 = fmaf(sum1, ivs[h], l1);
            }
            // O += P V, 16 keys at a time
            const int tail = cur.len - k0;  // rows of V from `tail` on are not keys: zero them
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[4][VW];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 2 * t + (i & 1) + 8 * (i >> 1);
                    if constexpr (D == 128) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(vs_at + (h ? second : 0u) + row * 128 + ((g ^ (row & 7)) << 4));
                        v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
                    } else {
                        const uint2 a = *reinterpret_cast<const uint2 *>(
                            vs_at + (h ? second : 0u) + row * 64 + ((((g >> 1) ^ ((row >> 1) & 3)) << 4) | ((g & 1) << 3)));
                        v[i][0] = a.x, v[i][1] = a.y;
                    }
                    if (tail < kStepKeys) {
#pragma unroll
                        for (int w = 0; w < VW; ++w) v[i][w] = row + 16 * h < tail ? v[i][w] : 0u;
                    }
                }
                if (partly) {
                    // A NaN among V must reach the rows that see its key and
                    // no other, but a row that does not still multiplies it,
                    // by 0: take it out of the product and put it into the
                    // rows that see it (the product of what each row sees
                    // with where V is NaN counts them).
                    uint32_t any = 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int w = 0; w < VW; ++w) any |= nan_bytes(v[i][w]);
                    if (__any_sync(0xffffffffu, any != 0u)) {
                        uint32_t see[4];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const int k = k0 + 16 * h + n * 8 + 2 * t;
                            see[2 * n] = (k < lim0 ? 0x3C00u : 0u) | (k + 1 < lim0 ? 0x3C000000u : 0u);
                            see[2 * n + 1] = (k < lim1 ? 0x3C00u : 0u) | (k + 1 < lim1 ? 0x3C000000u : 0u);
                        }
#pragma unroll
                        for (int w = 0; w < VW; ++w) {
                            uint32_t ind[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t m = nan_bytes(v[i][w]) >> 7;
                                ind[i] = m * 0x38u;  // e4m3's 1
                                v[i][w] &= ~(m * 0xFFu);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t sel = e < 2 ? 0x5140u : 0x7362u;
                                const uint32_t lo = __byte_perm(ind[0], ind[1], sel) >> (16 * (e & 1));
                                const uint32_t hi = __byte_perm(ind[2], ind[3], sel) >> (16 * (e & 1));
                                float c[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816(c, see[0], see[1], see[2], see[3], e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(hi));
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    acc[4 * w + e][k] = c[k] > 0.f ? __int_as_float(0x7FC00000) : acc[4 * w + e][k];
                            }
                        }
                    }
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    const uint32_t lo0 = __byte_perm(v[0][w], v[1][w], 0x5140), hi0 = __byte_perm(v[0][w], v[1][w], 0x7362);
                    const uint32_t lo1 = __byte_perm(v[2][w], v[3][w], 0x5140), hi1 = __byte_perm(v[2][w], v[3][w], 0x7362);
                    const uint32_t(&a)[4] = pa[h];
                    mma16816(acc[4 * w], a[0], a[1], a[2], a[3], e4m3x2_to_f16x2(lo0), e4m3x2_to_f16x2(lo1));
                    mma16816(acc[4 * w + 1], a[0], a[1], a[2], a[3], e4m3x2_to_f16x2(lo0 >> 16), e4m3x2_to_f16x2(lo1 >> 16));
                    mma16816(acc[4 * w + 2], a[0], a[1], a[2], a[3], e4m3x2_to_f16x2(hi0), e4m3x2_to_f16x2(hi1));
                    mma16816(acc[4 * w + 3], a[0], a[1], a[2], a[3], e4m3x2_to_f16x2(hi0 >> 16), e4m3x2_to_f16x2(hi1 >> 16));
                }
            }
        }
        __syncwarp();  // every lane has read the stage
        if (ok && loaded) {
            if (lane == 0) mbar_arrive(empty_bar(st));
            ++used;
        }

        const bool item_ends = cur.j + 1 == cur.n;
        if (item_ends || it + 1 == n_units) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const int nr = min(kKv8Tile, p.rows - cur.tile * kKv8Tile);
            const int64_t first_unit = u0 + it - cur.j;  // of the item
            const bool whole = first_unit >= u0 && item_ends;
            const int64_t part = part_at(2 * static_cast<int64_t>(blockIdx.x) + (first_unit > u0 ? 1 : 0), hw);
            const int64_t row0 = row_at(p, cur.b, cur.hg * p.heads + hw, cur.tile * kKv8Tile);
            // a lane's columns of row g: 2 NO consecutive ones from 2 t NO on, acc[i][0] then acc[i][1]
            if (shares == 1) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int r = g + 8 * hh;
                    if (r >= nr) continue;
                    const float m = hh ? m1 : m0, l = hh ? l1 : l0;
                    const float inv = !whole ? 1.f : (l == 0.f ? 0.f : 1.f / l);
                    float4 v[NO / 2];
#pragma unroll
                    for (int i = 0; i < NO; i += 4) {
                        v[i / 4] = make_float4(acc[i][2 * hh] * inv, acc[i + 1][2 * hh] * inv, acc[i + 2][2 * hh] * inv,
                                               acc[i + 3][2 * hh] * inv);
                        v[NO / 4 + i / 4] = make_float4(acc[i][2 * hh + 1] * inv, acc[i + 1][2 * hh + 1] * inv,
                                                        acc[i + 2][2 * hh + 1] * inv, acc[i + 3][2 * hh + 1] * inv);
                    }
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.o) + (row0 + r) * D + 2 * t * NO);
#pragma unroll
                        for (int i = 0; i < NO / 2; i += 2)
                            dst[i / 2] = make_uint4(Pair<T>::put(v[i].x, v[i].y), Pair<T>::put(v[i].z, v[i].w),
                                                    Pair<T>::put(v[i + 1].x, v[i + 1].y), Pair<T>::put(v[i + 1].z, v[i + 1].w));
                        if (t == 0 && p.lse) p.lse[row0 + r] = lse_of(m, l);
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(p.o_part + (part + r) * D + 2 * t * NO);
#pragma unroll
                        for (int i = 0; i < NO / 2; ++i) dst[i] = v[i];
                        if (t == 0) *reinterpret_cast<float2 *>(p.ml_part + (part + r) * 2) = make_float2(m, l);
                    }
                }
            } else {
                // the warps of one head join their parts
                float2 *ml = reinterpret_cast<float2 *>(smem + C::ML_OFF);
                float *ob = reinterpret_cast<float *>(smem + C::O_OFF);
                if (t == 0) {
                    ml[warp * 16 + g] = make_float2(m0, l0);
                    ml[warp * 16 + g + 8] = make_float2(m1, l1);
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {  // eight rows at a time
                    if (8 * hh >= nr) break;
                    if (g + 8 * hh < nr) {
                        float *dst = ob + (warp * 8 + g) * D + 2 * t * NO;
#pragma unroll
                        for (int i = 0; i < NO; i += 4) {
                            *reinterpret_cast<float4 *>(dst + i) =
                                make_float4(acc[i][2 * hh], acc[i + 1][2 * hh], acc[i + 2][2 * hh], acc[i + 3][2 * hh]);
                            *reinterpret_cast<float4 *>(dst + NO + i) = make_float4(
                                acc[i][2 * hh + 1], acc[i + 1][2 * hh + 1], acc[i + 2][2 * hh + 1], acc[i + 3][2 * hh + 1]);
                        }
                    }
                    named_barrier(1, kWarps * 32);
                    for (int i = kshare * 32 + lane; i < min(8, nr - 8 * hh) * (D / 4); i += shares * 32) {
                        const int r8 = i / (D / 4), c4 = i % (D / 4), r = r8 + 8 * hh;
                        float mx = -INFINITY, l = 0.f;
                        for (int w = hw; w < kWarps; w += p.heads) mx = fmaxf(mx, ml[w * 16 + r].x);
                        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int w = hw; w < kWarps; w += p.heads) {
                            const float2 a = ml[w * 16 + r];
                            const float f = a.x == mx ? 1.f : ex2_approx(a.x - mx);
                            const float4 v = *reinterpret_cast<const float4 *>(ob + (w * 8 + r8) * D + c4 * 4);
                            o.x = fmaf(v.x, f, o.x);
                            o.y = fmaf(v.y, f, o.y);
                            o.z = fmaf(v.z, f, o.z);
                            o.w = fmaf(v.w, f, o.w);
                            l = fmaf(a.y, f, l);
                        }
                        if (whole) {
                            const float inv = l == 0.f ? 0.f : 1.f / l;
                            store4<D, T>(static_cast<T *>(p.o) + (row0 + r) * D + c4 * 4,
                                         make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                            if (c4 == 0 && p.lse) p.lse[row0 + r] = lse_of(mx, l);
                        } else {
                            *reinterpret_cast<float4 *>(p.o_part + (part + r) * D + c4 * 4) = o;
                            if (c4 == 0) *reinterpret_cast<float2 *>(p.ml_part + (part + r) * 2) = make_float2(mx, l);
                        }
                    }
                    named_barrier(1, kWarps * 32);
                }
            }
        }
        if (it + 1 == n_units && threadIdx.x == 0) {
            // the item that this CTA begins and others go on with, if there is one
            const int64_t first_unit = u0 + it - cur.j;
            Kv8Cut c = {0, 0, 0, 0, 0};
            if (!item_ends && first_unit >= u0) {
                c.parts = static_cast<int>(shared_out.owner(first_unit + cur.n - 1) - blockIdx.x) + 1;
                c.second = first_unit > u0 ? 1 : 0;
                c.b = cur.b;
                c.hg = cur.hg;
                c.tile = cur.tile;
            }
            p.cut[blockIdx.x] = c;
        }
        next_unit(p, cur);
    }
}

// Joins the parts of an item that several CTAs share: blockIdx.x is the CTA
// that begins the item, blockIdx.y the head of its group.  Few rows: several
// warps share a row's parts and add up what they have, in a fixed order.
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_kv8_join_kernel(const __grid_constant__ Kv8Params p)
{
    constexpr int VEC = D / 32;
    constexpr int LOADS = kKv8MaxCtas / 32;
    __shared__ float weight[kKv8MaxCtas][kKv8Tile];  // of each part in each row
    __shared__ float red[8][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
    const Kv8Cut cut = p.cut[blockIdx.x];
    const int n = cut.parts;
    if (n == 0) return;
    const int hw = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nr = min(kKv8Tile, p.rows - cut.tile * kKv8Tile);
    auto part_of = [&](int k) { return part_at(2 * (static_cast<int64_t>(blockIdx.x) + k) + (k == 0 ? cut.second : 0), hw); };
    const int64_t row0 = row_at(p, cut.b, cut.hg * p.heads + hw, cut.tile * kKv8Tile);
    for (int r = warp; r < nr; r += 8) {
        float2 a[LOADS];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int k = lane + 32 * i;
            a[i] = k < n ? __ldcg(reinterpret_cast<const float2 *>(p.ml_part + (part_of(k) + r) * 2)) : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, a[i].x);
        }
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            a[i].x = a[i].x == m ? 1.f : ex2_approx(a[i].x - m);
            l = fmaf(a[i].y, a[i].x, l);
        }
        l = row_sum<32>(l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (lane + 32 * i < n) weight[lane + 32 * i][r] = a[i].x * inv;
        if (lane == 0 && p.lse) p.lse[row0 + r] = lse_of(m, l);
    }
    __syncthreads();
    const int wide = nr >= 8 ? 8 : (nr > 2 ? (nr > 4 ? 8 : 4) : nr);  // warps that have rows of their own
    const int sub = warp / wide, subs = 8 / wide;
    for (int r0 = 0; r0 < nr; r0 += wide) {
        const int r = r0 + warp % wide;
        float o[VEC] = {};
        if (r < nr) {
#pragma unroll 8
            for (int k = sub; k < n; k += subs) {
                const float f = weight[k][r];
                const float *src = p.o_part + (part_of(k) + r) * D + lane * VEC;
                if constexpr (VEC == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                    o[0] = fmaf(v.x, f, o[0]), o[1] = fmaf(v.y, f, o[1]), o[2] = fmaf(v.z, f, o[2]), o[3] = fmaf(v.w, f, o[3]);
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                    o[0] = fmaf(v.x, f, o[0]), o[1] = fmaf(v.y, f, o[1]);
                }
            }
        }
        if (subs > 1) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) red[warp][lane * VEC + i] = o[i];
            __syncthreads();
            if (sub == 0)
                for (int q = 1; q < subs; ++q)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o[i] += red[warp + q * wide][lane * VEC + i];
            __syncthreads();
        }
        if (sub == 0 && r < nr) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(p.o) + (row0 + r) * D + lane * VEC);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) dst[i] = Pair<T>::put(o[2 * i], o[2 * i + 1]);
        }
    }
}

template <int D, typename T>
cudaError_t launch_kv8_t(const Kv8LaunchArgs &a)
{
    auto kern = attn_kv8_kernel<D, T>;
    std::atomic<int> &ready = a.attr_ready[(D == 64 ? 0 : 2) + (Elem<T>::BF16 ? 1 : 0)];
    cudaError_t e;
    if (ready.load(std::memory_order_acquire) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Kv8Cfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    kern<<<a.grid, kThreads, Kv8Cfg<D>::SMEM, a.stream>>>(a.k, a.v, a.p);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.grid < 2) return e;
    // the join may be brought up while the last parts are computed; it waits for them itself
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.grid), static_cast<unsigned>(a.p.heads));
    cfg.blockDim = dim3(256);
    cfg.stream = a.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kv8_join_kernel<D, T>, a.p);
}

}  // namespace

cudaError_t launch_kv8(const Kv8LaunchArgs &a, int d, bool bf16)
{
    if (d == 64) return bf16 ? launch_kv8_t<64, __nv_bfloat16>(a) : launch_kv8_t<64, __half>(a);
    return bf16 ? launch_kv8_t<128, __nv_bfloat16>(a) : launch_kv8_t<128, __half>(a);
}

}  // namespace attn
