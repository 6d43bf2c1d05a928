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
// stride reached 2.2 of 6.8 TB/s).  An item is 8 or 16 query rows of such a group
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
// head meet at an item's end only.  Per 32 keys a warp computes S^T = K Q^T
// and O^T += V^T P^T: keys, and values of the head, are the 16 rows of a
// matrix instruction and the query rows its 8 columns (one or two sets of
// them), so that few query rows waste little.
//   K and V enter as fp16, converted (exactly) in registers.  The order of
//   the head's values in a dot product is free, so a lane takes 32 contiguous
//   ones (d = 128) of a key's row in two 16-byte loads.
//   Q enters as fp16: fp16 inputs as they are, bf16 inputs times a power of
//   two for each row that puts the row's largest value at 2^14, which keeps
//   all 8 significant bits of every value down to 2^-21 of the largest, and
//   rounds smaller ones at 2^-39 of it.
//   P is rounded to fp16 (2^-11 relative, between 2^-14 and 2^14) and
//   transposed in registers.
// (e4m3 products of these matrix instructions are no way round the
// conversions: 16 of them, one after another, take 560 clocks, the fp16
// products they would replace 224.)
//
// Softmax, in log2: s = ks scale log2(e) (q . k8), x = s + log2(vs).  A key's
// weight is 2^(s - m + 6), summed in fp32, and what meets its values is P =
// 2^(x - m + 6), so O needs no product with their scale.  m follows the
// maximum of x lazily: it is raised (and O and the sum rescaled) only when some
// x exceeds it by more than 8, so P <= 2^14.  In m a scale below 2^-64, zero
// among them, counts as that: zeros weigh in the sum, and do not raise m above
// the values beside them.  One exponential gives both, of x where vs >= 1 (to
// its power of two) and of s where it is smaller: whichever is larger, so that
// neither falls out of fp32 for the other's sake.
//
// What bounds it: the bytes of the cache.  8 caches of 1 to 16383 tokens (8
// key heads, d = 128, 127 MB, 18.7 us at a copy's rate): 31.8 us, of which the
// join 5; the same copies without any arithmetic take 24.6.  1001 tokens of
// one cache: 9.9 a call, two launches and their chains of loads.
#include "attn_kv8_common.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;                         // consumers
constexpr int kThreads = (kWarps + 4) * 32;       // and a warpgroup of which one warp copies
constexpr int kConsumerRegs = 216, kProducerRegs = 72;  // 256 * 216 + 128 * 72 = 384 * 168
constexpr int kStepKeys = 32;                     // keys of a warp's step

template <int D>
struct Kv8Cfg {
    static constexpr int KBYTES = kStepKeys * D;           // a warp's K (or V) rows of a step
    static constexpr int STAGE = 2 * kWarps * KBYTES;      // K of all warps, then V
    static constexpr int STAGES = D == 128 ? 2 : 4;        // 128 KB in flight
    static constexpr int O_OFF = STAGES * STAGE;           // where the warps of one head meet [warps][8 rows][D]
    static constexpr int ML_OFF = O_OFF + kWarps * 8 * D * 4;     // [warps][8] float2
    static constexpr int SC_OFF = ML_OFF + kWarps * 8 * 8;        // [STAGES][warps] scales: K, K, V, V
    static constexpr int BAR_OFF = SC_OFF + kWarps * STAGES * 16; // [STAGES] full, then empty
    static constexpr int CTL_OFF = BAR_OFF + 2 * STAGES * 8;
    static constexpr int SMEM = CTL_OFF + 16 + 1024;       // +1 KiB for alignment
    static_assert(SMEM <= 232448, "shared memory budget");
};

// c += A B: A 16 x 16, B 16 x 8, fp16.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 tile of 16-bit values, two of a row to a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

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

// Keys [0, end) are seen by some row of the tile, keys [0, all) by every one.
struct Seen {
    int end, all;
};

__device__ __forceinline__ Seen seen_keys(const Kv8Params &p, const Place &c)
{
    if (!p.causal) return {c.len, c.len};
    const int r0 = c.tile * p.tile_rows, r1 = min(r0 + p.tile_rows, p.rows) - 1;
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

template <int D, typename T>
__device__ __forceinline__ void store4(T *o, float4 v)
{
    *reinterpret_cast<uint2 *>(o) = make_uint2(Pair<T>::put(v.x, v.y), Pair<T>::put(v.z, v.w));
}

template <int D, typename T, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kv8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ Kv8Params p)
{
    using C = Kv8Cfg<D>;
    constexpr int STAGES = C::STAGES;
    constexpr int KS = D / 16;      // k-steps of S, and words of a lane's share of a K row
    constexpr int VW = D / 32;      // words of a lane's share of a V row
    constexpr int NO = D / 16;      // row tiles of O^T
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
    await_previous();

    const Shares shared_out(total_units(p), static_cast<int>(gridDim.x));
    if (blockIdx.x >= shared_out.ctas) {
        if (threadIdx.x == 0) p.cut[blockIdx.x].parts = 0;
        return;
    }
    const int64_t u0 = shared_out.start(blockIdx.x);
    const int n_units = static_cast<int>(shared_out.start(blockIdx.x + 1) - u0);
    Place cur = place_of(p, u0);
    // of the unit of a CTA's warps; all of them come to the same answer
    auto place_in_bounds = [&](const Place &c) {
        const bool ok = ATTN_OPS_IN_BOUNDS(c.b >= 0 && c.b < p.b && c.hg >= 0 && c.hg < p.head_groups && c.tile >= 0 &&
                                               c.tile < p.tiles && c.j >= 0 && c.j < c.n, p, SITE_OPS_UNIT);
        if (!ok) *abort_flag = 1u;
        return ok;
    };

    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
        if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
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
        if (warp == kWarps) {
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
                if (!place_in_bounds(cur)) break;
                end = seen_keys(p, cur).end;
                table = p.block_table + static_cast<int64_t>(cur.b) * p.pages_per_seq;
                head_scales = scales + static_cast<int64_t>(cur.hg * p.heads + hw) * blocks_per_page;
            }
            const int u_key = cur.j * p.unit_keys;
            if (u_key < end) {
                const int shares = min((end - u_key + kStepKeys - 1) / kStepKeys, kWarps >> head_shift);
                const int k = u_key + kshare * kStepKeys + 16 * half;
                const int pg = page_shift >= 0 ? k >> page_shift : k / p.page_size, off = k - pg * p.page_size;
                const int page = k < end ? table[pg] : -1;
                const bool in = page >= 0 && page < p.num_pages;
                const uint32_t st = issued % STAGES, bar = full_bar(st);
                if (!__all_sync(0xffffffffu, wait(empty_bar(st), ((issued / STAGES) & 1u) ^ 1u, SITE_KV8_EMPTY))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar, shares * p.heads * (2 * C::KBYTES));
                if (copies && kshare < shares)
                    // a page outside the pool is read at the token past its end: the copy fills zeros
                    tma_load_3d(base + st * C::STAGE + to, map, bar, 0, in ? page * p.page_size + off : nowhere,
                                cur.hg * p.heads, pol);
                const uint32_t sc = base + C::SC_OFF + st * (kWarps * 16) + (w * 4 + kv * 2 + half) * 4;
                const int64_t from = static_cast<int64_t>(page) * p.h_kv * blocks_per_page + (off >> p.block_shift);
                if (in && scale_in_bounds(p, head_scales - scales + from)) {
                    cp_async4(sc, head_scales + from);
                    cp_async_arrive(bar);
                } else {
                    // a page outside the pool, which reads as zeros, or no key that any row sees
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc), "f"(0.f) : "memory");
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
        }
    } else {
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
    // A lane's share: of keys, g and g + 8 of each 16; of query rows, 2 t and
    // 2 t + 1 of each 8; of O's columns, 2 NO from 2 NO g on.
    uint32_t qb[NT][KS][2];
    float acc[NT][NO][4];   // [.][.][0], [1]: an even column of rows 2 t, 2 t + 1; [2], [3]: the odd one after it
    float m[NT][2], l[NT][2], coef[NT][2];
    int lim[NT][2];
    // One step of 32 keys from k0 on, in stage st.  PARTLY: some query row
    // does not see some of the keys.
    Place at = cur;
    auto step = [&](int k0, uint32_t st, auto partly) __attribute__((always_inline)) {
        constexpr bool PARTLY = decltype(partly)::value;
        const uint8_t *ks_at = mine + st * C::STAGE, *vs_at = ks_at + kWarps * C::KBYTES;
        const float4 sc = sc_ptr[st * kWarps];
        // of the two halves: log2 of the values' scales as it enters the reference; e = 2^(s + lift - m + 6), of which
        // a key's weight is e * weigh and its P e * times
        float lv[2], lift[2], weigh[2], times[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float vs = h ? sc.w : sc.z;
            lv[h] = log2_scale(fmaxf(vs, kLeastScale));
            const int up = min(max(static_cast<int>(__float_as_uint(vs) << 1 >> 24), 127), 253);  // 1 at least, biased
            lift[h] = static_cast<float>(up - 127);
            weigh[h] = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
            times[h] = vs * weigh[h];
        }
        // S^T: two tiles of 16 keys
        float s[2][NT][4];
        {
            uint32_t w0[2][KS], w1[2][KS];  // of keys g and g + 8
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < KS / 4; ++c) {  // 16 bytes of the lane's share of each
                    const uint8_t *src = ks_at + (h ? second : 0u) +
                                         (D == 128 ? g * 128 + (((2 * t + c) ^ g) << 4) : g * 64 + ((t ^ ((g >> 1) & 3)) << 4));
                    const uint4 a = *reinterpret_cast<const uint4 *>(src);
                    const uint4 b = *reinterpret_cast<const uint4 *>(src + 8 * D);  // the swizzle repeats
                    w0[h][4 * c] = a.x, w0[h][4 * c + 1] = a.y, w0[h][4 * c + 2] = a.z, w0[h][4 * c + 3] = a.w;
                    w1[h][4 * c] = b.x, w1[h][4 * c + 1] = b.y, w1[h][4 * c + 2] = b.z, w1[h][4 * c + 3] = b.w;
                }
            // two sums for each tile, so that a product waits for its own only
            float c2[2][NT][2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) c2[h][nt][0][i] = c2[h][nt][1][i] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16(w0[h][k], a0, a2);
                    e4m3x4_to_f16(w1[h][k], a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(c2[h][nt][k & 1], a0, a1, a2, a3, qb[nt][k][0], qb[nt][k][1]);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[h][nt][i] = (c2[h][nt][0][i] + c2[h][nt][1][i]) * (coef[nt][i & 1] * (h ? sc.y : sc.x));
        }
        if constexpr (PARTLY) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k0 + 16 * h + g + 8 * (i >> 1) >= lim[nt][i & 1]) s[h][nt][i] = -INFINITY;
        }
        bool over = false;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[nt][i] = fmaxf(fmaxf(s[0][nt][i], s[0][nt][2 + i]) + lv[0], fmaxf(s[1][nt][i], s[1][nt][2 + i]) + lv[1]);
                over = over || top[nt][i] > m[nt][i] + kSlack;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float n = top[nt][i];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, off));
                    n = fmaxf(n, m[nt][i]);
                    const float fh = half_step(m[nt][i], n), f = fh * fh;
                    m[nt][i] = n;
                    l[nt][i] = l[nt][i] * fh * fh;
#pragma unroll
                    for (int j = 0; j < NO; ++j) {
                        acc[nt][j][i] *= f;
                        acc[nt][j][2 + i] *= f;
                    }
                }
        }
        uint32_t pb[2][NT][2];  // P^T: two keys of query row g
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kOffset;
            const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kOffset;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float a0 = b0 - lift[h], a1 = b1 - lift[h];
                const float2 e0 = make_float2(ex2_approx(s[h][nt][0] - a0), ex2_approx(s[h][nt][1] - a1));
                const float2 e1 = make_float2(ex2_approx(s[h][nt][2] - a0), ex2_approx(s[h][nt][3] - a1));
                l[nt][0] = fmaf(e0.x + e1.x, weigh[h], l[nt][0]);
                l[nt][1] = fmaf(e0.y + e1.y, weigh[h], l[nt][1]);
                const float2 f = make_float2(times[h], times[h]), p0 = __fmul2_rn(e0, f), p1 = __fmul2_rn(e1, f);
                pb[h][nt][0] = transposed(Pair<__half>::put(p0.x, p0.y));
                pb[h][nt][1] = transposed(Pair<__half>::put(p1.x, p1.y));
            }
        }
        // O^T += V^T P^T, 16 keys at a time
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v[4][VW];  // of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 2 * t + (i & 1) + 8 * (i >> 1);
                const uint8_t *at = vs_at + (h ? second : 0u);
                if constexpr (D == 128) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(at + row * 128 + ((g ^ (row & 7)) << 4));
                    v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
                } else {
                    const uint2 a = *reinterpret_cast<const uint2 *>(
                        at + row * 64 + ((((g >> 1) ^ ((row >> 1) & 3)) << 4) | ((g & 1) << 3)));
                    v[i][0] = a.x, v[i][1] = a.y;
                }
            }
            if constexpr (PARTLY) {
                // Rows from the length on are no keys: zero them.  A NaN
                // among V must reach the query rows that see its key and
                // no other, but a row that does not still multiplies it,
                // by 0: take it out of the product and put it into the
                // rows that see it (the product of where V is NaN with
                // what each row sees counts them).
                uint32_t any = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        if (k0 + 16 * h + 2 * t + (i & 1) + 8 * (i >> 1) >= at.len) v[i][w] = 0u;
                        any |= nan_bytes(v[i][w]);
                    }
                if (__any_sync(0xffffffffu, any != 0u)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        // limit of query row g of the set: lane (g >> 1) of the shares has it
                        const int l0 = __shfl_sync(0xffffffffu, lim[nt][0], g >> 1), l1 = __shfl_sync(0xffffffffu, lim[nt][1], g >> 1);
                        const int lg = (g & 1) ? l1 : l0, k = k0 + 16 * h + 2 * t;
                        const uint32_t see0 = (k < lg ? 0x3C00u : 0u) | (k + 1 < lg ? 0x3C000000u : 0u);
                        const uint32_t see1 = (k + 8 < lg ? 0x3C00u : 0u) | (k + 9 < lg ? 0x3C000000u : 0u);
#pragma unroll
                        for (int j = 0; j < NO; ++j) {
                            const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
                            uint32_t ind[4];  // e4m3's 1 where V is NaN
#pragma unroll
                            for (int i = 0; i < 4; ++i) ind[i] = (nan_bytes(v[i][j >> 1]) >> 7) * 0x38u;
                            const uint32_t a = __byte_perm(ind[0], ind[1], sel), b = __byte_perm(ind[2], ind[3], sel);
                            float c[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16(c, e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(b), e4m3x2_to_f16x2(b >> 16),
                                    see0, see1);
#pragma unroll
                            for (int k2 = 0; k2 < 4; ++k2)
                                acc[nt][j][k2] = c[k2] > 0.f ? __int_as_float(0x7FC00000) : acc[nt][j][k2];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int w = 0; w < VW; ++w) v[i][w] &= ~((nan_bytes(v[i][w]) >> 7) * 0xFFu);
                }
            }
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
                const uint32_t a = __byte_perm(v[0][j >> 1], v[1][j >> 1], sel), b = __byte_perm(v[2][j >> 1], v[3][j >> 1], sel);
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16(a, a0, a1);
                e4m3x4_to_f16(b, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][j], a0, a1, a2, a3, pb[h][nt][0], pb[h][nt][1]);
            }
        }
    };
    for (int it = 0; it < n_units;) {
        // an item begins, or goes on from the CTA before
        if (!place_in_bounds(at)) break;
        const Seen seen = seen_keys(p, at);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = at.tile * p.tile_rows + nt * 8 + g;  // the query row whose values this lane prepares
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const T *>(p.q) + row_at(p, at.b, at.hg * p.heads + hw, r < p.rows ? r : 0) * D + t * (D / 4));
            uint32_t w[D / 8];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 v = r < p.rows ? src[i] : make_uint4(0u, 0u, 0u, 0u);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
            float down = 1.f;
            if constexpr (Elem<T>::BF16) {
                uint32_t mx = 0u;  // largest magnitude of the row, as the bits of a non-negative bf16
#pragma unroll
                for (int i = 0; i < D / 8; ++i) mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int e = max(static_cast<int>(mx >> 7) - 127, -100);
                const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
                down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float2 v = Pair<T>::get(w[i]);
                    w[i] = Pair<__half>::put(v.x * up, v.y * up);
                }
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                qb[nt][i][0] = w[2 * i];
                qb[nt][i][1] = w[2 * i + 1];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                coef[nt][i] = p.sl2e * __shfl_sync(0xffffffffu, down, (2 * t + i) * 4);
                const int ri = at.tile * p.tile_rows + nt * 8 + 2 * t + i;
                lim[nt][i] = p.causal ? at.len - p.sq + ri % p.sq + 1 : at.len;
                m[nt][i] = -INFINITY;
                l[nt][i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < NO; ++j) acc[nt][j][0] = acc[nt][j][1] = acc[nt][j][2] = acc[nt][j][3] = 0.f;
        }
        const int j_end = min(at.n, at.j + n_units - it);
        // units of which some row sees a key; steps whose keys every row sees
        const int j_seen = min(j_end, (seen.end + p.unit_keys - 1) / p.unit_keys);
        const int whole_keys = seen.all - (kshare + 1) * kStepKeys;
        const int j_whole = whole_keys < 0 ? 0 : min(j_seen, whole_keys / p.unit_keys + 1);
        const int j_first = at.j;
        int j = j_first;
        auto unit = [&](auto partly) __attribute__((always_inline)) {
            const uint32_t st = used % STAGES;
            const int k0 = j * p.unit_keys + kshare * kStepKeys;
            if (ok) ok = __all_sync(0xffffffffu, wait(full_bar(st), (used / STAGES) & 1u, SITE_KV8_FULL));
            if (ok) {
                if (!decltype(partly)::value || k0 < seen.end) step(k0, st, partly);
                __syncwarp();  // every lane has read the stage
                if (lane == 0) mbar_arrive(empty_bar(st));
                ++used;
            }
        };
#pragma unroll 1
        for (; j < j_whole; ++j) unit(std::false_type());
#pragma unroll 1
        for (; j < j_seen; ++j) unit(std::true_type());
        it += j_end - j_first;
        // the item ends, or goes on in the next CTA
        const bool item_ends = j_end == at.n;
        {
            const int nr = min(p.tile_rows, p.rows - at.tile * p.tile_rows);
            const int64_t first_unit = u0 + it - j_end;  // of the item
            const bool whole = first_unit >= u0 && item_ends;
            const int64_t part = part_at(2 * static_cast<int64_t>(blockIdx.x) + (first_unit > u0 ? 1 : 0), hw);
            const int64_t row0 = row_at(p, at.b, at.hg * p.heads + hw, at.tile * p.tile_rows);
            float2 *ml = reinterpret_cast<float2 *>(smem + C::ML_OFF);
            float *ob = reinterpret_cast<float *>(smem + C::O_OFF);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (8 * nt >= nr) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], off);
                    const int r = nt * 8 + 2 * t + i;
                    if (shares == 1) {
                        if (r >= nr) continue;
                        const float inv = !whole ? 1.f : (l[nt][i] == 0.f ? 0.f : 1.f / l[nt][i]);
                        if (whole) {
                            uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(p.o) + (row0 + r) * D + 2 * NO * g);
#pragma unroll
                            for (int j = 0; j < NO; j += 4)
                                *reinterpret_cast<uint4 *>(dst + j) =
                                    make_uint4(Pair<T>::put(acc[nt][j][i] * inv, acc[nt][j][2 + i] * inv),
                                               Pair<T>::put(acc[nt][j + 1][i] * inv, acc[nt][j + 1][2 + i] * inv),
                                               Pair<T>::put(acc[nt][j + 2][i] * inv, acc[nt][j + 2][2 + i] * inv),
                                               Pair<T>::put(acc[nt][j + 3][i] * inv, acc[nt][j + 3][2 + i] * inv));
                            if (g == 0 && p.lse) p.lse[row0 + r] = lse_of(m[nt][i], l[nt][i]);
                        } else {
                            float *dst = p.o_part + (part + r) * D + 2 * NO * g;
#pragma unroll
                            for (int j = 0; j < NO; j += 2)
                                *reinterpret_cast<float4 *>(dst + 2 * j) =
                                    make_float4(acc[nt][j][i], acc[nt][j][2 + i], acc[nt][j + 1][i], acc[nt][j + 1][2 + i]);
                            if (g == 0) *reinterpret_cast<float2 *>(p.ml_part + (part + r) * 2) = make_float2(m[nt][i], l[nt][i]);
                        }
                    } else {
                        // several warps have parts of this head's rows: eight rows of each meet in shared memory
                        if (g == 0) ml[warp * 8 + 2 * t + i] = make_float2(m[nt][i], l[nt][i]);
                        float *dst = ob + (warp * 8 + 2 * t + i) * D + 2 * NO * g;
#pragma unroll
                        for (int j = 0; j < NO; j += 2)
                            *reinterpret_cast<float4 *>(dst + 2 * j) =
                                make_float4(acc[nt][j][i], acc[nt][j][2 + i], acc[nt][j + 1][i], acc[nt][j + 1][2 + i]);
                    }
                }
                if (shares == 1) continue;
                named_barrier(1, kWarps * 32);
                for (int i = kshare * 32 + lane; i < min(8, nr - 8 * nt) * (D / 4); i += shares * 32) {
                    const int r8 = i / (D / 4), c4 = i % (D / 4), r = r8 + 8 * nt;
                    float mx = -INFINITY, lx = 0.f;
                    for (int w = hw; w < kWarps; w += p.heads) mx = fmaxf(mx, ml[w * 8 + r8].x);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int w = hw; w < kWarps; w += p.heads) {
                        const float2 a = ml[w * 8 + r8];
                        const float fh = half_step(a.x, mx), f = fh * fh;
                        const float4 v = *reinterpret_cast<const float4 *>(ob + (w * 8 + r8) * D + c4 * 4);
                        o.x = fmaf(v.x, f, o.x);
                        o.y = fmaf(v.y, f, o.y);
                        o.z = fmaf(v.z, f, o.z);
                        o.w = fmaf(v.w, f, o.w);
                        lx = fmaf(a.y * fh, fh, lx);
                    }
                    if (whole) {
                        const float inv = lx == 0.f ? 0.f : 1.f / lx;
                        store4<D, T>(static_cast<T *>(p.o) + (row0 + r) * D + c4 * 4,
                                     make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                        if (c4 == 0 && p.lse) p.lse[row0 + r] = lse_of(mx, lx);
                    } else {
                        *reinterpret_cast<float4 *>(p.o_part + (part + r) * D + c4 * 4) = o;
                        if (c4 == 0) *reinterpret_cast<float2 *>(p.ml_part + (part + r) * 2) = make_float2(mx, lx);
                    }
                }
                named_barrier(1, kWarps * 32);
            }
        }
        if (it == n_units && threadIdx.x == 0) {
            // the item that this CTA begins and others go on with, if there is one
            const int64_t first_unit = u0 + it - j_end;
            Kv8Cut c = {0, 0, 0, 0};
            if (!item_ends && first_unit >= u0) {
                c.parts = static_cast<int>(shared_out.owner(first_unit + at.n - 1) - blockIdx.x) + 1;
                if (first_unit > u0) c.parts = -c.parts;
                c.b = at.b;
                c.hg = at.hg;
                c.tile = at.tile;
            }
            p.cut[blockIdx.x] = c;
        }
        at.j = at.n - 1;
        next_unit(p, at);
    }
    }
}

// VEC consecutive fp32 values, past L1 (another kernel wrote them).
template <int VEC>
__device__ __forceinline__ void load_part(const float *src, float (&v)[VEC])
{
    if constexpr (VEC == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
        v[0] = x.x, v[1] = x.y;
    }
}

constexpr int kJoinAhead = 8, kRounds = 2;

// Joins the parts of an item that several CTAs share: the blockIdx.x-th of
// such items, blockIdx.y the head of its group and which `rows` of its rows.
// The shares are added up in a fixed order.
//
// Of two parts, as most items have when there are more items than CTAs, a
// warp takes four rows at a time, of three or four two.  Of more, a warp takes
// a row and, when there are few rows, a share of its parts: the first parts'
// values are on their way while it forms the weights of all of them.
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_kv8_join_kernel(const __grid_constant__ Kv8Params p, int grid, int rows)
{
    constexpr int VEC = D / 32, LOADS = kKv8MaxCtas / 32, AHEAD = kJoinAhead;
    __shared__ float red[8][D], weight[8][kKv8MaxCtas];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    await_previous();
    int64_t cta = -1;  // the one that begins the item
    Kv8Cut cut;
    {
        int4 c[LOADS];
        int before = 0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            c[i] = lane + 32 * i < grid ? __ldcg(reinterpret_cast<const int4 *>(p.cut + lane + 32 * i)) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint32_t cuts = __ballot_sync(0xffffffffu, c[i].x != 0);
            const bool it_is = c[i].x != 0 && before + __popc(cuts & ((1u << lane) - 1u)) == static_cast<int>(blockIdx.x);
            const uint32_t found = __ballot_sync(0xffffffffu, it_is);
            if (found != 0u) {
                const int src = __ffs(found) - 1;
                cta = 32 * i + src;
                cut.parts = __shfl_sync(0xffffffffu, c[i].x, src);
                cut.b = __shfl_sync(0xffffffffu, c[i].y, src);
                cut.hg = __shfl_sync(0xffffffffu, c[i].z, src);
                cut.tile = __shfl_sync(0xffffffffu, c[i].w, src);
            }
            before += __popc(cuts);
        }
    }
    if (cta < 0) return;
    const int n = abs(cut.parts);
    if (!ATTN_OPS_IN_BOUNDS(cta + n <= grid && cut.b >= 0 && cut.b < p.b && cut.tile >= 0 && cut.tile < p.tiles && cut.hg >= 0 &&
                                cut.hg < (p.tile_rows > kKv8Tile ? p.h_kv : p.head_groups), p, SITE_OPS_PART))
        return;
    const bool many = p.tile_rows > kKv8Tile;
    const int pieces = p.tile_rows / rows, hw = blockIdx.y / pieces;
    const int in_item = (blockIdx.y - hw * pieces) * rows;         // of its rows, the block's first
    const int first = cut.tile * p.tile_rows + in_item;            // of its key head's rows
    const int nr = min(rows, p.rows - first);
    if (nr <= 0) return;
    auto part_of = [&](int k) {
        return (2 * (cta + k) + (k == 0 && cut.parts < 0 ? 1 : 0)) * (many ? kKv8WideRows : kWarps * kKv8Tile) + hw * kKv8Tile +
               in_item;
    };
    const int64_t row0 = row_at(p, cut.b, many ? cut.hg : cut.hg * p.heads + hw, first);
    auto store = [&](int r, const float (&o)[VEC], float inv) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(p.o) + (row0 + r) * D + lane * VEC);
        if constexpr (VEC == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(Pair<T>::put(o[0] * inv, o[1] * inv), Pair<T>::put(o[2] * inv, o[3] * inv));
        else
            *dst = Pair<T>::put(o[0] * inv, o[1] * inv);
    };
    auto join_few = [&](auto parts_, auto at_once_) {
        constexpr int N = decltype(parts_)::value, AT_ONCE = decltype(at_once_)::value;
        int64_t part[N];
#pragma unroll
        for (int k = 0; k < N; ++k) part[k] = part_of(k);
        for (int r0 = warp; r0 < nr; r0 += 8 * AT_ONCE) {
            float2 ml[AT_ONCE][N];
            float v[AT_ONCE][N][VEC];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int r = r0 + 8 * i;
                if (r >= nr) continue;
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    ml[i][k] = __ldcg(reinterpret_cast<const float2 *>(p.ml_part + (part[k] + r) * 2));
                    load_part<VEC>(p.o_part + (part[k] + r) * D + lane * VEC, v[i][k]);
                }
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int r = r0 + 8 * i;
                if (r >= nr) continue;
                float m = ml[i][0].x, l = 0.f, o[VEC] = {};
#pragma unroll
                for (int k = 1; k < N; ++k) m = fmaxf(m, ml[i][k].x);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float fh = half_step(ml[i][k].x, m), f = fh * fh;
                    l = fmaf(ml[i][k].y * fh, fh, l);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] = fmaf(v[i][k][e], f, o[e]);
                }
                store(r, o, l == 0.f ? 0.f : 1.f / l);
                if (lane == 0 && p.lse) p.lse[row0 + r] = lse_of(m, l);
            }
        }
    };
    if (n == 2) return join_few(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
    if (n == 3) return join_few(std::integral_constant<int, 3>(), std::integral_constant<int, 2>());
    if (n == 4) return join_few(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    const int wide = nr > 4 ? 8 : (nr > 2 ? 4 : nr);  // warps that have rows of their own
    const int sub = warp / wide, subs = 8 / wide;
    for (int r0 = 0; r0 < nr; r0 += wide) {
        const int r = r0 + warp % wide;
        const bool have = r < nr;
        float v[AHEAD][VEC];
        auto load = [&](int k0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (have && k0 + i * subs < n) load_part<VEC>(p.o_part + (part_of(k0 + i * subs) + r) * D + lane * VEC, v[i]);
        };
        load(sub);
        float2 a[LOADS];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int k = lane + 32 * i;
            a[i] = have && k < n ? __ldcg(reinterpret_cast<const float2 *>(p.ml_part + (part_of(k) + r) * 2))
                                 : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, a[i].x);
        }
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const float fh = half_step(a[i].x, m);
            a[i].x = fh * fh;
            l = fmaf(a[i].y * fh, fh, l);
        }
        l = row_sum<32>(l);
        if (have && sub == 0 && lane == 0 && p.lse) p.lse[row0 + r] = lse_of(m, l);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) weight[warp][lane + 32 * i] = a[i].x;
        __syncwarp();
        float o[VEC] = {};
        for (int k = sub; have && k < n;) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (k + i * subs < n) {
                    const float f = weight[warp][k + i * subs];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] = fmaf(v[i][e], f, o[e]);
                }
            k += AHEAD * subs;
            load(k);
        }
        __syncwarp();
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
        if (sub == 0 && have) store(r, o, l == 0.f ? 0.f : 1.f / l);
    }
}

template <int D, typename T, int NT>
cudaError_t launch_kv8_t(const Kv8LaunchArgs &a)
{
    auto kern = attn_kv8_kernel<D, T, NT>;
    std::atomic<int> &ready = a.attr_ready[(D == 64 ? 0 : 4) + (Elem<T>::BF16 ? 2 : 0) + NT - 1];
    cudaError_t e;
    if (ready.load(std::memory_order_acquire) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Kv8Cfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    e = launch_overlapped(kern, dim3(a.grid), kThreads, Kv8Cfg<D>::SMEM, a.stream, a.k, a.v, a.p);
    return e == cudaSuccess ? launch_kv8_join(a, D, Elem<T>::BF16) : e;
}

template <int D, typename T>
cudaError_t launch_join_t(const Kv8LaunchArgs &a)
{
    if (a.grid < 2) return cudaSuccess;
    const bool many = a.p.tile_rows > kKv8Tile;
    // no more items are cut than there are items, or cuts
    const int64_t items = static_cast<int64_t>(a.p.b) * (many ? a.p.h_kv : a.p.head_groups) * a.p.tiles;
    // Rows of a block.  Of items of few parts as many as keep the GPU full of blocks, up to 64; of many parts eight, one
    // for each warp, and fewer while there are not enough blocks for the GPU and a warp would go through its share of a
    // row's parts in more than kRounds rounds.  In us for the whole call, 16 rows and this: 256 rows of 256 items, 151 of
    // them cut in two 488 and 442 (the join itself 39 and 14); one cache of 16383 tokens, 8 key heads, 4 rows 17.2 and
    // 13.5; two of 16000, one key head, 256 rows 49.2 and 41.6.
    const int64_t cuts = items < a.grid - 1 ? items : a.grid - 1;
    const int heads = many ? 1 : a.p.heads, used = a.p.rows < a.p.tile_rows ? a.p.rows : a.p.tile_rows;
    const int64_t parts = a.grid / items + 2;  // of an item, about
    auto blocks_of = [&](int r) { return cuts * heads * ((used + r - 1) / r); };
    auto warps_a_row = [&](int r) { const int n = r < used ? r : used; return n > 4 ? 1 : (n > 2 ? 2 : 8 / n); };
    int rows = parts > 4 ? 8 : (many ? 4 * kKv8Tile : a.p.tile_rows);
    if (parts <= 4)
        while (rows > 8 && blocks_of(rows) < 2 * a.grid) rows /= 2;
    while (rows > 1 && blocks_of(rows) < a.grid && parts > kRounds * kJoinAhead * warps_a_row(rows)) rows /= 2;
    const dim3 blocks(static_cast<unsigned>(cuts), static_cast<unsigned>(heads * (a.p.tile_rows / rows)));
    return launch_overlapped(attn_kv8_join_kernel<D, T>, blocks, 256, 0, a.stream, a.p, a.grid, rows);
}

template <int D, typename T>
cudaError_t launch_kv8_rows(const Kv8LaunchArgs &a)
{
    return a.p.tile_rows == 8 ? launch_kv8_t<D, T, 1>(a) : launch_kv8_t<D, T, 2>(a);
}

}  // namespace

cudaError_t launch_kv8_join(const Kv8LaunchArgs &a, int d, bool bf16)
{
    if (d == 64) return bf16 ? launch_join_t<64, __nv_bfloat16>(a) : launch_join_t<64, __half>(a);
    return bf16 ? launch_join_t<128, __nv_bfloat16>(a) : launch_join_t<128, __half>(a);
}

cudaError_t launch_kv8(const Kv8LaunchArgs &a, int d, bool bf16)
{
    if (d == 64) return bf16 ? launch_kv8_rows<64, __nv_bfloat16>(a) : launch_kv8_rows<64, __half>(a);
    return bf16 ? launch_kv8_rows<128, __nv_bfloat16>(a) : launch_kv8_rows<128, __half>(a);
}

}  // namespace attn
