// Attention of many new queries over an e4m3 paged cache (chunks of a
// prompt, long drafts; more than 48 rows of a key head): the operation of
// attn_kv8.cu on the tensor cores' tcgen05 path.
//
// Work.  An item is 256 query rows of one key head of one batch element
// (rows of the query heads that share it, one after another); a unit is 128
// of the keys that some of its rows see.  The units of all items are dealt to
// the CTAs in equal contiguous shares, as there, and an item that several
// CTAs share is joined by the same kernel: 256 items of a 2048-token chunk
// fill 152 CTAs evenly, which whole items would not (two rounds, 84%).
//
// A CTA, 16 warps:
//   warps 0-3, 4-7  softmax group t, one thread to a row of Q tile t (128
//                   rows); its warps also bring Q's rows and store O's
//   warp  8         issues the matrix products
//   warp  9         copies raw K and V tiles (128 keys, TMA) and their scales
//   warps 10-15     convert raw tiles, even ones K's and odd ones V's, to fp16
//                   in the swizzled layout that the products read
// S_t = Q_t K_j^T and O_t += P_t V_j accumulate in tensor memory (128 lanes x
// 128 or d columns of fp32 for each tile); the softmax group overwrites S_t
// with P_t in fp16.  While one group works on its tile, the tensor cores work
// on the other's.
//
// Types.  The products are fp16: e4m3 values are exact in it; bf16 queries
// are scaled by a power of two for each row, as in attn_kv8.cu.  A tile's
// blocks of tokens enter as multiples of the largest scale among them (1 for
// a block of 128 tokens, an exact power of two for scales that are; a factor
// below 2^-15 loses what is below 2^-34 of the tile's largest value), and that
// scale enters the softmax's exponent: x = ks scale log2(e) (q . k) +
// log2(vs), with the sum of the weights divided by vs, tile by tile.  Of
// values it is 2^-64 at least: the quotients stay within fp32.
//
// What bounds it, at the last 2048 of 16384 tokens (causal, 32 heads on
// 8 key heads, d = 128): 437 us, 1.18 of 1.91 PFLOP/s, of which the join 14;
// the tensor cores are at work half of the time.  Without the conversion (raw
// tiles fed as they are, wrong results) 50 to 70 less: a tile of 128 keys
// serves two Q tiles only, so its conversion (16 KB read, 32 KB written and
// read again by the products) takes the shared memory's time away from them.
// The rest is the softmax, one exponential for each score, in step with the
// tensor cores.  A CTA with little to do is bound by its chain: 3 us until it
// knows its share, 4 until Q is in place, 3 to the second tile's scores, 2 a
// tile from there on, 4 to store 128 KB of a part.  At 64 rows (8 caches of up to 16383 tokens, 8 key heads) 101
// to 106 us: the bytes of the cache and their conversion.
#include "attn_kv8_common.cuh"

namespace attn {

namespace {

constexpr int kTileRows = 128, kItemRows = 2 * kTileRows, kTileKeys = 128;
constexpr int kTeam = 3;  // warps that convert K tiles, and as many V tiles (1: 681 us at the chunk above, 3: 498 in the same run)
constexpr int kThreads = (10 + 2 * kTeam) * 32;
static_assert(kThreads % 128 == 0, "whole warpgroups: registers are dealt out by them");
constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;  // 256 * 200 + 256 * 56 = 512 * 128
constexpr int kRefRing = 8;

template <int D>
struct WideCfg {
    static constexpr int PANEL = kTileRows * 128;        // 128 rows of 64 fp16 values, 128-byte swizzle
    static constexpr int TILE = PANEL * (D / 64);        // a Q tile, or a converted K or V tile
    static constexpr int RAW = kTileKeys * D;            // a raw tile
    // without a second Q tile there is room for two raw slots more (d = 128): 119 -> 101 us at 64 rows
    static constexpr int CONV_SLOTS = 4, RAW_SLOTS = D == 128 ? 2 : 8, RAW_SLOTS_ONE = D == 128 ? 4 : 8;
    static constexpr int CTL = 1024;
    static constexpr int Q_OFF = CTL;
    static constexpr int CONV_OFF = Q_OFF + 2 * TILE;
    static constexpr int RAW_OFF = CONV_OFF + CONV_SLOTS * TILE;
    static_assert((RAW_SLOTS_ONE - RAW_SLOTS) * RAW <= TILE, "the second Q tile's room");
    static constexpr int SMEM = RAW_OFF + RAW_SLOTS * RAW + 1024;  // +1 KiB for alignment
    static constexpr int TMEM_O = 2 * kTileKeys;         // O_t at TMEM_O + t * 128
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct WideCtl {
    uint64_t raw_full[8], raw_empty[8];
    uint64_t conv_full[4], conv_empty[4];
    uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], mma_done;
    float scales[8][16];      // of each raw slot's eight groups of 16 keys (a K slot: V's behind them)
    float2 refs[kRefRing];    // {K, V} reference scales of recent tiles
    uint32_t tmem_base, abort, v_nan;
};
static_assert(sizeof(WideCtl) <= 1024, "control block");

// Where in the work a unit lies: block `blk` of key head `kvh`, its units
// [0, n), unit j.
struct WidePlace {
    int b, kvh, blk;
    int j, n;
    int len;
};

struct WideSeen {
    int end, all;  // some row sees keys [0, end); every row sees keys [0, all)
};

__device__ __forceinline__ WideSeen wide_seen(const Kv8Params &p, int len, int blk)
{
    if (!p.causal) return {len, len};
    const int r0 = blk * kItemRows, r1 = min(r0 + kItemRows, p.rows) - 1;
    const int h0 = r0 / p.sq, h1 = r1 / p.sq;  // the rows of one query head are consecutive
    const int i0 = h0 != h1 ? 0 : r0 - h0 * p.sq, i1 = h0 != h1 ? p.sq - 1 : r1 - h1 * p.sq;
    return {max(len - p.sq + i1 + 1, 0), max(len - p.sq + i0 + 1, 0)};
}

// Units of a block: one at least, which writes the rows of a block that sees no key.
__device__ __forceinline__ int wide_units(const Kv8Params &p, int len, int blk)
{
    return max((wide_seen(p, len, blk).end + kTileKeys - 1) / kTileKeys, 1);
}

// Units of one head of batch element b (0 past the last element).
__device__ __forceinline__ int64_t wide_head_units(const Kv8Params &p, int b)
{
    if (b >= p.b) return 0;
    const int len = cached_len(p, b);
    if (!p.causal) return static_cast<int64_t>(p.tiles) * wide_units(p, len, 0);
    int64_t n = 0;
    for (int k = 0; k < p.tiles; ++k) n += wide_units(p, len, k);
    return n;
}

__device__ __forceinline__ int64_t wide_total(const Kv8Params &p)
{
    const int lane = threadIdx.x & 31;
    int64_t t = 0;
    for (int b = lane; b < p.b; b += 32) t += wide_head_units(p, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t * p.h_kv;
}

// Inclusive sums over the lanes; the first lane whose sum exceeds u, with
// what comes before it taken from u, or -1 (and all taken).
__device__ __forceinline__ int lane_of(int64_t v, int64_t &u)
{
    const int lane = threadIdx.x & 31;
    int64_t inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, inc > u);
    const int src = past ? __ffs(past) - 1 : 32;
    const int64_t before = __shfl_sync(0xffffffffu, inc, src > 0 ? src - 1 : 0);
    if (src > 0) u -= before;
    return past ? src : -1;
}

__device__ __forceinline__ WidePlace wide_place(const Kv8Params &p, int64_t u)
{
    const int lane = threadIdx.x & 31;
    WidePlace c{0, 0, 0, 0, 1, 0};
    for (int b0 = 0; b0 < p.b; b0 += 32) {
        const int64_t per = wide_head_units(p, b0 + lane);
        const int src = lane_of(per * p.h_kv, u);
        if (src < 0) continue;
        c.b = b0 + src;
        const int64_t one = __shfl_sync(0xffffffffu, per, src);
        const int64_t kvh = quotient(u, one);
        c.kvh = static_cast<int>(kvh);
        u -= kvh * one;
        break;
    }
    c.len = cached_len(p, c.b);
    for (int k0 = 0; k0 < p.tiles; k0 += 32) {
        const int n = k0 + lane < p.tiles ? wide_units(p, c.len, k0 + lane) : 0;
        const int src = lane_of(n, u);
        if (src < 0) continue;
        c.blk = k0 + src;
        c.n = __shfl_sync(0xffffffffu, n, src);
        break;
    }
    c.j = static_cast<int>(u);
    return c;
}

// The first unit of the next item.
__device__ __forceinline__ void wide_next(const Kv8Params &p, WidePlace &c)
{
    c.j = 0;
    if (++c.blk == p.tiles) {
        c.blk = 0;
        if (++c.kvh == p.h_kv) {
            c.kvh = 0;
            if (++c.b == p.b) return;
            c.len = cached_len(p, c.b);
        }
    }
    c.n = wide_units(p, c.len, c.blk);
}

// A store into a converted tile, ordered with the fence and the arrival that
// follow it (volatile statements keep their order) but not with the reads of
// the raw tile, which the compiler may move ahead of it.
__device__ __forceinline__ void st_tile(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d));
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kv8_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ Kv8Params p)
{
    using C = WideCfg<D>;
    constexpr uint32_t IDESC_QK = idesc_f16(128, kTileKeys, false, false);
    constexpr uint32_t IDESC_PV = idesc_f16(128, D, false, true);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    WideCtl *ctl = reinterpret_cast<WideCtl *>(smem);
    // with rows for one Q tile only, the converted tiles begin where the second
    // would lie and more raw tiles are on their way
    const bool one = p.rows <= kTileRows && C::RAW_SLOTS_ONE != C::RAW_SLOTS;
    const uint32_t raw_slots = one ? C::RAW_SLOTS_ONE : C::RAW_SLOTS;  // a power of two
    const uint32_t raw_shift = 31 - __clz(raw_slots);
    const uint32_t sQ = base + C::Q_OFF, sConv = base + C::CONV_OFF - (one ? C::TILE : 0);
    const uint32_t raw_off = one ? C::RAW_OFF - C::TILE : C::RAW_OFF, sRaw = base + raw_off;
    auto B = [&](const uint64_t &bar) { return smem_addr(&bar); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t *abort_flag = &ctl->abort;

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
    auto warp_waits = [&](uint32_t bar, uint32_t parity, uint32_t site) {
        return static_cast<bool>(__all_sync(0xffffffffu, wait(bar, parity, site)));
    };

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < raw_slots; ++i) {
            // the bytes' announcement and the scales: K's and V's with K (even slots), V's with V
            mbar_init(B(ctl->raw_full[i]), i % 2 == 0 ? 17 : 9);
            mbar_init(B(ctl->raw_empty[i]), kTeam);  // the warps that convert its tile
        }
        for (int i = 0; i < C::CONV_SLOTS; ++i) {
            mbar_init(B(ctl->conv_full[i]), kTeam);
            mbar_init(B(ctl->conv_empty[i]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(B(ctl->q_full[t]), 4);
            mbar_init(B(ctl->s_full[t]), 1);
            mbar_init(B(ctl->p_half[t]), 4);
            mbar_init(B(ctl->p_full[t]), 4);
            mbar_init(B(ctl->o_full[t]), 1);
        }
        mbar_init(B(ctl->mma_done), 1);
        ctl->abort = 0u;
        ctl->v_nan = 0u;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_addr(&ctl->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == 9 && lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    await_previous();

    const Shares shared_out(wide_total(p), static_cast<int>(gridDim.x));
    const bool works = blockIdx.x < shared_out.ctas;
    // (a CTA that gives up on a wait leaves it so: the join must not meet what was in the workspace)
    if (threadIdx.x == 0) p.cut[blockIdx.x].parts = 0;
    const int64_t u0 = works ? shared_out.start(blockIdx.x) : 0;
    const int n_units = works ? static_cast<int>(shared_out.start(blockIdx.x + 1) - u0) : 0;
    WidePlace at = wide_place(p, u0);
    // of an item that a warp begins or goes on with; all of a CTA's come to the same answer
    auto place_in_bounds = [&]() {
        const bool ok = ATTN_OPS_IN_BOUNDS(at.b >= 0 && at.b < p.b && at.kvh >= 0 && at.kvh < p.h_kv && at.blk >= 0 &&
                                               at.blk < p.tiles && at.j >= 0 && at.j < at.n, p, SITE_OPS_UNIT);
        if (!ok) *abort_flag = 1u;
        return ok;
    };

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9) {
            // -------------------------------------------------------- copies
            // Lane i < 8 looks after keys 16 i .. 16 i + 15 of a tile: where a
            // copy begins there it starts it, and it fetches their scale, K's
            // with K and V's with V; lane 8 + i fetches V's with K, since the
            // softmax wants a tile's largest V scale with its scores.
            const int blocks_per_page = p.page_size >> p.block_shift;
            const int page_shift = (p.page_size & (p.page_size - 1)) == 0 ? 31 - __clz(p.page_size) : -1;
            const int nowhere = p.num_pages * p.page_size;
            const uint64_t pol = l2_evict_normal();
            uint32_t n = 0u;  // raw tiles filled
            bool ok = true;
            for (int it = 0; ok && it < n_units;) {
                if (!place_in_bounds()) break;
                const int end = wide_seen(p, at.len, at.blk).end;
                const int j_end = min(at.n, at.j + n_units - it);
                const int32_t *table = p.block_table + static_cast<int64_t>(at.b) * p.pages_per_seq;
                for (int j = at.j; ok && end > 0 && j < j_end; ++j) {
                    const int left = min(at.len - j * kTileKeys, kTileKeys);  // cached keys of the tile
                    const int group = lane & 7, k = j * kTileKeys + 16 * group;
                    const bool there = lane < 16 && 16 * group < left;
                    const int pg = page_shift >= 0 ? k >> page_shift : k / p.page_size, off = k - pg * p.page_size;
                    const int page = there ? table[pg] : -1;
                    const bool in = page >= 0 && page < p.num_pages;
                    const int tok = in ? page * p.page_size + off : nowhere;
                    const bool copies = there && lane < 8 && (16 * group) % p.box == 0;
                    const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, copies));
                    const int64_t sc = (static_cast<int64_t>(page) * p.h_kv + at.kvh) * blocks_per_page + (off >> p.block_shift);
#pragma unroll 1
                    for (int kv = 0; ok && kv < 2; ++kv, ++n) {
                        const uint32_t st = n & (raw_slots - 1), bar = B(ctl->raw_full[st]);
                        ok = warp_waits(B(ctl->raw_empty[st]), ((n >> raw_shift) & 1u) ^ 1u, SITE_KV8_EMPTY);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * p.box * D);
                        if (copies)
                            tma_load_3d(sRaw + st * C::RAW + 16 * lane * D, kv ? &tmV : &tmK, bar, 0, tok, at.kvh, pol);
                        if (lane < (kv ? 8 : 16)) {
                            float *to = &ctl->scales[st][lane];
                            if (in && scale_in_bounds(p, sc)) {
                                cp_async4(smem_addr(to), (kv || lane >= 8 ? p.v_scale : p.k_scale) + sc);
                                cp_async_arrive(bar);
                            } else {
                                // keys past the end, and the zeros of a page outside the pool, take no part
                                // in the tile's largest scale
                                *to = 0.f;
                                mbar_arrive(bar);
                            }
                        }
                        __syncwarp();
                    }
                }
                it += j_end - at.j;
                wide_next(p, at);
            }
            for (uint32_t i = n > raw_slots ? n - raw_slots : 0u; i < n; ++i)
                drain_wait(B(ctl->raw_full[i & (raw_slots - 1)]), (i >> raw_shift) & 1u, p.timeout_ns);
        } else if (warp >= 10) {
            // -------------------------------------------------------- conversion
            // kTeam warps convert the K tiles and as many the V tiles, eight
            // keys at a time: 16 values to a lane, which for odd keys are the
            // other half of the row than for even ones, so that neither the
            // raw reads nor the writes of eight lanes meet in a bank.
            const int kv = warp & 1, wi = (warp - 10) >> 1;
            constexpr int PASSES = D == 128 ? 2 : 1;
            // where a lane's 16 values lie in eight raw rows, and where their two halves go
            uint32_t raw_at[PASSES], out_at[PASSES][2];
#pragma unroll
            for (int h = 0; h < PASSES; ++h) {
                const int r = lane >> 2, c = (lane & 3) + (D == 128 ? 4 * ((r & 1) ^ h) : 0);
                raw_at[h] = r * D + (D == 128 ? c ^ r : c ^ ((r >> 1) & 3)) * 16;
#pragma unroll
                for (int i = 0; i < 2; ++i) out_at[h][i] = (c >> 2) * C::PANEL + r * 128 + (((2 * (c & 3) + i) ^ r) << 4);
            }
            uint32_t tiles = 0u;
            bool ok = true;
            for (int it = 0; ok && it < n_units;) {
                if (!place_in_bounds()) break;
                const WideSeen seen = wide_seen(p, at.len, at.blk);
                const int j_end = min(at.n, at.j + n_units - it);
                for (int j = at.j; ok && seen.end > 0 && j < j_end; ++j, ++tiles) {
                    const int left = at.len - j * kTileKeys;                         // cached keys from the tile's first on
                    const bool whole = (j + 1) * kTileKeys <= (kv ? seen.all : at.len);  // nothing to take out
                    const uint32_t n = 2u * tiles + kv, rs = n & (raw_slots - 1), cs = n % C::CONV_SLOTS;
                    ok = warp_waits(B(ctl->raw_full[rs]), (n >> raw_shift) & 1u, SITE_KV8_FULL);
                    if (!ok) break;
                    const float sc = ctl->scales[rs][lane & 15];
                    float ref = sc;
#pragma unroll
                    for (int off = 4; off > 0; off >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, off));
                    const float vref = __shfl_sync(0xffffffffu, ref, 8);  // of a K slot
                    if (kv == 1) ref = fmaxf(ref, kLeastScale);
                    if (kv == 0 && wi == 0 && lane == 0)
                        ctl->refs[tiles % kRefRing] = make_float2(ref, vref > 0.f ? fmaxf(vref, kLeastScale) : 0.f);
                    const float mul = ref > 0.f ? sc / ref : 0.f;  // lanes 0..7: of keys 16 lane ..
                    ok = warp_waits(B(ctl->conv_empty[cs]), ((n / C::CONV_SLOTS) & 1u) ^ 1u, SITE_KV8_CONV);
                    if (!ok) break;
                    const uint8_t *raw = smem + raw_off + rs * C::RAW;
                    const uint32_t out = sConv + cs * C::TILE;
                    uint32_t nans = 0u;
                    // eight keys at a time: a lane's row is 8 q + (lane >> 2), so only q moves its addresses
#pragma unroll 1
                    for (int q = wi; q < 16; q += kTeam) {
                        const float m = __shfl_sync(0xffffffffu, mul, q >> 1);
                        uint4 v[PASSES];
#pragma unroll
                        for (int h = 0; h < PASSES; ++h) v[h] = *reinterpret_cast<const uint4 *>(raw + raw_at[h] + q * 8 * D);
#pragma unroll
                        for (int h = 0; h < PASSES; ++h) {
                            uint32_t x[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
                            if (!whole) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if (q * 8 + (lane >> 2) >= left) x[e] = 0u;
                                    if (kv == 1) {
                                        // a NaN that some row does not see must not reach it by way of 0 * NaN: it is
                                        // taken out here and put into the rows that see it when they are stored
                                        const uint32_t nb = nan_bytes(x[e]);
                                        nans |= nb;
                                        x[e] &= ~((nb >> 7) * 0xFFu);
                                    }
                                }
                            }
                            uint32_t y[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) e4m3x4_to_f16(x[e], y[2 * e], y[2 * e + 1]);
                            if (m != 1.f) {
                                const uint32_t mm = Pair<__half>::put(m, m);
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const __half2 z = __hmul2(*reinterpret_cast<const __half2 *>(&y[e]),
                                                              *reinterpret_cast<const __half2 *>(&mm));
                                    y[e] = *reinterpret_cast<const uint32_t *>(&z);
                                }
                            }
                            st_tile(out + out_at[h][0] + q * 1024, y[0], y[1], y[2], y[3]);
                            st_tile(out + out_at[h][1] + q * 1024, y[4], y[5], y[6], y[7]);
                        }
                    }
                    if (nans) *reinterpret_cast<volatile uint32_t *>(&ctl->v_nan) = 1u;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(B(ctl->conv_full[cs]));
                        mbar_arrive(B(ctl->raw_empty[rs]));
                    }
                }
                it += j_end - at.j;
                wide_next(p, at);
            }
        } else if (warp == 8) {
            // -------------------------------------------------------- matrix products
            uint32_t n = 0u, q_it[2] = {0u, 0u}, p_it[2] = {0u, 0u};
            bool ok = true;
            auto conv_wait = [&](uint32_t &slot) {
                slot = n % C::CONV_SLOTS;
                const bool r = warp_waits(B(ctl->conv_full[slot]), (n / C::CONV_SLOTS) & 1u, SITE_KV8_CONV);
                ++n;
                return r;
            };
            const uint32_t dq0 = desc_lo(sQ, 16), dk0 = desc_lo(sConv, 16), dv0 = desc_lo(sConv, C::PANEL);
            auto issue_qk = [&](int t, uint32_t slot) {
                const uint32_t a0 = dq0 + ((t * C::TILE) >> 4), b0 = dk0 + ((slot * C::TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {  // 16 values of the head a step
                    const uint32_t off = ((kk / 4) * C::PANEL + (kk % 4) * 32) >> 4;
                    mma_ss(tmem + t * kTileKeys, a0 + off, b0 + off, IDESC_QK, kk > 0 ? 1u : 0u);
                }
            };
            auto issue_pv = [&](int t, uint32_t slot, bool accumulate, int half) {
                const uint32_t b0 = dv0 + ((slot * C::TILE) >> 4);
#pragma unroll
                for (int k2 = 0; k2 < kTileKeys / 32; ++k2) {  // 16 keys a step
                    const int kk = half * (kTileKeys / 32) + k2;
                    mma_ts(tmem + C::TMEM_O + t * 128, tmem + t * kTileKeys + kk * 8, b0 + ((kk * 16 * 128) >> 4), IDESC_PV,
                           (accumulate || kk > 0) ? 1u : 0u);
                }
            };
            for (int it = 0; ok && it < n_units;) {
                if (!place_in_bounds()) break;
                const int end = wide_seen(p, at.len, at.blk).end;
                const int j_end = min(at.n, at.j + n_units - it);
                const int tiles = end > 0 ? j_end - at.j : 0;
                const bool two = at.blk * kItemRows + kTileRows < p.rows;  // Q tile 1 has rows
                if (tiles > 0) {
                    ok = warp_waits(B(ctl->q_full[0]), q_it[0]++ & 1u, SITE_KV8_Q);
                    if (ok && two) ok = warp_waits(B(ctl->q_full[1]), q_it[1]++ & 1u, SITE_KV8_Q);
                    uint32_t ks = 0u;
                    ok = ok && conv_wait(ks);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        issue_qk(0, ks);
                        tc_commit(B(ctl->s_full[0]));
                        if (two) {
                            issue_qk(1, ks);
                            tc_commit(B(ctl->s_full[1]));
                        }
                        tc_commit(B(ctl->conv_empty[ks]));
                    }
                    __syncwarp();
                }
                for (int i = 0; ok && i < tiles; ++i) {
                    const bool more = i + 1 < tiles;
                    uint32_t vs = 0u, ks = 0u;
                    if (!(ok = conv_wait(vs))) break;
                    if (more && !(ok = conv_wait(ks))) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && !two) break;
                        const bool last = t == 1 || !two;  // of the tile's products
                        if (!(ok = warp_waits(B(ctl->p_half[t]), p_it[t] & 1u, SITE_KV8_P))) break;
                        tc_fence_after();
                        if (elect_one()) issue_pv(t, vs, i > 0, 0);
                        __syncwarp();
                        if (!(ok = warp_waits(B(ctl->p_full[t]), p_it[t]++ & 1u, SITE_KV8_P))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_pv(t, vs, true, 1);
                            if (last) tc_commit(B(ctl->conv_empty[vs]));
                            if (more) {
                                issue_qk(t, ks);
                                tc_commit(B(ctl->s_full[t]));
                                if (last) tc_commit(B(ctl->conv_empty[ks]));
                            } else {
                                tc_commit(B(ctl->o_full[t]));
                            }
                        }
                        __syncwarp();
                    }
                }
                it += j_end - at.j;
                wide_next(p, at);
            }
            // every product completes before tensor memory is freed
            if (elect_one()) tc_commit(B(ctl->mma_done));
            __syncwarp();
            drain_wait(B(ctl->mma_done), 0u, p.timeout_ns);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<kSoftmaxRegs>();
        const int t = warp >> 2, row_in_tile = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * kTileKeys, tO = tmem + lane_off + C::TMEM_O + t * 128;
        uint32_t s_it = 0u, o_it = 0u, tiles = 0u;
        bool ok = true;
        for (int it = 0; ok && it < n_units;) {
            if (!place_in_bounds()) break;
            const WideSeen seen = wide_seen(p, at.len, at.blk);
            const int j_end = min(at.n, at.j + n_units - it);
            const int n = seen.end > 0 ? j_end - at.j : 0;
            const int r = at.blk * kItemRows + t * kTileRows + row_in_tile;  // of the key head's rows
            const bool valid = r < p.rows;
            const int64_t row0 = (static_cast<int64_t>(at.b) * p.h_kv + at.kvh) * p.rows;
            const int warp_row = r - lane;  // of the key head's rows, the warp's first
            const bool tile_has_rows = at.blk * kItemRows + t * kTileRows < p.rows;
            float m = -INFINITY, l = 0.f, coef = 0.f;
            const int lim = p.causal ? at.len - p.sq + r % p.sq + 1 : at.len;  // keys this row sees
            if (n > 0 && tile_has_rows) {
                // The warp's 32 rows of Q, all on their way at once, in fp16 into the tile.  LPR lanes share a
                // row, so that an access is of whole rows (a row to a lane: 32 lines an access, 2 us an item more).
                constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows of an access
                const int c = lane % LPR;
                // a negative scale turns Q's signs, so that a masked score is -inf in every case
                const uint32_t turn = p.sl2e < 0.f ? 0x80008000u : 0u;
                uint4 q[LPR];
#pragma unroll
                for (int i = 0; i < LPR; ++i) {
                    const int rr = warp_row + i * RPI + lane / LPR;
                    q[i] = rr < p.rows ? reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + (row0 + rr) * D)[c]
                                       : make_uint4(0u, 0u, 0u, 0u);
                }
                float down = 1.f;  // of the row that is this lane's in the softmax
#pragma unroll
                for (int i = 0; i < LPR; ++i) {
                    uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
                    if constexpr (Elem<T>::BF16) {
                        uint32_t mx = 0u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx = max(mx, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
#pragma unroll
                        for (int off = LPR / 2; off > 0; off >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const int e2 = max(static_cast<int>(mx >> 7) - 127, -100);  // the row's largest at 2^14
                        const float up = __uint_as_float(static_cast<uint32_t>(14 - e2 + 127) << 23);
                        const int own = __shfl_sync(0xffffffffu, e2, (lane % RPI) * LPR);
                        if (lane / RPI == i) down = __uint_as_float(static_cast<uint32_t>(own - 14 + 127) << 23);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = Pair<T>::get(w[e]);
                            w[e] = Pair<__half>::put(f.x * up, f.y * up);
                        }
                    }
                    const int in_tile = (warp & 3) * 32 + i * RPI + lane / LPR;
                    st_shared_v4(sQ + t * C::TILE + (c >> 3) * C::PANEL + in_tile * 128 + (((c & 7) ^ (in_tile & 7)) << 4),
                                 w[0] ^ turn, w[1] ^ turn, w[2] ^ turn, w[3] ^ turn);
                }
                coef = fabsf(p.sl2e) * down;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(B(ctl->q_full[t]));
                for (int i = 0; i < n; ++i) {
                    ok = warp_waits(B(ctl->s_full[t]), s_it & 1u, SITE_KV8_S);
                    if (!ok) break;
                    ++s_it;
                    tc_fence_after();
                    const float2 ref = *const_cast<const float2 *>(&ctl->refs[(tiles + i) % kRefRing]);
                    const float c = fmaxf(coef * ref.x, 1e-30f);
                    const int vis = lim - (at.j + i) * kTileKeys;  // columns >= vis are masked
                    const bool masked = __any_sync(0xffffffffu, vis < kTileKeys);
                    uint32_t s[128];
                    tmem_ld128_wait(tS, s);
                    if (masked) mask_columns(s, vis, false);
                    const float raw = row_extreme<false>(s);
                    float lv, ivs;
                    if (ref.y > 0.f) {
                        lv = log2_scale(ref.y);
                        ivs = rcp_approx(ref.y);
                    } else {
                        // No values but zeros: only the weights matter, and any scale will do: a power of two that keeps
                        // them within fp32 without raising the reference, which would push the P of values that are small
                        // towards fp16's subnormals.
                        lv = rintf(fminf(fmaxf(m - 16.f - raw * c, -64.f), 100.f));
                        ivs = ex2_approx(-lv);
                    }
                    const float mx = fmaf(raw, c, lv);
                    const float m_new = fmaxf(m, mx);
                    const bool need = m_new > m + kSlack;
                    if (__any_sync(0xffffffffu, need)) {
                        const float f = half_step(m, m_new);
                        if (i > 0) rescale_rows<D>(tO, f * f);
                        l = l * f * f;
                        m = m_new;
                    }
                    const float use = (m == -INFINITY ? 0.f : m - kOffset) - lv;
                    const float2 sums = exp_store_tile<__half, false, false>(s, 0, c, use, tS, B(ctl->p_half[t]));
                    l = fmaf(sums.x, ivs, l);
                    warp_announce_tmem(B(ctl->p_full[t]));
                }
                if (!ok) break;
                ok = warp_waits(B(ctl->o_full[t]), o_it & 1u, SITE_KV8_O);
                if (!ok) break;
                ++o_it;
                tc_fence_after();
            }
            tiles += n;
            // the item ends, or goes on in the next CTA
            const bool item_ends = j_end == at.n;
            const int64_t first_unit = u0 + it - at.j;  // of the item
            const bool whole = first_unit >= u0 && item_ends;
            if (tile_has_rows) {
                // columns in which a key that this row sees has a NaN that was taken out of the products
                uint32_t nan_at[D / 32] = {};
                if (n > 0 && *const_cast<volatile uint32_t *>(&ctl->v_nan) != 0u) {
                    const int32_t *table = p.block_table + static_cast<int64_t>(at.b) * p.pages_per_seq;
                    const int first = seen.all / kTileKeys * kTileKeys;
                    const int k1 = min(valid ? lim : 0, j_end * kTileKeys);
                    for (int k = max(first, at.j * kTileKeys); k < k1; ++k) {
                        const int page = table[k / p.page_size];
                        if (page < 0 || page >= p.num_pages) continue;
                        const uint4 *v = reinterpret_cast<const uint4 *>(
                            p.v_pool + ((static_cast<int64_t>(page) * p.page_size + k % p.page_size) * p.h_kv + at.kvh) * D);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            const uint4 a = v[2 * c], b = v[2 * c + 1];
                            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t nb = nan_bytes(w[e]) >> 7;  // a bit for each byte, to one for each column
                                nan_at[c] |= ((nb & 1u) | (nb >> 7 & 2u) | (nb >> 14 & 4u) | (nb >> 21 & 8u)) << (4 * e);
                            }
                        }
                    }
                }
                const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + (first_unit > u0 ? 1 : 0)) * kItemRows;
                const float inv = !whole ? 1.f : (l == 0.f ? 0.f : 1.f / l);
                // 32 columns at a time pass through the warp's rows of the Q tile, whose products are done, so that the
                // stores are of 128 (64) bytes of a row (a row to a lane: 32 lines a store, 4 us an item more)
                const uint32_t pass = sQ + t * C::TILE + (warp & 3) * (32 * 128);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32_wait(tO + c * 32, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    if (nan_at[c] != 0u) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = nan_at[c] >> e & 1u ? 0x7FC00000u : o[e];
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        st_shared_v4(pass + lane * 128 + ((e ^ (lane & 7)) << 4), o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // rows 4 k .., eight lanes to a row
                        const int in_warp = 4 * k + (lane >> 3), rr = warp_row + in_warp, col = c * 32 + (lane & 7) * 4;
                        const float4 v = ld_shared_f4(pass + in_warp * 128 + (((lane & 7) ^ (in_warp & 7)) << 4));
                        if (rr >= p.rows) continue;
                        if (whole)
                            *reinterpret_cast<uint2 *>(static_cast<T *>(p.o) + (row0 + rr) * D + col) =
                                make_uint2(Pair<T>::put(v.x, v.y), Pair<T>::put(v.z, v.w));
                        else
                            *reinterpret_cast<float4 *>(p.o_part + (part0 + rr - at.blk * kItemRows) * D + col) = v;
                    }
                    __syncwarp();
                }
                if (valid) {
                    if (!whole) *reinterpret_cast<float2 *>(p.ml_part + (part0 + r - at.blk * kItemRows) * 2) = make_float2(m, l);
                    else if (p.lse) p.lse[row0 + r] = lse_of(m, l);
                }
                tc_fence_before();
            }
            it += j_end - at.j;
            if (it == n_units && threadIdx.x == 0) {
                // the item that this CTA begins and others go on with, if there is one
                Kv8Cut c = {0, 0, 0, 0};
                if (!item_ends && first_unit >= u0) {
                    c.parts = static_cast<int>(shared_out.owner(first_unit + at.n - 1) - blockIdx.x) + 1;
                    if (first_unit > u0) c.parts = -c.parts;
                    c.b = at.b;
                    c.hg = at.kvh;
                    c.tile = at.blk;
                }
                p.cut[blockIdx.x] = c;
            }
            wide_next(p, at);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, typename T>
cudaError_t launch_wide_t(const Kv8LaunchArgs &a)
{
    auto kern = attn_kv8_wide_kernel<D, T>;
    std::atomic<int> &ready = a.attr_ready[8 + (D == 64 ? 0 : 2) + (Elem<T>::BF16 ? 1 : 0)];
    if (ready.load(std::memory_order_acquire) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, WideCfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    return launch_overlapped(kern, dim3(a.grid), kThreads, WideCfg<D>::SMEM, a.stream, a.k, a.v, a.p);
}

}  // namespace

cudaError_t launch_kv8_wide(const Kv8LaunchArgs &a, int d, bool bf16)
{
    cudaError_t e;
    if (d == 64) e = bf16 ? launch_wide_t<64, __nv_bfloat16>(a) : launch_wide_t<64, __half>(a);
    else e = bf16 ? launch_wide_t<128, __nv_bfloat16>(a) : launch_wide_t<128, __half>(a);
    return e == cudaSuccess ? launch_kv8_join(a, d, bf16) : e;
}

}  // namespace attn
