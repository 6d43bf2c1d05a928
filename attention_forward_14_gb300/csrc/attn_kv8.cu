// Attention of new queries over an e4m3 paged cache:
//   O = softmax(scale Q K^T [+ causal mask]) V,  K = ks k8,  V = vs v8,
// with one scale ks, vs for each block of tokens (16, 32, 64 or 128) and key
// head.  A key head serves `group` query heads, so its keys meet
// rows = group * sq query rows.
//
// Work.  An item is 16 query rows of one key head of one batch element; a
// unit is 128 of its keys.  The units of all items, in order, are dealt to
// the CTAs in equal contiguous shares, from the lengths that the device
// holds: ragged batches need no split count and leave no CTA behind.  An
// item that several CTAs share is written as partial results, which a second
// kernel joins.
//
// A CTA.  Eight warps; each takes 16 keys of every unit, whose K and V rows
// an elected lane copies into the warp's own ring of shared-memory stages
// (TMA, swizzled), several units ahead and across items.  Warps share
// nothing until an item's end.  Per 16 keys a warp computes S = Q K^T
// (16 x 16) and O += P V with fp16 matrix instructions on e4m3 values
// converted to fp16 (exact) in registers.  The order of the head's values in
// a dot product is free, so a lane takes 32 contiguous ones (d = 128) of its
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

constexpr int kWarps = 8;
constexpr int kGroupKeys = 16;                    // keys of a warp's step
constexpr int kUnitKeys = kWarps * kGroupKeys;    // 128
constexpr int kStages = 5;
constexpr float kOffset = 10.f, kSlack = 4.f;
constexpr uint32_t SITE_KV8_LOAD = 40;

template <int D>
struct Kv8Cfg {
    static constexpr int KBYTES = kGroupKeys * D;          // K (or V) rows of a stage
    static constexpr int STAGE = 2 * KBYTES;
    static constexpr int RING = kStages * STAGE;           // per warp
    static constexpr int O_OFF = kWarps * RING;            // merge buffer [warps][16][D]
    static constexpr int ML_OFF = O_OFF + kWarps * 16 * D * 4;  // [warps][16] float2
    static constexpr int SC_OFF = ML_OFF + kWarps * 16 * 8;     // [warps][kStages] float2 scales
    static constexpr int BAR_OFF = SC_OFF + kWarps * kStages * 8;
    static constexpr int CTL_OFF = BAR_OFF + kWarps * kStages * 8;
    static constexpr int SMEM = CTL_OFF + 16 + 1024;       // +1 KiB for alignment
    static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float lg2_approx(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int cached_len(const Kv8Params &p, int b) { return min(max(p.seqlens[b], 0), p.cap); }

// The top bit of every byte that is an e4m3 NaN (0x7F, 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Units of one item of a batch element with n keys: an item that sees no
// key still has one, which writes its rows.
__device__ __forceinline__ int units_of(int n) { return max((n + kUnitKeys - 1) / kUnitKeys, 1); }

// Where in the work a unit lies.
struct Place {
    int b, kvh, tile;
    int j, n;    // unit of the item, units of the item
    int len;     // cached keys of the batch element
};

__device__ __forceinline__ int64_t total_units(const Kv8Params &p)
{
    const int lane = threadIdx.x & 31;
    int64_t t = 0;
    for (int i = lane; i < p.b; i += 32) t += units_of(cached_len(p, i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t * p.h_kv * p.tiles;
}

// The place of unit u (< total), by every lane of a warp.
__device__ __forceinline__ Place place_of(const Kv8Params &p, int64_t u)
{
    const int lane = threadIdx.x & 31;
    const int64_t per = static_cast<int64_t>(p.h_kv) * p.tiles;
    Place c;
    for (int b0 = 0;; b0 += 32) {
        const int len = b0 + lane < p.b ? cached_len(p, b0 + lane) : 0;
        int64_t inc = b0 + lane < p.b ? units_of(len) * per : 0;
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
    c.n = units_of(c.len);
    const int64_t item = u / c.n;
    c.j = static_cast<int>(u - item * c.n);
    c.kvh = static_cast<int>(item / p.tiles);
    c.tile = static_cast<int>(item - static_cast<int64_t>(c.kvh) * p.tiles);
    return c;
}

__device__ __forceinline__ void next_unit(const Kv8Params &p, Place &c)
{
    if (++c.j < c.n) return;
    c.j = 0;
    if (++c.tile < p.tiles) return;
    c.tile = 0;
    if (++c.kvh < p.h_kv) return;
    c.kvh = 0;
    if (++c.b >= p.b) return;
    c.len = cached_len(p, c.b);
    c.n = units_of(c.len);
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

// Element offset of row r of the key head's rows in q and o.
__device__ __forceinline__ int64_t row_at(const Kv8Params &p, const Place &c, int r)
{
    return (static_cast<int64_t>(c.b) * p.h_kv + c.kvh) * p.rows + r;
}

// The rows of an item's partial results.
template <int D>
__device__ __forceinline__ float *o_slot(const Kv8Params &p, int64_t slot) { return p.o_part + slot * (kKv8Tile * D); }

template <int D, typename T>
__device__ __forceinline__ void store4(T *o, float4 v)
{
    *reinterpret_cast<uint2 *>(o) = make_uint2(Pair<T>::put(v.x, v.y), Pair<T>::put(v.z, v.w));
}

template <int D, typename T>
__global__ void __launch_bounds__(kWarps * 32, 1)
    attn_kv8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ Kv8Params p)
{
    using C = Kv8Cfg<D>;
    constexpr int KS = D / 16;      // k-steps of S, and words of a lane's share of a K row
    constexpr int VW = D / 32;      // words of a lane's share of a V row
    constexpr int NO = D / 8;       // column tiles of O
    constexpr bool BF16 = Elem<T>::BF16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + C::CTL_OFF);
    const uint32_t ring = base + warp * C::RING;
    const uint32_t bars = base + C::BAR_OFF + warp * kStages * 8;
    const uint32_t scs = base + C::SC_OFF + warp * kStages * 8;
    const float2 *sc_ptr = reinterpret_cast<const float2 *>(smem + C::SC_OFF + warp * kStages * 8);

    if (threadIdx.x == 0) {
        *abort_flag = 0u;
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(bars + s * 8, 1);
        fence_barrier_init();
    }
    __syncthreads();

    const int64_t total = total_units(p);
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
    if (blockIdx.x >= ctas) return;
    const int64_t u0 = blockIdx.x * total / ctas, u1 = (blockIdx.x + 1) * total / ctas;
    const int n_units = static_cast<int>(u1 - u0);
    Place cur = place_of(p, u0), ahead = cur;
    uint32_t issued = 0u, used = 0u;  // stages filled and taken by this warp

    // copy this warp's keys of the unit at `ahead` (nothing when no row sees them)
    auto issue = [&](int it) {
        const int k0 = ahead.j * kUnitKeys + warp * kGroupKeys;
        if (k0 < seen_keys(p, ahead).end) {
            const uint32_t st = issued % kStages;
            if (lane == 0) {
                const int pg = k0 / p.page_size, off = k0 - pg * p.page_size;
                const int page = p.block_table[static_cast<int64_t>(ahead.b) * p.pages_per_seq + pg];
                const bool in = page >= 0 && page < p.num_pages;
                // a page outside the pool is read at the token past its end: the copy fills zeros
                const int tok = in ? page * p.page_size + off : p.num_pages * p.page_size;
                const int64_t sc = (static_cast<int64_t>(in ? page : 0) * p.h_kv + ahead.kvh) * (p.page_size >> p.block_shift) +
                                   (off >> p.block_shift);
                if (in) {
                    cp_async4(scs + st * 8, p.k_scale + sc);
                    cp_async4(scs + st * 8 + 4, p.v_scale + sc);
                } else {
                    asm volatile("st.shared.v2.f32 [%0], {%1, %1};" ::"r"(scs + st * 8), "f"(1.f) : "memory");
                }
                mbar_arrive_expect_tx(bars + st * 8, C::STAGE);
                const uint64_t pol = l2_evict_normal();
                tma_load_3d(ring + st * C::STAGE, &tmK, bars + st * 8, 0, ahead.kvh, tok, pol);
                tma_load_3d(ring + st * C::STAGE + C::KBYTES, &tmV, bars + st * 8, 0, ahead.kvh, tok, pol);
            }
            ++issued;
        }
        cp_async_commit();
        if (it + 1 < n_units) next_unit(p, ahead);
    };
    int it_ahead = 0;
    for (; it_ahead < kStages && it_ahead < n_units; ++it_ahead) issue(it_ahead);
    for (int i = it_ahead; i < kStages; ++i) cp_async_commit();

    bool ok = true;
    auto wait_full = [&](uint32_t bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = global_timer_ns();
        while (true) {
            for (int i = 0; i < 64; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > p.timeout_ns) {
                *abort_flag = 1u;
                record_status(p.status, STATUS_TIMEOUT, SITE_KV8_LOAD);
                return false;
            }
        }
    };

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
                                                                   row_at(p, cur, rr < p.rows ? rr : 0) * D + t * (D / 4));
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
        const int k0 = cur.j * kUnitKeys + warp * kGroupKeys;
        cp_async_wait<kStages - 1>();  // the scales of this unit
        const uint32_t st = used % kStages;
        if (ok && k0 < seen.end) ok = __all_sync(0xffffffffu, wait_full(bars + st * 8, (used / kStages) & 1u));
        __syncwarp();
        if (ok && k0 < seen.end) {
            ++used;
            const uint32_t ks_at = ring + st * C::STAGE, vs_at = ks_at + C::KBYTES;
            const float2 sc = sc_ptr[st];
            float vs = sc.y;
            const bool vzero = vs < 1.1754944e-38f;  // a block of zeros
            if (vzero) vs = 1.f;
            const float lv = lg2_approx(vs), ivs = __frcp_rn(vs);
            // S: two tiles of eight keys
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
                const int row = n * 8 + g;
                uint32_t w[KS];
                if constexpr (D == 128) {
                    const uint4 a = lds128(ks_at + row * 128 + (((2 * t) ^ g) << 4));
                    const uint4 b = lds128(ks_at + row * 128 + (((2 * t + 1) ^ g) << 4));
                    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
                } else {
                    const uint4 a = lds128(ks_at + row * 64 + ((t ^ ((row >> 1) & 3)) << 4));
                    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
                }
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    mma16816(s[n], qa[k][0], qa[k][1], qa[k][2], qa[k][3], e4m3x2_to_f16x2(w[k]), e4m3x2_to_f16x2(w[k] >> 16));
            }
            const float a0 = c0 * sc.x, a1 = c1 * sc.x;
            float x[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                x[n][0] = fmaf(s[n][0], a0, lv);
                x[n][1] = fmaf(s[n][1], a0, lv);
                x[n][2] = fmaf(s[n][2], a1, lv);
                x[n][3] = fmaf(s[n][3], a1, lv);
            }
            const bool partly = k0 + kGroupKeys > seen.all;  // some row does not see some of these keys
            if (partly) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int k = k0 + n * 8 + 2 * t;
                    x[n][0] = k < lim0 ? x[n][0] : -INFINITY;
                    x[n][1] = k + 1 < lim0 ? x[n][1] : -INFINITY;
                    x[n][2] = k < lim1 ? x[n][2] : -INFINITY;
                    x[n][3] = k + 1 < lim1 ? x[n][3] : -INFINITY;
                }
            }
            const float t0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
            const float t1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
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
            float sum0 = 0.f, sum1 = 0.f;
            uint32_t pa[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float p0 = ex2_approx(x[n][0] - b0), p1 = ex2_approx(x[n][1] - b0);
                const float p2 = ex2_approx(x[n][2] - b1), p3 = ex2_approx(x[n][3] - b1);
                sum0 += p0 + p1;
                sum1 += p2 + p3;
                pa[2 * n] = vzero ? 0u : Pair<__half>::put(p0, p1);
                pa[2 * n + 1] = vzero ? 0u : Pair<__half>::put(p2, p3);
            }
            l0 = fmaf(sum0, ivs, l0);
            l1 = fmaf(sum1, ivs, l1);
            // O += P V
            const int tail = cur.len - k0;  // rows of V from `tail` on are not keys: zero them
            uint32_t v[4][VW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 2 * t + (i & 1) + 8 * (i >> 1);
                if constexpr (D == 128) {
                    const uint4 a = lds128(vs_at + row * 128 + ((g ^ (row & 7)) << 4));
                    v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
                } else {
                    const uint2 a = lds64(vs_at + row * 64 + ((((g >> 1) ^ ((row >> 1) & 3)) << 4) | ((g & 1) << 3)));
                    v[i][0] = a.x, v[i][1] = a.y;
                }
                if (tail < kGroupKeys) {
#pragma unroll
                    for (int w = 0; w < VW; ++w) v[i][w] = row < tail ? v[i][w] : 0u;
                }
            }
            if (partly) {
                // A NaN among V must reach the rows that see its key and no
                // other, but a row that does not still multiplies it, by 0:
                // take it out of the product and put it into the rows that
                // see it (the product of what each row sees with where V is
                // NaN counts them).
                uint32_t any = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < VW; ++w) any |= nan_bytes(v[i][w]);
                if (__any_sync(0xffffffffu, any != 0u)) {
                    uint32_t see[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int k = k0 + n * 8 + 2 * t;
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
                            for (int k = 0; k < 4; ++k) acc[4 * w + e][k] = c[k] > 0.f ? __int_as_float(0x7FC00000) : acc[4 * w + e][k];
                        }
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                const uint32_t lo0 = __byte_perm(v[0][w], v[1][w], 0x5140), hi0 = __byte_perm(v[0][w], v[1][w], 0x7362);
                const uint32_t lo1 = __byte_perm(v[2][w], v[3][w], 0x5140), hi1 = __byte_perm(v[2][w], v[3][w], 0x7362);
                mma16816(acc[4 * w], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(lo0), e4m3x2_to_f16x2(lo1));
                mma16816(acc[4 * w + 1], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(lo0 >> 16), e4m3x2_to_f16x2(lo1 >> 16));
                mma16816(acc[4 * w + 2], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(hi0), e4m3x2_to_f16x2(hi1));
                mma16816(acc[4 * w + 3], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(hi0 >> 16), e4m3x2_to_f16x2(hi1 >> 16));
            }
        }
        __syncwarp();  // every lane has read the stage (and its scales) before they are filled again
        if (ok && it_ahead < n_units) issue(it_ahead++);
        else cp_async_commit();

        const bool item_ends = cur.j + 1 == cur.n;
        if (item_ends || it + 1 == n_units) {
            // join the warps' parts of the item
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const int nr = min(kKv8Tile, p.rows - cur.tile * kKv8Tile);
            float2 *ml = reinterpret_cast<float2 *>(smem + C::ML_OFF);
            float *ob = reinterpret_cast<float *>(smem + C::O_OFF);
            if (t == 0) {
                ml[warp * 16 + g] = make_float2(m0, l0);
                ml[warp * 16 + g + 8] = make_float2(m1, l1);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                if (g + 8 * hh >= nr) continue;
                // column of acc[i][0]: 2t * NO + i; of acc[i][1]: NO further on
                float *dst = ob + (warp * 16 + g + 8 * hh) * D + 2 * t * NO;
#pragma unroll
                for (int i = 0; i < NO; i += 4) {
                    *reinterpret_cast<float4 *>(dst + i) = make_float4(acc[i][2 * hh], acc[i + 1][2 * hh], acc[i + 2][2 * hh],
                                                                       acc[i + 3][2 * hh]);
                    *reinterpret_cast<float4 *>(dst + NO + i) = make_float4(acc[i][2 * hh + 1], acc[i + 1][2 * hh + 1],
                                                                            acc[i + 2][2 * hh + 1], acc[i + 3][2 * hh + 1]);
                }
            }
            __syncthreads();
            const int64_t first_unit = u0 + it - cur.j;  // of the item
            const bool whole = first_unit >= u0 && item_ends;
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (first_unit > u0 ? 1 : 0);
            for (int i = threadIdx.x; i < nr * (D / 4); i += kWarps * 32) {
                const int r = i / (D / 4), c4 = i % (D / 4);
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml[w * 16 + r].x);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 a = ml[w * 16 + r];
                    const float f = a.x == -INFINITY ? (a.y == 0.f ? 0.f : 1.f) : ex2_approx(a.x - mx);
                    const float4 v = *reinterpret_cast<const float4 *>(ob + (w * 16 + r) * D + c4 * 4);
                    o.x = fmaf(v.x, f, o.x);
                    o.y = fmaf(v.y, f, o.y);
                    o.z = fmaf(v.z, f, o.z);
                    o.w = fmaf(v.w, f, o.w);
                    l = fmaf(a.y, f, l);
                }
                if (whole) {
                    const int64_t row = row_at(p, cur, cur.tile * kKv8Tile + r);
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    store4<D, T>(static_cast<T *>(p.o) + row * D + c4 * 4,
                                 make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                    if (c4 == 0 && p.lse)
                        p.lse[row] = l == 0.f ? -INFINITY : (mx - kOffset + log2f(l)) * 0.69314718055994531f;
                } else {
                    *reinterpret_cast<float4 *>(o_slot<D>(p, slot) + r * D + c4 * 4) = o;
                    if (c4 == 0) *reinterpret_cast<float2 *>(p.ml_part + (slot * kKv8Tile + r) * 2) = make_float2(mx, l);
                }
            }
            __syncthreads();
        }
        next_unit(p, cur);
    }
    // copies still in flight (only after a wait that gave up) land before the CTA goes
    for (; used < issued; ++used) drain_wait(bars + (used % kStages) * 8, (used / kStages) & 1u, p.timeout_ns);
}

// Joins the parts of an item that several CTAs share.  Block c - 1 looks at
// the boundary between the shares of CTAs c - 1 and c; the first boundary
// inside an item joins all of its parts, in order.
template <int D, typename T>
__global__ void __launch_bounds__(128) attn_kv8_join_kernel(const __grid_constant__ Kv8Params p, int grid)
{
    const int64_t total = total_units(p);
    const int64_t ctas = min(static_cast<int64_t>(grid), total);
    const int64_t c = blockIdx.x + 1;
    if (c >= ctas) return;
    const int64_t u = c * total / ctas;
    const Place at = place_of(p, u);
    const int64_t s = u - at.j, e = s + at.n;       // the item's units
    const int64_t prev = (c - 1) * total / ctas;    // where CTA c - 1 begins
    if (at.j == 0 || prev > s) return;              // no item is cut here, or it was cut before
    const int64_t c_first = c - 1;
    const int nr = min(kKv8Tile, p.rows - at.tile * kKv8Tile);
    for (int i = threadIdx.x; i < nr * (D / 4); i += blockDim.x) {
        const int r = i / (D / 4), c4 = i % (D / 4);
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int64_t k = c_first; k < ctas && (k == c_first || k * total / ctas < e); ++k) {
            const int64_t slot = 2 * k + (k == c_first && prev < s ? 1 : 0);
            const float2 a = *reinterpret_cast<const float2 *>(p.ml_part + (slot * kKv8Tile + r) * 2);
            const float4 v = *reinterpret_cast<const float4 *>(o_slot<D>(p, slot) + r * D + c4 * 4);
            const float n = fmaxf(m, a.x);
            const float f0 = m == n ? 1.f : ex2_approx(m - n), f1 = a.x == n ? 1.f : ex2_approx(a.x - n);
            o.x = o.x * f0 + v.x * f1;
            o.y = o.y * f0 + v.y * f1;
            o.z = o.z * f0 + v.z * f1;
            o.w = o.w * f0 + v.w * f1;
            l = l * f0 + a.y * f1;
            m = n;
        }
        const int64_t row = row_at(p, at, at.tile * kKv8Tile + r);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        store4<D, T>(static_cast<T *>(p.o) + row * D + c4 * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (c4 == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m - kOffset + log2f(l)) * 0.69314718055994531f;
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
    kern<<<a.grid, kWarps * 32, Kv8Cfg<D>::SMEM, a.stream>>>(a.k, a.v, a.p);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.grid < 2) return e;
    attn_kv8_join_kernel<D, T><<<a.grid - 1, 128, 0, a.stream>>>(a.p, a.grid);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8(const Kv8LaunchArgs &a, int d, bool bf16)
{
    if (d == 64) return bf16 ? launch_kv8_t<64, __nv_bfloat16>(a) : launch_kv8_t<64, __half>(a);
    return bf16 ? launch_kv8_t<128, __nv_bfloat16>(a) : launch_kv8_t<128, __half>(a);
}

}  // namespace attn
