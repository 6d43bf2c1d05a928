// New keys, rotated by their positions on the way, and new values into a
// paged cache: row t of batch element e goes to logical position
// L + t, L = clamp(seqlens[e], 0, capacity), for t < new_seqlens[e]; rows at
// or past the capacity, and rows of pages outside the pool, are not written.
//
// 16-bit pool: the rotated row, rounded once.
//
// e4m3 pool: one scale for each block of tokens and head.  A block's scale
// is the smallest power of two 2^n >= kMinScale with max|x| / 2^n <= 448
// (e4m3's largest value) over the finite values of the block's rows, so a
// stored value is x / 2^n (exact) rounded once to e4m3.  Rows that are in
// the block already keep their scale s when the new ones fit it; otherwise
// they are stored again at the new one: their value times s / 2^n, exact but
// for what falls below e4m3's smallest normal.  A power of two costs an e4m3
// value no precision, since its rounding is relative.
//
// Measured, of 6.80 TB/s (a copy): 16-bit pool 6.2 TB/s at 8 x 1000 tokens of
// 32 heads, d64 (21.4 us); e4m3 pool 3.3 TB/s at 4 x 4001 tokens of 8 heads,
// d128, blocks of 16 (13.0 us: 42 MB are six microseconds of memory, and the
// angles, the rotation done twice and the conversions take half of the issue
// slots meanwhile).
#include "kv_append.h"

#include <type_traits>

#include "rows.cuh"
#include "stream_order.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kMinScaleExp = -64;

// Cached tokens of element e, and how many of its new ones are there and fit.
struct NewRows {
    int start, end;  // logical positions [start, end)
};

__device__ __forceinline__ NewRows new_rows(const KvAppendParams &p, int e)
{
    const int cap = static_cast<int>(p.pages_per_seq) * p.page_size;
    const int count = p.new_seqlens ? min(max(p.new_seqlens[e], 0), static_cast<int>(p.s)) : static_cast<int>(p.s);
    const int start = min(max(p.seqlens[e], 0), cap);
    return {start, static_cast<int>(min(static_cast<int64_t>(start) + count, static_cast<int64_t>(cap)))};
}

// Pool row (token) of logical position `pos` of element e, or -1.
__device__ __forceinline__ int pool_token(const KvAppendParams &p, int e, int pos)
{
    const int pg = pos / p.page_size;
    const int page = p.block_table[static_cast<int64_t>(e) * p.pages_per_seq + pg];
    if (page < 0 || page >= p.num_pages) return -1;
    return page * p.page_size + (pos - pg * p.page_size);
}

// 16-bit pool.  A unit is one new token and RPW * ROWS of its 2 * heads rows
// (the keys' first), one warp.
template <int D, typename T, bool ADJACENT>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = 4;
    await_previous();
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t groups = (p.heads + RPW * ROWS - 1) / (RPW * ROWS);
    const uint32_t tok = unit / (2 * groups), gi = unit - tok * 2 * groups;
    if (tok >= p.b * p.s) return;
    const int kv = gi >= groups ? 1 : 0;
    const int h0 = static_cast<int>(gi - kv * groups) * RPW * ROWS;
    const int e = static_cast<int>(tok / static_cast<uint32_t>(p.s)), t = static_cast<int>(tok - e * static_cast<uint32_t>(p.s));
    if (!ATTN_OPS_IN_BOUNDS(e < p.b && t < p.s && h0 < p.heads, p, SITE_OPS_UNIT)) return;
    const RowLane rl = row_lane<ADJACENT>(l, kv == 0 ? p.rot : 0);
    const T *x = static_cast<const T *>(p.x[kv]) + e * p.xb[kv] + t * p.xs[kv];
    uint2 raw[ROWS][2];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int h = h0 + i * RPW + sub;
        raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
        if (h < p.heads) load_row<ADJACENT>(x + h * p.xh[kv], rl, raw[i]);
    }
    const NewRows nr = new_rows(p, e);
    const int pos = nr.start + t;
    if (pos >= nr.end) return;
    const int token = pool_token(p, e, pos);
    if (token < 0 || !ATTN_OPS_IN_BOUNDS(token < p.num_pages * p.page_size, p, SITE_OPS_PAGE)) return;
    T *dst = static_cast<T *>(p.pool[kv]) + static_cast<int64_t>(token) * p.heads * D;
    float c[4], s[4];
    load_angles(p.cos, p.sin, static_cast<int64_t>(pos) * (p.rot / 2), rl, c, s);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int h = h0 + i * RPW + sub;
        if (rl.on) {  // a row that is not rotated is a copy, bit for bit
            float2 v[4];
            unpack_pairs<T>(raw[i], v);
            rotate<ADJACENT>(v, c, s);
            pack_pairs<T>(v, raw[i]);
        }
        if (h < p.heads) store_row<ADJACENT>(dst + h * D, rl, raw[i]);
    }
}

// Largest |x| of eight values (of the FINITE ones; else of those that are no
// NaN), and m.
template <bool FINITE>
__device__ __forceinline__ float amax8(const float2 (&v)[4], float m)
{
    auto size = [](float x) { return !FINITE || fabsf(x) < INFINITY ? fabsf(x) : 0.f; };
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max3f(m, size(v[i].x), size(v[i].y));
    return m;
}

// Exponent of the smallest power of two >= 2^kMinScaleExp that brings a to at
// most 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(uint32_t a)
{
    const int e = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(e, kMinScaleExp);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ uint32_t to_e4m3(float2 a, float2 b, float f)
{
    a = __fmul2_rn(a, make_float2(f, f)), b = __fmul2_rn(b, make_float2(f, f));
    return pack_e4m3x2(a.x, a.y) | (pack_e4m3x2(b.x, b.y) << 16);
}

// e4m3 pool.  A unit is one block of one head of the keys or of the values,
// WPU warps of 16 rows.  A warp loads all of its new rows before it looks at
// them, finds the largest value, and once the unit's warps have agreed on the
// scale rotates the rows again (from registers, with angles that the first
// time left in L1) and stores them: holding the rotated fp32 values instead
// would take twice the registers.  Consecutive units are consecutive heads,
// so a block's stores are contiguous in the pool.
// (Four blocks on an SM, which takes nine registers of a thread: an append of
// one token to 64 caches 4.3 us and not 4.8.)
template <int D, typename T, bool ADJACENT, int WPU>
__global__ void __launch_bounds__(kThreads, 4) kv_append_e4m3_kernel(const __grid_constant__ KvAppendParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ITER = 16 / RPW, BLOCK = 16 * WPU, UPC = kThreads / 32 / WPU;
    __shared__ uint32_t warp_max[kThreads / 32];
    await_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
    const int kv = blockIdx.y;
    uint32_t u = blockIdx.x * UPC + warp / WPU;
    const uint32_t eh = u / p.nblk_heads;
    const int e = static_cast<int>(eh);
    u -= eh * p.nblk_heads;
    const int j = static_cast<int>(u / static_cast<uint32_t>(p.heads)), h = static_cast<int>(u - j * static_cast<uint32_t>(p.heads));
    // new rows [lo, hi) of the warp's 16, rows [0, old) of them cached before
    int start = 0, first = 0, lo = 0, hi = 0, old = 0;
    bool fresh = true;  // the block holds nothing from before
    if (e < p.b) {
        const NewRows nr = new_rows(p, e);
        start = nr.start;
        first = (nr.start / BLOCK + j) * BLOCK;
        if (first < nr.end && nr.start < nr.end) {
            const int base = first + (warp % WPU) * 16;
            lo = min(max(nr.start - base, 0), 16);
            hi = max(min(nr.end - base, 16), lo);
            old = lo;
            fresh = nr.start <= first;
        }
    }
    const bool any = hi > lo || old > 0;
    const RowLane rl = row_lane<ADJACENT>(l, kv == 0 ? p.rot : 0);
    const int row0 = (warp % WPU) * 16 + sub;  // of the block; the lane's rows are RPW apart
    int token = any ? pool_token(p, e, first) : -1;
    if (!ATTN_OPS_IN_BOUNDS(token + BLOCK <= p.num_pages * p.page_size, p, SITE_OPS_PAGE)) token = -1;
    uint2 raw[ITER][2];
    if (hi > lo) {
        const T *x = static_cast<const T *>(p.x[kv]) + e * p.xb[kv] + h * p.xh[kv] +
                     static_cast<int64_t>(first + row0 - start) * p.xs[kv];
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int r = i * RPW + sub;
            raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
            if (r >= lo && r < hi && ATTN_OPS_IN_BOUNDS(first + row0 + i * RPW - start < p.s && h < p.heads, p, SITE_OPS_ROW))
                load_row<ADJACENT>(x + i * RPW * p.xs[kv], rl, raw[i]);
        }
    }
    float *scale_at = nullptr;
    float was = 0.f;
    if (token >= 0) {
        const int page = token / p.page_size;
        scale_at = p.scale[kv] + (static_cast<int64_t>(page) * p.heads + h) * (p.page_size / BLOCK) + (token - page * p.page_size) / BLOCK;
        if (!ATTN_OPS_IN_BOUNDS(scale_at - p.scale[kv] < p.num_pages * p.heads * (p.page_size / BLOCK), p, SITE_OPS_SCALE)) token = -1;
        else if (!fresh) was = *scale_at;
    }
    auto value = [&](int i, float2 (&v)[4]) {
        unpack_pairs<T>(raw[i], v);
        if (rl.on) {
            float c[4], s[4];
            const int r = i * RPW + sub;
            load_angles(p.cos, p.sin, static_cast<int64_t>(first + (r >= lo && r < hi ? i * RPW + row0 : 0)) * (p.rot / 2), rl, c, s);
            rotate<ADJACENT>(v, c, s);
        }
    };
    auto largest = [&](auto finite) {
        float top = 0.f;
        if (hi > lo) {
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                if (i * RPW + RPW <= lo || i * RPW >= hi) continue;
                float2 v[4];
                value(i, v);
                top = amax8<decltype(finite)::value>(v, top);
            }
        }
        // the bits of non-negative floats compare like integers
        return __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    };
    uint32_t m = largest(std::false_type());
    if (m >= 0x7F800000u) m = largest(std::true_type());  // an infinity among them: look again, past it
    if constexpr (WPU > 1) {
        if (lane == 0) warp_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPU; ++i) m = max(m, warp_max[warp / WPU * WPU + i]);
    }
    if (token < 0) return;
    const int ex = scale_exponent(m);
    const float need = pow2(ex);
    const bool grows = need > was;  // false too for a stored NaN: its rows are left
    const bool keep = !fresh && !grows;
    const float inv = keep ? 1.f / was : pow2(-ex);
    // (every warp of the unit has read the scale: the barrier above; and every lane of this one)
    __syncwarp();
    if (warp % WPU == 0 && lane == 0) *scale_at = keep ? was : need;
    uint8_t *dst = static_cast<uint8_t *>(p.pool[kv]) + (static_cast<int64_t>(token + row0) * p.heads + h) * D;
    const int64_t step = static_cast<int64_t>(RPW) * p.heads * D;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        if (i * RPW + RPW <= lo || i * RPW >= hi) continue;
        const int r = i * RPW + sub;
        float2 v[4];
        value(i, v);
        if (r >= lo && r < hi) {
            const uint32_t a = to_e4m3(v[0], v[1], inv), b = to_e4m3(v[2], v[3], inv);
            if constexpr (ADJACENT) {
                *reinterpret_cast<uint2 *>(dst + i * step + rl.lo) = make_uint2(a, b);
            } else {
                *reinterpret_cast<uint32_t *>(dst + i * step + rl.lo) = a;
                *reinterpret_cast<uint32_t *>(dst + i * step + rl.hi) = b;
            }
        }
    }
    if (!fresh && grows) {  // the rows from before, at the new scale
        const float f = was * inv;
        for (int i = 0; i * RPW < old; ++i) {
            if (i * RPW + sub >= old) break;
            uint2 *at = reinterpret_cast<uint2 *>(dst + i * step + 8 * l);
            const uint2 w = *at;
            auto scaled = [&](uint32_t x) {
                return to_e4m3(Pair<__half>::get(e4m3x2_to_f16x2(x)), Pair<__half>::get(e4m3x2_to_f16x2(x >> 16)), f);
            };
            *at = make_uint2(scaled(w.x), scaled(w.y));
        }
    }
}

template <int D, typename T, bool ADJACENT>
cudaError_t launch_e4m3(const KvAppendParams &p, cudaStream_t stream)
{
    const int wpu = 1 << (p.block_shift - 4), upc = kThreads / 32 / wpu;
    const int64_t units = p.b * static_cast<int64_t>(p.nblk_heads);
    const dim3 grid(static_cast<unsigned>((units + upc - 1) / upc), 2);
    auto kernel = kv_append_e4m3_kernel<D, T, ADJACENT, 8>;
    switch (wpu) {
    case 1: kernel = kv_append_e4m3_kernel<D, T, ADJACENT, 1>; break;
    case 2: kernel = kv_append_e4m3_kernel<D, T, ADJACENT, 2>; break;
    case 4: kernel = kv_append_e4m3_kernel<D, T, ADJACENT, 4>; break;
    }
    return launch_overlapped(kernel, grid, kThreads, 0, stream, p);
}

template <int D, typename T, bool ADJACENT>
cudaError_t launch_16bit(const KvAppendParams &p, cudaStream_t stream)
{
    constexpr int HPU = 4 * (32 / (D / 8));
    const int64_t units = p.b * p.s * 2 * ((p.heads + HPU - 1) / HPU);
    const unsigned blocks = static_cast<unsigned>((units + kThreads / 32 - 1) / (kThreads / 32));
    return launch_overlapped(kv_append_kernel<D, T, ADJACENT>, dim3(blocks), kThreads, 0, stream, p);
}

template <int D, typename T>
cudaError_t launch_t(const KvAppendParams &p, bool e4m3, cudaStream_t stream)
{
    if (e4m3) return p.interleaved ? launch_e4m3<D, T, true>(p, stream) : launch_e4m3<D, T, false>(p, stream);
    return p.interleaved ? launch_16bit<D, T, true>(p, stream) : launch_16bit<D, T, false>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams &p, int d, bool bf16, bool e4m3, cudaStream_t stream)
{
    if (d == 64) return bf16 ? launch_t<64, __nv_bfloat16>(p, e4m3, stream) : launch_t<64, __half>(p, e4m3, stream);
    return bf16 ? launch_t<128, __nv_bfloat16>(p, e4m3, stream) : launch_t<128, __half>(p, e4m3, stream);
}

}  // namespace attn
