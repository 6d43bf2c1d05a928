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
#include "kv_append.h"

#include "attn_fwd_kernel.cuh"
#include "rows.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kMinScaleExp = -64;

__device__ __forceinline__ int64_t start_of(const KvAppendParams &p, int64_t e, int64_t cap)
{
    return min(max(static_cast<int64_t>(p.seqlens[e]), int64_t(0)), cap);
}

__device__ __forceinline__ int64_t count_of(const KvAppendParams &p, int64_t e)
{
    return p.new_seqlens ? min(max(static_cast<int64_t>(p.new_seqlens[e]), int64_t(0)), p.s) : p.s;
}

// Pool row (token) of logical position `pos` of element e, or -1.
__device__ __forceinline__ int64_t pool_token(const KvAppendParams &p, int64_t e, int64_t pos)
{
    const int64_t page = p.block_table[e * p.pages_per_seq + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) return -1;
    return page * p.page_size + pos % p.page_size;
}

// 16-bit pool.  A unit is one new token and RPW * 4 of its 2 * heads rows
// (the keys' first), one warp.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = 4;
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const int64_t unit = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    const int groups = (p.heads + RPW * ROWS - 1) / (RPW * ROWS);
    const int64_t tok = unit / (2 * groups);
    if (tok >= p.b * p.s) return;
    const int gi = static_cast<int>(unit - tok * 2 * groups);
    const int kv = gi >= groups ? 1 : 0;
    const int h0 = (gi - kv * groups) * RPW * ROWS;
    const int64_t e = tok / p.s, t = tok - e * p.s;
    const T *x = static_cast<const T *>(p.x[kv]) + e * p.xb[kv] + t * p.xs[kv] + l * 8;
    uint4 raw[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int h = h0 + i * RPW + sub;
        raw[i] = h < p.heads ? __ldcs(reinterpret_cast<const uint4 *>(x + h * p.xh[kv])) : make_uint4(0u, 0u, 0u, 0u);
    }
    const int64_t cap = p.pages_per_seq * p.page_size;
    const int64_t pos = start_of(p, e, cap) + t;
    if (t >= count_of(p, e) || pos >= cap) return;
    const int64_t token = pool_token(p, e, pos);
    if (token < 0) return;
    T *dst = static_cast<T *>(p.pool[kv]) + token * p.heads * D + l * 8;
    const bool il = p.interleaved != 0;
    const RotLane rl = rot_lane(lane, l, p.cos && kv == 0 ? p.rot : 0, il);
    float c[8], s[8];
    load_angles(p.cos, p.sin, pos * (p.rot / 2), rl, il, c, s);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int h = h0 + i * RPW + sub;
        float v[8], o[8];
        unpack8<T>(raw[i], v);
        unpack8<T>(shfl4(raw[i], rl.partner), o);
        rotate8<false>(v, o, c, s, rl, il);
        // a row that is not rotated is a copy, bit for bit
        if (h < p.heads) *reinterpret_cast<uint4 *>(dst + h * D) = rl.on ? pack8<T>(v) : raw[i];
    }
}

// Largest |x| of the finite ones of eight values, as the bits of a
// non-negative float (which compare like integers).
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[8], uint32_t m)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        if (a < 0x7F800000u) m = max(m, a);
    }
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

__device__ __forceinline__ uint2 to_e4m3(const float (&v)[8], float f)
{
    const uint32_t a = pack_e4m3x2(v[0] * f, v[1] * f), b = pack_e4m3x2(v[2] * f, v[3] * f);
    const uint32_t c = pack_e4m3x2(v[4] * f, v[5] * f), d = pack_e4m3x2(v[6] * f, v[7] * f);
    return make_uint2(a | (b << 16), c | (d << 16));
}

// e4m3 pool.  A unit is one block of one head of the keys or of the values:
// BLOCK rows of D values, eight to a lane, ITEMS of them to a thread.
template <int D, typename T, int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS) kv_append_e4m3_kernel(const __grid_constant__ KvAppendParams p)
{
    constexpr int LPR = D / 8;
    constexpr int BLOCK = THREADS * ITEMS / LPR;
    __shared__ uint32_t warp_max[THREADS / 32];
    const int lane = threadIdx.x & 31, l = lane % LPR;
    const int kv = blockIdx.y;
    int64_t u = blockIdx.x;
    const int h = static_cast<int>(u % p.heads);
    u /= p.heads;
    const int64_t j = u % p.nblk, e = u / p.nblk;
    const int64_t cap = p.pages_per_seq * p.page_size;
    const int64_t start = start_of(p, e, cap);
    const int64_t end = min(start + count_of(p, e), cap);
    const int64_t first = (start / BLOCK + j) * BLOCK;  // logical position of the block's first row
    if (first >= end || start >= end) return;
    const int64_t token = pool_token(p, e, first);
    if (token < 0) return;

    const int r_new = static_cast<int>(max(start - first, int64_t(0)));        // the block's rows [r_new, r_end) are new
    const int r_end = static_cast<int>(min(end - first, int64_t(BLOCK)));
    const T *x = static_cast<const T *>(p.x[kv]) + e * p.xb[kv] + h * p.xh[kv] + (first - start) * p.xs[kv] + l * 8;
    const bool il = p.interleaved != 0;
    const RotLane rl = rot_lane(lane, l, p.cos && kv == 0 ? p.rot : 0, il);
    uint4 raw[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int row = (i * THREADS + threadIdx.x) / LPR;
        raw[i] = row >= r_new && row < r_end ? __ldcs(reinterpret_cast<const uint4 *>(x + row * p.xs[kv]))
                                             : make_uint4(0u, 0u, 0u, 0u);
    }
    float *scale_at = p.scale[kv] + (token / p.page_size * p.heads + h) * static_cast<int64_t>(p.page_size / BLOCK) +
                      token % p.page_size / BLOCK;
    const float was = r_new > 0 ? *scale_at : 0.f;
    auto value = [&](int i, float (&v)[8]) {
        const int row = (i * THREADS + threadIdx.x) / LPR;
        float o[8], c[8], s[8];
        unpack8<T>(raw[i], v);
        unpack8<T>(shfl4(raw[i], rl.partner), o);
        if (row >= r_new && row < r_end) {
            load_angles(p.cos, p.sin, (first + row) * (p.rot / 2), rl, il, c, s);
            rotate8<false>(v, o, c, s, rl, il);
        }
    };
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        float v[8];
        value(i, v);
        m = amax_bits(v, m);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) m = max(m, warp_max[i]);
    const int ex = scale_exponent(m);
    const float need = pow2(ex);
    const bool grows = need > was;  // false too for a stored NaN: its rows are left
    const bool keep = r_new > 0 && !grows;
    const float now = keep ? was : need;
    const float inv = keep ? 1.f / was : pow2(-ex);
    if (threadIdx.x == 0) *scale_at = now;
    uint8_t *dst = static_cast<uint8_t *>(p.pool[kv]) + (token * p.heads + h) * D + l * 8;
    const int64_t row_bytes = static_cast<int64_t>(p.heads) * D;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int row = (i * THREADS + threadIdx.x) / LPR;
        float v[8];
        value(i, v);
        if (row >= r_new && row < r_end)
            *reinterpret_cast<uint2 *>(dst + row * row_bytes) = to_e4m3(v, inv);
        else if (row < r_new && grows) {
            const uint2 old = *reinterpret_cast<const uint2 *>(dst + row * row_bytes);
            const uint32_t w[2] = {old.x, old.y};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t hh = e4m3x2_to_f16x2(w[q >> 1] >> (16 * (q & 1)));
                const float2 f = Pair<__half>::get(hh);
                v[2 * q] = f.x;
                v[2 * q + 1] = f.y;
            }
            *reinterpret_cast<uint2 *>(dst + row * row_bytes) = to_e4m3(v, was * inv);
        }
    }
}

template <int D, typename T>
cudaError_t launch_e4m3(const KvAppendParams &p, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(p.b * p.nblk * p.heads), 2);
    constexpr int L = D / 8;  // lanes per row; a block of 16 rows is 16 * L threads
    switch (p.block_shift) {
    case 4: kv_append_e4m3_kernel<D, T, 16 * L, 1><<<grid, 16 * L, 0, stream>>>(p); break;
    case 5: kv_append_e4m3_kernel<D, T, 256, 32 * L / 256><<<grid, 256, 0, stream>>>(p); break;
    case 6: kv_append_e4m3_kernel<D, T, 256, 64 * L / 256><<<grid, 256, 0, stream>>>(p); break;
    default: kv_append_e4m3_kernel<D, T, 256, 128 * L / 256><<<grid, 256, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

template <int D, typename T>
cudaError_t launch_16bit(const KvAppendParams &p, cudaStream_t stream)
{
    constexpr int HPU = 4 * (32 / (D / 8));
    const int64_t units = p.b * p.s * 2 * ((p.heads + HPU - 1) / HPU);
    const unsigned blocks = static_cast<unsigned>((units + kThreads / 32 - 1) / (kThreads / 32));
    kv_append_kernel<D, T><<<blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams &p, int d, bool bf16, bool e4m3, cudaStream_t stream)
{
    if (e4m3) {
        if (d == 64) return bf16 ? launch_e4m3<64, __nv_bfloat16>(p, stream) : launch_e4m3<64, __half>(p, stream);
        return bf16 ? launch_e4m3<128, __nv_bfloat16>(p, stream) : launch_e4m3<128, __half>(p, stream);
    }
    if (d == 64) return bf16 ? launch_16bit<64, __nv_bfloat16>(p, stream) : launch_16bit<64, __half>(p, stream);
    return bf16 ? launch_16bit<128, __nv_bfloat16>(p, stream) : launch_16bit<128, __half>(p, stream);
}

}  // namespace attn
