// Rows of one head of one token, held by the lanes of a warp: loads, the
// rotary rotation and the sums that the q/k norm, the rotated cache append
// and their gradients share.
//
// A row of D 16-bit values is D/8 lanes of eight values, so a warp holds
// 32 / (D/8) rows: four at D = 64, two at D = 128.
//
// Rotation of the first `rot` values of a row by the angles of its position
// (cos/sin tables of rot/2 columns; rot a multiple of 16):
//   pairs (i, i + rot/2), or adjacent pairs (2i, 2i + 1):
//   (a, b) -> (a cos - b sin, b cos + a sin);  its transpose has -sin.
// A lane's eight values are two runs of four, placed so that both of a pair
// are the same lane's: no value is fetched from another lane or twice, and a
// lane needs four columns of the tables.  The price is two 8-byte accesses
// for a 16-byte one.
// In `rotate` the products and the sum are rounded one by one (no fused
// multiply-add), so that a key appended to a cache equals the formula
// evaluated step by step in fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_fwd_kernel.cuh"

namespace attn {

// Checked build (ATTN_CHECKED=1): the operators that use this file compare
// what they decode and index with its bounds; a violation is recorded in the
// status word, with its site, and the access is left out.
enum : uint32_t {
    SITE_OPS_UNIT = 70,   // decoded unit outside the problem
    SITE_OPS_ROW = 71,    // row of an input
    SITE_OPS_PAGE = 72,   // row of the pool
    SITE_OPS_SCALE = 73,  // scale of a block
    SITE_OPS_PART = 74,   // partial result
};
#if ATTN_CHECKED
#define ATTN_OPS_IN_BOUNDS(cond, p, site) ops_in_bounds((cond), (p).status, (site))
__device__ __forceinline__ bool ops_in_bounds(bool ok, uint32_t *status, uint32_t site)
{
    if (!ok) record_status(status, STATUS_BOUNDS, site);
    return ok;
}
#else
#define ATTN_OPS_IN_BOUNDS(cond, p, site) true
#endif

template <typename T>
struct Pair;
template <>
struct Pair<__half> {
    static __device__ __forceinline__ float2 get(uint32_t u)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    static __device__ __forceinline__ uint32_t put(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 get(uint32_t u)
    {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t put(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Four 16-bit values as fp32.
template <typename T>
__device__ __forceinline__ void unpack4(const uint2 &u, float *x)
{
    const float2 a = Pair<T>::get(u.x), b = Pair<T>::get(u.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// Where the two runs of a lane's values lie in its row, and what it does in
// the rotation (x[0..3] from `lo`, x[4..7] from `hi`).
struct RowLane {
    int lo, hi;
    bool on;   // rotated, by columns [col, col + 4) of the tables
    int col;
};

// `l`: the lane within its row.
template <bool ADJACENT>
__device__ __forceinline__ RowLane row_lane(int l, int rot)
{
    RowLane r;
    r.on = 8 * l < rot;
    r.col = 4 * l;
    r.lo = ADJACENT || !r.on ? 8 * l : 4 * l;
    r.hi = r.lo + (ADJACENT || !r.on ? 4 : rot >> 1);
    return r;
}

// Both runs of a row at `row`, read once (streaming) or written.
template <bool ADJACENT, typename T>
__device__ __forceinline__ void load_row(const T *row, const RowLane &r, uint2 (&u)[2])
{
    if constexpr (ADJACENT) {  // one run of eight
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(row + r.lo));
        u[0] = make_uint2(v.x, v.y), u[1] = make_uint2(v.z, v.w);
    } else {
        u[0] = __ldcs(reinterpret_cast<const uint2 *>(row + r.lo));
        u[1] = __ldcs(reinterpret_cast<const uint2 *>(row + r.hi));
    }
}

template <bool ADJACENT, typename T>
__device__ __forceinline__ void store_row(T *row, const RowLane &r, const uint2 (&u)[2])
{
    if constexpr (ADJACENT) {
        *reinterpret_cast<uint4 *>(row + r.lo) = make_uint4(u[0].x, u[0].y, u[1].x, u[1].y);
    } else {
        *reinterpret_cast<uint2 *>(row + r.lo) = u[0];
        *reinterpret_cast<uint2 *>(row + r.hi) = u[1];
    }
}

// The lane's columns of one position's cos and sin, at element `at` of the tables.
__device__ __forceinline__ void load_angles(const float *cos_t, const float *sin_t, int64_t at, const RowLane &r,
                                            float (&c)[4], float (&s)[4])
{
    if (!r.on) return;
    const float4 a = *reinterpret_cast<const float4 *>(cos_t + at + r.col);
    const float4 b = *reinterpret_cast<const float4 *>(sin_t + at + r.col);
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
    s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
}

// u rotated; u[0..1] is the lane's first run, u[2..3] its second.  The
// products are formed two at a time and the sums one at a time: of packed
// products and a packed sum the compiler makes fused multiply-adds, which
// round once and not twice.
template <bool ADJACENT>
__device__ __forceinline__ void rotate(float2 (&u)[4], const float (&c)[4], const float (&s)[4])
{
    if constexpr (ADJACENT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __fmul2_rn(u[i], make_float2(c[i], c[i])), q = __fmul2_rn(u[i], make_float2(s[i], s[i]));
            u[i] = make_float2(__fsub_rn(p.x, q.y), __fadd_rn(p.y, q.x));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 co = make_float2(c[2 * i], c[2 * i + 1]), si = make_float2(s[2 * i], s[2 * i + 1]);
            const float2 ac = __fmul2_rn(u[i], co), as = __fmul2_rn(u[i], si);
            const float2 bc = __fmul2_rn(u[i + 2], co), bs = __fmul2_rn(u[i + 2], si);
            u[i] = make_float2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y));
            u[i + 2] = make_float2(__fadd_rn(bc.x, as.x), __fadd_rn(bc.y, as.y));
        }
    }
}

// The same with fused multiply-adds (fewer instructions, one rounding less):
// a Turn is what it needs of the angles, and of a weight for each value that
// is folded into them: out = u * a + partner(u) * b.
struct Turn {
    float2 a[4], b[4];
};

template <bool ADJACENT, bool BACK>
__device__ __forceinline__ Turn make_turn(const float (&c)[4], const float (&s)[4], const float (&w)[8])
{
    Turn t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (ADJACENT) {  // the partner of a value is the other one of its register pair
            const float si = BACK ? -s[i] : s[i];
            t.a[i] = make_float2(w[2 * i] * c[i], w[2 * i + 1] * c[i]);
            t.b[i] = make_float2(-w[2 * i + 1] * si, w[2 * i] * si);
        } else {                   // u[i] and u[i ^ 2]
            const int k = 2 * (i & 1);
            const bool upper = i >= 2;
            const float s0 = upper != BACK ? s[k] : -s[k], s1 = upper != BACK ? s[k + 1] : -s[k + 1];
            const int own = (upper ? 4 : 0) + k, other = (upper ? 0 : 4) + k;
            t.a[i] = make_float2(w[own] * c[k], w[own + 1] * c[k + 1]);
            t.b[i] = make_float2(w[other] * s0, w[other + 1] * s1);
        }
    }
    return t;
}

template <bool ADJACENT>
__device__ __forceinline__ void turned(float2 (&u)[4], const Turn &t)
{
    float2 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 other = ADJACENT ? make_float2(u[i].y, u[i].x) : u[i ^ 2];
        o[i] = __ffma2_rn(other, t.b[i], __fmul2_rn(u[i], t.a[i]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = o[i];
}

template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint2 (&r)[2], float2 (&u)[4])
{
    u[0] = Pair<T>::get(r[0].x), u[1] = Pair<T>::get(r[0].y);
    u[2] = Pair<T>::get(r[1].x), u[3] = Pair<T>::get(r[1].y);
}

template <typename T>
__device__ __forceinline__ void pack_pairs(const float2 (&u)[4], uint2 (&r)[2])
{
    r[0] = make_uint2(Pair<T>::put(u[0].x, u[0].y), Pair<T>::put(u[1].x, u[1].y));
    r[1] = make_uint2(Pair<T>::put(u[2].x, u[2].y), Pair<T>::put(u[3].x, u[3].y));
}

// Sum of the products of the lane's values.
__device__ __forceinline__ float dot8(const float2 (&x)[4], const float2 (&y)[4])
{
    const float2 p = __ffma2_rn(x[1], y[1], __fmul2_rn(x[0], y[0])), q = __ffma2_rn(x[3], y[3], __fmul2_rn(x[2], y[2]));
    const float2 t = __fadd2_rn(p, q);
    return t.x + t.y;
}

// Sum over the LPR lanes of each row, the same in every lane.
template <int LPR>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

}  // namespace attn
