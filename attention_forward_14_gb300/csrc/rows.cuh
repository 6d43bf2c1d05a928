// Rows of one head of one token, held by the lanes of a warp: loads, the
// rotary rotation and the sums that the q/k norm, the rotated cache append
// and their gradients share.
//
// A row of D 16-bit values is D/8 lanes of eight values (one 16-byte piece
// each), so a warp holds 32 / (D/8) rows: four at D = 64, two at D = 128.
//
// Rotation of the first `rot` values of a row by the angles of its position
// (cos/sin tables of rot/2 columns; rot a multiple of 16):
//   pairs (i, i + rot/2), or adjacent pairs (2i, 2i + 1):
//   (a, b) -> (a cos - b sin, b cos + a sin);  its transpose has -sin.
// The products and the sum are rounded one by one (no fused multiply-add),
// so the result is the same whichever of the two orders a caller writes, and
// equals the formula evaluated step by step in fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace attn {

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

// Eight 16-bit values (a 16-byte piece of a row) as fp32.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Pair<T>::get(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(Pair<T>::put(x[0], x[1]), Pair<T>::put(x[2], x[3]), Pair<T>::put(x[4], x[5]),
                      Pair<T>::put(x[6], x[7]));
}

// Which part of the rotation this lane of a row does.
struct RotLane {
    bool on;        // the lane's values are rotated
    bool upper;     // pairs (i, i + rot/2): the lane holds the second of each pair
    int partner;    // lane (of the warp) that holds the other of each pair
    int col;        // first column of the cos/sin tables
};

// `l`: the lane within its row; `lane`: within the warp.
__device__ __forceinline__ RotLane rot_lane(int lane, int l, int rot, bool interleaved)
{
    RotLane r;
    r.on = 8 * l < rot;
    r.upper = false;
    r.partner = lane;
    r.col = 4 * l;
    if (!interleaved) {
        const int half = rot >> 4;  // lanes that hold the first of each pair
        r.upper = r.on && l >= half;
        r.partner = !r.on ? lane : (r.upper ? lane - half : lane + half);
        r.col = 8 * (r.upper ? l - half : l);
    }
    return r;
}

// The lane's columns of one position's cos and sin: eight, or four (adjacent
// pairs) of which the others are not used.
__device__ __forceinline__ void load_angles(const float *cos_t, const float *sin_t, int64_t at, const RotLane &r,
                                            bool interleaved, float (&c)[8], float (&s)[8])
{
    if (!r.on) return;
    const float4 *cp = reinterpret_cast<const float4 *>(cos_t + at + r.col);
    const float4 *sp = reinterpret_cast<const float4 *>(sin_t + at + r.col);
    const float4 c0 = __ldg(cp), s0 = __ldg(sp);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w;
    if (!interleaved) {
        const float4 c1 = __ldg(cp + 1), s1 = __ldg(sp + 1);
        c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
        s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
    }
}

// x rotated (back, when `BACK`); `other` holds the partner lane's values
// (pairs (i, i + rot/2); not read for adjacent pairs).
template <bool BACK>
__device__ __forceinline__ void rotate8(float (&x)[8], const float (&other)[8], const float (&c)[8],
                                        const float (&s)[8], const RotLane &r, bool interleaved)
{
    if (!r.on) return;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            const float ac = __fmul_rn(a, c[i]), bs = __fmul_rn(b, s[i]);
            const float bc = __fmul_rn(b, c[i]), as = __fmul_rn(a, s[i]);
            x[2 * i] = BACK ? __fadd_rn(ac, bs) : __fsub_rn(ac, bs);
            x[2 * i + 1] = BACK ? __fsub_rn(bc, as) : __fadd_rn(bc, as);
        }
        return;
    }
    const bool plus = r.upper != BACK;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float xc = __fmul_rn(x[i], c[i]), os = __fmul_rn(other[i], s[i]);
        x[i] = plus ? __fadd_rn(xc, os) : __fsub_rn(xc, os);
    }
}

__device__ __forceinline__ uint4 shfl4(const uint4 &u, int src)
{
    return make_uint4(__shfl_sync(0xffffffffu, u.x, src), __shfl_sync(0xffffffffu, u.y, src),
                      __shfl_sync(0xffffffffu, u.z, src), __shfl_sync(0xffffffffu, u.w, src));
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
