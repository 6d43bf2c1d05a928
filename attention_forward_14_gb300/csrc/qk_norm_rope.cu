// RMS norm of every query and key head and the rotary rotation in one pass,
// and the gradients.  For one head x of one token (d values), with a norm
// weight w and the rotation R of the token's position:
//   r = (mean(x^2) + eps)^(-1/2),  n = r x,  y = w n,  out = R y
//   dy = R^T dout,  dw = sum over tokens and heads of dy n,  dn = w dy,
//   dx = r (dn - n mean(dn n))
// Everything in fp32 from the 16-bit inputs, rounded once at the store.
//
// Both passes read and write each value once and do about ten operations on
// it, so they are bound by HBM.  A unit of work is one token and a few of its
// heads: the token's cos and sin are read once for all of the unit's heads
// and stay in registers, and the unit's rows are loaded before the first of
// them is used, which keeps enough bytes in flight.
#include "qk_norm_rope.h"

#include "attn_fwd_kernel.cuh"
#include "rows.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsInFlight = 4;  // rows that each lane group loads ahead

template <int D>
constexpr int heads_per_unit() { return kRowsInFlight * (32 / (D / 8)); }

// Position of token `tok`; false when it lies outside the tables (the
// token's rows are then zeros, and a position past the end is reported).
__device__ __forceinline__ bool token_position(const NormRopeParams &p, int64_t bi, int64_t si, int &pos)
{
    pos = p.pos ? p.pos[bi * p.pos_b + si] : static_cast<int>(si);
    if (p.cos == nullptr) return true;
    if (pos >= p.table_len) record_status(p.status, 4u, 0u);
    return pos >= 0 && pos < p.table_len;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, HPU = heads_per_unit<D>();
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const int64_t unit = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    const int groups = p.side[0].groups + p.side[1].groups;
    const int64_t tok = unit / groups;
    if (tok >= p.tokens) return;
    const int gi = static_cast<int>(unit - tok * groups);
    const bool key = gi >= p.side[0].groups;
    const NormRopeSide &sd = p.side[key ? 1 : 0];
    const int h0 = (key ? gi - p.side[0].groups : gi) * HPU;
    const int64_t bi = tok / p.s, si = tok - bi * p.s;

    const T *x = static_cast<const T *>(sd.x) + bi * sd.xb + si * sd.xs + l * 8;
    uint4 raw[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        const int h = h0 + i * RPW + sub;
        raw[i] = h < sd.heads ? __ldcs(reinterpret_cast<const uint4 *>(x + h * sd.xh)) : make_uint4(0u, 0u, 0u, 0u);
    }
    int pos;
    const bool valid = token_position(p, bi, si, pos);
    const bool il = p.interleaved != 0;
    const RotLane rl = rot_lane(lane, l, p.cos ? p.rot : 0, il);
    float c[8], s[8];
    if (valid) load_angles(p.cos, p.sin, static_cast<int64_t>(pos) * (p.rot / 2), rl, il, c, s);
    float w[8], wo[8];
    if (sd.w) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(sd.w) + l * 8));
        unpack8<T>(u, w);
        unpack8<T>(shfl4(u, rl.partner), wo);
    }
    T *out = static_cast<T *>(sd.out) + bi * sd.ob + si * sd.os + l * 8;
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        const int h = h0 + i * RPW + sub;
        float v[8], o[8];
        unpack8<T>(raw[i], v);
        unpack8<T>(shfl4(raw[i], rl.partner), o);
        if (sd.w) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
            const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= r * w[e];
                o[e] *= r * wo[e];
            }
        }
        rotate8<false>(v, o, c, s, rl, il);
        if (h < sd.heads) {
            const uint4 y = valid ? pack8<T>(v) : make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(out + h * sd.oh) = y;
        }
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, HPU = heads_per_unit<D>();
    __shared__ float acc_s[kThreads / 32][2][D];
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const int groups = p.side[0].groups + p.side[1].groups;
    const int64_t units = p.tokens * groups;
    const bool il = p.interleaved != 0;
    const RotLane rl = rot_lane(lane, l, p.cos ? p.rot : 0, il);
    float dw[2][8] = {};
    for (int64_t unit = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); unit < units;
         unit += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const int64_t tok = unit / groups;
        const int gi = static_cast<int>(unit - tok * groups);
        const bool key = gi >= p.side[0].groups;
        const NormRopeSide &sd = p.side[key ? 1 : 0];
        const int h0 = (key ? gi - p.side[0].groups : gi) * HPU;
        const int64_t bi = tok / p.s, si = tok - bi * p.s;
        const T *x = static_cast<const T *>(sd.x) + bi * sd.xb + si * sd.xs + l * 8;
        const T *g = static_cast<const T *>(sd.g) + bi * sd.gb + si * sd.gs + l * 8;
        uint4 rx[kRowsInFlight], rg[kRowsInFlight];
#pragma unroll
        for (int i = 0; i < kRowsInFlight; ++i) {
            const int h = h0 + i * RPW + sub;
            const bool in = h < sd.heads;
            rx[i] = in ? __ldcs(reinterpret_cast<const uint4 *>(x + h * sd.xh)) : make_uint4(0u, 0u, 0u, 0u);
            rg[i] = in ? __ldcs(reinterpret_cast<const uint4 *>(g + h * sd.gh)) : make_uint4(0u, 0u, 0u, 0u);
        }
        int pos;
        const bool valid = token_position(p, bi, si, pos);
        float c[8], s[8];
        if (valid) load_angles(p.cos, p.sin, static_cast<int64_t>(pos) * (p.rot / 2), rl, il, c, s);
        float w[8];
        if (sd.w) unpack8<T>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(sd.w) + l * 8)), w);
        T *out = static_cast<T *>(sd.out) + bi * sd.ob + si * sd.os + l * 8;
#pragma unroll
        for (int i = 0; i < kRowsInFlight; ++i) {
            const int h = h0 + i * RPW + sub;
            float dy[8], o[8];
            unpack8<T>(rg[i], dy);
            unpack8<T>(shfl4(rg[i], rl.partner), o);
            rotate8<true>(dy, o, c, s, rl, il);
            if (sd.w) {
                float n[8];
                unpack8<T>(rx[i], n);
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(n[e], n[e], ss);
                    dot = fmaf(dy[e] * w[e], n[e], dot);
                }
                const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
                const float mean = row_sum<LPR>(dot) * r * (1.f / D);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[e] *= r;
                    const float t = valid ? dy[e] * n[e] : 0.f;  // rows past the last head are zeros
                    if (key) dw[1][e] += t;
                    else dw[0][e] += t;
                    dy[e] = r * (dy[e] * w[e] - n[e] * mean);
                }
            }
            if (h < sd.heads)
                *reinterpret_cast<uint4 *>(out + h * sd.oh) = valid ? pack8<T>(dy) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (p.dw_part == nullptr) return;
    // the block's sums, in a fixed order: the lane groups of a warp, then the warps
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = dw[k][e];
#pragma unroll
            for (int off = 16; off >= LPR; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (sub == 0) acc_s[threadIdx.x >> 5][k][l * 8 + e] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int wi = 0; wi < kThreads / 32; ++wi) v += acc_s[wi][i / D][i % D];
        p.dw_part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = v;
    }
}

// The blocks' partial sums added up: 32 columns a block, the rows dealt to
// the warps and joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float *part, int blocks, int d, float *dwq, float *dwk)
{
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float v = 0.f;
    for (int r = warp; r < blocks; r += 32) v += part[static_cast<int64_t>(r) * 2 * d + col];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][lane];
        float *dst = col < d ? dwq : dwk;
        if (dst) dst[col < d ? col : col - d] = t;
    }
}

NormRopeParams with_groups(const NormRopeParams &p, int d)
{
    NormRopeParams q = p;
    const int hpu = d == 64 ? heads_per_unit<64>() : heads_per_unit<128>();
    for (NormRopeSide &sd : q.side) sd.groups = (sd.heads + hpu - 1) / hpu;
    return q;
}

int64_t unit_blocks(const NormRopeParams &p)
{
    const int64_t units = p.tokens * (p.side[0].groups + p.side[1].groups);
    return (units + kThreads / 32 - 1) / (kThreads / 32);
}

}  // namespace

int norm_rope_bwd_blocks(const NormRopeParams &p, int d, int sm_count)
{
    const int64_t n = unit_blocks(with_groups(p, d));
    int64_t cap = static_cast<int64_t>(sm_count) * 4;
    if (cap > kNormRopeMaxBlocks) cap = kNormRopeMaxBlocks;
    return static_cast<int>(n < cap ? n : cap);
}

cudaError_t launch_norm_rope(const NormRopeParams &p0, int d, bool bf16, cudaStream_t stream)
{
    const NormRopeParams p = with_groups(p0, d);
    const unsigned blocks = static_cast<unsigned>(unit_blocks(p));
    if (d == 64) {
        if (bf16) norm_rope_kernel<64, __nv_bfloat16><<<blocks, kThreads, 0, stream>>>(p);
        else norm_rope_kernel<64, __half><<<blocks, kThreads, 0, stream>>>(p);
    } else {
        if (bf16) norm_rope_kernel<128, __nv_bfloat16><<<blocks, kThreads, 0, stream>>>(p);
        else norm_rope_kernel<128, __half><<<blocks, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_norm_rope_bwd(const NormRopeParams &p0, int d, bool bf16, int sm_count, cudaStream_t stream)
{
    const NormRopeParams p = with_groups(p0, d);
    const int blocks = norm_rope_bwd_blocks(p0, d, sm_count);
    if (d == 64) {
        if (bf16) norm_rope_bwd_kernel<64, __nv_bfloat16><<<blocks, kThreads, 0, stream>>>(p);
        else norm_rope_bwd_kernel<64, __half><<<blocks, kThreads, 0, stream>>>(p);
    } else {
        if (bf16) norm_rope_bwd_kernel<128, __nv_bfloat16><<<blocks, kThreads, 0, stream>>>(p);
        else norm_rope_bwd_kernel<128, __half><<<blocks, kThreads, 0, stream>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.dw_part == nullptr) return e;
    norm_rope_dw_kernel<<<2 * d / 32, 1024, 0, stream>>>(p.dw_part, blocks, d, p.dw[0], p.dw[1]);
    return cudaGetLastError();
}

}  // namespace attn
