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

#include "attn_fwd.h"
#include "rows.cuh"
#include "stream_order.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kBwdBlocks = 2;  // of the backward on an SM; the grid is what fits at a time

// Rows that each lane group loads ahead, and the heads of a unit.
template <int D>
constexpr int heads_per_unit(int rows) { return rows * (32 / (D / 8)); }

// False when a position lies outside the tables (the token's rows are then
// zeros, and a position past the end is reported).
__device__ __forceinline__ bool known_position(const NormRopeParams &p, int pos)
{
    if (p.cos == nullptr) return true;
    if (pos >= p.table_len) record_status(p.status, ATTN_STATUS_POSITION, 0u);
    return pos >= 0 && pos < p.table_len;
}

// The unit of a warp: a token and ROWS rows of each of the warp's lane groups.
struct NormUnit {
    bool key;
    int h0;           // its first head
    int64_t bi, si;   // its token
};

__device__ __forceinline__ NormUnit norm_unit(const NormRopeParams &p, uint32_t unit, int hpu)
{
    const uint32_t groups = p.side[0].groups + p.side[1].groups;
    const uint32_t tok = unit / groups, gi = unit - tok * groups;
    NormUnit u;
    u.key = gi >= static_cast<uint32_t>(p.side[0].groups);
    u.h0 = static_cast<int>(u.key ? gi - p.side[0].groups : gi) * hpu;
    const uint32_t s = static_cast<uint32_t>(p.s), bi = tok / s;
    u.bi = bi;
    u.si = tok - bi * s;
    return u;
}

// The lane's values of a norm weight, or ones.
template <typename T>
__device__ __forceinline__ void load_weight(const void *w, const RowLane &rl, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
    if (w) {
        unpack4<T>(__ldg(reinterpret_cast<const uint2 *>(static_cast<const T *>(w) + rl.lo)), v);
        unpack4<T>(__ldg(reinterpret_cast<const uint2 *>(static_cast<const T *>(w) + rl.hi)), v + 4);
    }
}

template <int D, typename T, bool ADJACENT, int ROWS>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    await_previous();
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (unit >= p.units) return;
    const NormUnit u = norm_unit(p, unit, heads_per_unit<D>(ROWS));
    const NormRopeSide &sd = p.side[u.key ? 1 : 0];
    if (!ATTN_OPS_IN_BOUNDS(u.bi * p.s + u.si < p.tokens && u.h0 < sd.heads, p, SITE_OPS_UNIT)) return;
    const RowLane rl = row_lane<ADJACENT>(l, p.rot);
    const int left = sd.heads - u.h0 - sub;  // row i of the lane group is there when i * RPW < left

    uint2 raw[ROWS][2];
    {
        const T *x = static_cast<const T *>(sd.x) + u.bi * sd.xb + u.si * sd.xs + (u.h0 + sub) * sd.xh;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
            if (i * RPW < left) load_row<ADJACENT>(x, rl, raw[i]);
            x += RPW * sd.xh;
        }
    }
    T *out = static_cast<T *>(sd.out) + u.bi * sd.ob + u.si * sd.os + (u.h0 + sub) * sd.oh;
    const int pos = p.pos ? __ldg(p.pos + u.bi * p.pos_b + u.si) : static_cast<int>(u.si);
    if (!known_position(p, pos)) {
        const uint2 zero[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
        for (int i = 0; i < ROWS; ++i, out += RPW * sd.oh)
            if (i * RPW < left) store_row<ADJACENT>(out, rl, zero);
        return;
    }
    float c[4], s[4], w[8];
    load_angles(p.cos, p.sin, static_cast<int64_t>(pos) * (p.rot / 2), rl, c, s);
    load_weight<T>(sd.w, rl, w);
    const Turn turn = make_turn<ADJACENT, false>(c, s, w);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (i * RPW >= sd.heads - u.h0) break;  // (by every lane)
        float2 v[4];
        unpack_pairs<T>(raw[i], v);
        float r = 1.f;
        if (sd.w) r = rsqrtf(row_sum<LPR>(dot8(v, v)) * (1.f / D) + p.eps);
        if (rl.on) {
            turned<ADJACENT>(v, turn);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __fmul2_rn(v[e], make_float2(w[2 * e], w[2 * e + 1]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __fmul2_rn(v[e], make_float2(r, r));
        pack_pairs<T>(v, raw[i]);
        if (i * RPW < left) store_row<ADJACENT>(out, rl, raw[i]);
        out += RPW * sd.oh;
    }
}

// The backward's blocks go over the units of the queries, then over those of
// the keys, so that a lane adds up one weight's gradient at a time.
template <int D, typename T, bool ADJACENT, int ROWS>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, HPU = heads_per_unit<D>(ROWS);
    __shared__ float acc_s[kThreads / 32][D];
    await_previous();
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR, warp = threadIdx.x >> 5;
    const RowLane rl = row_lane<ADJACENT>(l, p.rot);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const NormRopeSide &sd = p.side[k];
        float2 dw[4] = {}, w[4];
        {
            float w8[8];
            load_weight<T>(sd.w, rl, w8);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = make_float2(w8[2 * e], w8[2 * e + 1]);
        }
        const uint32_t units = static_cast<uint32_t>(p.tokens) * sd.groups;
        // a unit's rows, its gradients' rows and its position, as they come from memory
        struct Fetched {
            uint2 x[ROWS][2], g[ROWS][2];
            int pos;
        };
        auto fetch = [&](uint32_t unit, Fetched &f) {
            const uint32_t tok = unit / sd.groups;
            const int h = static_cast<int>(unit - tok * sd.groups) * HPU + sub;
            const uint32_t bi = tok / static_cast<uint32_t>(p.s), si = tok - bi * static_cast<uint32_t>(p.s);
            f.pos = p.pos ? __ldg(p.pos + bi * p.pos_b + si) : static_cast<int>(si);
            const T *x = static_cast<const T *>(sd.x) + bi * sd.xb + si * sd.xs + h * sd.xh;
            const T *g = static_cast<const T *>(sd.g) + bi * sd.gb + si * sd.gs + h * sd.gh;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                f.x[i][0] = f.x[i][1] = f.g[i][0] = f.g[i][1] = make_uint2(0u, 0u);
                if (h + i * RPW < sd.heads) {
                    load_row<ADJACENT>(g, rl, f.g[i]);
                    if (sd.w) load_row<ADJACENT>(x, rl, f.x[i]);
                }
                x += RPW * sd.xh;
                g += RPW * sd.gh;
            }
        };
        const uint32_t stride = gridDim.x * (kThreads / 32);
        for (uint32_t unit = blockIdx.x * (kThreads / 32) + warp; unit < units; unit += stride) {
            const uint32_t tok = unit / sd.groups;
            const int h = static_cast<int>(unit - tok * sd.groups) * HPU + sub;
            if (!ATTN_OPS_IN_BOUNDS(tok < p.tokens && h - sub < sd.heads, p, SITE_OPS_UNIT)) continue;
            Fetched cur;
            fetch(unit, cur);
            const int left = sd.heads - h;
            const uint32_t bi = tok / static_cast<uint32_t>(p.s), si = tok - bi * static_cast<uint32_t>(p.s);
            T *out = static_cast<T *>(sd.out) + bi * sd.ob + si * sd.os + h * sd.oh;
            const int pos = cur.pos;
            if (!known_position(p, pos)) {
                const uint2 zero[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
                for (int i = 0; i < ROWS; ++i, out += RPW * sd.oh)
                    if (i * RPW < left) store_row<ADJACENT>(out, rl, zero);
                continue;
            }
            float c[4], s[4];
            load_angles(p.cos, p.sin, static_cast<int64_t>(pos) * (p.rot / 2), rl, c, s);
            const float ones[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            const Turn turn = make_turn<ADJACENT, true>(c, s, ones);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                if (i * RPW >= sd.heads - (h - sub)) break;  // (by every lane)
                float2 dy[4];
                unpack_pairs<T>(cur.g[i], dy);
                if (rl.on) turned<ADJACENT>(dy, turn);
                if (sd.w) {
                    float2 x[4], wdy[4];
                    unpack_pairs<T>(cur.x[i], x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) wdy[e] = __fmul2_rn(dy[e], w[e]);
                    const float r0 = rsqrtf(row_sum<LPR>(dot8(x, x)) * (1.f / D) + p.eps);
                    const float r = i * RPW < left ? r0 : 0.f;  // (no row: with eps 0 an infinity, times zeros)
                    // dx = r (wdy - n mean(wdy n)), n = r x: x enters with -r^3 mean(wdy x)
                    const float f = row_sum<LPR>(dot8(wdy, x)) * (-1.f / D) * r * r * r;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // rows past the last head are zeros
                        dw[e] = __ffma2_rn(dy[e], __fmul2_rn(x[e], make_float2(r, r)), dw[e]);
                        dy[e] = __ffma2_rn(x[e], make_float2(f, f), __fmul2_rn(wdy[e], make_float2(r, r)));
                    }
                }
                uint2 y[2];
                pack_pairs<T>(dy, y);
                if (i * RPW < left) store_row<ADJACENT>(out, rl, y);
                out += RPW * sd.oh;
            }
        }
        if (p.dw_part == nullptr) continue;
        // the block's sums, in a fixed order: the lane groups of a warp, then the warps
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = e & 1 ? dw[e >> 1].y : dw[e >> 1].x;
#pragma unroll
            for (int off = 16; off >= LPR; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (sub == 0) acc_s[warp][(e < 4 ? rl.lo : rl.hi - 4) + e] = v;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < D; i += kThreads) {
            if (!ATTN_OPS_IN_BOUNDS(blockIdx.x < kNormRopeMaxBlocks, p, SITE_OPS_PART)) break;
            float v = 0.f;
#pragma unroll
            for (int wi = 0; wi < kThreads / 32; ++wi) v += acc_s[wi][i];
            p.dw_part[(static_cast<int64_t>(blockIdx.x) * 2 + k) * D + i] = v;
        }
        __syncthreads();
    }
}

// The blocks' partial sums added up: 32 columns a block, the rows dealt to
// the warps and joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float *part, int blocks, int d, float *dwq, float *dwk)
{
    __shared__ float s[32][33];
    await_previous();
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

NormRopeParams with_units(const NormRopeParams &p, int d, int rows)
{
    NormRopeParams q = p;
    const int hpu = d == 64 ? heads_per_unit<64>(rows) : heads_per_unit<128>(rows);
    for (NormRopeSide &sd : q.side) sd.groups = (sd.heads + hpu - 1) / hpu;
    q.units = static_cast<uint32_t>(q.tokens * (q.side[0].groups + q.side[1].groups));
    return q;
}

int blocks_of(const NormRopeParams &p) { return static_cast<int>((static_cast<int64_t>(p.units) + kThreads / 32 - 1) / (kThreads / 32)); }

constexpr int kFwdRows = 4, kBwdRows = 4;  // 2 rows ahead: +14% and +7% at b2 h32 s4096 d128; 8: +15% (forward)

template <int D, typename T>
cudaError_t launch_fwd_t(const NormRopeParams &p0, cudaStream_t stream)
{
    const NormRopeParams p = with_units(p0, D, kFwdRows);
    return launch_overlapped(p.interleaved ? norm_rope_kernel<D, T, true, kFwdRows> : norm_rope_kernel<D, T, false, kFwdRows>,
                             dim3(blocks_of(p)), kThreads, 0, stream, p);
}

template <int D, typename T>
cudaError_t launch_bwd_t(const NormRopeParams &p0, int sm_count, cudaStream_t stream)
{
    const NormRopeParams p = with_units(p0, D, kBwdRows);
    int blocks = blocks_of(p);
    const int cap = sm_count * kBwdBlocks < kNormRopeMaxBlocks ? sm_count * kBwdBlocks : kNormRopeMaxBlocks;
    if (blocks > cap) blocks = cap;
    const cudaError_t e = launch_overlapped(
        p.interleaved ? norm_rope_bwd_kernel<D, T, true, kBwdRows> : norm_rope_bwd_kernel<D, T, false, kBwdRows>,
        dim3(blocks), kThreads, 0, stream, p);
    if (e != cudaSuccess || p.dw_part == nullptr) return e;
    return launch_overlapped(norm_rope_dw_kernel, dim3(2 * D / 32), 1024, 0, stream, p.dw_part, blocks, D, p.dw[0], p.dw[1]);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, int d, bool bf16, cudaStream_t stream)
{
    if (d == 64) return bf16 ? launch_fwd_t<64, __nv_bfloat16>(p, stream) : launch_fwd_t<64, __half>(p, stream);
    return bf16 ? launch_fwd_t<128, __nv_bfloat16>(p, stream) : launch_fwd_t<128, __half>(p, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeParams &p, int d, bool bf16, int sm_count, cudaStream_t stream)
{
    if (d == 64)
        return bf16 ? launch_bwd_t<64, __nv_bfloat16>(p, sm_count, stream) : launch_bwd_t<64, __half>(p, sm_count, stream);
    return bf16 ? launch_bwd_t<128, __nv_bfloat16>(p, sm_count, stream) : launch_bwd_t<128, __half>(p, sm_count, stream);
}

}  // namespace attn
