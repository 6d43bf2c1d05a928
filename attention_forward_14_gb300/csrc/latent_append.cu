// New tokens of latent attention into its paged cache: token t of batch
// element e, [latent (512) | key part (64)], goes to logical position L + t,
// L = clamp(seqlens[e], 0, capacity), for t < new_seqlens[e]:
//   latent: w * x * (mean(x^2) + eps)^(-1/2)   (no weight: x, bit for bit)
//   key part: rotated by the angles of position L + t (no tables: as it is)
// rounded once to 16 bits.  Tokens at or past the capacity, and tokens of
// pages outside the pool, are not written.
//
// A warp takes a token: 32 bytes of the latent and two values of the key part
// to a lane, so that both of a rotated pair are one lane's and the sum of the
// squares is five shuffles.  Bound by the copies: 1152 bytes in, 1152 out and
// 256 of angles a token; four times up to 4001 tokens, fp16: 4.8 us.  Single
// tokens are bound by the launch and a chain of loads (length, page, token):
// 64 requests 2.7 us.
#include "latent.h"
#include "rows.cuh"
#include "stream_order.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const __grid_constant__ LatentAppendParams p)
{
    await_previous();
    const int lane = threadIdx.x & 31;
    const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), s_new = static_cast<uint32_t>(p.s);
    const uint32_t e = unit / s_new;
    const int t = static_cast<int>(unit - e * s_new);
    if (e >= p.b) return;
    const T *x = static_cast<const T *>(p.x) + e * p.xb + t * p.xs;
    // (read before the lengths are known: a padded token's row is there, and left out below)
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(x) + lane), b = __ldcs(reinterpret_cast<const uint4 *>(x) + 32 + lane);
    // the lane's pair of the key part: values 2 l, 2 l + 1, or l and l + 32
    const int k0 = kLatent + (p.interleaved ? 2 * lane : lane), k1 = k0 + (p.interleaved ? 1 : 32);
    const uint16_t *xr = reinterpret_cast<const uint16_t *>(x);
    const uint32_t key = xr[k0] | static_cast<uint32_t>(xr[k1]) << 16;

    const int cap = static_cast<int>(p.pages_per_seq) * p.page_size;
    const int count = p.new_seqlens ? min(max(p.new_seqlens[e], 0), static_cast<int>(p.s)) : static_cast<int>(p.s);
    const int64_t pos = static_cast<int64_t>(min(max(p.seqlens[e], 0), cap)) + t;
    if (t >= count || pos >= cap) return;
    const int pg = static_cast<int>(pos) / p.page_size;
    const int page = p.block_table[static_cast<int64_t>(e) * p.pages_per_seq + pg];
    if (page < 0 || page >= p.num_pages) return;
    const int64_t token = static_cast<int64_t>(page) * p.page_size + (static_cast<int>(pos) - pg * p.page_size);
    if (!ATTN_OPS_IN_BOUNDS(token < p.num_pages * p.page_size && pos >= 0, p, SITE_OPS_PAGE)) return;
    T *dst = static_cast<T *>(p.pool) + token * kLatentToken;

    uint4 out[2] = {a, b};
    if (p.weight) {
        const uint4 *w = static_cast<const uint4 *>(p.weight);
        const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        float2 v[8];
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = Pair<T>::get(in[i]);
            sum = __ffma2_rn(v[i], v[i], sum);
        }
        const float r = rsqrtf(row_sum<32>(sum.x + sum.y) * (1.f / kLatent) + p.eps);
        const uint4 wa = w[lane], wb = w[32 + lane];
        const uint32_t wi[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 n = __fmul2_rn(__fmul2_rn(v[i], make_float2(r, r)), Pair<T>::get(wi[i]));
            y[i] = Pair<T>::put(n.x, n.y);
        }
        out[0] = make_uint4(y[0], y[1], y[2], y[3]);
        out[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
    reinterpret_cast<uint4 *>(dst)[lane] = out[0];
    reinterpret_cast<uint4 *>(dst)[32 + lane] = out[1];
    uint32_t turned = key;
    if (p.cos) {
        const float c = p.cos[pos * 32 + lane], s = p.sin[pos * 32 + lane];
        const float2 v = Pair<T>::get(key);
        turned = Pair<T>::put(__fsub_rn(__fmul_rn(v.x, c), __fmul_rn(v.y, s)), __fadd_rn(__fmul_rn(v.y, c), __fmul_rn(v.x, s)));
    }
    uint16_t *dr = reinterpret_cast<uint16_t *>(dst);
    if (p.interleaved) {
        *reinterpret_cast<uint32_t *>(dr + k0) = turned;
    } else {
        dr[k0] = static_cast<uint16_t>(turned);
        dr[k1] = static_cast<uint16_t>(turned >> 16);
    }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams &p, bool bf16, cudaStream_t stream)
{
    const int64_t per = kThreads / 32;
    const dim3 grid(static_cast<unsigned>((p.b * p.s + per - 1) / per));
    return bf16 ? launch_overlapped(latent_append_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, p)
                : launch_overlapped(latent_append_kernel<__half>, grid, kThreads, 0, stream, p);
}

}  // namespace attn
