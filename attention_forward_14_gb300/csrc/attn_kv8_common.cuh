// What the two kernels of the attention over an e4m3 paged cache share on the
// device: conversions, small copies, and how work is dealt out.
#pragma once

#include "attn_kv8.h"
#include "rows.cuh"
#include "stream_order.cuh"

namespace attn {

// P = 2^(x - m + kOffset) against a reference m that is raised when some x
// exceeds it by more than kSlack: P <= 2^14, within fp16.
constexpr float kOffset = 6.f, kSlack = 8.f;
// Values with a smaller scale count as multiples of this one (it is the
// smallest that an append gives a block), so that neither its logarithm nor
// the weights divided by it leave fp32's range.
constexpr float kLeastScale = 0x1p-64f;
enum : uint32_t { SITE_KV8_FULL = 60, SITE_KV8_EMPTY = 61, SITE_KV8_Q = 62, SITE_KV8_CONV = 63, SITE_KV8_S = 64,
                  SITE_KV8_P = 65, SITE_KV8_O = 66 };

// fp16 of the e4m3 values in the low and in the high half of a word.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Arrives on `bar` when this thread's earlier cp.async have landed (the
// barrier's count includes it).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// log2 of a scale (a normal number): exact for a power of two.  (Of the whole
// number at once the approximation is off by 2^-22 of the result, which for a
// scale of 2^-64 is 2^-16 of every weight.)
__device__ __forceinline__ float log2_scale(float x)
{
    const uint32_t b = __float_as_uint(x);
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u)));
    return static_cast<float>(static_cast<int>(b >> 23) - 127) + y;
}

// (with subnormal results: x may be above 2^126)
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int cached_len(const Kv8Params &p, int b) { return min(max(p.seqlens[b], 0), p.cap); }

// Whether the scale at `i` is one of the pool's.
__device__ __forceinline__ bool scale_in_bounds(const Kv8Params &p, int64_t i)
{
    return ATTN_OPS_IN_BOUNDS(i >= 0 && i < static_cast<int64_t>(p.num_pages) * p.h_kv * (p.page_size >> p.block_shift), p,
                              SITE_OPS_SCALE);
}

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The top bit of every byte that is an e4m3 NaN (0x7F, 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// a / b of non-negative numbers that mostly fit 32 bits (a 64-bit division
// is a hundred instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The units dealt to the CTAs: the first `rem` get one more than `per`.  No
// more CTAs than there are units, and none with fewer than kMinUnits of them
// when that leaves a CTA (1: one request of 1001 tokens 0.5 us slower; 4: 1.7).
constexpr int kMinUnits = 2;
struct Shares {
    int64_t per, rem;
    int ctas;
    __device__ __forceinline__ Shares(int64_t total, int grid, int min_units = kMinUnits)
    {
        ctas = static_cast<int>(min(static_cast<int64_t>(grid), max(total / min_units, int64_t(1))));
        per = quotient(total, ctas);
        rem = total - per * ctas;
    }
    __device__ __forceinline__ int64_t start(int64_t c) const { return c * per + min(c, rem); }
    // the CTA that has unit u
    __device__ __forceinline__ int64_t owner(int64_t u) const
    {
        const int64_t big = rem * (per + 1);
        return u < big ? quotient(u, per + 1) : rem + quotient(u - big, per);
    }
};

// The square root of 2^(m - top), by which a sum with reference m is
// multiplied twice to have reference top.  (At once 2^-126 and less would be
// 0, while the sum itself may be 2^70: of keys whose values are zeros, before
// any whose scale is large.)
__device__ __forceinline__ float half_step(float m, float top) { return m == top ? 1.f : ex2_approx(0.5f * (m - top)); }

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Natural log-sum-exp of a row from its reference and sum.  With the scales of
// the values the two are large and opposite (a scale of 2^-64: some -64 and
// 2^70), so the sum's exponent meets the reference before its logarithm does.
__device__ __forceinline__ float lse_of(float m, float l)
{
    int e;
    const float f = frexpf(l, &e);
    return l == 0.f ? -INFINITY : (m - kOffset + static_cast<float>(e) + log2f(f)) * 0.69314718055994531f;
}

}  // namespace attn
