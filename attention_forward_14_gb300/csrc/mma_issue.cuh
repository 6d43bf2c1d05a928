// Products of the tensor cores issued from code that the whole warp runs: one
// lane's predicate guards the instruction, not a branch around it.  In the
// branch of one lane the compiler keeps descriptors and addresses in vector
// registers and moves them over to uniform ones product by product; where the
// warp stays together it computes them there.  Twelve products of a loop,
// beside eight busy warps: 54 clk each in a branch, 21 so (N = 32, of which
// the tensor cores need 16; of N = 64 they need 32).
#pragma once

#include "ptx.cuh"

namespace attn {

// The lane that issues; 1 there, 0 in the others.  (Called once: products and
// the commits that track them are one thread's.)
__device__ __forceinline__ uint32_t issuing_lane() { return elect_one() ? 1u : 0u; }

// D(tmem) (+)= A(smem desc) * B(smem desc), kind::f16, fp32 accumulate.
__device__ __forceinline__ void mma_ss_by(uint32_t lane, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi), "r"(lane)
        : "memory");
}

// D(tmem) (+)= A(tmem) * B(smem desc), kind::f16, fp32 accumulate.
__device__ __forceinline__ void mma_ts_by(uint32_t lane, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi), "r"(lane)
        : "memory");
}

// Arrive (once) on `bar` when the issuing lane's earlier products have completed.
__device__ __forceinline__ void tc_commit_by(uint32_t lane, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lane)
        : "memory");
}

}  // namespace attn
