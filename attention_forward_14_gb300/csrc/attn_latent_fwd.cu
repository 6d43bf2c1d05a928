// Latent attention, expanded form, over packed sequences:
//   S = scale (Q_nope K_h^T + Q_rope K_rope^T) [+ causal mask],  O = softmax(S) V
// with 192 values of a query, 128 of a head's own keys, 64 of the key part
// that all heads share, and 128 of a value.  The keys are never put together
// in memory: a tile's three 64-value panels in shared memory come from two
// tensors.
//
// A CTA takes 256 query rows of one head of one sequence, 12 warps:
//   warps 0-3, 4-7  softmax of Q tile t (128 rows), one thread to a row
//   warp  8         issues the products
//   warp  9         copies Q and, panel by panel through a ring of eight,
//                   K_0, V_0, K_1, V_1, .. (128 keys; 3 and 2 panels)
// S_t = Q_t K_j^T and O_t += P_t V_j accumulate in tensor memory (128 columns
// of fp32 each); the softmax group overwrites S_t with P_t.  While one group
// works on its tile, the tensor cores work on the other's.  Units are blocks
// of the grid: the hardware deals them out, the heaviest of some heads first,
// heads together whose keys the L2 holds.
//
// What bounds it: the round from a tile's scores over its weights to its
// products; the tensor cores would take 2560 clocks for two tiles of scores,
// which take 3500, and are active for 61% of the time.  Two sequences of 4096
// tokens, 32 heads, causal: 242 us a call in bursts of eight, at 2070 MHz, 1.42
// PFLOP/s; 259 to 266 back to back, which keeps the GPU at its power limit
// (1.79 to 1.84 GHz).  (Timed without them, the exponentials cost nothing, the
// sum of the weights as rounded 11 us: it stays, since with a reference up to
// 2^8 below a row's maximum the rounding of one large weight would show.  Two
// warps to a row's keys, sixteen in all: 370 us.)  One sequence of 300 tokens,
// 8 heads: 10.3 us, the chain of a launch and of three tiles.
#include "latent.h"

#include "attn_kv8_common.cuh"
#include "latent_seq.cuh"
#include "mma_issue.cuh"

namespace attn {

namespace {

constexpr int kRows = 128, kKeys = 128, kUnitRows = 2 * kRows;
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // 256 * 216 + 128 * 72 = 384 * 168
constexpr int kPanel = 128 * 128;                   // 128 rows of 64 values
constexpr int kQPanels = 3, kKPanels = 3, kVPanels = 2, kSlots = 8;
constexpr int kCtl = 1024, kQOff = kCtl, kRingOff = kQOff + 2 * kQPanels * kPanel;
constexpr int kSmem = kRingOff + kSlots * kPanel + 1024;  // +1 KiB for alignment
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kTmO = 256;  // O_t at kTmO + t * 128; S_t at t * 128

enum : uint32_t { SITE_LF_EMPTY = 90, SITE_LF_FULL = 91, SITE_LF_Q = 92, SITE_LF_S = 93, SITE_LF_P = 94, SITE_LF_O = 95 };

struct FwdCtl {
    uint64_t k_full[2], v_full[2], empty[kSlots];  // of even and of odd tiles; of each panel's slot
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], mma_done;
    uint32_t tmem_base, abort;
};
static_assert(sizeof(FwdCtl) <= kCtl, "control block");

// p = 2^(s * c - m) for the 128 scores of a row, rounded to T into the first 64
// tensor-memory columns at tS (asynchronous stores).  Returns the sum of p and
// the sum of p as rounded.
template <typename T>
__device__ __forceinline__ float2 store_weights(const uint32_t (&s)[128], float c, float m, uint32_t tS)
{
    const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
    float2 l[2];
    float lr[4] = {0.f, 0.f, 0.f, 0.f};
    l[0] = l[1] = make_float2(0.f, 0.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int e = 64 * h + 2 * i;
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, m2);
            const float2 v = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            l[i & 1] = __fadd2_rn(l[i & 1], v);
            pk[i] = Pair<T>::put(v.x, v.y);
            lr[i & 3] = add_halves<T>(pk[i], lr[i & 3]);
        }
        tmem_st32(tS + 32 * h, pk);
    }
    const float2 a = __fadd2_rn(l[0], l[1]);
    return make_float2(a.x + a.y, (lr[0] + lr[1]) + (lr[2] + lr[3]));
}

template <typename T, bool CAUSAL>
__global__ void __launch_bounds__(kThreads, 1)
    attn_latent_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ LatentFwdParams p)
{
    constexpr bool BF16 = Elem<T>::BF16;
    constexpr uint32_t IDESC_QK = idesc_f16(kRows, kKeys, BF16, false);
    constexpr uint32_t IDESC_PV = idesc_f16(kRows, 128, BF16, true), IDESC_PV_HALF = idesc_f16(kRows, 64, BF16, true);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    FwdCtl *ctl = reinterpret_cast<FwdCtl *>(smem);
    const uint32_t sQ = base + kQOff, sRing = base + kRingOff;
    auto B = [&](const uint64_t &bar) { return smem_addr(&bar); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmR);
        tma_prefetch_desc(&tmV);
    }
    await_previous();
    const LatentCu cu = latent_cu(p.s);  // in its memory's time, what follows
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(B(ctl->empty[i]), 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(B(ctl->k_full[t]), 1);
            mbar_init(B(ctl->v_full[t]), 1);
            mbar_init(B(ctl->q_full[t]), 1);
            mbar_init(B(ctl->s_full[t]), 1);
            mbar_init(B(ctl->p_full[t]), 4);
            mbar_init(B(ctl->o_full[t]), 1);
        }
        mbar_init(B(ctl->mma_done), 1);
        ctl->abort = 0u;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_addr(&ctl->tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const auto done = [&]() {
        if (warp == 8) tmem_dealloc(tmem, 512);
    };

    // rows row0 .. of sequence seq: heads of a group together, heaviest blocks first
    const LatentUnit un = latent_unit<kUnitRows, false>(p.s, cu, blockIdx.x, p.slots, p.group);
    if (un.row0 >= un.sq) return done();
    const int last = min(un.row0 + kUnitRows, un.sq) - 1;
    const int kend = CAUSAL ? max(min(un.sk, last + 1 + un.sk - un.sq), 0) : un.sk;
    const int n = (kend + kKeys - 1) / kKeys;
    const bool two = un.row0 + kRows < un.sq;  // Q tile 1 has rows
    if (!ATTN_OPS_IN_BOUNDS(un.head < p.s.h && un.q0 + un.sq <= p.s.total_q && un.k0 + un.sk <= p.s.total_k, p.s, SITE_OPS_UNIT)) return done();
    if (n == 0) {  // rows that see no key
        for (int i = threadIdx.x; i < kUnitRows * (kLatentValue / 8); i += kThreads) {
            const int r = un.row0 + i / (kLatentValue / 8);
            if (r >= un.sq) break;
            reinterpret_cast<uint4 *>(static_cast<T *>(p.o) + (un.q0 + r) * p.ot + un.head * p.oh)[i % (kLatentValue / 8)] =
                make_uint4(0u, 0u, 0u, 0u);
        }
        for (int r = un.row0 + threadIdx.x; p.lse && r <= last; r += kThreads)
            p.lse[static_cast<int64_t>(un.head) * p.s.total_q + un.q0 + r] = -INFINITY;
        return done();
    }
    BoundedWaits waits{&ctl->abort, p.s.status, p.s.timeout_ns};

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9) {
            // -------------------------------------------------------- copies
            const uint64_t pol = l2_evict_normal();
            uint32_t np = 0u;
            bool ok = true;
            // the first panel of a tile announces the bytes of all of them
            auto panel = [&](const CUtensorMap *map, uint32_t bar, int first_of, int c0, int c1, int tok) {
                const uint32_t st = np % kSlots;
                if (ok) ok = waits.warp(B(ctl->empty[st]), ((np / kSlots) & 1u) ^ 1u, SITE_LF_EMPTY);
                if (!ok) return;
                if (elect_one()) {
                    if (first_of > 0) mbar_arrive_expect_tx(bar, first_of * kPanel);
                    tma_load_3d(sRing + st * kPanel, map, bar, c0, c1, tok, pol);
                }
                __syncwarp();
                ++np;
            };
            auto q_tile = [&](int t) {
                if (elect_one()) {
                    mbar_arrive_expect_tx(B(ctl->q_full[t]), kQPanels * kPanel);
                    for (int pn = 0; pn < kQPanels; ++pn)
                        tma_load_3d(sQ + (t * kQPanels + pn) * kPanel, &tmQ, B(ctl->q_full[t]), pn * 64, un.head,
                                    un.q0 + un.row0 + t * kRows, pol);
                }
                __syncwarp();
            };
            q_tile(0);
            int j = 0;
            for (; ok && j < n; ++j) {
                const int tok = un.k0 + j * kKeys;
                const uint32_t kb = B(ctl->k_full[j & 1]), vb = B(ctl->v_full[j & 1]);
                panel(&tmK, kb, kKPanels, 0, un.head, tok);
                panel(&tmK, kb, 0, 64, un.head, tok);
                panel(&tmR, kb, 0, 0, 0, tok);
                if (j == 0 && two) q_tile(1);
                panel(&tmV, vb, kVPanels, 0, un.head, tok);
                panel(&tmV, vb, 0, 64, un.head, tok);
            }
            // wait (bounded) for the last copies, so that none lands after the CTA
            for (int k = max(j - 2, 0); k < j; ++k) {
                drain_wait(B(ctl->k_full[k & 1]), (k >> 1) & 1u, p.s.timeout_ns);
                drain_wait(B(ctl->v_full[k & 1]), (k >> 1) & 1u, p.s.timeout_ns);
            }
            drain_wait(B(ctl->q_full[0]), 0u, p.s.timeout_ns);
            if (two) drain_wait(B(ctl->q_full[1]), 0u, p.s.timeout_ns);
        } else if (warp == 8) {
            const uint32_t leader = issuing_lane();
            // -------------------------------------------------------- products
            bool ok = true;
            const uint32_t dq = desc_lo(sQ, 16), dk = desc_lo(sRing, 16), dv = desc_lo(sRing, kPanel);
            // K_j's panels are numbers 5 j .. 5 j + 2, V_j's 5 j + 3 and 5 j + 4
            auto let_go = [&](uint32_t panel) { tc_commit_by(leader, B(ctl->empty[panel % kSlots])); };
            auto issue_qk = [&](int t, uint32_t first, bool final) {
#pragma unroll
                for (int kk = 0; kk < 12; ++kk) {  // 16 values a step
                    mma_ss_by(leader, tmem + t * 128, dq + (((t * kQPanels + kk / 4) * kPanel + (kk % 4) * 32) >> 4),
                              dk + ((((first + kk / 4) % kSlots) * kPanel + (kk % 4) * 32) >> 4), IDESC_QK, kk > 0 ? 1u : 0u);
                    if (kk % 4 == 3 && final) let_go(first + kk / 4);
                }
                tc_commit_by(leader, B(ctl->s_full[t]));
            };
            auto issue_pv = [&](int t, uint32_t first, bool accumulate) {
                const uint32_t o = tmem + kTmO + t * 128, pt = tmem + t * 128, v = first % kSlots;
                if (v + 1u < kSlots) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // 16 keys a step
                        mma_ts_by(leader, o, pt + kk * 8, dv + ((v * kPanel + kk * 2048) >> 4), IDESC_PV, (accumulate || kk > 0) ? 1u : 0u);
                } else {  // the ring's last slot and its first, a panel at a time
#pragma unroll 1
                    for (uint32_t pn = 0; pn < 2; ++pn)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ts_by(leader, o + pn * 64, pt + kk * 8, dv + ((((v + pn) % kSlots) * kPanel + kk * 2048) >> 4), IDESC_PV_HALF,
                                      (accumulate || kk > 0) ? 1u : 0u);
                }
            };
            ok = waits.warp(B(ctl->q_full[0]), 0u, B(ctl->k_full[0]), 0u, SITE_LF_Q);
            if (ok) {
                tc_fence_after();
                issue_qk(0, 0u, !two);
            }
            if (ok && two) {
                ok = waits.warp(B(ctl->q_full[1]), 0u, SITE_LF_Q);
                tc_fence_after();
                if (ok) issue_qk(1, 0u, true);
            }
            for (int j = 0; ok && j < n; ++j) {
                const uint32_t vs = 5u * j + 3u, ks = vs + 2u, par = j & 1u;
                const bool more = j + 1 < n;
                if (!(ok = waits.warp(B(ctl->v_full[par]), (j >> 1) & 1u, SITE_LF_FULL))) break;
                // keys past the end of the sequence: their weights are 0, and so must be what they meet
                if (un.sk - j * kKeys < kKeys)
                    for (int pn = 0; pn < kVPanels; ++pn) zero_panel_rows(sRing + ((vs + pn) % kSlots) * kPanel, un.sk - j * kKeys, kKeys);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t == 1 && !two) break;
                    const bool final = t == 1 || !two;  // of the tile's products
                    if (!(ok = waits.warp(B(ctl->p_full[t]), par, SITE_LF_P))) break;
                    tc_fence_after();
                    issue_pv(t, vs, j > 0);
                    if (t == 0 && more && !(ok = waits.warp(B(ctl->k_full[par ^ 1u]), ((j + 1) >> 1) & 1u, SITE_LF_FULL))) break;
                    if (final) let_go(vs), let_go(vs + 1u);
                    if (more) issue_qk(t, ks, final);
                    else tc_commit_by(leader, B(ctl->o_full[t]));
                }
            }
            // every product completes before tensor memory is freed
            tc_commit_by(leader, B(ctl->mma_done));
            __syncwarp();
            drain_wait(B(ctl->mma_done), 0u, p.s.timeout_ns);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<kSoftmaxRegs>();
        const int t = warp >> 2, in_tile = (warp & 3) * 32 + lane;
        if (t == 0 || two) {
            const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lane_off + t * 128, tO = tmem + lane_off + kTmO + t * 128;
            const int row = un.row0 + t * kRows + in_tile;
            // (a scale of 0, or next to it, as the smallest that still turns -inf into -inf)
            const float c = fabsf(p.s.sl2e) < 1e-30f ? 1e-30f : p.s.sl2e;
            const bool neg = c < 0.f;
            const int lim = CAUSAL ? min(row + 1 + un.sk - un.sq, un.sk) : un.sk;  // keys this row sees
            float m = -INFINITY, l = 0.f, lr = 0.f;
            bool ok = true;
            for (int j = 0; j < n; ++j) {
                if (!(ok = waits.warp(B(ctl->s_full[t]), j & 1u, SITE_LF_S))) break;
                tc_fence_after();
                const int vis = lim - j * kKeys;  // columns >= vis are masked
                // (two instances: of one, the compiler makes selects that every tile pays for)
                auto tile = [&](auto masked) __attribute__((always_inline)) {
                    uint32_t s[128];
                    tmem_ld128_wait(tS, s);
                    if constexpr (decltype(masked)::value) mask_columns(s, vis, neg);
                    const float mx = (neg ? row_extreme<true>(s) : row_extreme<false>(s)) * c;
                    const float m_new = fmaxf(m, mx);
                    if (__any_sync(0xffffffffu, m_new > m + 8.f)) {
                        const float f = m_new == m ? 1.f : ex2_approx(m - m_new);
                        if (j > 0) rescale_rows<kLatentValue>(tO, f);
                        l *= f;
                        lr *= f;
                        m = m_new;
                    }
                    const float2 sums = store_weights<T>(s, c, m == -INFINITY ? 0.f : m, tS);
                    l += sums.x;
                    lr += sums.y;
                    warp_announce_tmem(B(ctl->p_full[t]));
                };
                if (__any_sync(0xffffffffu, vis < kKeys)) tile(std::true_type());
                else tile(std::false_type());
            }
            if (ok) ok = waits.warp(B(ctl->o_full[t]), 0u, SITE_LF_O);
            if (ok) {
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / lr;
                if (row < un.sq && p.lse)
                    p.lse[static_cast<int64_t>(un.head) * p.s.total_q + un.q0 + row] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                // 64 columns at a time pass through the warp's rows of the Q tile, whose products are done, so that a
                // store is of 128 bytes of a row
                const uint32_t pass = sQ + t * kQPanels * kPanel + (warp & 3) * 4096;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[64];
                    tmem_ld64_wait(tO + h * 64, o);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = l == 0.f ? 0u : Pair<T>::put(__uint_as_float(o[8 * e + 2 * i]) * inv, __uint_as_float(o[8 * e + 2 * i + 1]) * inv);
                        st_shared_v4(pass + lane * 128 + ((e ^ (lane & 7)) << 4), v[0], v[1], v[2], v[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // rows 4 k .., eight lanes to a row
                        const int r = 4 * k + (lane >> 3), rr = un.row0 + t * kRows + (warp & 3) * 32 + r;
                        const uint4 v = ld_shared_u4(pass + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                        if (rr < un.sq)
                            *reinterpret_cast<uint4 *>(static_cast<T *>(p.o) + (un.q0 + rr) * p.ot + un.head * p.oh + h * 64 + (lane & 7) * 8) = v;
                    }
                    __syncwarp();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, bool CAUSAL>
cudaError_t launch_t(const LatentFwdArgs &a)
{
    auto kern = attn_latent_fwd_kernel<T, CAUSAL>;
    std::atomic<int> &ready = a.attr_ready[(Elem<T>::BF16 ? 2 : 0) + (CAUSAL ? 1 : 0)];
    if (ready.load(std::memory_order_acquire) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    return launch_overlapped(kern, dim3(a.units), kThreads, kSmem, a.stream, a.q, a.k, a.r, a.v, a.p);
}

}  // namespace

cudaError_t launch_latent_fwd(const LatentFwdArgs &a, bool bf16)
{
    if (bf16) return a.p.s.causal ? launch_t<__nv_bfloat16, true>(a) : launch_t<__nv_bfloat16, false>(a);
    return a.p.s.causal ? launch_t<__half, true>(a) : launch_t<__half, false>(a);
}

}  // namespace attn
