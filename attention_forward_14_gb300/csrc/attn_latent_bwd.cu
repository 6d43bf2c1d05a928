// Gradients of the expanded form of latent attention (attn_latent_fwd.cu),
// for the gradient dO of its outputs:
//   P = exp(scale S - LSE),  D = rowsum(dO * O),  dS = P * (dO V^T - D)
//   dV = P^T dO,  dQ = scale dS [K_nope | K_rope],
//   dK_nope = scale dS^T Q_nope,  dK_rope = scale sum over heads of dS^T Q_rope
//
// Three launches, in which every sum is added up in a fixed order:
//   D of every row;
//   the units of keys, and behind them those of queries, which fill the SMs
//   that the last of keys leave;
//   the sum over the heads of the shared key part's gradient.
// A unit of keys (dK, dV) is 128 keys of one head, to which the queries that
// see them are streamed, 64 at a time.  Keys are the lanes of tensor memory:
// S^T and dP^T (64 columns each), whose places P^T and dS^T take as 16-bit
// operands, the sums dV (128 columns) and dK (192), and V as an operand (64):
// all 512.  A head's share of the shared key part's gradient is written in
// fp32.
// A unit of queries (dQ) is 128 queries of one head, to which the keys that
// they see are streamed, 64 at a time: S (64 columns), two tiles' dP (64
// each), whose places dS takes, the sum dQ (192), and Q as an operand (96).
// It computes S and dP again: 38% more products than one pass would take.  One
// pass over keys has no room in tensor memory for a running dQ beside dK's 192
// columns; it would add up each tile's in global memory, in an order that is
// not fixed or that units wait for.  That pass has not been built and measured
// here; two give equal calls equal bits without either.
// In both, the softmax warps work on P while the tensor cores work on the sums
// of the tile before, and on dS while they work on the next tile's scores.
//
// What bounds it: the tensor cores and the round between them and the softmax
// warps.  A tile of a unit of keys takes 1690 clocks, its products 1470; one
// of a unit of queries 1500, its products 1150.  Two sequences of 4096 tokens,
// 32 heads, causal: 864 us a call in bursts of eight (23 of them for D, 13 for
// the sum over heads; the two kinds of units in launches of their own took 512
// and 370), 1.03 PFLOP/s of what one pass needs, 1.43 of what is computed; 920
// to 934 back to back, at the power limit.  4001 packed tokens, 16 heads: 126
// us.  (Persistent CTAs that claim units and bring the next one's operands
// meanwhile took 525 us for dK and dV and 326 for dQ, in two launches.)
#include "latent.h"

#include "attn_kv8_common.cuh"
#include "latent_seq.cuh"
#include "mma_issue.cuh"
#include "tmem_cols.cuh"

namespace attn {

namespace {

constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // 256 * 216 + 128 * 72 = 384 * 168
constexpr int kPanel = 128 * 128;                   // 128 rows of 64 values
constexpr float kLog2e = 1.4426950408889634f;

enum : uint32_t { SITE_LB_EMPTY = 100, SITE_LB_FULL = 101, SITE_LB_KV = 102, SITE_LB_S = 104, SITE_LB_P = 105,
                  SITE_LB_DP = 106, SITE_LB_DS = 107, SITE_LB_ACC = 108 };

// ---------------------------------------------------------------- D

// 16 lanes to a row of a head, eight values each.
template <typename T>
__global__ void __launch_bounds__(256) latent_dsum_kernel(const __grid_constant__ LatentBwdParams p)
{
    await_previous();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const int l = threadIdx.x & 15;
    const int64_t tok = row / p.s.h;
    const int head = static_cast<int>(row - tok * p.s.h);
    float sum = 0.f;
    if (tok < p.s.total_q) {
        const uint4 a = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.o) + tok * p.ot + head * p.oh)[l];
        const uint4 b = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.dout) + tok * p.gt + head * p.gh)[l];
        const float2 x[4] = {Pair<T>::get(a.x), Pair<T>::get(a.y), Pair<T>::get(a.z), Pair<T>::get(a.w)};
        const float2 y[4] = {Pair<T>::get(b.x), Pair<T>::get(b.y), Pair<T>::get(b.z), Pair<T>::get(b.w)};
        sum = dot8(x, y);
    }
    sum = row_sum<16>(sum);
    if (l == 0 && tok < p.s.total_q) p.dsum[static_cast<int64_t>(head) * p.s.total_q + tok] = sum;
}

// log2 of a row's sum of weights; infinite for a row that sees no key, whose weights are 0.
__device__ __forceinline__ float lse_log2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// 32 columns of the accumulator at `taddr`, times `f`, to 16-bit rows: the
// warp's 32 rows pass through 2 KB at `pass` so that a store is of 64 bytes of
// a row.  `row`: where the row of a lane's number begins, or nullptr.
template <typename T, typename F>
__device__ __forceinline__ void store_piece(uint32_t taddr, float f, uint32_t pass, F row)
{
    const int lane = threadIdx.x & 31;
    uint32_t v[32];
    tmem_ld32_wait(taddr, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = Pair<T>::put(__uint_as_float(v[8 * e + 2 * i]) * f, __uint_as_float(v[8 * e + 2 * i + 1]) * f);
        st_shared_v4(pass + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // rows 8 k .., four lanes to a row
        const int r = 8 * k + (lane >> 2);
        const uint4 w = ld_shared_u4(pass + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
        T *to = row(r);
        if (to) reinterpret_cast<uint4 *>(to)[lane & 3] = w;
    }
    __syncwarp();
}

// Row `row` of a panel of 64 values to 32 columns of this thread's lane.
__device__ __forceinline__ void move_panel_row(uint32_t panel, int row, uint32_t taddr)
{
    uint32_t v[32];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint4 x = ld_shared_u4(panel + row * 128 + ((e ^ (row & 7)) << 4));
        v[4 * e] = x.x, v[4 * e + 1] = x.y, v[4 * e + 2] = x.z, v[4 * e + 3] = x.w;
    }
    tmem_st32(taddr, v);
}

// ---------------------------------------------------------------- dK, dV

constexpr int kKeys = 128, kQueries = 64;  // of a unit, of a tile
struct KeysCfg {
    static constexpr int HALF = kQueries * 128;           // a panel of a tile of queries
    static constexpr int STAGE = 5 * HALF, STAGES = 3;    // Q (3 panels), dO (2)
    static constexpr int LD_OFF = 1024;                   // of each stage: -LSE in log2 [64], -D [64]
    static constexpr int K_OFF = 4096, V_OFF = K_OFF + 3 * kPanel, Q_OFF = V_OFF + 2 * kPanel;
    static constexpr int SMEM = Q_OFF + STAGES * STAGE + 1024;
    // P^T and dS^T take the place of S^T and dP^T, each half of the queries that of its own scores
    static constexpr int TM_DV = 0, TM_DK = 128, TM_S = 320, TM_DP = 384, TM_V = 448;
    static_assert(SMEM <= 232448 && LD_OFF + STAGES * 512 <= K_OFF, "shared memory budget");
};

struct KeysCtl {
    uint64_t v_full, k_full, v_moved, full[3], empty[3], ld_full[3];
    uint64_t s_full, dp_full, p_full, ds_full, acc_full;
    uint32_t tmem_base, abort;
};
static_assert(sizeof(KeysCtl) <= KeysCfg::LD_OFF, "control block");

template <typename T, bool CAUSAL>
__device__ __forceinline__ void latent_bwd_keys(const CUtensorMap &tmQ, const CUtensorMap &tmG, const CUtensorMap &tmK, const CUtensorMap &tmR,
                                 const CUtensorMap &tmV, const LatentBwdParams &p, unsigned unit)
{
    using C = KeysCfg;
    constexpr bool BF16 = Elem<T>::BF16;
    constexpr uint32_t IDESC_S = idesc_f16(kKeys, kQueries, BF16, false);
    constexpr uint32_t IDESC_DV = idesc_f16(kKeys, 128, BF16, true), IDESC_DK = idesc_f16(kKeys, 192, BF16, true);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    KeysCtl *ctl = reinterpret_cast<KeysCtl *>(smem);
    auto B = [&](const uint64_t &bar) { return smem_addr(&bar); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const LatentCu cu = latent_cu(p.s);  // in its memory's time, what follows
    if (threadIdx.x == 0) {
        mbar_init(B(ctl->v_full), 1);
        mbar_init(B(ctl->k_full), 1);
        mbar_init(B(ctl->v_moved), 8);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(B(ctl->full[i]), 1);
            mbar_init(B(ctl->empty[i]), 1);
            mbar_init(B(ctl->ld_full[i]), 1);
        }
        mbar_init(B(ctl->s_full), 1);
        mbar_init(B(ctl->dp_full), 1);
        mbar_init(B(ctl->p_full), 8);
        mbar_init(B(ctl->ds_full), 8);
        mbar_init(B(ctl->acc_full), 1);
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

    const LatentUnit un = latent_unit<kKeys, true>(p.s, cu, unit, p.k_slots, p.group);
    if (un.row0 >= un.sk) return done();
    const int key0 = un.row0, off = un.sk - un.sq;  // query i sees keys j <= i + off
    if (!ATTN_OPS_IN_BOUNDS(un.head < p.s.h && un.q0 + un.sq <= p.s.total_q && un.k0 + un.sk <= p.s.total_k, p.s, SITE_OPS_UNIT)) return done();
    const int first = CAUSAL ? max(key0 - off, 0) / kQueries : 0;  // tile of queries
    const int n = max((un.sq + kQueries - 1) / kQueries - first, 0);

    auto dv_row = [&](int key) { return static_cast<T *>(p.dv) + (un.k0 + key) * p.dvt + un.head * p.dvh; };
    auto dkn_row = [&](int key) { return static_cast<T *>(p.dkn) + (un.k0 + key) * p.dknt + un.head * p.dknh; };
    auto dkr_row = [&](int key) { return p.kr_part + (static_cast<int64_t>(un.head) * p.s.total_k + un.k0 + key) * kLatentRope; };
    if (n == 0) {  // keys that no query sees
        for (int i = threadIdx.x; i < kKeys * 16; i += kThreads) {
            const int key = key0 + i / 16, c = i % 16;
            if (key >= un.sk) break;
            reinterpret_cast<uint4 *>(dv_row(key))[c] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4 *>(dkn_row(key))[c] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4 *>(dkr_row(key))[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        return done();
    }
    const BoundedWaits waits{&ctl->abort, p.s.status, p.s.timeout_ns};

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9) {
            // -------------------------------------------------------- copies
            const uint64_t pol = l2_evict_normal();
            if (elect_one()) {
                uint32_t bar = B(ctl->v_full);
                mbar_arrive_expect_tx(bar, 2 * kPanel);
                for (int pn = 0; pn < 2; ++pn) tma_load_3d(base + C::V_OFF + pn * kPanel, &tmV, bar, pn * 64, un.head, un.k0 + key0, pol);
                bar = B(ctl->k_full);
                mbar_arrive_expect_tx(bar, 3 * kPanel);
                tma_load_3d(base + C::K_OFF, &tmK, bar, 0, un.head, un.k0 + key0, pol);
                tma_load_3d(base + C::K_OFF + kPanel, &tmK, bar, 64, un.head, un.k0 + key0, pol);
                tma_load_3d(base + C::K_OFF + 2 * kPanel, &tmR, bar, 0, 0, un.k0 + key0, pol);
            }
            __syncwarp();
            int i = 0;
            for (; i < n; ++i) {
                const uint32_t st = i % C::STAGES, bar = B(ctl->full[st]), at = base + C::Q_OFF + st * C::STAGE;
                const int tok = un.q0 + (first + i) * kQueries;
                if (!waits.warp(B(ctl->empty[st]), ((i / C::STAGES) & 1u) ^ 1u, SITE_LB_EMPTY)) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, C::STAGE);
                    for (int pn = 0; pn < 3; ++pn) tma_load_3d(at + pn * C::HALF, &tmQ, bar, pn * 64, un.head, tok, pol);
                    for (int pn = 0; pn < 2; ++pn) tma_load_3d(at + (3 + pn) * C::HALF, &tmG, bar, pn * 64, un.head, tok, pol);
                }
                __syncwarp();
            }
            // wait (bounded) for the last copies, so that none lands after the CTA
            for (int k = max(i - C::STAGES, 0); k < i; ++k) drain_wait(B(ctl->full[k % C::STAGES]), (k / C::STAGES) & 1u, p.s.timeout_ns);
            drain_wait(B(ctl->v_full), 0u, p.s.timeout_ns);
            drain_wait(B(ctl->k_full), 0u, p.s.timeout_ns);
        } else if (warp == 10) {
            // -------------------------------------------------------- LSE and D of a tile's queries
            const int64_t row0 = static_cast<int64_t>(un.head) * p.s.total_q + un.q0;
            for (int i = 0; i < n; ++i) {
                const uint32_t st = i % C::STAGES;
                if (!waits.warp(B(ctl->empty[st]), ((i / C::STAGES) & 1u) ^ 1u, SITE_LB_EMPTY)) break;
                float *to = reinterpret_cast<float *>(smem + C::LD_OFF + st * 512);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int q = (first + i) * kQueries + h * 32 + lane;
                    to[h * 32 + lane] = q < un.sq ? -lse_log2(p.lse[row0 + q]) : -INFINITY;
                    to[64 + h * 32 + lane] = q < un.sq ? -p.dsum[row0 + q] : 0.f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(B(ctl->ld_full[st]));
            }
        } else if (warp == 8) {
            const uint32_t leader = issuing_lane();
            // -------------------------------------------------------- products
            const uint32_t dk = desc_lo(base + C::K_OFF, 16);
            const uint32_t dq_k = desc_lo(base + C::Q_OFF, 16), dq_mn = desc_lo(base + C::Q_OFF, C::HALF);
            auto stage_full = [&](int i) { return B(ctl->full[i % C::STAGES]); };
            auto stage_parity = [&](int i) { return static_cast<uint32_t>(i / C::STAGES) & 1u; };
            auto clean = [&](int i) {
                const uint32_t st = i % C::STAGES;
                // queries past the end of the sequence: their weights are 0, and so must be what they meet
                const int valid = un.sq - (first + i) * kQueries;
                if (valid < kQueries)
                    for (int pn = 0; pn < 5; ++pn) zero_panel_rows(base + C::Q_OFF + st * C::STAGE + pn * C::HALF, valid, kQueries);
                tc_fence_after();
            };
            auto issue_s = [&](uint32_t st) {
#pragma unroll
                for (int kk = 0; kk < 12; ++kk)
                    mma_ss_by(leader, tmem + C::TM_S, dk + (((kk / 4) * kPanel + (kk % 4) * 32) >> 4),
                           dq_k + ((st * C::STAGE + (kk / 4) * C::HALF + (kk % 4) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
                tc_commit_by(leader, B(ctl->s_full));
            };
            auto issue_dp = [&](uint32_t st) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ts_by(leader, tmem + C::TM_DP, tmem + C::TM_V + kk * 8,
                           dq_k + ((st * C::STAGE + (3 + kk / 4) * C::HALF + (kk % 4) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
                tc_commit_by(leader, B(ctl->dp_full));
            };
            // k-step kk of a tile's queries, 16 of them, in P^T or dS^T: 32 queries to each half
            auto at_step = [](int kk) { return (kk / 2) * 32 + (kk % 2) * 8; };
            bool ok = waits.warp(B(ctl->k_full), 0u, stage_full(0), 0u, SITE_LB_KV);
            if (ok) {
                clean(0);
                issue_s(0u);
                ok = waits.warp(B(ctl->v_moved), 0u, SITE_LB_KV);
                tc_fence_after();
                if (ok) issue_dp(0u);
            }
            for (int i = 0; ok && i < n; ++i) {
                const uint32_t st = i % C::STAGES, next = (i + 1) % C::STAGES;
                const bool more = i + 1 < n;
                ok = more ? waits.warp(B(ctl->p_full), i & 1u, stage_full(i + 1), stage_parity(i + 1), SITE_LB_P)
                          : waits.warp(B(ctl->p_full), i & 1u, SITE_LB_P);
                if (!ok) break;
                if (more) clean(i + 1);
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 16 queries a step
                    mma_ts_by(leader, tmem + C::TM_DV, tmem + C::TM_S + at_step(kk), dq_mn + ((st * C::STAGE + 3 * C::HALF + kk * 2048) >> 4), IDESC_DV,
                           (i > 0 || kk > 0) ? 1u : 0u);
                if (more) issue_s(next);
                if (!(ok = waits.warp(B(ctl->ds_full), i & 1u, SITE_LB_DS))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts_by(leader, tmem + C::TM_DK, tmem + C::TM_DP + at_step(kk), dq_mn + ((st * C::STAGE + kk * 2048) >> 4), IDESC_DK,
                           (i > 0 || kk > 0) ? 1u : 0u);
                tc_commit_by(leader, B(ctl->empty[st]));
                if (more) issue_dp(next);
            }
            // every product completes before the sums are read and tensor memory is freed
            tc_commit_by(leader, B(ctl->acc_full));
            __syncwarp();
            drain_wait(B(ctl->acc_full), 0u, p.s.timeout_ns);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ P^T and dS^T: a key to a thread, half of the queries
        regs_inc<kSoftmaxRegs>();
        const int w = warp >> 2, in_unit = (warp & 3) * 32 + lane, key = key0 + in_unit;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16, at = tmem + lane_off;
        // the keys' values as an operand in tensor memory, half of them by each group
        bool ok = waits.warp(B(ctl->v_full), 0u, SITE_LB_KV);
        if (ok) {
            move_panel_row(base + C::V_OFF + w * kPanel, in_unit, at + C::TM_V + w * 32);
            warp_announce_tmem(B(ctl->v_moved));
        }
        for (int i = 0; ok && i < n; ++i) {
            const uint32_t st = i % C::STAGES;
            const float *ld = reinterpret_cast<const float *>(smem + C::LD_OFF + st * 512) + w * 32;
            const int q0 = (first + i) * kQueries + w * 32;
            ok = waits.warp(B(ctl->ld_full[st]), (i / C::STAGES) & 1u, B(ctl->s_full), i & 1u, SITE_LB_S);
            if (!ok) break;
            tc_fence_after();
            // queries [lo, hi) of the 32 see this key
            const int lo = CAUSAL ? key - off - q0 : 0, hi = un.sq - q0;
            // (two instances: of one, the compiler makes selects that every tile pays for, a third of the instructions)
            auto tile = [&](auto masked) __attribute__((always_inline)) {
                constexpr bool MASKED = decltype(masked)::value;
                const float2 scale2 = make_float2(p.s.sl2e, p.s.sl2e);
                float2 pr[16];
                uint32_t s[32], pk[16];
                tmem_ld32_wait(at + C::TM_S + w * 32, s);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2,
                                                reinterpret_cast<const float2 *>(ld)[c]);
                    pr[c] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    if constexpr (MASKED) {
                        pr[c].x = 2 * c >= lo && 2 * c < hi ? pr[c].x : 0.f;
                        pr[c].y = 2 * c + 1 >= lo && 2 * c + 1 < hi ? pr[c].y : 0.f;
                    }
                    pk[c] = Pair<T>::put(pr[c].x, pr[c].y);
                }
                tmem_st16(at + C::TM_S + w * 32, pk);
                warp_announce_tmem(B(ctl->p_full));
                if (!(ok = waits.warp(B(ctl->dp_full), i & 1u, SITE_LB_DP))) return;
                tc_fence_after();
                tmem_ld32_wait(at + C::TM_DP + w * 32, s);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    float2 x = __fmul2_rn(pr[c], __fadd2_rn(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])),
                                                            reinterpret_cast<const float2 *>(ld + 64)[c]));
                    if constexpr (MASKED) {  // (a masked dP may be anything)
                        x.x = 2 * c >= lo && 2 * c < hi ? x.x : 0.f;
                        x.y = 2 * c + 1 >= lo && 2 * c + 1 < hi ? x.y : 0.f;
                    }
                    pk[c] = Pair<T>::put(x.x, x.y);
                }
                tmem_st16(at + C::TM_DP + w * 32, pk);
                warp_announce_tmem(B(ctl->ds_full));
            };
            if (__any_sync(0xffffffffu, lo > 0 || hi < 32)) tile(std::true_type());
            else tile(std::false_type());
            if (!ok) break;
        }
        if (ok) ok = waits.warp(B(ctl->acc_full), 0u, SITE_LB_ACC);
        if (ok) {
            tc_fence_after();
            // ten pieces of 32 columns: dV 0..3, dK_nope 4..7, the key part 8, 9; the keys' tile is not needed any more
            const uint32_t pass = base + C::K_OFF + warp * 4096;
            const int warp_key = key0 + (warp & 3) * 32;
#pragma unroll 1
            for (int piece = w; piece < 10; piece += 2) {
                if (piece < 4) {
                    store_piece<T>(at + C::TM_DV + piece * 32, 1.f, pass,
                                   [&](int r) { return warp_key + r < un.sk ? dv_row(warp_key + r) + piece * 32 : nullptr; });
                } else if (piece < 8) {
                    store_piece<T>(at + C::TM_DK + (piece - 4) * 32, p.s.scale, pass,
                                   [&](int r) { return warp_key + r < un.sk ? dkn_row(warp_key + r) + (piece - 4) * 32 : nullptr; });
                } else {
                    uint32_t v[32];
                    tmem_ld32_wait(at + C::TM_DK + 128 + (piece - 8) * 32, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = __float_as_uint(__uint_as_float(v[4 * e + k]) * p.s.scale);
                        st_shared_v4(pass + lane * 128 + ((e ^ (lane & 7)) << 4), x[0], x[1], x[2], x[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // rows 4 k .., eight lanes to a row
                        const int r = 4 * k + (lane >> 3);
                        const uint4 x = ld_shared_u4(pass + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                        if (warp_key + r < un.sk) reinterpret_cast<uint4 *>(dkr_row(warp_key + r) + (piece - 8) * 32)[lane & 7] = x;
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

// ---------------------------------------------------------------- dQ

struct QueriesCfg {
    static constexpr int TILE = 64;                       // keys
    static constexpr int HALF = TILE * 128;               // a panel of a tile of keys
    static constexpr int STAGE = 5 * HALF, STAGES = 4;    // K (3 panels), V (2)
    static constexpr int G_OFF = 1024, KV_OFF = G_OFF + 2 * kPanel;
    // Q's three panels pass through the last stage, and what is behind it, on their way to tensor memory
    static constexpr int Q_OFF = KV_OFF + (STAGES - 1) * STAGE;
    static constexpr int SMEM = Q_OFF + 3 * kPanel + 1024;
    // dS takes the place of dP, each half of the keys that of its own; two tiles' dP
    static constexpr int TM_DQ = 0, TM_S = 192, TM_DP = 256, TM_Q = 384;
    static_assert(3 * kPanel >= STAGE && SMEM <= 232448, "shared memory budget");
};

struct QueriesCtl {
    uint64_t q_full, g_full, q_moved, full[4], empty[4];
    // (of dP and dS one for each of the two tiles: a tile's dP may be there
    // before the slowest warp has looked for that of the tile before, and one
    // barrier's phase would then be the other again)
    uint64_t s_full, s_free, dp_full[2], ds_full[2], acc_full;
    uint32_t tmem_base, abort;
};
static_assert(sizeof(QueriesCtl) <= QueriesCfg::G_OFF, "control block");

template <typename T, bool CAUSAL>
__device__ __forceinline__ void latent_bwd_queries(const CUtensorMap &tmQ, const CUtensorMap &tmG, const CUtensorMap &tmK, const CUtensorMap &tmR,
                                    const CUtensorMap &tmV, const LatentBwdParams &p, unsigned unit)
{
    using C = QueriesCfg;
    constexpr int ROWS = 128, TILE = C::TILE;
    constexpr bool BF16 = Elem<T>::BF16;
    constexpr uint32_t IDESC_S = idesc_f16(ROWS, TILE, BF16, false), IDESC_DQ = idesc_f16(ROWS, 192, BF16, true);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    QueriesCtl *ctl = reinterpret_cast<QueriesCtl *>(smem);
    auto B = [&](const uint64_t &bar) { return smem_addr(&bar); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const LatentCu cu = latent_cu(p.s);  // in its memory's time, what follows
    if (threadIdx.x == 0) {
        mbar_init(B(ctl->q_full), 1);
        mbar_init(B(ctl->g_full), 1);
        mbar_init(B(ctl->q_moved), 8);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(B(ctl->full[i]), 1);
            mbar_init(B(ctl->empty[i]), 1);
        }
        mbar_init(B(ctl->s_full), 1);
        mbar_init(B(ctl->s_free), 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(B(ctl->dp_full[i]), 1);
            mbar_init(B(ctl->ds_full[i]), 8);
        }
        mbar_init(B(ctl->acc_full), 1);
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

    const LatentUnit un = latent_unit<ROWS, false>(p.s, cu, unit, p.q_slots, p.group);
    if (un.row0 >= un.sq) return done();
    if (!ATTN_OPS_IN_BOUNDS(un.head < p.s.h && un.q0 + un.sq <= p.s.total_q && un.k0 + un.sk <= p.s.total_k, p.s, SITE_OPS_UNIT)) return done();
    const int last = min(un.row0 + ROWS, un.sq) - 1;
    const int kend = CAUSAL ? max(min(un.sk, last + 1 + un.sk - un.sq), 0) : un.sk;
    const int n = (kend + TILE - 1) / TILE;
    auto dq_row = [&](int q) { return static_cast<T *>(p.dq) + (un.q0 + q) * p.dqt + un.head * p.dqh; };
    if (n == 0) {  // rows that see no key
        for (int i = threadIdx.x; i < ROWS * (kLatentKey / 8); i += kThreads) {
            const int q = un.row0 + i / (kLatentKey / 8);
            if (q >= un.sq) break;
            reinterpret_cast<uint4 *>(dq_row(q))[i % (kLatentKey / 8)] = make_uint4(0u, 0u, 0u, 0u);
        }
        return done();
    }
    const BoundedWaits waits{&ctl->abort, p.s.status, p.s.timeout_ns};

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9) {
            // -------------------------------------------------------- copies: Q, dO, the keys and values
            const uint64_t pol = l2_evict_normal();
            const int tok = un.q0 + un.row0;
            if (elect_one()) {
                uint32_t bar = B(ctl->q_full);
                mbar_arrive_expect_tx(bar, 3 * kPanel);
                for (int pn = 0; pn < 3; ++pn) tma_load_3d(base + C::Q_OFF + pn * kPanel, &tmQ, bar, pn * 64, un.head, tok, pol);
            }
            __syncwarp();
            int j = 0;
            for (; j < n; ++j) {
                const uint32_t st = j % C::STAGES, bar = B(ctl->full[st]), at = base + C::KV_OFF + st * C::STAGE;
                const int key = un.k0 + j * TILE;
                if (j == C::STAGES - 1 && !waits.warp(B(ctl->q_moved), 0u, SITE_LB_KV)) break;
                if (!waits.warp(B(ctl->empty[st]), ((j / C::STAGES) & 1u) ^ 1u, SITE_LB_EMPTY)) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, C::STAGE);
                    for (int pn = 0; pn < 2; ++pn) tma_load_3d(at + pn * C::HALF, &tmK, bar, pn * 64, un.head, key, pol);
                    tma_load_3d(at + 2 * C::HALF, &tmR, bar, 0, 0, key, pol);
                    for (int pn = 0; pn < 2; ++pn) tma_load_3d(at + (3 + pn) * C::HALF, &tmV, bar, pn * 64, un.head, key, pol);
                    if (j == 0) {
                        mbar_arrive_expect_tx(B(ctl->g_full), 2 * kPanel);
                        for (int pn = 0; pn < 2; ++pn)
                            tma_load_3d(base + C::G_OFF + pn * kPanel, &tmG, B(ctl->g_full), pn * 64, un.head, tok, pol);
                    }
                }
                __syncwarp();
            }
            // wait (bounded) for the last copies, so that none lands after the CTA
            for (int k = max(j - C::STAGES, 0); k < j; ++k) drain_wait(B(ctl->full[k % C::STAGES]), (k / C::STAGES) & 1u, p.s.timeout_ns);
            drain_wait(B(ctl->q_full), 0u, p.s.timeout_ns);
            if (j > 0) drain_wait(B(ctl->g_full), 0u, p.s.timeout_ns);
        } else if (warp == 8) {
            const uint32_t leader = issuing_lane();
            // -------------------------------------------------------- products
            const uint32_t dg = desc_lo(base + C::G_OFF, 16), dkv = desc_lo(base + C::KV_OFF, 16);
            const uint32_t dk_mn = desc_lo(base + C::KV_OFF, C::HALF);
            auto scores = [&](int j) {  // S and dP of tile j
                const uint32_t st = j % C::STAGES, kv = dkv + ((st * C::STAGE) >> 4);
                const uint32_t full = B(ctl->full[st]), par = (j / C::STAGES) & 1u;
                // the scores of the tile before have been read
                if (!(j > 0 ? waits.warp(full, par, B(ctl->s_free), (j - 1) & 1u, SITE_LB_FULL) : waits.warp(full, par, SITE_LB_FULL)))
                    return false;
                // keys past the end of the sequence: dS is 0 there, and so must be what it meets
                if (un.sk - j * TILE < TILE)
                    for (int pn = 0; pn < 3; ++pn)
                        zero_panel_rows(base + C::KV_OFF + st * C::STAGE + pn * C::HALF, un.sk - j * TILE, TILE);
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 12; ++kk)
                    mma_ts_by(leader, tmem + C::TM_S, tmem + C::TM_Q + kk * 8, kv + (((kk / 4) * C::HALF + (kk % 4) * 32) >> 4), IDESC_S,
                           kk > 0 ? 1u : 0u);
                tc_commit_by(leader, B(ctl->s_full));
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss_by(leader, tmem + C::TM_DP + (j & 1) * 64, dg + (((kk / 4) * kPanel + (kk % 4) * 32) >> 4),
                           kv + (((3 + kk / 4) * C::HALF + (kk % 4) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
                tc_commit_by(leader, B(ctl->dp_full[j & 1]));
                return true;
            };
            bool ok = waits.warp(B(ctl->q_moved), 0u, SITE_LB_KV) && waits.warp(B(ctl->g_full), 0u, SITE_LB_KV) && scores(0);
            for (int j = 0; ok && j < n; ++j) {
                if (j + 1 < n && !(ok = scores(j + 1))) break;
                if (!(ok = waits.warp(B(ctl->ds_full[j & 1]), (j >> 1) & 1u, SITE_LB_DS))) break;
                tc_fence_after();
                {
                    const uint32_t st = j % C::STAGES;
#pragma unroll
                    for (int kk = 0; kk < TILE / 16; ++kk)  // 16 keys a step, 32 to each half
                        mma_ts_by(leader, tmem + C::TM_DQ, tmem + C::TM_DP + (j & 1) * 64 + (kk / 2) * 32 + (kk % 2) * 8,
                               dk_mn + ((st * C::STAGE + kk * 2048) >> 4), IDESC_DQ, (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit_by(leader, B(ctl->empty[st]));
                }
            }
            tc_commit_by(leader, B(ctl->acc_full));
            __syncwarp();
            drain_wait(B(ctl->acc_full), 0u, p.s.timeout_ns);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ dS: a query to a thread, half of the keys
        regs_inc<kSoftmaxRegs>();
        const int w = warp >> 2, in_unit = (warp & 3) * 32 + lane, q = un.row0 + in_unit;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16, at = tmem + lane_off;
        const int64_t stat = static_cast<int64_t>(un.head) * p.s.total_q + un.q0 + q;
        const float lse = q < un.sq ? lse_log2(p.lse[stat]) : INFINITY, d = q < un.sq ? p.dsum[stat] : 0.f;
        const int lim = CAUSAL ? min(q + 1 + un.sk - un.sq, un.sk) : un.sk;
        const float2 scale2 = make_float2(p.s.sl2e, p.s.sl2e), lse2 = make_float2(-lse, -lse), d2 = make_float2(-d, -d);
        // Q as an operand in tensor memory
        bool ok = waits.warp(B(ctl->q_full), 0u, SITE_LB_KV);
        if (ok) {
            for (int pn = w; pn < 3; pn += 2) move_panel_row(base + C::Q_OFF + pn * kPanel, in_unit, at + C::TM_Q + pn * 32);
            warp_announce_tmem(B(ctl->q_moved));
        }
        for (int j = 0; ok && j < n; ++j) {
            if (!(ok = waits.warp(B(ctl->s_full), j & 1u, SITE_LB_S))) break;
            tc_fence_after();
            const int vis = lim - j * TILE - w * 32;  // columns >= vis are masked
            auto tile = [&](auto masked) __attribute__((always_inline)) {
                uint32_t s[32], pk[16];
                tmem_ld32_wait(at + C::TM_S + w * 32, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B(ctl->s_free));
                float2 pr[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, lse2);
                    pr[c] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                }
                if (!(ok = waits.warp(B(ctl->dp_full[j & 1]), (j >> 1) & 1u, SITE_LB_DP))) return;
                tc_fence_after();
                const uint32_t tDP = at + C::TM_DP + (j & 1) * 64 + w * 32;
                tmem_ld32_wait(tDP, s);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    float2 x = __fmul2_rn(pr[c], __fadd2_rn(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), d2));
                    if constexpr (decltype(masked)::value) {
                        x.x = 2 * c < vis ? x.x : 0.f;
                        x.y = 2 * c + 1 < vis ? x.y : 0.f;
                    }
                    pk[c] = Pair<T>::put(x.x, x.y);
                }
                tmem_st16(tDP, pk);
                warp_announce_tmem(B(ctl->ds_full[j & 1]));
            };
            if (__any_sync(0xffffffffu, vis < 32)) tile(std::true_type());
            else tile(std::false_type());
        }
        if (ok) ok = waits.warp(B(ctl->acc_full), 0u, SITE_LB_ACC);
        if (ok) {
            tc_fence_after();
            const uint32_t pass = base + C::G_OFF + warp * 4096;  // dO's rows are not needed any more
            const int warp_q = un.row0 + (warp & 3) * 32;
#pragma unroll 1
            for (int piece = w; piece < 6; piece += 2)
                store_piece<T>(at + C::TM_DQ + piece * 32, p.s.scale, pass,
                               [&](int r) { return warp_q + r < un.sq ? dq_row(warp_q + r) + piece * 32 : nullptr; });
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Both: the units of keys, and behind them those of queries, which fill the SMs that the last of keys leave.
template <typename T, bool CAUSAL>
__global__ void __launch_bounds__(kThreads, 1)
    latent_bwd_kernel(const __grid_constant__ LatentBwdMaps m, const __grid_constant__ LatentBwdParams p, unsigned key_units)
{
    const bool keys = blockIdx.x < key_units;
    if (threadIdx.x == 0)
        for (const CUtensorMap *map : {keys ? &m.q_half : &m.q, keys ? &m.dout_half : &m.dout, keys ? &m.k : &m.k_half,
                                       keys ? &m.r : &m.r_half, keys ? &m.v : &m.v_half})
            tma_prefetch_desc(map);
    await_previous();
    if (keys)
        latent_bwd_keys<T, CAUSAL>(m.q_half, m.dout_half, m.k, m.r, m.v, p, blockIdx.x);
    else
        latent_bwd_queries<T, CAUSAL>(m.q, m.dout, m.k_half, m.r_half, m.v_half, p, blockIdx.x - key_units);
}

// ---------------------------------------------------------------- the shared key part

// 16 keys of a sequence to a block: their heads' shares, summed in the heads' order.
template <typename T>
__global__ void __launch_bounds__(256) latent_rope_sum_kernel(const __grid_constant__ LatentBwdParams p)
{
    await_previous();
    const LatentUnit un = latent_slot<kKeys, true>(p.s, latent_cu(p.s), blockIdx.x / 8);
    const int key = un.row0 + (blockIdx.x % 8) * 16 + (threadIdx.x >> 4), c = threadIdx.x & 15, k0 = un.k0;
    if (key >= un.sk) return;
    const float4 *x = reinterpret_cast<const float4 *>(p.kr_part + static_cast<int64_t>(k0 + key) * kLatentRope) + c;
    const int64_t step = static_cast<int64_t>(p.s.total_k) * (kLatentRope / 4);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = 0; h < p.s.h; ++h) {
        const float4 v = __ldcs(x + h * step);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    reinterpret_cast<uint2 *>(static_cast<T *>(p.dkr) + (k0 + key) * p.dkrt)[c] =
        make_uint2(Pair<T>::put(sum.x, sum.y), Pair<T>::put(sum.z, sum.w));
}

template <typename K>
cudaError_t opt_in(std::atomic<int> &ready, K kernel, int smem)
{
    if (ready.load(std::memory_order_acquire) != 0) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) ready.store(1, std::memory_order_release);
    return e;
}

template <typename T, bool CAUSAL>
cudaError_t launch_t(const LatentBwdArgs &a)
{
    const LatentSeqs &s = a.p.s;
    constexpr int SMEM = KeysCfg::SMEM > QueriesCfg::SMEM ? KeysCfg::SMEM : QueriesCfg::SMEM;
    cudaError_t e = opt_in(a.attr_ready[(Elem<T>::BF16 ? 2 : 0) + (CAUSAL ? 1 : 0)], latent_bwd_kernel<T, CAUSAL>, SMEM);
    const unsigned key_units = static_cast<unsigned>(s.h) * a.p.k_slots, units = key_units + static_cast<unsigned>(s.h) * a.p.q_slots;
    if (e == cudaSuccess && s.total_q > 0)
        e = launch_overlapped(latent_dsum_kernel<T>, dim3(static_cast<unsigned>((static_cast<int64_t>(s.total_q) * s.h + 15) / 16)), 256, 0,
                              a.stream, a.p);
    if (e == cudaSuccess && units > 0)
        e = launch_overlapped(latent_bwd_kernel<T, CAUSAL>, dim3(units), kThreads, SMEM, a.stream, a.maps, a.p, key_units);
    if (e == cudaSuccess && key_units > 0)
        e = launch_overlapped(latent_rope_sum_kernel<T>, dim3(static_cast<unsigned>(a.p.k_slots) * 8), 256, 0, a.stream, a.p);
    return e;
}

}  // namespace

cudaError_t launch_latent_bwd(const LatentBwdArgs &a, bool bf16)
{
    if (bf16) return a.p.s.causal ? launch_t<__nv_bfloat16, true>(a) : launch_t<__nv_bfloat16, false>(a);
    return a.p.s.causal ? launch_t<__half, true>(a) : launch_t<__half, false>(a);
}

}  // namespace attn
