// Latent attention: a token's keys and values are one vector that all heads
// share, [latent (512) | rotated key part (64)].  Parameters and launches of
// the append to its paged cache, of the attention over that cache, and of the
// expanded form (a head's keys are 128 values of its own and the shared 64,
// its values 128) with its gradients.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

constexpr int kLatent = 512, kLatentRope = 64, kLatentToken = kLatent + kLatentRope;

// ---------------------------------------------------------------- append

struct LatentAppendParams {
    const void *x;               // [b, s, 576] by strides (elements)
    int64_t xb, xs;
    void *pool;                  // [num_pages, page_size, 576]
    const void *weight;          // [512] or nullptr: no norm
    const float *cos, *sin;      // [>= capacity, 32], or nullptr: no rotation
    const int32_t *seqlens;      // [b] cached tokens
    const int32_t *new_seqlens;  // [b] new tokens, or nullptr: s
    const int32_t *block_table;  // [b, pages_per_seq]
    uint32_t *status;
    int64_t b, s, num_pages, pages_per_seq;
    int page_size, interleaved;
    float eps;
};

cudaError_t launch_latent_append(const LatentAppendParams &p, bool bf16, cudaStream_t stream);

// ---------------------------------------------------------------- paged attention

// An item that a team of CTAs begins and later teams go on with.
struct alignas(16) LatentCut {
    int32_t parts;  // teams that have a part (0: there is no such item); negated when it is not this team's first
    int32_t entry;  // which item
    int32_t pad[2];
};

enum LatentMask { LATENT_MASK_NONE = 0, LATENT_MASK_CAUSAL = 1, LATENT_MASK_TREE = 2 };

struct LatentPagedParams {
    const void *q;               // [b, h, sq, 576] by strides (elements)
    void *o;                     // [b, h, sq, 512] by strides
    int64_t qb, qh, qs, ob, oh, os;
    float *lse;                  // [b, h, sq] or nullptr
    const uint8_t *pool;         // [num_pages, page_size, 576] (copied through its map, prefetched directly)
    const int32_t *seqlens;      // [b]
    const int32_t *block_table;  // [b, pages_per_seq]
    const int32_t *tree;         // [b, sq, tree_words] or nullptr
    uint32_t *status;
    float *o_part;               // [2 * grid][tile rows][512]: parts of the items that several teams share
    float4 *ml_part;             // [2 * grid][tile rows]: their reference (log2), sum, sum as rounded
    LatentCut *cut;              // [teams]
    float sl2e;                  // scale * log2(e)
    int32_t b, h, sq, rows;      // rows = h * sq, row i * h + head
    int32_t tiles;               // ceil(rows / tile rows)
    int32_t team, groups;        // CTAs that work on the same keys, a tile of rows each; ceil(tiles / team)
    int32_t cap, page_size, pages_per_seq, num_pages;
    int32_t mask, tree_words;
    int32_t box;                 // tokens of a copy: 128, 64, 32 or 16, a divisor of page_size
    uint64_t timeout_ns;
};

// What an item's beginning and end (its first weights, its store, the way to
// the next one) cost, in units.  The teams' shares are equal with it: for 64
// rows 0, 1, 2, 3, 4 of them took 60, 49, 45, 45, 47 us for trees of 13 tokens
// (8 requests, 300 to 4000 tokens, 32 heads), and 49, 43, 43, 45, 45 for 64
// requests of 100 to 1024 tokens, 128 heads; for 16 rows 0 to 3 24.0, 22.8,
// 22.9, 25.7 for those requests with 16 heads; for 32 rows 0 to 3 43.3, 42.5,
// 43.0, 43.6 for 48 of 100 to 2048 tokens.
__host__ __device__ constexpr int latent_item_cost(int tile_rows) { return tile_rows == 64 ? 2 : 1; }

constexpr int kLatentMaxCtas = 160;  // CTAs of a launch at most (sizes the workspace)
constexpr int kLatentMaxTeam = 12;
constexpr int kLatentPagedInstances = 6;  // {fp16, bf16} x {16, 32, 64 rows}

struct LatentPagedArgs {
    CUtensorMap pool;
    LatentPagedParams p;
    int tile_rows, grid;
    cudaStream_t stream;
    std::atomic<int> *attr_ready;  // the library's flags, for the current device: shared-memory opt-in set, per instance
};

cudaError_t launch_latent_paged(const LatentPagedArgs &a, bool bf16);

// ---------------------------------------------------------------- expanded form

constexpr int kLatentNope = 128, kLatentKey = kLatentNope + kLatentRope, kLatentValue = 128;

// Packed sequences: queries [total_q, h, 192], keys [total_k, h, 128] and
// [total_k, 64], values [total_k, h, 128]; the tensors by strides.
struct LatentSeqs {
    const int32_t *cu_q, *cu_k;  // [batch + 1]
    int32_t batch, h;
    int32_t total_q, total_k;
    int32_t causal;
    float sl2e;                  // scale * log2(e)
    float scale;
    uint32_t *status;
    uint64_t timeout_ns;
};

struct LatentFwdParams {
    LatentSeqs s;
    void *o;                     // [total_q, h, 128] by strides (elements)
    int64_t ot, oh;              // of a token, of a head
    float *lse;                  // [h, total_q] or nullptr
    int32_t slots;               // of 256 queries: total_q / 256 + batch
    int32_t group;               // heads whose units are taken together
};

struct LatentFwdArgs {
    CUtensorMap q, k, r, v;
    LatentFwdParams p;
    unsigned units;
    cudaStream_t stream;
    std::atomic<int> *attr_ready;
};

constexpr int kLatentFwdInstances = 4;  // {fp16, bf16} x {causal, not}

cudaError_t launch_latent_fwd(const LatentFwdArgs &a, bool bf16);

struct LatentBwdParams {
    LatentSeqs s;
    const void *o, *dout;        // [total_q, h, 128] by strides (elements)
    int64_t ot, oh, gt, gh;
    const float *lse;            // [h, total_q]
    float *dsum;                 // [h, total_q]: sum over a row of dO * O
    float *kr_part;              // [h, total_k, 64]: each head's gradient of the shared key part
    void *dq, *dkn, *dkr, *dv;   // by strides of a token and of a head
    int64_t dqt, dqh, dknt, dknh, dkrt, dvt, dvh;
    int32_t q_slots, k_slots;    // of 128 queries, of 128 keys (0: there are none)
    int32_t group;               // heads whose units are taken together
};

struct LatentBwdMaps {
    CUtensorMap q, dout, k, r, v;                           // 128 rows a copy
    CUtensorMap q_half, dout_half, k_half, r_half, v_half;  // 64 rows a copy
};

struct LatentBwdArgs {
    LatentBwdMaps maps;
    LatentBwdParams p;
    cudaStream_t stream;
    std::atomic<int> *attr_ready;
};

constexpr int kLatentBwdInstances = 4;  // {fp16, bf16} x {causal, not}

cudaError_t launch_latent_bwd(const LatentBwdArgs &a, bool bf16);

}  // namespace attn
