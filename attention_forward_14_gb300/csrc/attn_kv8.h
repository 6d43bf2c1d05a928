// Attention over an e4m3 paged cache with a scale for each block of tokens
// and head: parameters and launches.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

// An item that a CTA begins and later CTAs go on with.
struct alignas(16) Kv8Cut {
    int32_t parts;        // CTAs that have a part (0: there is no such item); negated when it is not this CTA's first
    int32_t b, hg, tile;  // batch element, group of key heads, tile of query rows
};

struct Kv8Params {
    const void *q;               // [b, h, sq, d] fp16 / bf16
    void *o;                     // the same
    float *lse;                  // [b, h, sq] or nullptr
    const uint8_t *v_pool;       // [num_pages, page_size, h_kv, d] (read directly for its NaNs only)
    const float *k_scale, *v_scale;  // [num_pages, h_kv, page_size >> block_shift]
    const int32_t *seqlens;      // [b]
    const int32_t *block_table;  // [b, pages_per_seq]
    uint32_t *status;
    float *o_part;               // [2 * grid][8][16][d], or [2 * grid][256][d]: parts of the items that several CTAs share
    float *ml_part;              // [2 * grid][8][16][2] or [2 * grid][256][2]: their reference (log2) and sum
    Kv8Cut *cut;                 // [grid]
    float sl2e;                  // scale * log2(e)
    int32_t b, h_kv;
    int32_t heads;               // key heads that a CTA works on at a time: 8, 4, 2 or 1, a divisor of h_kv
    int32_t head_groups;         // h_kv / heads
    int32_t unit_keys;           // 32 * 8 / heads
    int32_t sq, rows;            // rows = (h / h_kv) * sq query rows of one key head
    int32_t tile_rows, tiles;    // query rows of an item: 8, 16 or 256; ceil(rows / tile_rows)
    int32_t box;                 // tokens of a copy (256 rows): 128, 64, 32 or 16, a divisor of page_size
    int32_t cap;                 // pages_per_seq * page_size
    int32_t page_size, pages_per_seq, num_pages, block_shift;
    int32_t causal;
    uint64_t timeout_ns;
};

constexpr int kKv8MaxCtas = 160;  // CTAs of a launch at most (sizes the workspace)
constexpr int kKv8Instances = 12;  // head dim {64, 128} x {fp16, bf16} x {8, 16, 256 rows}
constexpr int kKv8Heads = 8;       // key heads of an item at most
constexpr int kKv8WideRows = 256;  // query rows of an item of the kernel for many
constexpr int kKv8Tile = 16;       // query rows of an item of the other, at most

struct Kv8LaunchArgs {
    CUtensorMap k, v;
    Kv8Params p;
    int grid;
    cudaStream_t stream;
    std::atomic<int> *attr_ready;  // the library's flags, for the current device: shared-memory opt-in set, per instance
};

cudaError_t launch_kv8(const Kv8LaunchArgs &a, int d, bool bf16);       // tile_rows 8 or 16
cudaError_t launch_kv8_wide(const Kv8LaunchArgs &a, int d, bool bf16);  // tile_rows 256
cudaError_t launch_kv8_join(const Kv8LaunchArgs &a, int d, bool bf16);

}  // namespace attn
