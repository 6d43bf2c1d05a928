// Append of rotated keys and of values to a paged cache: parameters, launch.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace attn {

struct KvAppendParams {
    const void *x[2];            // k_new, v_new: [b, heads, s, d] by strides (elements), d contiguous
    int64_t xb[2], xh[2], xs[2];
    void *pool[2];               // [num_pages, page_size, heads, d], 16-bit or e4m3
    float *scale[2];             // e4m3: [num_pages, heads, page_size / block]
    const int32_t *seqlens;      // [b] cached tokens
    const int32_t *new_seqlens;  // [b] new tokens, or nullptr: s
    const int32_t *block_table;  // [b, pages_per_seq]
    const float *cos, *sin;      // [>= capacity, rot / 2], or nullptr: no rotation
    int64_t b, s, num_pages, pages_per_seq;
    int heads, page_size, block_shift;  // a block of the scales is 1 << block_shift tokens
    int rot, interleaved;
    uint32_t *status;
    uint32_t nblk_heads;         // e4m3: blocks that a request's new rows can touch, times heads
};

cudaError_t launch_kv_append(const KvAppendParams &p, int d, bool bf16, bool e4m3, cudaStream_t stream);

}  // namespace attn
