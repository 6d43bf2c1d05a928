// RMS norm of every query and key head with the rotary rotation in the same
// pass, and its gradients: parameters and launches.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace attn {

// One of the two tensors (queries, keys).  Strides count elements; the
// values of a head are contiguous.
struct NormRopeSide {
    const void *x = nullptr;    // forward: input; backward: the forward's input
    const void *g = nullptr;    // backward: gradient of the output
    void *out = nullptr;        // forward: output; backward: gradient of the input
    const void *w = nullptr;    // norm weight [d], or nullptr: no norm
    int64_t xb = 0, xh = 0, xs = 0;
    int64_t gb = 0, gh = 0, gs = 0;
    int64_t ob = 0, oh = 0, os = 0;
    int heads = 0;
    int groups = 0;             // units that a token's heads make
};

struct NormRopeParams {
    NormRopeSide side[2];
    const float *cos = nullptr, *sin = nullptr;  // [table_len, rot / 2], or nullptr: no rotation
    const int32_t *pos = nullptr;                // position of token (b, s) at pos[b * pos_b + s]; nullptr: s
    int64_t pos_b = 0;
    int64_t tokens = 0;                          // b * s
    uint32_t units = 0;                          // units of work
    int64_t s = 0;
    int table_len = 0;
    int rot = 0;
    int interleaved = 0;
    float eps = 0.f;
    uint32_t *status = nullptr;
    float *dw_part = nullptr;                    // backward: [blocks][2][d] partial sums of the weights' gradients
    float *dw[2] = {nullptr, nullptr};           // backward: gradient of each weight [d], or nullptr
};

constexpr int kNormRopeMaxBlocks = 640;  // partial sums of the weights' gradients at most

cudaError_t launch_norm_rope(const NormRopeParams &p, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(const NormRopeParams &p, int d, bool bf16, int sm_count, cudaStream_t stream);

}  // namespace attn
