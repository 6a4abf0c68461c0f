// norm_rope.h -- parameters of the kernels that norm and turn heads in one pass, and of
// their gradients (norm_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "rope.h"

namespace apex {

constexpr int kNormThreads = 128, kNormSumThreads = 256;
constexpr int kNormCtas = 5, kNormGradCtas = 4;  // of an SM, where rows go 16 bytes at a time
constexpr int kNormBatch = 4;                    // heads of a token that a lane takes, whose loads are in flight together
constexpr int kNormFastRow = 512;      // widest row of the kernels that go 16 bytes at a time
constexpr int kNormHeads = 128;        // heads with weights of their own that a block takes, times lanes of a row
constexpr int kNormGradBlocks = 1024;  // blocks of a gradient at most (but for one of each group),
constexpr int kNormGradHeads = 8;      // and partial sums of weights of each at most

// Rows at x + b * x_b + h * x_h + s * x_s, likewise dy (gradients) and out (the result, or x's gradient).
struct NormTensor {
    const uint16_t *x, *dy;
    uint16_t *out;
    long long x_b, x_h, x_s, dy_b, dy_h, dy_s, out_b, out_h, out_s;
    const void *weight;   // bf16 or fp32; NULL: ones
    int weight_f32;
    int weight_h;         // entries between the weights of two heads (0: the same for all)
    int n_heads, d_row;
    int per, n_groups;    // heads of a group, groups
    int blocks;           // blocks of each group
    int tile, tiles;      // tokens of a tile, tiles of a sequence (rows that go 16 bytes at a time)
    int batch;            // heads of a token that a slot takes, where there are as many
    int norm;             // 0: rows copied (values)
    int append;           // rows go to row0[b] + s when row0 is given
    float inv_d;
    float *partial;       // gradients: sums of weights, [n_groups * blocks][d_row], or [n_heads][blocks][d_row]
    float *dweight;       // [d_row] or [n_heads][d_row]
};

struct NormRopeParams {
    NormTensor t[3];  // q, k, v (those present, in this order)
    const int *positions;
    long long pos_stride;
    const int *row0;
    int out_rows;
    int B, S;
    int rot_start, d_rot;  // d_rot 0: nothing turns
    int n_tensors;
    float eps, sign;
    uint64_t turns[kRopeMaxPairs];
};
static_assert(sizeof(NormRopeParams) <= 4096, "kernel parameters");

// half: pair layout; lanes: lanes of a row (4, 8, 16 or 32; 0: rows that go 2 bytes at a time)
cudaError_t launch_norm_rope(const NormRopeParams &p, bool half, int lanes, cudaStream_t stream);
cudaError_t launch_norm_rope_grad(const NormRopeParams &p, bool half, int lanes, cudaStream_t stream);

}  // namespace apex
