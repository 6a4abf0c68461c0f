// rope.h -- parameters of the rotary-position kernel (rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace apex {

constexpr int kRopeMaxPairs = 256;   // d_rot <= 512
constexpr int kRopeMaxGroups = 48;   // head groups of one launch
constexpr int kRopeThreads = 256;    // threads per block

enum RopeKind { kRopeInterleaved, kRopeHalf, kRopePairs };

struct RopeTensor {
    const uint16_t *in;
    uint16_t *out;
    long long in_b, in_h, in_s, out_b, out_h, out_s;  // strides in elements
    int d_row;
    int rotate;  // 0: rows copied (values)
    int append;  // rows go to row0[b] + s when row0 is given
};

// Heads [h0, h0 + n) of one tensor: what one block row of the grid works on.
struct RopeGroup {
    int tensor, h0, n;
};

struct RopeParams {
    RopeTensor t[3];  // q, k, v (those present, in this order)
    RopeGroup groups[kRopeMaxGroups];
    const int *positions;
    long long pos_stride;
    const int *row0;
    int out_rows;
    int B, S;
    int rot_start, d_rot, half;
    int n_groups;
    float sign;
    uint64_t turns[kRopeMaxPairs];  // theta_i as fractions of a turn, 0.64 fixed point
};
static_assert(sizeof(RopeParams) <= 4096, "kernel parameters");

cudaError_t launch_rope(const RopeParams &p, int kind, int grid_x, cudaStream_t stream);

}  // namespace apex
