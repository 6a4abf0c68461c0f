// bits4.h -- caches held in 4 bits: their layout, and parameters of the kernels that write
// them, read them back (bits4.cu) and attend to them (decode4.cu).
//
// A row of d entries is d / 2 bytes of e2m1 values, entry 2i in the low half of byte i, and
// d / 16 e4m3 scales, one for 16 neighbouring entries; an entry stands for
//   value * scale * factor,
// factor an fp32 number of the KV head (1 without).  value * scale has six significant bits at
// most, so it is exact in fp16 and in bf16.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_attn.h"

namespace apex {

constexpr int kBits4Threads = 128;
constexpr int kBits4Block = 16;    // entries of a scale
constexpr int kBits4MaxRow = 512;  // widest row that is written and read back

// Rows of one tensor: bf16 at x + b * x_b + h * x_h + s * x_s and packed rows of a cache
// [B, H, S_cap, d / 2], [B, H, S_cap, d / 16].
struct Bits4Tensor {
    uint16_t *x;
    long long x_b, x_h, x_s;
    uint8_t *bytes, *scales;
    const float *factor;
    int d;
    int wide;             // bytes that the addresses of 16 entries of x are multiples of: 32, 16 or less
    int per, inv_blocks;  // rows of a block at a time; 2^16 / (d / 16), rounded up (set by the launch)
};

struct Bits4Params {
    Bits4Tensor t[2];  // k, v
    const int *row0;   // first row of each sequence; NULL: 0
    int B, H, S, S_cap;
};

cudaError_t launch_append4(Bits4Params &p, cudaStream_t stream);
cudaError_t launch_unpack4(Bits4Params &p, cudaStream_t stream);

// ---------------------------------------------------------------- attention
struct Decode4Params {
    CacheAttnParams c;  // sizes, lengths, masks, schedule and workspace, as for bf16 caches
    const uint16_t *q;
    const uint8_t *k, *v, *k_scale, *v_scale;
    const float *k_factor;  // the values': c.v_factor
};

// Rows of a KV head's queries that are worked on together: they share each key's conversion.  Up
// to 16 on mma.sync (decode4.cu), more on tcgen05 (decode4_wide.cu).
inline int decode4_group(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 128; }

// CTAs of an SM: with 16 rows the sums of outputs take twice the registers.  8 caches of 9001 to
// 32768 keys, 16 rows: 56 us with 2, 58 with 3 and the queries in shared memory, 70 with 4.
constexpr int decode4_ctas(int group) { return group == 8 ? 4 : group == 16 ? 2 : 1; }
constexpr int kDecode4MaxCtas = 4 * kCacheMaxCtas;

// shares of a call at most: a tile each
inline int decode4_shares(long long units, int S_cap, int ctas)
{
    const long long tiles = units * ((S_cap + kCacheTileKeys - 1) / kCacheTileKeys);
    return (int)std::min<long long>(std::min(ctas, kDecode4MaxCtas), tiles);
}

// Whether short caches are better not cut: without cuts the joining kernel is not launched (3 us), but
// few units leave SMs idle, where a tile takes 0.8 us (1.2 with groups of 128 rows).  `keys`: what a unit of
// a full cache can reach, under a window the window, the sinks and two tiles beside them.  Measured cut / whole at d = 128, 32/8 heads, one token: 1 cache of 500 keys 7.5 / 6.8 us, of
// 760 7.5 / 8.5; 8 of 1020 10.6 / 10.3, of 1500 11.0 / 13.4; 32 of 1000 15.9 / 13.0, of 2000 21.3 /
// 21.2; 128 of 1000 40.0 / 38.0, of 2000 63.5 / 65.7; four tokens: 1 of 500 9.5 / 9.0, of 1000 9.6 /
// 13.0, 32 of 1000 22.1 / 16.7; sixteen: 1 of 250 11.8 / 11.4, of 500 12.1 / 14.3, 8 of 1000 18.4 / 17.6.
inline bool decode4_whole(long long units, int keys, int group)
{
    const int tiles = (keys + kCacheTileKeys - 1) / kCacheTileKeys;
    return tiles <= (units >= 48 ? 8 : group == 128 ? 2 : 4);
}

struct Decode4Workspace {
    size_t ml, units, bytes;
    int rows_cap, n_groups;
};

inline Decode4Workspace decode4_workspace(int B, int H_q, int H_kv, int T, int S_cap, int d_v)
{
    Decode4Workspace w;
    const int R = H_q / H_kv * T, group = decode4_group(R);
    w.rows_cap = std::min(R, group);
    w.n_groups = (R + group - 1) / group;
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    const long long units = (long long)B * H_kv * w.n_groups;
    const size_t slots = (size_t)2 * decode4_shares(units, S_cap, decode4_ctas(group) * kCacheMaxCtas) * w.rows_cap;
    w.ml = up(slots * d_v * sizeof(float));
    w.units = w.ml + up(slots * sizeof(float2));
    w.bytes = w.units + up((size_t)units * sizeof(int2));
    return w;
}

// the attention of groups of 128 rows alone (the caller joins)
cudaError_t launch_decode4_wide(const Decode4Params &p, int grid, cudaStream_t stream);
// chooses the kernel and how the work is cut (p.c.whole), launches it and what joins it
cudaError_t launch_decode4(Decode4Params &p, int sm_count, cudaStream_t stream);

}  // namespace apex
