// evict.h -- parameters of the cache eviction kernels (evict.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace apex {

struct EvictParams {
    uint4 *k, *v;  // [B*H_kv][S_cap][ck], [..][cv] 16-byte chunks
    int ck, cv;
    const float *acc;
    const int *positions;  // NULL: row index
    const int *lens, *next_pos;
    int newest;  // next_pos holds lens: the rows' positions may be past it
    float *acc_out;
    int *positions_out;
    int *lens_out;
    int *holes, *sources;   // [B*H_kv][cap] destination and source rows, ascending
    int cap;
    int B, H_kv, S_cap, budget, n_sink, n_recent;
};

struct EvictWorkspace {
    size_t sources, bytes;
    int cap;
};

// At most min(budget, S_cap - budget) rows of a (sequence, KV head) move.
inline EvictWorkspace evict_workspace(int units, int S_cap, int budget)
{
    EvictWorkspace w;
    w.cap = std::max(0, std::min(budget, S_cap - budget));
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    w.sources = up((size_t)units * w.cap * sizeof(int));
    w.bytes = std::max<size_t>(256, 2 * w.sources);
    return w;
}

cudaError_t launch_evict(const EvictParams &p, int sm_count, cudaStream_t stream);

}  // namespace apex
