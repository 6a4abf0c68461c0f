// cache_attn.h -- parameters of the attention kernels over caches of rotated keys
// (cache_attn.cu): drafted trees, and decode that accumulates attention weights.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kernel_params.h"

namespace apex {

constexpr int kTreeMaxDrafts = 64;  // one mask word per draft

struct CacheAttnParams {
    const uint16_t *q;  // [B, H_q, T, d_qk]
    const uint16_t *k;  // [B, H_kv, S_cap, d_qk]
    const uint16_t *v;  // [B, H_kv, S_cap, d_v]
    uint16_t *out;      // [B, H_q, T, d_v]
    int B, H_q, H_kv, G, T, S_cap, d_qk, d_v;
    const int *lens;
    const uint64_t *tree_mask;
    long long mask_stride;
    const int *positions;
    int window;  // 0: none
    int drafts;  // draft rows behind lens[b]: T, or 0 for the decode
    float *acc;  // [B, H_kv, S_cap], or NULL
    float scale_log2;
    WaitCtl wait;
    float *lse;  // [B*H_q] log2 of the softmax denominators (with acc)
};

struct CacheAttnWorkspace {
    size_t bytes;
};

inline CacheAttnWorkspace cache_attn_workspace(int B, int H_q, int, int T, int, int, bool weights)
{
    CacheAttnWorkspace w;
    w.bytes = weights ? ((size_t)B * H_q * T * sizeof(float) + 255) & ~size_t(255) : 256;
    return w;
}

inline void cache_attn_bind(CacheAttnParams &p, const CacheAttnWorkspace &, void *workspace)
{
    p.lse = static_cast<float *>(workspace);
}

cudaError_t launch_cache_attn(const CacheAttnParams &p, int sm_count, cudaStream_t stream);

}  // namespace apex
