// cache_attn.h -- parameters of the attention kernels over caches of rotated keys
// (cache_attn.cu): drafted trees, and decode that accumulates attention weights.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "kernel_params.h"

namespace apex {

constexpr int kTreeMaxDrafts = 64;    // one mask word per draft
constexpr int kCacheTileKeys = 128;   // keys per tile
constexpr int kCacheMaxCtas = 160;    // CTAs of a call at most

struct CacheAttnParams {
    uint16_t *out;  // [B, H_q, T, d_v]
    int B, H_q, H_kv, G, T, S_cap, d_qk, d_v;
    const int *lens;
    const uint64_t *tree_mask;
    long long mask_stride;
    const int *positions;
    int window;  // 0: none
    int n_sink;  // first keys that stay visible behind a window
    int drafts;  // draft rows behind lens[b]: T, or 0 for the decode
    float *acc;  // [B, H_kv, S_cap], or NULL
    float scale_log2;
    const float *v_factor;  // [H_kv] of the values, for the rows once they are joined, or NULL: 1
    WaitCtl wait;
    int R;          // query rows of a KV head, G * T
    int group;      // rows of a row group
    int n_groups;   // row groups of a KV head
    int rows_cap;   // rows of a partial result, min(R, group)
    int whole;      // units are not cut: nothing to join
    // workspace
    float *ws_o;    // [2 * shares][d_v / 4][rows_cap][4] partial outputs (unnormalised)
    float2 *ws_ml;  // [2 * shares][rows_cap]             their (max in log2 units, sum)
    int2 *units;    // [B * H_kv * n_groups]              first and last share of each unit
    float *lse;     // [B * H_q]                          log2 of the softmax denominators (with acc)
    float *scores;  // [B * H_q][S_pad]                   scores (with acc)
    int S_pad;
};

// Which kernel, by the rows R = G * T of a KV head's queries.  Up to 128 rows: one M tile
// on one CTA, bound by the cache's bytes.  More: pairs of CTAs that share each K/V tile,
// with one M tile each up to 256 rows and two from there on, as the tensor cores read the
// tile from shared memory once for both CTAs.  d_v = 64, whose halves of a V tile would be
// narrower than the 128-byte swizzle, stays on one CTA with two M tiles.
// Measured at d = 128 on pairs / on single CTAs with two M tiles (an instance built for the
// comparison; rows of 192 leave it one stage).  512 rows, 8 x 8000 keys: 90 / 106 us; 1024
// rows, 4 x 8192: 94 / 108, ragged 4100 to 8192: 76 / 82.  Up to 256 rows neither leads
// throughout: 32 units (32 caches of 500 to 4000 keys, one KV head) 144 rows 20.2 / 23.7,
// 256 rows 21.2 / 30.3; 64 units (8 x 8000) 144 rows 54.7 / 50.7, 256 rows 57.2 / 55.7,
// 8 x 30000 keys 256 rows 172 / 170; 128 units (16 caches of 500 to 4000) 144 rows
// 47.4 / 37.0, 256 rows 51.4 / 44.8.
inline bool cache_attn_pairs(int R, int d_v) { return R > 128 && d_v == 128; }
inline int cache_attn_group(int R, int d_v) { return R <= 128 ? 128 : (R <= 256 || d_v != 128) ? 256 : 512; }

// What starting a unit costs in the schedule, in tiles: the pipeline fills and drains once
// more.  32 caches of 100 to 2000 keys, 4 drafts, 32/8 heads: 36.3 us counting 0, 29.5 at 1,
// 28.5 at 2, 28.8 at 3; a tree of 64 on 128/8 heads, 4 x 8192 keys: 95.9, 94.6, 94.0, 94.4,
// 4 x 4100 to 8192: 77.8, 78.7, 76.3, 77.0; 8 long caches are indifferent (102.9 to 103.5).
constexpr int kCacheUnitCost = 2;

// Most shares of a call: one per tile, one per CTA or pair at most.
inline int cache_attn_shares(int B, int H_kv, int n_groups, int S_cap, bool pairs)
{
    const long long tiles = (long long)B * H_kv * n_groups * ((S_cap + kCacheTileKeys - 1) / kCacheTileKeys);
    return (int)std::min<long long>(pairs ? kCacheMaxCtas / 2 : kCacheMaxCtas, tiles);
}

// Whether short caches are better not cut: without cuts the joining kernel is not
// launched, which is worth about 3.5 tiles, but the CTAs' loads are less even.  Judged on
// full caches; past 6 tiles a ragged batch could lose more than that.  Measured cut / whole
// at d = 128, 32/8 heads, 4 drafts: 1 cache of 376 keys 8.5 / 7.7 us, of 504 8.6 / 8.5, of
// 632 8.5 / 9.3; 8 caches of 504 keys 10.8 / 8.7; 32 of 248 14.0 / 11.7, of 760 21.8 / 20.0;
// 640 rows, 4 caches of 480 keys on pairs 22.6 / 15.9.
inline bool cache_attn_whole(long long units, int keys, int shares)
{
    const long long tiles = (keys + kCacheTileKeys - 1) / kCacheTileKeys, cost = tiles + kCacheUnitCost;
    if (tiles == 1) return true;
    const long long rounds = (units + shares - 1) / shares;
    const long long cut = std::max<long long>(1 + kCacheUnitCost, units * cost / shares);
    return tiles <= 6 && 2 * rounds * cost <= 2 * cut + 7;
}

struct CacheAttnWorkspace {
    size_t ml, units, lse, scores, bytes;
    int rows_cap, n_groups, S_pad;
};

inline CacheAttnWorkspace cache_attn_workspace(int B, int H_q, int H_kv, int T, int S_cap, int d_v, bool weights)
{
    CacheAttnWorkspace w;
    const int R = H_q / H_kv * T, group = cache_attn_group(R, d_v);
    w.rows_cap = std::min(R, group);
    w.n_groups = (R + group - 1) / group;
    w.S_pad = (S_cap + kCacheTileKeys - 1) / kCacheTileKeys * kCacheTileKeys;
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    const size_t slots = (size_t)2 * cache_attn_shares(B, H_kv, w.n_groups, S_cap, cache_attn_pairs(R, d_v)) * w.rows_cap;
    w.ml = up(slots * d_v * sizeof(float));
    w.units = w.ml + up(slots * sizeof(float2));
    w.lse = w.units + up((size_t)B * H_kv * w.n_groups * sizeof(int2));
    w.scores = w.lse + (weights ? up((size_t)B * H_q * sizeof(float)) : 0);
    w.bytes = w.scores + (weights ? up((size_t)B * H_q * w.S_pad * sizeof(float)) : 0);
    return w;
}

inline void cache_attn_bind(CacheAttnParams &p, const CacheAttnWorkspace &w, void *workspace)
{
    char *base = static_cast<char *>(workspace);
    p.R = p.G * p.T;
    p.group = cache_attn_group(p.R, p.d_v);
    p.n_groups = w.n_groups;
    p.rows_cap = w.rows_cap;
    p.S_pad = w.S_pad;
    p.ws_o = reinterpret_cast<float *>(base);
    p.ws_ml = reinterpret_cast<float2 *>(base + w.ml);
    p.units = reinterpret_cast<int2 *>(base + w.units);
    p.lse = reinterpret_cast<float *>(base + w.lse);
    p.scores = reinterpret_cast<float *>(base + w.scores);
}

struct CacheAttnLaunch {
    // 3-D maps, boxes of 128 rows x 64 entries (k on pairs: 64 x 64), 128-byte swizzle: q as
    // [B*H_kv][R][d_qk] (the rows of a KV head's query heads are adjacent), k and v
    // [B*H_kv][S_cap][d]
    CUtensorMap tm_q, tm_k, tm_v;
    CacheAttnParams p;
};

// chooses the kernel and how the work is cut (L.p.whole), launches it and what joins it
cudaError_t launch_cache_attn(CacheAttnLaunch &L, int sm_count, cudaStream_t stream);
// the attention kernel on CTA pairs alone (the caller joins)
cudaError_t launch_cache_pair(const CacheAttnLaunch &L, int pairs, cudaStream_t stream);
// joins the partial results that `shares` shares left
cudaError_t launch_cache_join(const CacheAttnParams &p, int shares, cudaStream_t stream);

}  // namespace apex
