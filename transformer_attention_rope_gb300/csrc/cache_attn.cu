// cache_attn.cu -- attention over caches of rotated keys: trees of drafted tokens,
// and single-query decode that accumulates attention weights.
//
// One block per (sequence, query head, draft); its warps take every fourth key.
#include <math.h>

#include "cache_attn.h"
#include "device_common.cuh"

namespace apex {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float bf16_at(const uint16_t *p, int i) { return bf16lo_to_f32(p[i]); }

// Which keys draft t of sequence b sees.
struct Sight {
    int len, total, lo;  // cached keys, keys with the drafts, first key inside the window
    uint64_t drafts;
    __device__ Sight(const CacheAttnParams &p, int b, int t)
    {
        len = min(max(p.lens[b], 0), p.S_cap);
        total = min(len + p.drafts, p.S_cap);
        lo = 0;
        drafts = 0;
        if (p.drafts == 0) return;
        drafts = p.tree_mask ? p.tree_mask[b * p.mask_stride + t] : (t == 63 ? ~0ull : (1ull << (t + 1)) - 1);
        if (p.drafts < 64) drafts &= (1ull << p.drafts) - 1;
        if (p.window > 0) {
            const int *pos = p.positions ? p.positions + (long long)b * p.T : nullptr;
            const long long m = pos ? max(pos[t], len) : len + t;
            lo = (int)max(0ll, m - p.window + 1);
            for (int u = 0; u < p.drafts; ++u) {
                const long long at = pos ? max(pos[u], len) : len + u;
                if (m - at >= p.window) drafts &= ~(1ull << u);
            }
        }
    }
    __device__ bool sees(int j) const { return j < len ? j >= lo : (j < total && ((drafts >> (j - len)) & 1)); }
};

__global__ void __launch_bounds__(32 * kWarps) cache_attn_kernel(const CacheAttnParams p)
{
    __shared__ float sq[192], sm[kWarps], sl[kWarps], so[kWarps][128];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t row = blockIdx.x;
    const int t = row % p.T, h = (int)(row / p.T % p.H_q), b = (int)(row / p.T / p.H_q);
    const size_t unit = (size_t)b * p.H_kv + h / p.G;
    for (int i = threadIdx.x; i < p.d_qk; i += blockDim.x) sq[i] = bf16_at(p.q + row * p.d_qk, i);
    __syncthreads();
    const Sight sight(p, b, t);
    const uint16_t *k = p.k + unit * p.S_cap * p.d_qk, *v = p.v + unit * p.S_cap * p.d_v;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = min(sight.lo, sight.len) + warp; j < sight.total; j += kWarps) {
        if (!sight.sees(j)) continue;
        float s = 0.f;
        for (int i = lane; i < p.d_qk; i += 32) s = fmaf(sq[i], bf16_at(k + (size_t)j * p.d_qk, i), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale_log2;
        const float m_new = fmaxf(m, s), a = m == -INFINITY ? 0.f : exp2f(m - m_new), w = exp2f(s - m_new);
        m = m_new;
        l = l * a + w;
        for (int e = 0; e * 32 < p.d_v; ++e) o[e] = o[e] * a + w * bf16_at(v + (size_t)j * p.d_v, e * 32 + lane);
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    for (int e = 0; e * 32 < p.d_v; ++e) so[warp][e * 32 + lane] = o[e];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kWarps; ++w) L += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - M);
    for (int i = threadIdx.x; i < p.d_v; i += blockDim.x) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += sm[w] == -INFINITY ? 0.f : so[w][i] * exp2f(sm[w] - M);
        p.out[row * p.d_v + i] = (uint16_t)pack_bf16x2(L > 0.f ? x / L : 0.f, 0.f);
    }
    if (p.acc && threadIdx.x == 0) p.lse[row] = M + log2f(L);
}

// acc[b, g, j] += sum over the heads of g of exp2(score - lse); one warp per key.
__global__ void __launch_bounds__(256) cache_weights_kernel(const CacheAttnParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const size_t unit = blockIdx.x;
    const int b = (int)(unit / p.H_kv);
    const int len = min(max(p.lens[b], 0), p.S_cap);
    for (int j = blockIdx.y * 8 + (threadIdx.x >> 5); j < len; j += gridDim.y * 8) {
        float w = 0.f;
        for (int g = 0; g < p.G; ++g) {
            const size_t row = unit * p.G + g;
            float s = 0.f;
            for (int i = lane; i < p.d_qk; i += 32)
                s = fmaf(bf16_at(p.q + row * p.d_qk, i), bf16_at(p.k + (unit * p.S_cap + j) * p.d_qk, i), s);
            for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            w += exp2f(s * p.scale_log2 - p.lse[row]);
        }
        if (lane == 0) p.acc[unit * p.S_cap + j] += w;
    }
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnParams &p, int sm_count, cudaStream_t stream)
{
    cudaError_t err = launch_dependent(cache_attn_kernel, p.B * p.H_q * p.T, 32 * kWarps, 0, stream, p);
    if (err != cudaSuccess || !p.acc) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.B * p.H_kv, 64);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, cache_weights_kernel, p);
}

}  // namespace apex
