// cache_attn.cu -- attention over caches of rotated keys on single CTAs (sm_103a): trees
// of drafted tokens of up to 128 rows per KV head (256 at d = 64), and single-query
// decode that also accumulates attention weights; the kernel that joins partial results.
// What is computed and how the work is dealt out: cache_attn.cuh.
//
// Warp roles: 4 softmax warps per M tile (thread i owns row i = TMEM lane i), a TMA
// warp for K and V, an MMA warp issuing S = Q K^T and O += P V on tcgen05 (S, O in TMEM,
// P over S as bf16) and a warp that loads the queries, so that the next fragment's keys
// are under way before this fragment's queries are done with.  With one M tile S has two
// buffers, so the product of the next tile runs under this tile's softmax; with two M
// tiles the tiles take turns.
//
// Bound: HBM.  8 caches of 9001 to 32768 keys, 8 drafts, 32/8 heads of 128: 104 us, 6.6 TB/s
// (a CTA's tile of 64 KB takes 1.3 us, its products 0.5 and its softmax 0.9 beside it); the
// same with weights kept and added, 12345 to 32768 keys: 122 us.  8 caches of 8000 keys of
// 192 / 128 entries, 128 rows: 57 us, 5.8 TB/s.  8 caches of 30000 keys at d = 64: 78 us,
// 6.3 TB/s.  One cache of 128 keys: 5.4 to 6.0 us.  With two M tiles at d = 64 the softmax, 0.9 us
// a tile and M tile beside products of 0.25, bounds: 256 rows over 8 x 30000 keys 136 us (the
// bytes 73), 1024 rows over 4 x 8192 keys 84 us (the products 36).
#include <math.h>

#include "cache_attn.cuh"

namespace apex {
namespace {

constexpr int kKeys = kCacheTileKeys;
constexpr int kBox = 128 * 128;  // [128 rows][64 bf16]

template <int DQK, int DV, int MT>
struct Cfg {
    static_assert(MT == 1 || DV == 64, "two M tiles at d = 64 only: wider rows run on pairs");
    static constexpr int kQBoxes = DQK / 64, kVBoxes = DV / 64;
    static constexpr int kQTile = kQBoxes * kBox, kKTile = kQBoxes * kBox, kVTile = kVBoxes * kBox;
    // ring depth: what 224 KB hold beside the queries
    static constexpr int kKStages = DQK == 64 ? 6 : (DQK == 128 ? 3 : 2);
    static constexpr int kVStages = kKStages;
    static constexpr int kThreads = 128 * MT + 96;
    static constexpr int kWarpTma = 4 * MT, kWarpMma = 4 * MT + 1, kWarpQ = 4 * MT + 2;
    static constexpr int kQOff = 0;
    static constexpr int kKOff = MT * kQTile;
    static constexpr int kVOff = kKOff + kKStages * kKTile;
    static constexpr int kBarOff = kVOff + kVStages * kVTile;
    static constexpr int kBarQFull = 0, kBarQEmpty = 1;
    static constexpr int kBarKFull = 2, kBarKEmpty = kBarKFull + kKStages;
    static constexpr int kBarVFull = kBarKEmpty + kKStages, kBarVEmpty = kBarVFull + kVStages;
    static constexpr int kBarSFull = kBarVEmpty + kVStages;  // [2] per S buffer
    static constexpr int kBarPReady = kBarSFull + 2;         // [2] per S buffer
    static constexpr int kBarPV = kBarPReady + 2;            // [MT] a phase per tile (MT = 1) or fragment
    static constexpr int kBarOEmpty = kBarPV + 2;            // [MT] one phase per fragment
    static constexpr int kNumBars = kBarOEmpty + 2;
    static constexpr int kSched = kBarOff + kNumBars * 8;
    static constexpr int kTmemSlot = kSched + 48;
    static constexpr int kSmemBytes = kTmemSlot + 16 + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    // TMEM columns: S buffers [0, 128), [128, 256); O of tile t from 256 + DV t
    __device__ static constexpr uint32_t col_s(int s) { return 128u * s; }
    __device__ static constexpr uint32_t col_o(int t) { return 256u + (uint32_t)DV * t; }
};

// ---------------------------------------------------------------- attention
template <int DQK, int DV, int MT, bool WEIGHTS, bool SINK>
__global__ void __launch_bounds__(Cfg<DQK, DV, MT>::kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CacheAttnParams p)
{
    using C = Cfg<DQK, DV, MT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sb + C::kBarOff + 8 * i; };
    // softmax warps of M tile t that hold rows
    auto live_warps = [&](int t) { return min(4, (p.rows_cap - 128 * t + 31) / 32); };

    if (threadIdx.x == 0) {
        mbar_init(bar(C::kBarQFull), 1);
        mbar_init(bar(C::kBarQEmpty), 1);
        for (int s = 0; s < C::kKStages; ++s) {
            mbar_init(bar(C::kBarKFull + s), 1);
            mbar_init(bar(C::kBarKEmpty + s), 1);
        }
        for (int s = 0; s < C::kVStages; ++s) {
            mbar_init(bar(C::kBarVFull + s), 1);
            mbar_init(bar(C::kBarVEmpty + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(C::kBarSFull + s), 1);
            mbar_init(bar(C::kBarPReady + s), live_warps(MT == 2 ? s : 0));
        }
        for (int t = 0; t < MT; ++t) {
            mbar_init(bar(C::kBarPV + t), 1);
            mbar_init(bar(C::kBarOEmpty + t), live_warps(t));
        }
        fence_mbarrier_init();
    }
    if (warp == C::kWarpMma) tmem_alloc(sb + C::kTmemSlot, 512);
    if (warp == C::kWarpTma && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // launched as a programmatic dependent: nothing in global memory is touched
    // before the stream's previous kernel is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Sched *sched = reinterpret_cast<Sched *>(smem + C::kSched);
    if (warp == C::kWarpTma) make_sched<SINK>(p, blockIdx.x, gridDim.x, sched);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kTmemSlot);

    Walk<SINK> walk(p, *sched);
    Frag f;
    if (warp == C::kWarpTma) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            // a cache that one row group reads is streamed once: its lines go first from L2
            uint64_t policy;
            if (p.n_groups == 1)
                asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
            else
                asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
            int g = 0;  // tiles so far
            while (walk.next(p, f)) {
                const int kv = f.b * p.H_kv + f.hk;
                if (f.head) p.units[f.unit] = make_int2(blockIdx.x, f.last);
                for (int j = 0; j < f.n; ++j, ++g) {
                    const int key0 = kKeys * f.tile<SINK>(j);
                    const int ks = g % C::kKStages, vs = g % C::kVStages;
                    mbar_wait(bar(C::kBarKEmpty + ks), ((g / C::kKStages) & 1) ^ 1, p.wait);
                    mbar_arrive_expect_tx(bar(C::kBarKFull + ks), C::kKTile);
#pragma unroll
                    for (int bx = 0; bx < C::kQBoxes; ++bx)
                        tma_load_3d_policy(sb + C::kKOff + ks * C::kKTile + bx * kBox, &tm_k, bar(C::kBarKFull + ks),
                                           64 * bx, key0, kv, policy);
                    mbar_wait(bar(C::kBarVEmpty + vs), ((g / C::kVStages) & 1) ^ 1, p.wait);
                    mbar_arrive_expect_tx(bar(C::kBarVFull + vs), C::kVTile);
#pragma unroll
                    for (int bx = 0; bx < C::kVBoxes; ++bx)
                        tma_load_3d_policy(sb + C::kVOff + vs * C::kVTile + bx * kBox, &tm_v, bar(C::kBarVFull + vs),
                                           64 * bx, key0, kv, policy);
                }
            }
        }
    } else if (warp == C::kWarpQ) {
        // ------------------------------------------------------------ queries
        if (lane == 0) {
            for (int fi = 0; walk.next(p, f); ++fi) {
                mbar_wait(bar(C::kBarQEmpty), (fi & 1) ^ 1, p.wait);
                mbar_arrive_expect_tx(bar(C::kBarQFull), MT * C::kQTile);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int bx = 0; bx < C::kQBoxes; ++bx)
                        tma_load_3d(sb + C::kQOff + t * C::kQTile + bx * kBox, &tm_q, bar(C::kBarQFull), 64 * bx,
                                    f.group * p.group + 128 * t, f.b * p.H_kv + f.hk);
            }
        }
    } else if (warp == C::kWarpMma) {
        // ------------------------------------------------------------ MMA issuer, which also mends V tiles
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kKeys, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DV, true);
        const bool one = elect_one();
        auto commit = [&](int i) {
            if (one) tc_commit(bar(i));
        };
        auto issue_qk = [&](int t, int s, int ks) {
            const uint64_t da = smem_desc_sw128(sb + C::kQOff + t * C::kQTile, 16, 1024);
            const uint64_t db = smem_desc_sw128(sb + C::kKOff + ks * C::kKTile, 16, 1024);
            if (one) {
#pragma unroll
                for (int i = 0; i < DQK / 16; ++i) {
                    const uint64_t off = ((i >> 2) * kBox + (i & 3) * 32) >> 4;
                    umma_ss(tmem + C::col_s(s), da + off, db + off, idesc_qk, i > 0 ? 1u : 0u);
                }
            }
            commit(C::kBarSFull + s);
        };
        auto issue_pv = [&](int t, int s, int vs, bool acc) {
            const uint64_t dv = smem_desc_sw128(sb + C::kVOff + vs * C::kVTile, kBox, 1024);
            if (one) {
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i)
                    umma_ts(tmem + C::col_o(t), tmem + C::col_s(s) + 8 * i, dv + (uint64_t)(i * 2048 >> 4), idesc_pv,
                            (acc || i > 0) ? 1u : 0u);
            }
        };
        int g = 0;
        for (int fi = 0; walk.next(p, f); ++fi) {
            mbar_wait(bar(C::kBarQFull), fi & 1, p.wait);
            mbar_wait(bar(C::kBarKFull + g % C::kKStages), (g / C::kKStages) & 1, p.wait);
            tc_fence_after();
            for (int t = 0; t < MT; ++t) issue_qk(t, MT == 2 ? t : (g & 1), g % C::kKStages);
            commit(C::kBarKEmpty + g % C::kKStages);
            if (f.n == 1) commit(C::kBarQEmpty);
            const Sight<SINK> some(p, f);
            for (int j = 0; j < f.n; ++j, ++g) {
                const int ks = (g + 1) % C::kKStages, vs = g % C::kVStages;
                const bool nxt = j + 1 < f.n;
                if (MT == 1 && nxt) {
                    mbar_wait(bar(C::kBarKFull + ks), ((g + 1) / C::kKStages) & 1, p.wait);
                    tc_fence_after();
                    issue_qk(0, (g + 1) & 1, ks);
                    commit(C::kBarKEmpty + ks);
                    if (j + 2 == f.n) commit(C::kBarQEmpty);
                }
                mbar_wait(bar(C::kBarVFull + vs), (g / C::kVStages) & 1, p.wait);
                mend_v<C::kVBoxes, SINK>(p, f, some, kKeys * f.tile<SINK>(j), smem + C::kVOff + vs * C::kVTile);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int s = MT == 2 ? t : (g & 1);
                    mbar_wait(bar(C::kBarPReady + s), (MT == 2 ? g : g >> 1) & 1, p.wait);
                    if (j == 0) mbar_wait(bar(C::kBarOEmpty + t), (fi & 1) ^ 1, p.wait);
                    tc_fence_after();
                    issue_pv(t, s, vs, j > 0);
                    if (MT == 1 || !nxt) commit(C::kBarPV + t);
                    if (t == MT - 1) commit(C::kBarVEmpty + vs);
                    if (MT == 2 && nxt) {
                        if (t == 0) {
                            mbar_wait(bar(C::kBarKFull + ks), ((g + 1) / C::kKStages) & 1, p.wait);
                            tc_fence_after();
                        }
                        issue_qk(t, t, ks);
                        if (t == 1) {
                            commit(C::kBarKEmpty + ks);
                            if (j + 2 == f.n) commit(C::kBarQEmpty);
                        }
                    }
                }
            }
        }
    } else if ((warp & 3) < live_warps(warp >> 2)) {
        // ------------------------------------------------------------ softmax + epilogue
        const int t = warp >> 2;
        const int i = (warp & 3) * 32 + lane;  // row of the M tile == TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_addr = lane_base + C::col_o(t);
        int g = 0;
        for (int fi = 0; walk.next(p, f); ++fi) {
            const int r = f.group * p.group + 128 * t + i;  // row of the KV head
            const bool row_ok = r < p.R;  // padding rows of the last M tile
            const int kv = f.b * p.H_kv + f.hk;
            int lo;
            const uint64_t drafts = draft_sight<SINK>(p, f.b, row_ok ? r % p.T : 0, f.s.len, f.s.total, lo);
            float m_run = -INFINITY, l_run = 0.f;
            float *scores = nullptr;
            if (WEIGHTS) scores = p.scores + ((size_t)kv * p.R + r) * p.S_pad;

            for (int j = 0; j < f.n; ++j, ++g) {
                const int s = MT == 2 ? t : (g & 1);
                const uint32_t s_addr = lane_base + C::col_s(s);
                const int key0 = kKeys * f.tile<SINK>(j);
                mbar_wait(bar(C::kBarSFull + s), (MT == 2 ? g : g >> 1) & 1, p.wait);
                tc_fence_after();
                // O's product of tile g - 1 must be done before O is touched.  With one S buffer a
                // tile these scores follow it; with two it is waited for, in every tile, so
                // that no phase of its barrier is skipped.
                softmax_tile<DV, WEIGHTS, SINK>(
                    p, s_addr, o_addr, key0, lo, f.s.len, drafts, m_run, l_run, row_ok ? scores : nullptr,
                    [&] { if (MT == 1 && g > 0) mbar_wait(bar(C::kBarPV + t), (g - 1) & 1, p.wait); }, [] {});
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarPReady + s));
            }

            // ---- epilogue: the finished row, or this fragment's partial result
            mbar_wait(bar(C::kBarPV + t), (MT == 1 ? g - 1 : fi) & 1, p.wait);
            tc_fence_after();
            write_row<DV, WEIGHTS>(p, o_addr, f.head && f.tail, row_ok, (size_t)kv * p.R + r,
                                   2 * blockIdx.x + (f.head ? 1 : 0), 128 * t + i, m_run, l_run);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarOEmpty + t));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- joining partial results
// max and sum of a row of a cut unit over its fragments, by a warp.  The fragments of a
// unit are the last of share c0 (slot 2 c0 + 1), then the first of each share up to c1
// (slots 2 c).
struct RowParts {
    const CacheAttnParams &p;
    int c0, n, rc;
    __device__ __forceinline__ size_t at(int i) const
    {
        return (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * p.rows_cap + rc;
    }
    __device__ __forceinline__ void stats(int lane, float &M, float &L) const
    {
        float2 mine = make_float2(-INFINITY, 0.f);
        if (lane < n) mine = p.ws_ml[at(lane)];
        M = mine.x;
        for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, p.ws_ml[at(i)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        L = mine.x == -INFINITY ? 0.f : exp2f(mine.x - M) * mine.y;
        for (int i = lane + 32; i < n; i += 32) {
            const float2 v = p.ws_ml[at(i)];
            L += v.x == -INFINITY ? 0.f : exp2f(v.x - M) * v.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    }
};

// Cut units: a thread takes eight entries of a row; consecutive threads take consecutive
// rows, as partial outputs lie.  SPLIT warps of a block share the fragments of the same 32
// threads' rows (few units, cut into many fragments), then their results are joined in turn.
template <int DV, int SPLIT>
__device__ __forceinline__ void join_rows(const CacheAttnParams &p, int blocks_per_unit, float (*sh)[10][32])
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / blocks_per_unit;
    const int idx = (blockIdx.x % blocks_per_unit) * (256 / SPLIT) + (SPLIT == 1 ? threadIdx.x : lane);
    const int rc = idx % p.rows_cap, chunk = idx / p.rows_cap;
    const int r = unit % p.n_groups * p.group + rc;
    const bool ok = chunk < DV / 8 && r < p.R;
    const int2 c = p.units[unit];
    if (c.x == c.y) return;
    const int n = c.y - c.x + 1, first = SPLIT == 1 ? 0 : warp;
    const float factor = p.v_factor ? p.v_factor[unit / p.n_groups % p.H_kv] : 1.f;
    auto slot = [&](int i) { return (size_t)(2 * (c.x + i) + (i == 0 ? 1 : 0)) * p.rows_cap; };
    float M = -INFINITY, L = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    // four fragments in flight: one round trip for their statistics and outputs
    for (int i0 = first; ok && i0 < n; i0 += 4 * SPLIT) {
        float2 ml[4];
        float4 a[4], b[4];
        float top = M;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + q * SPLIT;
            ml[q] = make_float2(-INFINITY, 0.f);
            if (i < n) {
                const float4 *o =
                    reinterpret_cast<const float4 *>(p.ws_o + slot(i) * DV) + (size_t)2 * chunk * p.rows_cap + rc;
                ml[q] = p.ws_ml[slot(i) + rc];
                a[q] = o[0];
                b[q] = o[p.rows_cap];
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) top = fmaxf(top, ml[q].x);
        const float keep = (M == -INFINITY) ? 0.f : exp2f(M - top);
        M = top;
        L *= keep;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= keep;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (ml[q].x == -INFINITY) continue;  // nothing seen, or no such fragment
            const float w = exp2f(ml[q].x - M);
            L = fmaf(w, ml[q].y, L);
            acc[0] = fmaf(w, a[q].x, acc[0]);
            acc[1] = fmaf(w, a[q].y, acc[1]);
            acc[2] = fmaf(w, a[q].z, acc[2]);
            acc[3] = fmaf(w, a[q].w, acc[3]);
            acc[4] = fmaf(w, b[q].x, acc[4]);
            acc[5] = fmaf(w, b[q].y, acc[5]);
            acc[6] = fmaf(w, b[q].z, acc[6]);
            acc[7] = fmaf(w, b[q].w, acc[7]);
        }
    }
    if (SPLIT > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sh[warp][e][lane] = acc[e];
        sh[warp][8][lane] = M;
        sh[warp][9][lane] = L;
        __syncthreads();
        if (warp > 0 || !ok) return;
        float top = M;
        for (int w = 1; w < SPLIT; ++w) top = fmaxf(top, sh[w][8][lane]);
        L = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        for (int w = 0; w < SPLIT; ++w) {
            const float m = sh[w][8][lane];
            const float x = (m == -INFINITY) ? 0.f : exp2f(m - top);
            L = fmaf(x, sh[w][9][lane], L);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(x, sh[w][e][lane], acc[e]);
        }
    }
    if (!ok) return;
    const float inv = (L > 0.f) ? factor / L : 0.f;
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((size_t)(unit / p.n_groups) * p.R + r) * DV) + chunk;
    *dst = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                      pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
}

// acc[b, g, j] += sum over the heads of g of 2^(scale score - lse), heads in order:
// a block takes 1024 keys of a (sequence, KV head), a thread four neighbours.
constexpr int kWeightKeys = 1024;
constexpr int kWeightHeads = 4;  // heads whose scores are in flight
__device__ __forceinline__ void add_weights(const CacheAttnParams &p, long long block, int chunks, float *lse)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = (int)(block / chunks);
    const int j0 = (int)(block % chunks) * kWeightKeys;
    const int j = j0 + 4 * threadIdx.x;
    const float *s = p.scores + (size_t)unit * p.G * p.S_pad + j;
    // the first heads' scores and the sums are under way before the statistics that they wait for
    float4 x[kWeightHeads];
#pragma unroll
    for (int g = 0; g < kWeightHeads; ++g) {
        x[g] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (g < p.G && j < p.S_pad) x[g] = *reinterpret_cast<const float4 *>(s + (size_t)g * p.S_pad);
    }
    float *acc = p.acc + (size_t)unit * p.S_cap + j;
    const bool wide = (reinterpret_cast<uintptr_t>(acc) & 15) == 0;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (wide && j + 4 <= p.S_cap) sum = *reinterpret_cast<const float4 *>(acc);
    const int len = min(max(p.lens[unit / p.H_kv], 0), p.S_cap);
    if (j0 >= len) return;
    const int2 c = p.units[unit];
    for (int g = warp; g < p.G; g += 8) {
        float at;
        if (c.x == c.y) {
            at = p.lse[(size_t)unit * p.G + g];
        } else {
            const RowParts parts{p, c.x, c.y - c.x + 1, g};
            float M, L;
            parts.stats(lane, M, L);
            at = M + log2f(L);
        }
        if (lane == 0) lse[g] = at;
    }
    __syncthreads();
    if (j >= len) return;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g0 = 0; g0 < p.G; g0 += kWeightHeads) {
#pragma unroll
        for (int g = 0; g < kWeightHeads; ++g)
            if (g0 + g < p.G) {
                // exp2f: weights below 2^-126 are kept, as the sums of a long service need them
                const float at = lse[g0 + g];
                w[0] += exp2f(fmaf(x[g].x, p.scale_log2, -at));
                w[1] += exp2f(fmaf(x[g].y, p.scale_log2, -at));
                w[2] += exp2f(fmaf(x[g].z, p.scale_log2, -at));
                w[3] += exp2f(fmaf(x[g].w, p.scale_log2, -at));
            }
#pragma unroll
        for (int g = 0; g < kWeightHeads; ++g)
            if (g0 + kWeightHeads + g < p.G)
                x[g] = *reinterpret_cast<const float4 *>(s + (size_t)(g0 + kWeightHeads + g) * p.S_pad);
    }
    if (wide && j + 4 <= len) {
        *reinterpret_cast<float4 *>(acc) = make_float4(sum.x + w[0], sum.y + w[1], sum.z + w[2], sum.w + w[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < len) acc[e] += w[e];
    }
}

// The first blocks join rows; with WEIGHTS the others add weights, each from its own
// join of the statistics.
template <int DV, int SPLIT, bool WEIGHTS>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheAttnParams p, int join_blocks, int blocks_per_unit,
                                                         int chunks)
{
    __shared__ float sh[SPLIT > 1 ? SPLIT : 1][10][32];
    __shared__ float lse[16];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!WEIGHTS || blockIdx.x < join_blocks)
        join_rows<DV, SPLIT>(p, blocks_per_unit, sh);
    else
        add_weights(p, blockIdx.x - join_blocks, chunks, lse);
}

template <int DQK, int DV, int MT, bool WEIGHTS, bool SINK>
cudaError_t launch_t(const CacheAttnLaunch &L, int grid, cudaStream_t stream)
{
    using C = Cfg<DQK, DV, MT>;
    auto kernel = cache_attn_kernel<DQK, DV, MT, WEIGHTS, SINK>;
    static KernelSetup setup;
    const cudaError_t err = setup(kernel, C::kSmemBytes);
    if (err != cudaSuccess) return err;
    return launch_dependent(kernel, grid, C::kThreads, C::kSmemBytes, stream, L.tm_q, L.tm_k, L.tm_v, L.p);
}

template <int DQK, int DV, int MT>
cudaError_t launch_sink(const CacheAttnLaunch &L, int grid, cudaStream_t stream)
{
    return L.p.n_sink > 0 ? launch_t<DQK, DV, MT, false, true>(L, grid, stream)
                          : launch_t<DQK, DV, MT, false, false>(L, grid, stream);
}

template <int DV, int SPLIT>
cudaError_t launch_join_t(const CacheAttnParams &p, cudaStream_t stream)
{
    const int n_units = p.B * p.H_kv * p.n_groups;
    const int per_unit = (p.rows_cap * (DV / 8) + 256 / SPLIT - 1) / (256 / SPLIT);
    // below 2^31 blocks: B * H_q <= 2^24 and B * H_kv * S_cap <= 2^40
    const int join_blocks = n_units * per_unit;
    const int chunks = (p.S_cap + kWeightKeys - 1) / kWeightKeys;
    if (p.acc)
        return launch_dependent(cache_join_kernel<DV, SPLIT, true>, join_blocks + n_units * chunks, 256, 0, stream, p,
                                join_blocks, per_unit, chunks);
    return launch_dependent(cache_join_kernel<DV, SPLIT, false>, join_blocks, 256, 0, stream, p, join_blocks, per_unit,
                            chunks);
}

template <int DV>
cudaError_t launch_join(const CacheAttnParams &p, int shares, cudaStream_t stream)
{
    // Few units: each is cut into many fragments, which the warps of a block then share.  8
    // units of 19 tiles, one or two a CTA: 9.9 us a call so, 12.4 with a thread for all
    // fragments; 64 long units of 2 or 3 fragments: 162.9 and 160.0; 64 of 512 rows: 120 and 77.
    return 4ll * p.B * p.H_kv * p.n_groups <= shares ? launch_join_t<DV, 8>(p, stream) : launch_join_t<DV, 1>(p, stream);
}

}  // namespace

cudaError_t launch_cache_attn(CacheAttnLaunch &L, int sm_count, cudaStream_t stream)
{
    CacheAttnParams &p = L.p;
    const bool pairs = cache_attn_pairs(p.R, p.d_v);
    const int n_units = p.B * p.H_kv * p.n_groups, room = pairs ? sm_count / 2 : sm_count;
    int shares = std::min(room, cache_attn_shares(p.B, p.H_kv, p.n_groups, p.S_cap, pairs));
    // keys that a unit can reach: a window bounds them, the drafts and a tile's slack beside it
    const long long sinks = p.n_sink > 0 ? (long long)p.n_sink + kKeys : 0;
    const int reach = p.window > 0 ? (int)std::min<long long>(p.S_cap, p.window + sinks + p.drafts + kKeys) : p.S_cap;
    p.whole = !p.acc && cache_attn_whole(n_units, reach, room);
    if (p.whole) shares = std::min(shares, n_units);
    cudaError_t err;
    if (pairs)
        err = launch_cache_pair(L, shares, stream);
    else if (p.d_qk == 64)
        err = p.acc              ? launch_t<64, 64, 1, true, false>(L, shares, stream)
              : p.group == 128 ? launch_sink<64, 64, 1>(L, shares, stream)
                               : launch_sink<64, 64, 2>(L, shares, stream);
    else if (p.d_qk == 128)
        err = p.acc ? launch_t<128, 128, 1, true, false>(L, shares, stream) : launch_sink<128, 128, 1>(L, shares, stream);
    else
        err = p.acc ? launch_t<192, 128, 1, true, false>(L, shares, stream) : launch_sink<192, 128, 1>(L, shares, stream);
    if (err != cudaSuccess) return err;
    return p.whole ? cudaSuccess : launch_cache_join(p, shares, stream);
}

cudaError_t launch_cache_join(const CacheAttnParams &p, int shares, cudaStream_t stream)
{
    return p.d_v == 64 ? launch_join<64>(p, shares, stream) : launch_join<128>(p, shares, stream);
}

}  // namespace apex
