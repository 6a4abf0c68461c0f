// cache_pair.cu -- attention of drafted trees with more than 128 query rows per KV head
// on CTA pairs (tcgen05 cta_group::2), value rows of 128 entries, query and key rows of
// 128 or 192.  What is computed and how the work is dealt out: cache_attn.cuh.
//
// On one CTA such a tree is bound by shared memory: a 128 x 128 product reads its A and
// B operands at the rate the tensor cores use them.  Here S_t = Q_t K^T and O_t += P_t V
// are M = 256 products over both CTAs (M tile 2 t of the row group on the leader, 2 t + 1
// on its peer) and B is split between the two shared memories: each CTA loads 64 of a
// tile's 128 keys of K and 64 of the 128 entries of V, so every K/V byte crosses L2 once
// for 256 (MT = 1) or 512 (MT = 2) rows and the operand traffic of B halves.
//
// Warps per CTA: two softmax warpgroups, then a TMA warp (K and V), an MMA warp (the
// leader's issues, both allocate TMEM), a warp that loads the queries, waits for what has
// landed here, mends V tiles and tells the leader, and an idle one.  The leader's MMA warp
// waits on its own barriers, which the peer reaches by remote arrivals; commits are
// multicast, so everybody waits on local barriers.
//
// Softmax: one warpgroup needs about 1 us for the 128 x 128 scores of a tile, the products
// half of that.  With MT = 2 each warpgroup has its own M tile.  With MT = 1 both work on
// the same rows, on every other key tile, each with its own S, running maximum, sum and O;
// the two results are joined when a fragment ends (both warpgroups reach the same TMEM
// lanes), each warpgroup writing half of the columns.
//
// Bound: the softmax beside the products from 257 rows on -- 64 drafts on 128/8 heads over
// 4 x 32768 keys 313 to 330 us, 1.67 to 1.76 PFLOP/s; over 4 x 4100 to 8192 keys 76 to 81 us
// with cut units joined (84 before O += P V started on half a tile); rows of 192 over 4 x 8192
// keys 108 us.  Below that the cycle of an S buffer -- product, 1 us of softmax, product --
// of which there are two: 256 rows over 8 x 8000 keys 57 us, where the bytes take 40 and the
// products 36 (65 us with one warpgroup); 208 rows of 192 63 us, where the bytes take 50.
#include <math.h>

#include "cache_attn.cuh"
#include "pair_common.cuh"

namespace apex {
namespace {

constexpr int DV = 128;
constexpr int kKeys = kCacheTileKeys;
constexpr int kQBox = 128 * 128;   // [128 rows][64 entries]
constexpr int kKBox = 64 * 128;    // [64 keys][64 entries]
constexpr int kVTile = 128 * 128;  // 128 keys x this CTA's 64 entries

template <int DQK, int MT>
struct PairCfg {
    static constexpr int kThreads = 3 * 128;
    static constexpr int kWarpTma = 8, kWarpMma = 9, kWarpReady = 10;
    // Two softmax warpgroups need more registers than an even split of 64 K gives: the
    // block is launched with kLaunchRegs a thread, which setmaxnreg redistributes.
    static constexpr int kLaunchRegs = 168, kRegsSoftmax = 200, kRegsCtl = 104;
    static_assert(2 * kRegsSoftmax + kRegsCtl <= 3 * kLaunchRegs, "register split");
    static constexpr int kBoxes = DQK / 64;
    static constexpr int kQTile = kBoxes * kQBox, kKTile = kBoxes * kKBox;
    static constexpr int kStage = kKTile + kVTile;  // K and V of a tile share a stage
    static constexpr int kStages = DQK == 128 ? 5 : (MT == 1 ? 4 : 3);
    static constexpr int kQOff = 0;
    static constexpr int kStageOff = MT * kQTile;
    static constexpr int kBarOff = kStageOff + kStages * kStage;
    static constexpr int kBarQFull = 0;                       // local TMA
    static constexpr int kBarQReady = 1;                      // leader: both CTAs
    static constexpr int kBarQEmpty = 2;                      // multicast commit
    static constexpr int kBarSFull = 3;                       // [2] multicast commit, per S buffer
    static constexpr int kBarPReady = 5;                      // [2] leader: live softmax warps, per S buffer
    static constexpr int kBarPV = 7;                          // [2] multicast commit, per O: its last product of a fragment
    static constexpr int kBarOEmpty = 9;                      // [MT] leader: live softmax warps, one phase per fragment
    static constexpr int kBarPHalf = 11;                      // [2] leader: the same, the first 64 keys' weights
    static constexpr int kBarFull = 13;                       // [stages] local TMA
    static constexpr int kBarReady = kBarFull + kStages;      // [stages] leader: both CTAs
    static constexpr int kBarEmpty = kBarReady + kStages;     // [stages] multicast commit
    static constexpr int kNumBars = kBarEmpty + kStages;
    static constexpr int kSched = kBarOff + kNumBars * 8;
    static constexpr int kTmemSlot = kSched + 48;
    static constexpr int kStatsOff = kTmemSlot + 16;          // MT = 1: [2 fragments][2 warpgroups][128] (max, sum)
    static constexpr int kSmemBytes = kStatsOff + (MT == 1 ? 4096 : 0) + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t col_s(int s) { return 128u * s; }
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + 128u * t; }

// Columns [c0, c0 + 64) of a row from both warpgroups' outputs, w0 O_0 + w1 O_1 (a weight of
// zero: that O may hold anything), finished or as a part of a cut unit's result.
__device__ __forceinline__ void join_half(const CacheAttnParams &p, uint32_t lane_cols, float w0, float w1, bool whole,
                                          bool row_ok, size_t row, int slot, int rc, int c0, float M, float L)
{
    const float inv = !whole ? 1.f : (L == 0.f) ? 0.f : 1.f / L;
    if (row_ok && !whole && c0 == 0) p.ws_ml[(size_t)slot * p.rows_cap + rc] = make_float2(M, L);
    uint4 *dst16 = reinterpret_cast<uint4 *>(p.out + row * DV + c0);
    float4 *dst32 = reinterpret_cast<float4 *>(p.ws_o + (size_t)slot * p.rows_cap * DV) + (size_t)(c0 / 4) * p.rows_cap + rc;
    w0 *= inv;
    w1 *= inv;
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
        uint32_t a[16], b[16];
        tmem_ld16(lane_cols + col_o(0) + 16 * ch, a);
        tmem_ld16(lane_cols + col_o(1) + 16 * ch, b);
        tmem_wait_ld();
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[e] = (w0 == 0.f ? 0.f : w0 * __uint_as_float(a[e])) + (w1 == 0.f ? 0.f : w1 * __uint_as_float(b[e]));
        if (row_ok && whole) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                dst16[2 * ch + q] =
                    make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                               pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
        } else if (row_ok) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                dst32[(size_t)(4 * ch + q) * p.rows_cap] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
    }
}

template <int DQK, int MT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg<DQK, MT>::kThreads, 1)
    cache_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CacheAttnParams p)
{
    using C = PairCfg<DQK, MT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int share = blockIdx.x >> 1, shares = gridDim.x >> 1;
    auto bar = [&](int i) -> uint32_t { return sb + C::kBarOff + 8 * i; };
    volatile uint32_t *abort = reinterpret_cast<volatile uint32_t *>(smem + C::kTmemSlot + 4);
    // softmax warps that hold rows of M tile T of the row group
    auto live_warps = [&](int T) { return max(0, min(4, (p.rows_cap - 128 * T + 31) / 32)); };

    if (threadIdx.x == 0) {
        *abort = 0u;
        mbar_init(bar(C::kBarQFull), 1);
        mbar_init(bar(C::kBarQReady), 2);
        mbar_init(bar(C::kBarQEmpty), 1);
        for (int s = 0; s < 2; ++s) {
            const int t = MT == 2 ? s : 0, live = live_warps(2 * t) + live_warps(2 * t + 1);
            mbar_init(bar(C::kBarSFull + s), 1);
            mbar_init(bar(C::kBarPReady + s), live);
            mbar_init(bar(C::kBarPHalf + s), live);
            mbar_init(bar(C::kBarPV + s), 1);
            mbar_init(bar(C::kBarOEmpty + s), MT == 2 ? live : 2 * live);
        }
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar(C::kBarFull + s), 1);
            mbar_init(bar(C::kBarReady + s), 2);
            mbar_init(bar(C::kBarEmpty + s), 1);
        }
        fence_mbarrier_init();
    }
    if (warp == C::kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + C::kTmemSlot),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == C::kWarpTma && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // launched as a programmatic dependent: nothing in global memory is touched
    // before the stream's previous kernel is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Sched *sched = reinterpret_cast<Sched *>(smem + C::kSched);
    if (warp == C::kWarpTma) make_sched(p, share, shares, sched);
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers initialised, TMEM allocated, schedules made
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kTmemSlot);

    Walk walk(p, *sched);
    Frag f;
    if (warp >= C::kWarpTma) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsCtl));
    if (warp == C::kWarpTma) {
        // ------------------------------------------------------------ K and V (both CTAs, a half each)
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
                if (f.head && rank == 0) p.units[f.unit] = make_int2(share, f.last);
                for (int j = 0; j < f.n; ++j, ++g) {
                    const int key0 = kKeys * (f.first + j);
                    const int st = g % C::kStages;
                    const uint32_t at = sb + C::kStageOff + st * C::kStage;
                    pair_wait(bar(C::kBarEmpty + st), ((g / C::kStages) & 1) ^ 1, p.wait, abort);
                    mbar_arrive_expect_tx(bar(C::kBarFull + st), C::kStage);
#pragma unroll
                    for (int bx = 0; bx < C::kBoxes; ++bx)
                        tma_load_3d_policy(at + bx * kKBox, &tm_k, bar(C::kBarFull + st), 64 * bx, key0 + 64 * rank, kv,
                                           policy);
                    tma_load_3d_policy(at + C::kKTile, &tm_v, bar(C::kBarFull + st), 64 * rank, key0, kv, policy);
                }
            }
        }
    } else if (warp == C::kWarpReady) {
        // ------------------------------------------------------------ queries, mended V tiles, word to the leader
        int g = 0;
        for (int fi = 0; walk.next(p, f); ++fi) {
            if (lane == 0) {
                pair_wait(bar(C::kBarQEmpty), (fi & 1) ^ 1, p.wait, abort);
                mbar_arrive_expect_tx(bar(C::kBarQFull), MT * C::kQTile);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int bx = 0; bx < C::kBoxes; ++bx)
                        tma_load_3d(sb + C::kQOff + t * C::kQTile + bx * kQBox, &tm_q, bar(C::kBarQFull), 64 * bx,
                                    f.group * p.group + 128 * (2 * t + rank), f.b * p.H_kv + f.hk);
            }
            __syncwarp();
            const Sight some(p, f);
            pair_wait(bar(C::kBarQFull), fi & 1, p.wait, abort);
            if (lane == 0) arrive_leader(bar(C::kBarQReady));
            for (int j = 0; j < f.n; ++j, ++g) {
                const int st = g % C::kStages;
                pair_wait(bar(C::kBarFull + st), (g / C::kStages) & 1, p.wait, abort);
                mend_v<1>(f, some, kKeys * (f.first + j), smem + C::kStageOff + st * C::kStage + C::kKTile);
                __syncwarp();
                if (lane == 0) arrive_leader(bar(C::kBarReady + st));
            }
        }
    } else if (warp == C::kWarpMma) {
        // ------------------------------------------------------------ MMA issuer (leader)
        if (rank == 0) {
            constexpr uint32_t idesc_qk = idesc_bf16_f32(256, kKeys, false);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(256, DV, true);
            const bool one = elect_one();
            auto commit = [&](int i) {
                if (one) commit_pair(bar(i));
            };
            auto issue_qk = [&](int t, int s, int st) {
                const uint64_t da = smem_desc_sw128(sb + C::kQOff + t * C::kQTile, 16, 1024);
                const uint64_t db = smem_desc_sw128(sb + C::kStageOff + st * C::kStage, 16, 1024);
                if (one) {
#pragma unroll
                    for (int i = 0; i < DQK / 16; ++i)
                        mma_ss_pair(tmem + col_s(s), da + (uint64_t)(((i >> 2) * kQBox + (i & 3) * 32) >> 4),
                                    db + (uint64_t)(((i >> 2) * kKBox + (i & 3) * 32) >> 4), idesc_qk, i > 0 ? 1u : 0u);
                }
                commit(C::kBarSFull + s);
            };
            // half h of the tile's keys: the first can start while the softmax still works on the second
            auto issue_pv = [&](int o, int s, int st, int h, bool acc) {
                const uint64_t dv =
                    smem_desc_sw128(sb + C::kStageOff + st * C::kStage + C::kKTile + h * 8192, kQBox, 1024);
                if (one) {
#pragma unroll
                    for (int i = 0; i < kKeys / 32; ++i)
                        mma_ts_pair(tmem + col_o(o), tmem + col_s(s) + 32 * h + 8 * i, dv + (uint64_t)(i * 2048 >> 4),
                                    idesc_pv, (acc || i > 0) ? 1u : 0u);
                }
            };
            int g = 0;
            for (int fi = 0; walk.next(p, f); ++fi) {
                pair_wait(bar(C::kBarQReady), fi & 1, p.wait, abort);
                pair_wait(bar(C::kBarReady + g % C::kStages), (g / C::kStages) & 1, p.wait, abort);
                tc_fence_after();
                for (int t = 0; t < MT; ++t) issue_qk(t, MT == 2 ? t : (g & 1), g % C::kStages);
                if (f.n == 1) commit(C::kBarQEmpty);
                for (int j = 0; j < f.n; ++j, ++g) {
                    const int st = g % C::kStages, st1 = (g + 1) % C::kStages;
                    const bool nxt = j + 1 < f.n;
                    if (MT == 1 && nxt) {
                        pair_wait(bar(C::kBarReady + st1), ((g + 1) / C::kStages) & 1, p.wait, abort);
                        tc_fence_after();
                        issue_qk(0, (g + 1) & 1, st1);
                        if (j + 2 == f.n) commit(C::kBarQEmpty);
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const int s = MT == 2 ? t : (g & 1);
                        const uint32_t ph = (MT == 2 ? g : g >> 1) & 1;
                        pair_wait(bar(C::kBarPHalf + s), ph, p.wait, abort);
                        if (j == 0) pair_wait(bar(C::kBarOEmpty + t), (fi & 1) ^ 1, p.wait, abort);
                        tc_fence_after();
                        // MT = 1: O s takes every other tile of the fragment
                        issue_pv(s, s, st, 0, j >= (MT == 2 ? 1 : 2));
                        pair_wait(bar(C::kBarPReady + s), ph, p.wait, abort);
                        tc_fence_after();
                        issue_pv(s, s, st, 1, true);
                        if (j + (MT == 2 ? 1 : 2) >= f.n) commit(C::kBarPV + s);
                        if (t == MT - 1) commit(C::kBarEmpty + st);
                        if (MT == 2 && nxt) {
                            if (t == 0) {
                                pair_wait(bar(C::kBarReady + st1), ((g + 1) / C::kStages) & 1, p.wait, abort);
                                tc_fence_after();
                            }
                            issue_qk(t, t, st1);
                            if (t == 1 && j + 2 == f.n) commit(C::kBarQEmpty);
                        }
                    }
                }
            }
        }
    } else if (warp < C::kWarpTma) {
        // ------------------------------------------------------------ softmax + epilogue (both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
        const int t = warp >> 2;
        const int T = MT == 2 ? 2 * t + rank : rank;  // M tile of the row group
        const int i = (warp & 3) * 32 + lane;         // its row == TMEM lane
        if ((warp & 3) < live_warps(T)) {
            const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            const uint32_t s_addr = lane_base + col_s(t), o_addr = lane_base + col_o(t);
            int g = 0;   // tiles so far
            int mine = 0;  // MT = 1: fragments so far that held a tile of this warpgroup
            for (int fi = 0; walk.next(p, f); ++fi) {
                const int r = f.group * p.group + 128 * T + i;  // row of the KV head
                const bool row_ok = r < p.R;                    // padding rows of the last M tile
                int lo;
                const uint64_t drafts = draft_sight(p, f.b, row_ok ? r % p.T : 0, f.s.len, f.s.total, lo);
                float m_run = -INFINITY, l_run = 0.f;
                for (int j = 0; j < f.n; ++j, ++g) {
                    if (MT == 1 && (g & 1) != t) continue;
                    pair_wait(bar(C::kBarSFull + t), (MT == 2 ? g : g >> 1) & 1, p.wait, abort);
                    tc_fence_after();
                    // O's last product came before the product that made these scores: O may be touched
                    softmax_tile<DV, false>(p, s_addr, o_addr, kKeys * (f.first + j), lo, f.s.len, drafts, m_run, l_run,
                                            nullptr, [] {}, [&] {
                                                tmem_wait_st();
                                                tc_fence_before();
                                                __syncwarp();
                                                if (lane == 0) arrive_leader(bar(C::kBarPHalf + t));
                                            });
                    __syncwarp();
                    if (lane == 0) arrive_leader(bar(C::kBarPReady + t));
                }
                const bool whole = f.head && f.tail;
                const size_t row = (size_t)(f.b * p.H_kv + f.hk) * p.R + r;
                const int slot = 2 * share + (f.head ? 1 : 0), rc = 128 * T + i;
                if (MT == 2) {
                    pair_wait(bar(C::kBarPV + t), fi & 1, p.wait, abort);
                    tc_fence_after();
                    write_row<DV, false>(p, o_addr, whole, row_ok, row, slot, rc, m_run, l_run);
                } else {
                    if (f.n > 1 || ((g - 1) & 1) == t) {
                        pair_wait(bar(C::kBarPV + t), mine & 1, p.wait, abort);
                        ++mine;
                    }
                    m_run = row_max(m_run, l_run);
                    float2 *stats = reinterpret_cast<float2 *>(smem + C::kStatsOff) + 256 * (fi & 1);
                    stats[128 * t + i] = make_float2(m_run, l_run);
                    tc_fence_before();
                    named_bar_sync(1, 64 * live_warps(T));  // both warpgroups are done with the fragment's tiles
                    tc_fence_after();
                    const float2 other = stats[128 * (t ^ 1) + i];
                    const float M = fmaxf(m_run, other.x);
                    const float ws = m_run == -INFINITY ? 0.f : fast_exp2(m_run - M);
                    const float wo = other.x == -INFINITY ? 0.f : fast_exp2(other.x - M);
                    const float L = ws * l_run + wo * other.y;
                    join_half(p, lane_base + 64 * t, t == 0 ? ws : wo, t == 0 ? wo : ws, whole, row_ok, row, slot, rc,
                              64 * t, M, L);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(bar(C::kBarOEmpty + (MT == 2 ? t : 0)));
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync();  // every product of the pair has completed and every remote arrival has landed
    if (warp == C::kWarpMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int DQK, int MT>
cudaError_t launch_t(const CacheAttnLaunch &L, int pairs, cudaStream_t stream)
{
    using C = PairCfg<DQK, MT>;
    auto kernel = cache_pair_kernel<DQK, MT>;
    static KernelSetup setup;
    const cudaError_t err = setup(kernel, C::kSmemBytes, C::kLaunchRegs);
    if (err != cudaSuccess) return err;
    return launch_dependent(kernel, 2 * pairs, C::kThreads, C::kSmemBytes, stream, L.tm_q, L.tm_k, L.tm_v, L.p);
}

}  // namespace

cudaError_t launch_cache_pair(const CacheAttnLaunch &L, int pairs, cudaStream_t stream)
{
    if (L.p.d_qk == 128) return L.p.group == 256 ? launch_t<128, 1>(L, pairs, stream) : launch_t<128, 2>(L, pairs, stream);
    return L.p.group == 256 ? launch_t<192, 1>(L, pairs, stream) : launch_t<192, 2>(L, pairs, stream);
}

}  // namespace apex
