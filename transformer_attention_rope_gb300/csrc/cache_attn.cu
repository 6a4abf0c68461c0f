// cache_attn.cu -- attention over caches of rotated keys (sm_103a): trees of drafted
// tokens, and single-query decode that also accumulates attention weights.
//
// Mathematics: the online softmax of Part 2, §6.2 over the keys a row sees, as
// partial results (max, sum, unnormalised output) over ranges of keys, joined by
// softmax's invariance to a shift.  A row that sees nothing has sum 0 and gives 0.
//
// Work: the G * T query rows of a KV head (G heads share it, T drafts) are adjacent
// in memory and form one or two 128-row M tiles, so a K/V tile is read once for all
// of them.  A unit is (sequence, KV head, row group); its key tiles are 128 keys each.
// All tiles of all units, in order, are dealt to the CTAs in equal contiguous shares,
// whatever the lengths -- which only the device knows -- so a ragged batch keeps every
// SM busy to the end.  A CTA's share cuts at most its first and its last unit; cut
// units leave partial results that cache_join_kernel joins, the others are finished
// in place.
//
// Warp roles: 4 softmax warps per M tile (thread i owns row i = TMEM lane i), a TMA
// warp, an MMA warp issuing S = Q K^T and O += P V on tcgen05 (S, O in TMEM, P over S
// as bf16).  With one M tile S has two buffers, so the product of the next tile runs
// under this tile's softmax; with two M tiles the tiles take turns.
//
// Keys that nobody sees -- behind the drafts, before every window, masked in the whole
// tree -- may hold anything: their scores are replaced by -inf, and their V rows are
// set to zero in shared memory before the product (0 * NaN would be NaN).
#include <math.h>

#include "cache_attn.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace apex {
namespace {

constexpr int kKeys = kCacheTileKeys;
constexpr int kBox = 128 * 128;  // [128 rows][64 bf16]

template <int DQK, int DV, int MT>
struct Cfg {
    static constexpr int kQBoxes = DQK / 64, kVBoxes = DV / 64;
    static constexpr int kQTile = kQBoxes * kBox, kKTile = kQBoxes * kBox, kVTile = kVBoxes * kBox;
    // ring depths: what 224 KB hold beside the queries
    static constexpr int kKStages = DQK == 64 ? 6 : (DQK == 128 ? 3 : 2);
    static constexpr int kVStages = DQK == 64 ? 6 : (MT == 1 ? (DQK == 128 ? 3 : 2) : (DQK == 128 ? 2 : 1));
    static constexpr int kThreads = 128 * MT + 64;
    static constexpr int kWarpTma = 4 * MT, kWarpMma = 4 * MT + 1;
    static constexpr int kQOff = 0;
    static constexpr int kKOff = MT * kQTile;
    static constexpr int kVOff = kKOff + kKStages * kKTile;
    static constexpr int kBarOff = kVOff + kVStages * kVTile;
    static constexpr int kBarQFull = 0, kBarQEmpty = 1;
    static constexpr int kBarKFull = 2, kBarKEmpty = kBarKFull + kKStages;
    static constexpr int kBarVFull = kBarKEmpty + kKStages, kBarVEmpty = kBarVFull + kVStages;
    static constexpr int kBarSFull = kBarVEmpty + kVStages;  // [2] per S buffer
    static constexpr int kBarPReady = kBarSFull + 2;         // [2] per S buffer
    static constexpr int kBarPV = kBarPReady + 2;            // [MT] one phase per tile
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

// ---------------------------------------------------------------- schedule
// Lengths of sequence b: cached keys, keys with its drafts, its first key tile and
// number of tiles (one at least, so that every unit writes its output).
struct Seq {
    int len, total, tile0, tiles;
    __device__ __forceinline__ void load(const CacheAttnParams &p, int b)
    {
        len = min(max(__ldg(p.lens + b), 0), p.S_cap);
        total = min(len + p.drafts, p.S_cap);
        const int lo = p.window > 0 ? max(0, len - p.window + 1) : 0;
        tile0 = lo / kKeys;
        tiles = max(1, (total + kKeys - 1) / kKeys - tile0);
    }
};

// Where a CTA's share starts, and how the shares are cut.
struct Sched {
    long long tile, total;  // first tile of the share, tiles of all units
    int left;               // tiles of the share
    int n_cta;              // CTAs that have a share
    int b, unit, off;       // sequence, unit within it and tile within the unit of the first tile
};

// One warp: the share of this CTA, tiles [total * c / n, total * (c + 1) / n).
__device__ __forceinline__ void make_sched(const CacheAttnParams &p, Sched *out)
{
    const int lane = threadIdx.x & 31;
    const int per_b = p.H_kv * p.n_groups;
    long long total = 0;
    Seq s;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        s.tiles = 0;
        if (b0 + lane < p.B) s.load(p, b0 + lane);
        total += __reduce_add_sync(0xffffffffu, s.tiles);
    }
    total *= per_b;
    Sched r;
    r.total = total;
    r.n_cta = (int)min((long long)gridDim.x, total);
    const int c = blockIdx.x;
    r.tile = c < r.n_cta ? total * c / r.n_cta : total;
    r.left = c < r.n_cta ? (int)(total * (c + 1) / r.n_cta - r.tile) : 0;
    r.b = r.unit = r.off = 0;
    if (r.left > 0) {
        long long before = 0;  // tiles of the sequences before b0
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            if (p.B > 32) {  // else the lanes still hold the lengths
                s.tiles = 0;
                if (b0 + lane < p.B) s.load(p, b0 + lane);
            }
            int incl = s.tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const long long end = before + (long long)incl * per_b;
            const uint32_t past = __ballot_sync(0xffffffffu, end > r.tile && b0 + lane < p.B);
            if (past) {
                const int w = __ffs(past) - 1;
                const int tiles = __shfl_sync(0xffffffffu, s.tiles, w);
                const long long start = __shfl_sync(0xffffffffu, end - (long long)s.tiles * per_b, w);
                r.b = b0 + w;
                r.unit = (int)((r.tile - start) / tiles);
                r.off = (int)((r.tile - start) % tiles);
                break;
            }
            before = __shfl_sync(0xffffffffu, end, 31);
        }
    }
    if (lane == 0) *out = r;
}

// The part of one unit that a CTA works on: n tiles from tile `first` of the sequence.
struct Frag {
    Seq s;
    int b, hk, group, unit;  // unit: index over all units
    int first, n;
    bool head, tail;         // holds the unit's first / last tile
};

struct Walk {
    Sched s;
    Seq seq;
    bool fresh;
    __device__ __forceinline__ Walk(const CacheAttnParams &p, const Sched &sched) : s(sched), fresh(true) {}
    __device__ __forceinline__ bool next(const CacheAttnParams &p, Frag &f)
    {
        if (s.left <= 0) return false;
        const int per_b = p.H_kv * p.n_groups;
        if (fresh) seq.load(p, s.b);
        fresh = false;
        f.s = seq;
        f.b = s.b;
        f.hk = s.unit / p.n_groups;
        f.group = s.unit % p.n_groups;
        f.unit = s.b * per_b + s.unit;
        f.first = seq.tile0 + s.off;
        f.n = min(seq.tiles - s.off, s.left);
        f.head = s.off == 0;
        f.tail = s.off + f.n == seq.tiles;
        s.left -= f.n;
        s.tile += f.n;
        s.off = 0;
        if (++s.unit == per_b) {
            s.unit = 0;
            ++s.b;
            fresh = true;
        }
        return true;
    }
};

// ---------------------------------------------------------------- masks
// Drafts that draft t of sequence b sees, and its first visible cached key.
__device__ __forceinline__ uint64_t draft_sight(const CacheAttnParams &p, int b, int t, int len, int total, int &lo)
{
    lo = 0;
    if (p.drafts == 0) return 0;
    uint64_t w = p.tree_mask ? p.tree_mask[b * p.mask_stride + t] : (~0ull >> (63 - t));
    const int n = total - len;  // drafts that the cache holds
    w = n >= 64 ? w : (w & ((1ull << n) - 1));
    if (p.window > 0) {
        const int *pos = p.positions ? p.positions + (long long)b * p.T : nullptr;
        const long long m = pos ? max(pos[t], len) : (long long)len + t;
        lo = (int)min((long long)len, max(0ll, m - p.window + 1));
        for (int u = 0; u < n; ++u) {
            const long long at = pos ? max(pos[u], len) : (long long)len + u;
            if (m - at >= p.window) w &= ~(1ull << u);
        }
    }
    return w;
}

__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// Visibility of the 128 keys of the tile at k0: cached keys [lo, len) and drafts.
__device__ __forceinline__ void sight_words(uint32_t (&w)[4], int k0, int lo, int len, uint64_t drafts)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bits_below(len - k0 - 32 * i) & ~bits_below(lo - k0 - 32 * i);
    const int s = len - k0;  // column of draft 0
    uint64_t d0 = 0, d1 = 0;
    if (s <= -64 || s >= 128) {
    } else if (s < 0) {
        d0 = drafts >> -s;
    } else if (s == 0) {
        d0 = drafts;
    } else if (s < 64) {
        d0 = drafts << s;
        d1 = drafts >> (64 - s);
    } else {
        d1 = drafts << (s - 64);
    }
    w[0] |= (uint32_t)d0;
    w[1] |= (uint32_t)(d0 >> 32);
    w[2] |= (uint32_t)d1;
    w[3] |= (uint32_t)(d1 >> 32);
}

__device__ __forceinline__ void tma_load_3d_policy(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y,
                                                   int z, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
        "{%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

// ---------------------------------------------------------------- attention
template <int DQK, int DV, int MT, bool WEIGHTS>
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
    static_assert(sizeof(Sched) <= 48, "schedule slot");
    if (warp == C::kWarpTma) make_sched(p, sched);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kTmemSlot);

    Walk walk(p, *sched);
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
            for (int fi = 0; walk.next(p, f); ++fi) {
                const int kv = f.b * p.H_kv + f.hk;
                if (f.head) {
                    // the CTAs that hold this unit's first and last tile
                    const long long end = walk.s.tile - f.n + f.s.tiles;
                    p.units[f.unit] = make_int2(blockIdx.x, (int)((end * walk.s.n_cta - 1) / walk.s.total));
                }
                mbar_wait(bar(C::kBarQEmpty), (fi & 1) ^ 1, p.wait);
                mbar_arrive_expect_tx(bar(C::kBarQFull), MT * C::kQTile);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int bx = 0; bx < C::kQBoxes; ++bx)
                        tma_load_3d(sb + C::kQOff + t * C::kQTile + bx * kBox, &tm_q, bar(C::kBarQFull), 64 * bx,
                                    f.group * p.group + 128 * t, kv);
                for (int j = 0; j < f.n; ++j, ++g) {
                    const int key0 = kKeys * (f.first + j);
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
    } else if (warp == C::kWarpMma) {
        // ------------------------------------------------------------ MMA issuer (lane 0; the warp mends V tiles)
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kKeys, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DV, true);
        // the empty asm keeps a descriptor's base a runtime value, stepped by its
        // address field, instead of one live register pair per tile and stage
        auto desc_base = [&](uint32_t addr, uint32_t lbo) -> uint64_t {
            uint64_t d = smem_desc_sw128(addr, lbo, 1024);
            asm volatile("" : "+l"(d));
            return d;
        };
        auto issue_qk = [&](int t, int s, int ks) {
            if (lane == 0) {
                const uint64_t da = desc_base(sb + C::kQOff + t * C::kQTile, 16);
                const uint64_t db = desc_base(sb + C::kKOff + ks * C::kKTile, 16);
#pragma unroll
                for (int i = 0; i < DQK / 16; ++i) {
                    const uint64_t off = ((i >> 2) * kBox + (i & 3) * 32) >> 4;
                    umma_ss(tmem + C::col_s(s), da + off, db + off, idesc_qk, i > 0 ? 1u : 0u);
                }
                tc_commit(bar(C::kBarSFull + s));
            }
        };
        auto issue_pv = [&](int t, int s, int vs, bool acc) {
            if (lane == 0) {
                const uint64_t dv = desc_base(sb + C::kVOff + vs * C::kVTile, kBox);
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i)
                    umma_ts(tmem + C::col_o(t), tmem + C::col_s(s) + 8 * i, dv + (uint64_t)(i * 2048 >> 4), idesc_pv,
                            (acc || i > 0) ? 1u : 0u);
                tc_commit(bar(C::kBarPV + t));
            }
        };
        auto commit = [&](int i) {
            if (lane == 0) tc_commit(bar(i));
        };
        int g = 0;
        for (int fi = 0; walk.next(p, f); ++fi) {
            // zero the V rows that no row sees, in the tiles that hold any
            const int lo_all = p.window > 0 ? max(0, f.s.len - p.window + 1) : 0;
            uint64_t any = 0;
            bool have_any = false;
            auto mend_v = [&](int key0, int vs) {
                if (key0 >= lo_all && key0 + kKeys <= f.s.len) return;
                if (!have_any) {
                    int lo;
                    for (int t = lane; t < p.T && p.drafts; t += 32)
                        any |= draft_sight(p, f.b, t, f.s.len, f.s.total, lo);
                    any = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)any) |
                          ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32);
                    have_any = true;
                }
                uint32_t w[4];
                sight_words(w, key0, lo_all, f.s.len, any);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((w[i] >> lane) & 1))
                        for (int bx = 0; bx < C::kVBoxes; ++bx) {
                            uint4 *row = reinterpret_cast<uint4 *>(smem + C::kVOff + vs * C::kVTile + bx * kBox +
                                                                   (32 * i + lane) * 128);
#pragma unroll
                            for (int c = 0; c < 8; ++c) row[(c + lane) & 7] = make_uint4(0, 0, 0, 0);
                        }
                fence_proxy_async_smem();
                __syncwarp();
            };
            mbar_wait(bar(C::kBarQFull), fi & 1, p.wait);
            mbar_wait(bar(C::kBarKFull + g % C::kKStages), (g / C::kKStages) & 1, p.wait);
            tc_fence_after();
            for (int t = 0; t < MT; ++t) issue_qk(t, MT == 2 ? t : (g & 1), g % C::kKStages);
            commit(C::kBarKEmpty + g % C::kKStages);
            if (f.n == 1) commit(C::kBarQEmpty);
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
                mend_v(kKeys * (f.first + j), vs);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int s = MT == 2 ? t : (g & 1);
                    mbar_wait(bar(C::kBarPReady + s), (MT == 2 ? g : g >> 1) & 1, p.wait);
                    if (j == 0) mbar_wait(bar(C::kBarOEmpty + t), (fi & 1) ^ 1, p.wait);
                    tc_fence_after();
                    issue_pv(t, s, vs, j > 0);
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
        // every product of this CTA is issued: the joining kernel's launch may overlap the rest
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    } else if ((warp & 3) < live_warps(warp >> 2)) {
        // ------------------------------------------------------------ softmax + epilogue
        const int t = warp >> 2;
        const int i = (warp & 3) * 32 + lane;  // row of the M tile == TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_addr = lane_base + C::col_o(t);
        int g = 0;
        for (int fi = 0; walk.next(p, f); ++fi) {
            const int r = f.group * p.group + 128 * t + i;  // row of the KV head
            const bool row_ok = r < p.R;
            const int kv = f.b * p.H_kv + f.hk;
            int lo;
            const uint64_t drafts = draft_sight(p, f.b, row_ok ? r % p.T : 0, f.s.len, f.s.total, lo);
            float m_run = -INFINITY, l_run = 0.f;
            float *scores = nullptr;
            if (WEIGHTS) scores = p.scores + ((size_t)kv * p.R + r) * p.S_pad;

            for (int j = 0; j < f.n; ++j, ++g) {
                const int s = MT == 2 ? t : (g & 1);
                const uint32_t s_addr = lane_base + C::col_s(s);
                const int key0 = kKeys * (f.first + j);
                mbar_wait(bar(C::kBarSFull + s), (MT == 2 ? g : g >> 1) & 1, p.wait);
                tc_fence_after();
                uint32_t v[128];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    tmem_ld32(s_addr + 32 * ch, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * ch]));
                tmem_wait_ld();
                if (!__all_sync(0xffffffffu, key0 >= lo && key0 + kKeys <= f.s.len)) {
                    uint32_t w[4];
                    sight_words(w, key0, lo, f.s.len, drafts);
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (!((w[e >> 5] >> (e & 31)) & 1)) v[e] = 0xff800000u;
                }
                if (WEIGHTS && row_ok) {
#pragma unroll
                    for (int e = 0; e < 128; e += 4)
                        *reinterpret_cast<uint4 *>(scores + key0 + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                float acc[8];
#pragma unroll
                for (int a = 0; a < 8; ++a) acc[a] = __uint_as_float(v[a]);
#pragma unroll
                for (int e = 8; e + 16 <= 128; e += 16)
#pragma unroll
                    for (int a = 0; a < 8; ++a)
                        acc[a] = fmax3(acc[a], __uint_as_float(v[e + a]), __uint_as_float(v[e + 8 + a]));
#pragma unroll
                for (int a = 0; a < 8; ++a) acc[a] = fmaxf(acc[a], __uint_as_float(v[120 + a]));
                const float mx = fmax3(fmax3(acc[0], acc[1], acc[2]), fmax3(acc[3], acc[4], acc[5]), fmaxf(acc[6], acc[7]));
                const float m_new = fmaxf(m_run, mx * p.scale_log2);
                // O is rescaled only when the maximum grew by more than 2^8: the final
                // O / l does not depend on the reference point
                const bool need = (m_run != -INFINITY) && (m_new > m_run + 8.f);
                // O's last product (of tile g - 1) must be done before O is touched; waited for in
                // every tile, so that no phase of the barrier is skipped
                if (g > 0) mbar_wait(bar(C::kBarPV + t), (g - 1) & 1, p.wait);
                if (__any_sync(0xffffffffu, need)) {
                    tc_fence_after();
                    const float alpha = (m_new == -INFINITY) ? 1.f : fast_exp2(m_run - m_new);
                    l_run *= alpha;
                    m_run = m_new;
#pragma unroll 1
                    for (int ch = 0; ch < DV / 16; ++ch) {
                        uint32_t o[16];
                        tmem_ld16(o_addr + 16 * ch, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st16(o_addr + 16 * ch, o);
                    }
                } else if (m_run == -INFINITY) {
                    m_run = m_new;
                }
                const float m_use = (m_run == -INFINITY) ? 0.f : m_run;
                const uint64_t SC = f2_pack(p.scale_log2, p.scale_log2);
                const uint64_t NM = f2_pack(-m_use, -m_use);
                uint64_t lacc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e2 = 0; e2 < 16; ++e2) {
                        const uint64_t x =
                            f2_pack(__uint_as_float(v[32 * q4 + 2 * e2]), __uint_as_float(v[32 * q4 + 2 * e2 + 1]));
                        float y0, y1;
                        f2_unpack(f2_fma(x, SC, NM), y0, y1);
                        const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                        lacc[e2 & 3] = f2_add(lacc[e2 & 3], f2_pack(p0, p1));
                        pk[e2] = pack_bf16x2(p0, p1);  // the tensor cores take bf16; the sum keeps fp32
                    }
                    tmem_st16(s_addr + 16 * q4, pk);
                }
                {
                    float a0, a1;
                    f2_unpack(f2_add(f2_add(lacc[0], lacc[1]), f2_add(lacc[2], lacc[3])), a0, a1);
                    l_run += a0 + a1;
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarPReady + s));
            }

            // ---- epilogue: the finished row, or this fragment's partial result
            mbar_wait(bar(C::kBarPV + t), (g - 1) & 1, p.wait);
            tc_fence_after();
            const bool whole = f.head && f.tail;
            const float inv = (l_run > 0.f) ? 1.f / l_run : 0.f;
            const int slot = 2 * blockIdx.x + (f.head ? 1 : 0);
            const size_t part = (size_t)slot * p.rows_cap + 128 * t + i;
            if (row_ok && !whole) p.ws_ml[part] = make_float2(m_run, l_run);
            if (WEIGHTS && row_ok && whole) p.lse[(size_t)kv * p.R + r] = m_run + log2f(l_run);
            uint4 *dst16 = reinterpret_cast<uint4 *>(p.out + ((size_t)kv * p.R + r) * DV);
            uint4 *dst32 = reinterpret_cast<uint4 *>(p.ws_o + part * DV);
#pragma unroll
            for (int ch = 0; ch < DV / 32; ++ch) {
                uint32_t v[32];
                tmem_ld32(o_addr + 32 * ch, v);
                tmem_wait_ld();
                if (row_ok && whole) {
                    uint32_t w2[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w2[e] = pack_bf16x2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        dst16[4 * ch + q4] = make_uint4(w2[4 * q4], w2[4 * q4 + 1], w2[4 * q4 + 2], w2[4 * q4 + 3]);
                } else if (row_ok) {
#pragma unroll
                    for (int q4 = 0; q4 < 8; ++q4)
                        dst32[8 * ch + q4] = make_uint4(v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]);
                }
            }
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
// max and sum of a row of a cut unit over its fragments, and the shift of this lane's
// fragment c0 + lane: the fragments of unit u are the last of CTA c0 (slot 2 c0 + 1),
// then the first of each CTA up to c1 (slots 2 c).
struct RowParts {
    const CacheAttnParams &p;
    int c0, n, rc;
    __device__ __forceinline__ size_t at(int i) const
    {
        return (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * p.rows_cap + rc;
    }
    // log2 of the sum of all fragments, relative to the maximum M
    __device__ __forceinline__ void stats(int lane, float &M, float &L, float2 &mine) const
    {
        mine = make_float2(-INFINITY, 0.f);
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

template <int E>
struct Vec;
template <>
struct Vec<2> {
    float2 v;
    __device__ __forceinline__ float at(int e) const { return e ? v.y : v.x; }
};
template <>
struct Vec<4> {
    float4 v;
    __device__ __forceinline__ float at(int e) const { return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w; }
};

template <int E>
__device__ __forceinline__ void store_row(uint16_t *out, int lane, const float (&acc)[E], float L)
{
    const float inv = (L > 0.f) ? 1.f / L : 0.f;
    uint32_t *dst = reinterpret_cast<uint32_t *>(out) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
}

// One row of a cut unit to a block: its 8 warps share the fragments (few units, cut
// into many).
template <int DV>
__device__ __forceinline__ void join_many(const CacheAttnParams &p, int n_units, float (*sh)[DV])
{
    constexpr int E = DV / 32;  // entries per lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / p.rows_cap, rc = blockIdx.x % p.rows_cap;
    const int r = unit % p.n_groups * p.group + rc;
    if (r >= p.R) return;
    const int2 c = p.units[unit];
    if (c.x == c.y) return;
    const RowParts parts{p, c.x, c.y - c.x + 1, rc};
    float M, L;
    float2 mine;
    parts.stats(lane, M, L, mine);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < parts.n; i += 8) {
        const Vec<E> o = *reinterpret_cast<const Vec<E> *>(p.ws_o + parts.at(i) * DV + lane * E);
        const float m = i < 32 ? __shfl_sync(0xffffffffu, mine.x, i & 31) : p.ws_ml[parts.at(i)].x;
        const float w = (m == -INFINITY) ? 0.f : exp2f(m - M);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, o.at(e), acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sh[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < 8; ++w)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += sh[w][lane * E + e];
    store_row<E>(p.out + ((size_t)(unit / p.n_groups) * p.R + r) * DV, lane, acc, L);
}

// 32 rows of a cut unit to a block, 4 to a warp (many units, cut into a few fragments
// each): lanes 8 k .. 8 k + 7 hold the statistics of row k's fragments, eight at a time.
template <int DV>
__device__ __forceinline__ void join_few(const CacheAttnParams &p, int row_blocks)
{
    constexpr int E = DV / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / row_blocks, rc0 = blockIdx.x % row_blocks * 32 + 4 * warp;
    const int r0 = unit % p.n_groups * p.group + rc0;
    const int rows = min(4, min(p.R - r0, p.rows_cap - rc0));
    if (rows <= 0) return;
    const int2 c = p.units[unit];
    if (c.x == c.y) return;
    const int n = c.y - c.x + 1;
    const RowParts stat{p, c.x, n, rc0 + min(lane >> 3, rows - 1)};  // this lane's row, for the statistics
    float M = -INFINITY;
    for (int i = lane & 7; i < n; i += 8) M = fmaxf(M, p.ws_ml[stat.at(i)].x);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float acc[4][E];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 8) {
        float w = 0.f;
        if (i0 + (lane & 7) < n) {
            const float2 v = p.ws_ml[stat.at(i0 + (lane & 7))];
            w = v.x == -INFINITY ? 0.f : exp2f(v.x - M);
            L += w * v.y;
        }
#pragma unroll 2
        for (int i = i0; i < min(i0 + 8, n); ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const RowParts part{p, c.x, n, rc0 + min(k, rows - 1)};
                const Vec<E> o = *reinterpret_cast<const Vec<E> *>(p.ws_o + part.at(i) * DV + lane * E);
                const float wk = __shfl_sync(0xffffffffu, w, 8 * k + i - i0);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[k][e] = fmaf(wk, o.at(e), acc[k][e]);
            }
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const size_t out0 = (size_t)(unit / p.n_groups) * p.R + r0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float Lk = __shfl_sync(0xffffffffu, L, 8 * k);
        if (k < rows) store_row<E>(p.out + (out0 + k) * DV, lane, acc[k], Lk);
    }
}

// acc[b, g, j] += sum over the heads of g of 2^(scale score - lse), heads in order:
// a block takes 1024 keys of a (sequence, KV head), a thread four neighbours.
constexpr int kWeightKeys = 1024;
__device__ __forceinline__ void add_weights(const CacheAttnParams &p, long long block, int chunks, float *lse)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = (int)(block / chunks);
    const int j0 = (int)(block % chunks) * kWeightKeys;
    const int len = min(max(p.lens[unit / p.H_kv], 0), p.S_cap);
    if (j0 >= len) return;
    const int2 c = p.units[unit];
    const int j = j0 + 4 * threadIdx.x;
    const float *s = p.scores + (size_t)unit * p.G * p.S_pad + j;
    for (int g = warp; g < p.G; g += 8) {
        float x;
        if (c.x == c.y) {
            x = p.lse[(size_t)unit * p.G + g];
        } else {
            const RowParts parts{p, c.x, c.y - c.x + 1, g};
            float M, L;
            float2 mine;
            parts.stats(lane, M, L, mine);
            x = M + log2f(L);
        }
        if (lane == 0) lse[g] = x;
    }
    __syncthreads();
    if (j >= len) return;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int g = 0; g < p.G; ++g) {
        // exp2f: weights below 2^-126 are kept, as the sums of a long service need them
        const float4 x = *reinterpret_cast<const float4 *>(s + (size_t)g * p.S_pad);
        w[0] += exp2f(fmaf(x.x, p.scale_log2, -lse[g]));
        w[1] += exp2f(fmaf(x.y, p.scale_log2, -lse[g]));
        w[2] += exp2f(fmaf(x.z, p.scale_log2, -lse[g]));
        w[3] += exp2f(fmaf(x.w, p.scale_log2, -lse[g]));
    }
    float *acc = p.acc + (size_t)unit * p.S_cap + j;
    if (j + 4 <= len && (reinterpret_cast<uintptr_t>(acc) & 15) == 0) {
        float4 a = *reinterpret_cast<float4 *>(acc);
        a.x += w[0];
        a.y += w[1];
        a.z += w[2];
        a.w += w[3];
        *reinterpret_cast<float4 *>(acc) = a;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < len) acc[e] += w[e];
    }
}

// The first blocks join rows; with WEIGHTS the others add weights, each from its own
// join of the statistics.
template <int DV, bool MANY, bool WEIGHTS>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheAttnParams p, int n_units, int join_blocks,
                                                         int row_blocks, int chunks)
{
    __shared__ float sh[MANY ? 8 : 1][DV];
    __shared__ float lse[16];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the next kernel's launch may overlap this one (it waits for it before it reads)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!WEIGHTS || blockIdx.x < join_blocks) {
        if (MANY)
            join_many<DV>(p, n_units, sh);
        else
            join_few<DV>(p, row_blocks);
    } else {
        add_weights(p, blockIdx.x - join_blocks, chunks, lse);
    }
}

template <int DQK, int DV, int MT, bool WEIGHTS>
cudaError_t launch_t(const CacheAttnLaunch &L, int grid, cudaStream_t stream)
{
    using C = Cfg<DQK, DV, MT>;
    auto kernel = cache_attn_kernel<DQK, DV, MT, WEIGHTS>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (err != cudaSuccess) return err;
    return launch_dependent(kernel, grid, C::kThreads, C::kSmemBytes, stream, L.tm_q, L.tm_k, L.tm_v, L.p);
}

template <int DQK, int DV>
cudaError_t launch_d(const CacheAttnLaunch &L, int grid, cudaStream_t stream)
{
    if (L.p.acc) return launch_t<DQK, DV, 1, true>(L, grid, stream);
    return L.p.group == 128 ? launch_t<DQK, DV, 1, false>(L, grid, stream) : launch_t<DQK, DV, 2, false>(L, grid, stream);
}

template <int DV, bool MANY>
cudaError_t launch_join_t(const CacheAttnParams &p, cudaStream_t stream)
{
    const int n_units = p.B * p.H_kv * p.n_groups;
    const int row_blocks = MANY ? p.rows_cap : (p.rows_cap + 31) / 32;
    const long long join_blocks = (long long)n_units * row_blocks;
    const int chunks = (p.S_cap + kWeightKeys - 1) / kWeightKeys;
    const long long blocks = join_blocks + (p.acc ? (long long)n_units * chunks : 0);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    if (p.acc)
        return launch_dependent(cache_join_kernel<DV, MANY, true>, (int)blocks, 256, 0, stream, p, n_units,
                                (int)join_blocks, row_blocks, chunks);
    return launch_dependent(cache_join_kernel<DV, MANY, false>, (int)blocks, 256, 0, stream, p, n_units,
                            (int)join_blocks, row_blocks, chunks);
}

template <int DV>
cudaError_t launch_join(const CacheAttnParams &p, int grid, cudaStream_t stream)
{
    // few units: each is cut into many fragments, which then share a block
    return 4ll * p.B * p.H_kv * p.n_groups <= grid ? launch_join_t<DV, true>(p, stream)
                                                   : launch_join_t<DV, false>(p, stream);
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnLaunch &L, int sm_count, cudaStream_t stream)
{
    const CacheAttnParams &p = L.p;
    const int grid = std::min(sm_count, cache_attn_ctas(p.B, p.H_kv, p.n_groups, p.S_cap));
    cudaError_t err = p.d_qk == 64    ? launch_d<64, 64>(L, grid, stream)
                      : p.d_qk == 128 ? launch_d<128, 128>(L, grid, stream)
                                      : launch_d<192, 128>(L, grid, stream);
    if (err != cudaSuccess) return err;
    return p.d_v == 64 ? launch_join<64>(p, grid, stream) : launch_join<128>(p, grid, stream);
}

}  // namespace apex
