// evict.cu -- cutting a cache down to a budget of rows per (sequence, KV head).
//
// One cluster of CTAs per (sequence, KV head), each warp with a contiguous part of its
// rows, whose weights and positions stay in registers.  A row's ranking key: rows
// that must stay (sinks, newest positions) have the largest, the others the order-
// preserving integer image of their weight.  A radix search over 8-bit digits, most
// significant first, finds the budget-th largest key: each CTA pushes its digit counts
// into every CTA of the cluster (distributed shared memory), so that a digit costs one
// cluster barrier and no remote read.  Of the rows that equal that key the lowest are
// kept.
//
// Kept rows past the budget (sources) pair up, in ascending order, with freed rows
// below it (holes); the cluster then copies each source's key, value, weight and
// position into its hole.  Sources and holes never meet, so the copies need no order
// among themselves, and a cache slightly over its budget moves only the few rows
// that are past it.
//
// Bound: latency of the search, about 2 us a digit and 4 for the two walks, then HBM for
// the moves.  64 caches of 4224 rows cut to 4096: 12.3 us; 32 of 32768 rows cut to 4096 with
// 110 MB moved: 37 us, 20 of them the moves at 5.5 TB/s.
#include <cooperative_groups.h>
#include <limits.h>

#include "device_common.cuh"
#include "evict.h"

namespace cg = cooperative_groups;

namespace apex {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMoveRows = 4;  // rows a warp has in flight
constexpr int kItems = 8;     // rows of a lane in one block of a warp's rows
constexpr int kBlock = 32 * kItems;
constexpr uint32_t kMust = 0xffffffffu;

struct Shared {
    uint32_t hist[4][256];                     // this CTA's digit counts
    uint32_t inbox[2][kMaxCluster][256];       // those of the whole cluster, by turns
    uint32_t warp[2][kWarps];
    uint32_t digit, above, equal;
    int len, next;      // of the sequence, in the first CTA
    int top[kWarps];    // the largest position of each warp's rows
    uint32_t count[2];  // this CTA's ties, then its holes and sources, for the cluster
};

// Order-preserving image of a weight; NaN below everything, -0 as +0.  No image
// is kMust (that would be a NaN's).
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sums of two counters over the warps before this one, and over all; every lane of a
// warp passes its warp's counts.
__device__ __forceinline__ void before_warp(Shared &sh, uint32_t c0, uint32_t c1, uint32_t &p0, uint32_t &p1,
                                            uint32_t &t0, uint32_t &t1)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) {
        sh.warp[0][warp] = c0;
        sh.warp[1][warp] = c1;
    }
    __syncthreads();
    const uint32_t a = lane < kWarps ? sh.warp[0][lane] : 0, b = lane < kWarps ? sh.warp[1][lane] : 0;
    p0 = __reduce_add_sync(0xffffffffu, lane < warp ? a : 0);
    p1 = __reduce_add_sync(0xffffffffu, lane < warp ? b : 0);
    t0 = __reduce_add_sync(0xffffffffu, a);
    t1 = __reduce_add_sync(0xffffffffu, b);
}

// chunk: rows of a CTA; seg: rows of a warp, a multiple of 32 (chunk <= kWarps * seg).
// ONE: seg <= kBlock, the rows are read once and kept; else they are read again, from
// L2, in each of the up to eight walks over them (64 caches of 4224 rows 12.3 us kept, 14.3
// read again; 32 of 32768 rows 37.5 and 40.1).
template <bool ONE>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictParams p, int chunk, int seg)
{
    __shared__ __align__(16) Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    const int unit = blockIdx.x / cs;
    const int b = unit / p.H_kv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 4 * 256; i += kThreads) (&sh.hist[0][0])[i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lo = min(rank * chunk, p.S_cap), hi = min(lo + chunk, p.S_cap);
    const int wlo = min(lo + warp * seg, hi), whi = min(wlo + seg, hi);  // this warp's rows
    const size_t base = (size_t)unit * p.S_cap;

    float w[kItems];
    int pos[kItems];
    auto load = [&](int j0) {  // rows j0 + 32 e + lane
#pragma unroll
        for (int e = 0; e < kItems; ++e) {
            const int j = j0 + 32 * e + lane;
            w[e] = 0.f;
            pos[e] = j;
            if (j < whi) {
                w[e] = p.acc[base + j];
                if (p.positions) pos[e] = p.positions[base + j];
            }
        }
    };
    // visit(j0) for the blocks of this warp's rows, in order
    auto blocks = [&](auto &&visit) {
        if (ONE) {
            visit(wlo);
        } else {
            for (int j0 = wlo; j0 < whi; j0 += kBlock) {
                load(j0);
                visit(j0);
            }
        }
    };
    if (ONE) load(wlo);

    // One CTA reads the length, so that the whole cluster walks the same path through its
    // barriers; the rows are under way meanwhile.
    if (rank == 0 && tid == 0) {
        sh.len = p.lens[b];
        sh.next = p.next_pos[b];
    }
    cluster.sync();  // every CTA runs, and its counts are clear
    const int n = min(max(*cluster.map_shared_rank(&sh.len, 0), 0), p.S_cap);
    long long next = *cluster.map_shared_rank(&sh.next, 0);
    const int wend = min(whi, n);  // this warp's rows that hold a key
    const int out_len = min(n, p.budget);
    auto key = [&](int e) -> uint32_t {
        return (pos[e] < p.n_sink || pos[e] >= next - p.n_recent) ? kMust : weight_key(w[e]);
    };

    uint32_t cut = 0;      // the budget-th largest key
    uint32_t ties = 0;     // rows equal to it that are kept
    bool all_ties = true;  // every row equal to it is kept
    if (n > p.budget) {    // the same for the whole cluster
        if (p.newest) {  // positions without next_pos: one past the largest, lens where that is more
            int top = INT_MIN;
            blocks([&](int j0) {
#pragma unroll
                for (int e = 0; e < kItems; ++e)
                    if (j0 + 32 * e + lane < wend) top = max(top, pos[e]);
            });
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) sh.top[warp] = top;
            cluster.sync();  // read by every CTA; not written again
            for (int i = lane; i < cs * kWarps; i += 32)
                top = max(top, *cluster.map_shared_rank(&sh.top[i % kWarps], i / kWarps));
            next = max(next, 1ll + __reduce_max_sync(0xffffffffu, top));
        }
        uint32_t want = p.budget;  // rows to take from those that match the prefix
#pragma unroll
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            blocks([&](int j0) {
#pragma unroll
                for (int e = 0; e < kItems; ++e) {
                    const uint32_t k = key(e);
                    if (j0 + 32 * e + lane < wend && (pass == 0 || ((k ^ cut) >> (shift + 8)) == 0))
                        atomicAdd(&sh.hist[pass][(k >> shift) & 255u], 1u);
                }
            });
            __syncthreads();
            // 64 threads push the counts to each CTA
            for (int i = tid; i < 64 * cs; i += kThreads)
                reinterpret_cast<uint4 *>(cluster.map_shared_rank(&sh.inbox[pass & 1][rank][0], i >> 6))[i & 63] =
                    reinterpret_cast<const uint4 *>(&sh.hist[pass][0])[i & 63];
            cluster.sync();
            uint32_t mine = 0, suffix = 0;  // rows with digit tid, with digit tid or larger in this warp
            if (tid < 256) {
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    if (r < cs) mine += sh.inbox[pass & 1][r][tid];
                suffix = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_down_sync(0xffffffffu, suffix, o);
                    if (lane + o < 32) suffix += x;
                }
                if (lane == 0) sh.warp[0][warp] = suffix;
            }
            __syncthreads();
            if (tid < 256) {
                const uint32_t later = __reduce_add_sync(0xffffffffu, lane < 8 && lane > warp ? sh.warp[0][lane] : 0);
                const uint32_t larger = later + suffix - mine;
                if (larger < want && larger + mine >= want) {
                    sh.digit = tid;
                    sh.above = larger;
                    sh.equal = mine;
                }
            }
            __syncthreads();
            cut |= sh.digit << shift;
            want -= sh.above;
            all_ties = sh.equal == want;
            // every row with this prefix stays: the digits below it do not matter (for weights
            // that differ, usually after three of four)
            if (all_ties) break;
        }
        ties = want;
    }

    // Rows equal to the cut in the parts and warps before this one, where not all stay
    uint32_t tie_base = 0;
    if (n > p.budget && !all_ties) {
        uint32_t mine = 0;
        blocks([&](int j0) {
#pragma unroll
            for (int e = 0; e < kItems; ++e)
                mine += __popc(__ballot_sync(0xffffffffu, j0 + 32 * e + lane < wend && key(e) == cut));
        });
        uint32_t before, unused, total, unused2;
        before_warp(sh, mine, 0, before, unused, total, unused2);
        if (tid == 0) sh.count[0] = total;
        cluster.sync();
        for (int r = 0; r < rank; ++r) tie_base += cluster.map_shared_rank(&sh.count[0], r)[0];
        tie_base += before;
        cluster.sync();
    }

    // A walk over this warp's rows in order: which are kept, which are holes and sources
    auto walk = [&](auto &&visit) {
        uint32_t seen = tie_base;
        blocks([&](int j0) {
#pragma unroll
            for (int e = 0; e < kItems; ++e) {
                const int j = j0 + 32 * e + lane;
                const bool there = j < wend;
                bool kept = there;
                if (n > p.budget) {
                    const uint32_t k = key(e);
                    kept = there && k >= cut;
                    if (!all_ties) {
                        const uint32_t tie = __ballot_sync(0xffffffffu, there && k == cut);
                        if (there && k == cut) kept = seen + __popc(tie & ((1u << lane) - 1u)) < ties;
                        seen += __popc(tie);
                    }
                }
                const bool hole = there && !kept && j < p.budget, src = kept && j >= p.budget;
                visit(j, e, kept, hole, src, __ballot_sync(0xffffffffu, hole), __ballot_sync(0xffffffffu, src));
            }
        });
    };
    uint32_t n_hole = 0, n_src = 0;
    if (n > p.budget)
        walk([&](int, int, bool, bool, bool, uint32_t bh, uint32_t bs) {
            n_hole += __popc(bh);
            n_src += __popc(bs);
        });
    uint32_t hole_at, src_at, t0, t1;
    before_warp(sh, n_hole, n_src, hole_at, src_at, t0, t1);
    if (tid == 0) {
        sh.count[0] = t0;
        sh.count[1] = t1;
    }
    cluster.sync();
    uint32_t moves = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < cs) {
            const uint32_t *c = cluster.map_shared_rank(&sh.count[0], r);
            const uint32_t h = c[0], s = c[1];
            hole_at += r < rank ? h : 0;
            src_at += r < rank ? s : 0;
            moves += h;
        }
    int *holes = p.holes + (size_t)unit * p.cap, *sources = p.sources + (size_t)unit * p.cap;
    walk([&](int j, int e, bool kept, bool hole, bool src, uint32_t bh, uint32_t bs) {
        const uint32_t below = (1u << lane) - 1u;
        if (hole) holes[hole_at + __popc(bh & below)] = j;
        if (src) sources[src_at + __popc(bs & below)] = j;
        hole_at += __popc(bh);
        src_at += __popc(bs);
        if (j < whi) {
            if (j >= out_len) {
                p.acc_out[base + j] = 0.f;
                p.positions_out[base + j] = -1;
            } else if (kept) {
                p.acc_out[base + j] = w[e];
                p.positions_out[base + j] = pos[e];
            }
        }
    });
    if (rank == 0 && tid == 0 && unit % p.H_kv == 0) p.lens_out[b] = out_len;
    // the lists are complete, and no CTA leaves while another may read its counters
    cluster.sync();

    // The moves, dealt to the cluster's warps: a row's key and value chunks across the lanes
    const int nw = cs * kWarps, first = rank * kWarps + warp;
    const int ct = p.ck + p.cv;
    for (int i0 = first; i0 < (int)moves; i0 += nw * kMoveRows) {
        size_t s[kMoveRows], d[kMoveRows];
#pragma unroll
        for (int e = 0; e < kMoveRows; ++e) {
            const int i = min(i0 + e * nw, (int)moves - 1);  // the last one again where none is left
            s[e] = base + __ldcg(sources + i);
            d[e] = base + __ldcg(holes + i);
        }
        for (int c = lane; c < ct; c += 32) {
            const bool is_k = c < p.ck;
            uint4 *cache = is_k ? p.k + c : p.v + (c - p.ck);
            const int w = is_k ? p.ck : p.cv;
            uint4 x[kMoveRows];
#pragma unroll
            for (int e = 0; e < kMoveRows; ++e) x[e] = cache[s[e] * w];
#pragma unroll
            for (int e = 0; e < kMoveRows; ++e)
                if (i0 + e * nw < (int)moves) cache[d[e] * w] = x[e];
        }
#pragma unroll
        for (int e = 0; e < kMoveRows; ++e)
            if (lane == e && i0 + e * nw < (int)moves) {
                p.acc_out[d[e]] = p.acc[s[e]];
                p.positions_out[d[e]] = p.positions ? p.positions[s[e]] : (int)(s[e] - base);
            }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sm_count, cudaStream_t stream)
{
    const int units = p.B * p.H_kv;
    // Parts of 4096 rows at most, as far as clusters of 8 go; smaller ones, down to 1024
    // rows, only while every CTA still has an SM of its own.  64 caches of 4224 rows cut to
    // 4096: 22 us as 64 CTAs, 12.3 as 128, 14.2 as 256; 8 caches of 4096 rows cut to half: 39 us
    // as 8 CTAs, 18.5 as 32, 16.3 as 64; 32 of 32768 cut to 4096: 106 us in clusters of 2, 59 of
    // 4, 37.5 of 8.  Where half of the rows go, more CTAs than SMs would move them faster: 64
    // caches of 8192 rows 63 us as 128 CTAs, 46 as 256; of 2048 rows 18.1 and 19.0.
    int cs = 1;
    auto part = [&](int c) { return (p.S_cap + c - 1) / c; };
    while (cs < kMaxCluster && (part(cs) > 16 * kBlock || (part(cs) > 1024 && (long long)units * cs * 2 <= sm_count)))
        cs *= 2;
    const int chunk = part(cs);
    const int seg = ((chunk + kWarps - 1) / kWarps + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * cs);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (seg <= kBlock) return cudaLaunchKernelEx(&cfg, evict_kernel<true>, p, chunk, seg);
    return cudaLaunchKernelEx(&cfg, evict_kernel<false>, p, chunk, seg);
}

}  // namespace apex
