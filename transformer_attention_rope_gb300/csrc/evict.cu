// evict.cu -- cutting a cache down to a budget of rows per (sequence, KV head).
//
// evict_select_kernel ranks the rows of one (sequence, KV head): rows that must
// stay (sinks, newest positions) have the largest key, the others the order-
// preserving integer image of their accumulated weight.  A radix search over
// 8-bit digits, most significant first, finds the budget-th largest key; of the
// rows that equal it the lowest are kept.  The rows are shared by a cluster of
// CTAs, each holding a contiguous part; digit histograms are summed over the
// cluster through distributed shared memory, so the rows are read once and the
// search costs four cluster barriers.
//
// Kept rows past the budget (sources) pair up, in ascending order, with freed rows
// below it (holes).  evict_move_kernel copies each source's key, value, weight and
// position into its hole: sources and holes never meet, so the moves need no order
// among themselves, and a cache slightly over its budget moves only the few rows
// that are past it.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "evict.h"

namespace cg = cooperative_groups;

namespace apex {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;
constexpr uint32_t kMust = 0xffffffffu;

struct SelShared {
    uint32_t hist[4][256];
    uint32_t warp[2][kSelWarps];
    uint32_t digit, above;
    uint32_t count[2];  // this CTA's holes and sources (or ties), for the cluster
};

// Order-preserving image of a weight; NaN below everything, -0 as +0.  No image
// is kMust (that would be a NaN's).
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix over the block of two flags, in thread order; the totals in t0, t1.
__device__ __forceinline__ void block_prefix(SelShared &sh, bool f0, bool f1, uint32_t &p0, uint32_t &p1, uint32_t &t0,
                                             uint32_t &t1)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t b0 = __ballot_sync(0xffffffffu, f0), b1 = __ballot_sync(0xffffffffu, f1);
    __syncthreads();
    if (lane == 0) {
        sh.warp[0][warp] = __popc(b0);
        sh.warp[1][warp] = __popc(b1);
    }
    __syncthreads();
    p0 = __popc(b0 & ((1u << lane) - 1u));
    p1 = __popc(b1 & ((1u << lane) - 1u));
    t0 = t1 = 0;
    for (int w = 0; w < kSelWarps; ++w) {
        const uint32_t c0 = sh.warp[0][w], c1 = sh.warp[1][w];
        if (w < warp) {
            p0 += c0;
            p1 += c1;
        }
        t0 += c0;
        t1 += c1;
    }
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p, int chunk, int in_smem)
{
    extern __shared__ uint32_t keys[];  // [chunk] when in_smem
    __shared__ SelShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    const int unit = blockIdx.x / cs;
    const int b = unit / p.H_kv;
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = min(max(p.lens[b], 0), p.S_cap);
    const int next = p.next_pos[b];
    const int lo = min(rank * chunk, p.S_cap), hi = min(lo + chunk, p.S_cap);
    const int end = min(hi, n);  // rows of this part that hold a key
    const size_t base = (size_t)unit * p.S_cap;
    const int out_len = min(n, p.budget);

    auto position = [&](int j) { return p.positions ? p.positions[base + j] : j; };
    auto make_key = [&](int j) -> uint32_t {
        const int pos = position(j);
        if (pos < p.n_sink || (long long)pos >= (long long)next - p.n_recent) return kMust;
        return weight_key(p.acc[base + j]);
    };

    uint32_t cut = 0;      // the budget-th largest key
    uint32_t ties = 0;     // rows equal to it that are kept
    bool all_ties = true;  // every row equal to it is kept
    if (n > p.budget) {    // the same for the whole cluster
        for (int i = tid; i < 4 * 256; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
        if (in_smem)
            for (int j = lo + tid; j < end; j += kSelThreads) keys[j - lo] = make_key(j);
        __syncthreads();
        uint32_t want = p.budget;  // rows to take from those that match the prefix
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int j = lo + tid; j < end; j += kSelThreads) {
                const uint32_t k = in_smem ? keys[j - lo] : make_key(j);
                if (pass == 0 || (k >> (shift + 8)) == (cut >> (shift + 8))) {
                    // neighbouring weights share their leading digit: one add per distinct digit of the warp
                    const uint32_t d = (k >> shift) & 255u;
                    const uint32_t same = __match_any_sync(__activemask(), d);
                    if ((threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&sh.hist[pass][d], __popc(same));
                }
            }
            cluster.sync();
            // thread d < 256 sums digit d over the cluster; rows with a larger digit come first
            uint32_t mine = 0;
            if (tid < 256)
                for (int r = 0; r < cs; ++r) mine += cluster.map_shared_rank(&sh.hist[pass][0], r)[tid];
            // inclusive suffix sums over the 256 digits: warp w holds digits [32 w, 32 w + 32)
            uint32_t suffix = mine;
            const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_down_sync(0xffffffffu, suffix, o);
                if (lane + o < 32) suffix += x;
            }
            if (lane == 0) sh.warp[0][warp] = suffix;
            __syncthreads();
            if (tid < 256) {
                for (int w = warp + 1; w < 8; ++w) suffix += sh.warp[0][w];
                if (suffix >= want && suffix - mine < want) {
                    sh.digit = tid;
                    sh.above = suffix - mine;
                    sh.count[0] = mine;
                }
            }
            __syncthreads();
            cut |= sh.digit << shift;
            want -= sh.above;
            all_ties = sh.count[0] == want;
            __syncthreads();
        }
        ties = want;
    }

    // which rows of this part are kept; ties beyond `ties` go, the highest rows first
    uint32_t tie_base = 0;
    if (n > p.budget && !all_ties) {
        uint32_t mine = 0;
        for (int j = lo + tid; j < end; j += kSelThreads) mine += (in_smem ? keys[j - lo] : make_key(j)) == cut;
        mine = __reduce_add_sync(0xffffffffu, mine);
        if ((tid & 31) == 0) sh.warp[0][tid >> 5] = mine;
        __syncthreads();
        if (tid == 0) {
            uint32_t t = 0;
            for (int w = 0; w < kSelWarps; ++w) t += sh.warp[0][w];
            sh.count[0] = t;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) tie_base += cluster.map_shared_rank(&sh.count[0], r)[0];
        cluster.sync();
    }

    // Two walks over the part in row order: the first counts its holes and sources,
    // the second, knowing the parts before it, writes the lists and the kept rows'
    // weights and positions.
    uint32_t hole_base = 0, src_base = 0;
    for (int walk = 0; walk < 2; ++walk) {
        uint32_t tie_seen = tie_base, n_hole = hole_base, n_src = src_base;
        for (int j0 = lo; j0 < hi; j0 += kSelThreads) {
            const int j = j0 + tid;
            const bool there = j < end;
            bool kept = there;
            if (n > p.budget) {
                const uint32_t k = there ? (in_smem ? keys[j - lo] : make_key(j)) : 0;
                kept = there && k >= cut;
                if (!all_ties) {
                    const bool tie = there && k == cut;
                    uint32_t before, unused, total, unused2;
                    block_prefix(sh, tie, false, before, unused, total, unused2);
                    if (tie) kept = tie_seen + before < ties;
                    tie_seen += total;
                }
            }
            const bool hole = there && !kept && j < p.budget;
            const bool src = kept && j >= p.budget;
            uint32_t ph, ps, th, ts;
            block_prefix(sh, hole, src, ph, ps, th, ts);
            if (walk == 1) {
                if (hole) p.holes[(size_t)unit * p.cap + n_hole + ph] = j;
                if (src) p.sources[(size_t)unit * p.cap + n_src + ps] = j;
                if (j < hi) {
                    if (j >= out_len) {
                        p.acc_out[base + j] = 0.f;
                        p.positions_out[base + j] = -1;
                    } else if (kept) {
                        p.acc_out[base + j] = p.acc[base + j];
                        p.positions_out[base + j] = position(j);
                    }
                }
            }
            n_hole += th;
            n_src += ts;
        }
        if (walk == 0) {
            if (tid == 0) {
                sh.count[0] = n_hole;
                sh.count[1] = n_src;
            }
            cluster.sync();
            uint32_t total = 0;
            for (int r = 0; r < cs; ++r) {
                const uint32_t *c = cluster.map_shared_rank(&sh.count[0], r);
                if (r < rank) {
                    hole_base += c[0];
                    src_base += c[1];
                }
                total += c[0];
            }
            if (rank == 0 && tid == 0) p.moved[unit] = (int)total;
        }
    }
    cluster.sync();  // no CTA leaves while another may still read its counters
}

// One warp per moved row, its key and value chunks across the lanes.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int units)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int warp = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5;
    const int n_warps = (gridDim.x * kMoveThreads) >> 5;
    for (int unit = blockIdx.y; unit < units; unit += gridDim.y) {
        const size_t base = (size_t)unit * p.S_cap;
        const int n = p.moved[unit];
        if (blockIdx.x == 0 && threadIdx.x == 0 && unit % p.H_kv == 0)
            p.lens_out[unit / p.H_kv] = min(min(max(p.lens[unit / p.H_kv], 0), p.S_cap), p.budget);
        for (int i = warp; i < n; i += n_warps) {
            const size_t d = base + p.holes[(size_t)unit * p.cap + i], s = base + p.sources[(size_t)unit * p.cap + i];
            for (int c = lane; c < p.ck; c += 32) p.k[d * p.ck + c] = p.k[s * p.ck + c];
            for (int c = lane; c < p.cv; c += 32) p.v[d * p.cv + c] = p.v[s * p.cv + c];
            if (lane == 0) {
                p.acc_out[d] = p.acc[s];
                p.positions_out[d] = p.positions ? p.positions[s] : (int)(s - base);
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sm_count, cudaStream_t stream)
{
    const int units = p.B * p.H_kv;
    int cs = 1;
    while (cs < 8 && (p.S_cap + cs - 1) / cs > 4096) cs *= 2;
    const int chunk = (p.S_cap + cs - 1) / cs;
    const size_t key_bytes = (size_t)chunk * sizeof(uint32_t);
    const int in_smem = key_bytes <= 160 * 1024;
    const size_t smem = in_smem ? key_bytes : 0;
    cudaError_t err = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * cs);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
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
    err = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, chunk, in_smem);
    if (err != cudaSuccess) return err;
    const int gy = std::min(units, 65535);
    const int want = std::max(1, (8 * sm_count + gy - 1) / gy);
    const int most = std::max(1, (p.cap + 7) / 8);
    cfg.gridDim = dim3(std::min(want, most), gy);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p, units);
}

}  // namespace apex
