// cache_attn.cuh -- device code shared by the attention kernels over caches of rotated
// keys (one CTA: cache_attn.cu, CTA pairs: cache_pair.cu): the schedule, the masks, the
// softmax of a tile and the epilogue.
//
// Mathematics: the online softmax of Part 2, §6.2 over the keys a row sees, as
// partial results (max, sum, unnormalised output) over ranges of keys, joined by
// softmax's invariance to a shift.  A row that sees nothing has sum 0 and gives 0.
//
// Work: the G * T query rows of a KV head (G heads share it, T drafts) are adjacent
// in memory and are worked on in groups of M tiles of 128 rows, so a K/V tile of 128
// keys is read once for all of a group.  A unit is (sequence, KV head, row group).
// All tiles of all units, in order, are dealt out in equal contiguous shares -- one to
// a CTA or CTA pair -- whatever the lengths, which only the device knows, so a ragged
// batch keeps every SM busy to the end.  A share cuts at most its first and its last
// unit; cut units leave partial results that cache_join_kernel joins, the others are
// finished in place.
//
// Keys that nobody sees -- behind the drafts, before every window, masked in the whole
// tree -- may hold anything: their scores are replaced by -inf, and their V rows are
// set to zero in shared memory before the product (0 * NaN would be NaN).
#pragma once

#include <atomic>

#include "cache_attn.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace apex {
namespace {

// Dynamic shared memory allowed to a kernel, once per device (a call takes a few
// microseconds on the host, of which this would be one).  launch_regs: registers a thread
// that setmaxnreg redistributes -- setmaxnreg.inc blocks until the block's own pool can
// serve it, so a kernel built with fewer is never launched.
struct KernelSetup {
    std::atomic<uint64_t> done{0};
    template <typename K>
    cudaError_t operator()(K kernel, int smem_bytes, int launch_regs = 0)
    {
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
        if (err != cudaSuccess) return err;
        cudaFuncAttributes fa;
        err = cudaFuncGetAttributes(&fa, kernel);
        if (err != cudaSuccess) return err;
        if (fa.numRegs < launch_regs) return cudaErrorInvalidConfiguration;
        done.fetch_or(bit, std::memory_order_release);
        return cudaSuccess;
    }
};

// ---------------------------------------------------------------- issuing products
// One lane of a converged warp.  The warp that issues products runs its loops as a whole and
// only the instructions are elected: descriptors are then the same in every lane and stay in
// the uniform registers that tcgen05.mma takes.  Under `if (lane == 0)` each was moved there
// anew, about 100 clocks a product: a tree of 64 on 128/8 heads over 4 x 32768 keys took
// 435 us so, and 341 us elected.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// ---------------------------------------------------------------- schedule
// Lengths of sequence b: cached keys, keys with its drafts, its first key tile and
// number of tiles (one at least, so that every unit writes its output).
struct Seq {
    int len, total, tile0, tiles;
    int cost;  // of a unit in the schedule: its tiles and kCacheUnitCost for its start; 1 when units stay whole
    __device__ __forceinline__ void load(const CacheAttnParams &p, int b)
    {
        len = min(max(p.lens[b], 0), p.S_cap);
        total = min(len + p.drafts, p.S_cap);
        const int lo = p.window > 0 ? max(0, len - p.window + 1) : 0;
        tile0 = lo / kCacheTileKeys;
        tiles = max(1, (total + kCacheTileKeys - 1) / kCacheTileKeys - tile0);
        cost = p.whole ? 1 : tiles + kCacheUnitCost;
    }
};

// Where a share starts, and how the shares are cut.  Positions count cost: a unit takes
// kCacheUnitCost for its start (filling and draining the pipeline once more) and then one
// for each tile.
struct Sched {
    long long at, total;  // start of the share, cost of all units
    int left;             // cost of the share
    int n;                // shares
    int b, unit, off;     // sequence, unit within it and cost within the unit where the share starts
};

// One warp: share c of n, cost [total * c / n, total * (c + 1) / n).  The lengths are read 32 at
// a time, and beyond 32 sequences twice, before the first tile: 512 caches of 256 to 512 keys
// take 1.29 times their bytes and 4096 of them 1.24, but 65536 caches of 8 keys, one KV head,
// 2.4 ms, nearly all of it here.
__device__ __forceinline__ void make_sched(const CacheAttnParams &p, int c, int n, Sched *out)
{
    const int lane = threadIdx.x & 31;
    const int per_b = p.H_kv * p.n_groups;
    long long total = 0;
    Seq s;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        s.cost = 0;
        if (b0 + lane < p.B) s.load(p, b0 + lane);
        total += __reduce_add_sync(0xffffffffu, s.cost);
    }
    total *= per_b;
    Sched r;
    r.total = total;
    r.n = (int)min((long long)n, total);
    r.at = c < r.n ? total * c / r.n : total;
    r.left = c < r.n ? (int)(total * (c + 1) / r.n - r.at) : 0;
    r.b = r.unit = r.off = 0;
    if (r.left > 0) {
        long long before = 0;  // cost of the sequences before b0
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            if (p.B > 32) {  // else the lanes still hold the lengths
                s.cost = 0;
                if (b0 + lane < p.B) s.load(p, b0 + lane);
            }
            int incl = s.cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const long long end = before + (long long)incl * per_b;
            const uint32_t past = __ballot_sync(0xffffffffu, end > r.at && b0 + lane < p.B);
            if (past) {
                const int w = __ffs(past) - 1;
                const int cost = __shfl_sync(0xffffffffu, s.cost, w);
                const long long start = __shfl_sync(0xffffffffu, end - (long long)s.cost * per_b, w);
                r.b = b0 + w;
                r.unit = (int)((r.at - start) / cost);
                r.off = (int)((r.at - start) % cost);
                break;
            }
            before = __shfl_sync(0xffffffffu, end, 31);
        }
    }
    if (lane == 0) *out = r;
}

// The part of one unit in a share: n tiles from tile `first` of the sequence.
struct Frag {
    Seq s;
    int b, hk, group, unit;  // unit: index over all units
    int first, n;
    bool head, tail;         // holds the unit's first / last tile
    int last;                // share of the unit's last tile
};

static_assert(sizeof(Sched) <= 48, "schedule slot");

struct Walk {
    Sched s;
    Seq seq;
    bool fresh;
    __device__ __forceinline__ Walk(const CacheAttnParams &p, const Sched &sched) : s(sched), fresh(true) {}
    __device__ __forceinline__ bool next(const CacheAttnParams &p, Frag &f)
    {
        const int per_b = p.H_kv * p.n_groups;
        while (s.left > 0) {
            if (fresh) seq.load(p, s.b);
            fresh = false;
            const int n = min(seq.cost - s.off, s.left);  // cost of this unit in the share
            const int t0 = p.whole ? 0 : max(0, s.off - kCacheUnitCost);
            const int t1 = p.whole ? seq.tiles : max(0, s.off + n - kCacheUnitCost);
            f.s = seq;
            f.b = s.b;
            f.hk = s.unit / p.n_groups;
            f.group = s.unit % p.n_groups;
            f.unit = s.b * per_b + s.unit;
            f.first = seq.tile0 + t0;
            f.n = t1 - t0;
            f.head = t0 == 0;
            f.tail = t1 == seq.tiles;
            // share of the unit's last tile, at end - 1: the last c with total * c / n <= end - 1
            f.last = (int)(((s.at - s.off + seq.cost) * s.n - 1) / s.total);
            s.left -= n;
            s.at += n;
            s.off += n;
            if (s.off == seq.cost) {
                s.off = 0;
                if (++s.unit == per_b) {
                    s.unit = 0;
                    ++s.b;
                    fresh = true;
                }
            }
            if (f.n > 0) return true;
        }
        return false;
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

// What some row of a unit sees: the drafts in `any` and the cached keys from `lo` on -- the
// first that any draft's window reaches, which is past len - window + 1 when every draft's
// position is past len.  Made once a fragment by one warp, while its first tile is on the way.
struct Sight {
    uint64_t any;
    int lo;
    __device__ __forceinline__ Sight(const CacheAttnParams &p, const Frag &f) : any(0), lo(0)
    {
        // keys that every row sees, but for a window and the drafts
        if (p.drafts == 0 || (p.window == 0 && kCacheTileKeys * (f.first + f.n) <= f.s.len)) return;
        int first = f.s.len;
        for (int t = threadIdx.x & 31; t < p.T; t += 32) {
            int from;
            any |= draft_sight(p, f.b, t, f.s.len, f.s.total, from);
            first = min(first, from);
        }
        any = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)any) |
              ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32);
        lo = __reduce_min_sync(0xffffffffu, first);
    }
};

// Zero the rows of a V tile in shared memory (NB boxes of [128 keys][64 entries]) whose
// key no row of the unit sees; by one warp.
template <int NB>
__device__ __forceinline__ void mend_v(const Frag &f, const Sight &some, int key0, uint8_t *tile)
{
    const int lane = threadIdx.x & 31;
    if (key0 >= some.lo && key0 + kCacheTileKeys <= f.s.len) return;
    uint32_t w[4];
    sight_words(w, key0, some.lo, f.s.len, some.any);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (!((w[i] >> lane) & 1))
            for (int bx = 0; bx < NB; ++bx) {
                uint4 *row = reinterpret_cast<uint4 *>(tile + bx * 128 * 128 + (32 * i + lane) * 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) row[(c + lane) & 7] = make_uint4(0, 0, 0, 0);
            }
    fence_proxy_async_smem();
    __syncwarp();
}

// ---------------------------------------------------------------- softmax of one tile
// Thread = row = TMEM lane: the row's 128 scores at s_addr become its weights, bf16 over
// the scores, relative to a running maximum in log2 units; m_run, l_run: that maximum and
// the sum of weights so far.  O (at o_addr) is rescaled only when the maximum grew by more
// than 2^8: the final O / l does not depend on the reference point.  scores: where the
// row's scores are kept, or NULL; wait_pv: waits until O may be touched;
// half_done: called once the first 64 keys' weights are stored.
template <int DV, bool WEIGHTS, typename WaitPV, typename Half>
__device__ __forceinline__ void softmax_tile(const CacheAttnParams &p, uint32_t s_addr, uint32_t o_addr, int key0,
                                             int lo, int len, uint64_t drafts, float &m_run, float &l_run,
                                             float *scores, WaitPV wait_pv, Half half_done)
{
    uint32_t v[128];
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
        tmem_ld32(s_addr + 32 * ch, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * ch]));
    tmem_wait_ld();
    if (!__all_sync(0xffffffffu, key0 >= lo && key0 + kCacheTileKeys <= len)) {
        uint32_t w[4];
        sight_words(w, key0, lo, len, drafts);
#pragma unroll
        for (int e = 0; e < 128; ++e)
            if (!((w[e >> 5] >> (e & 31)) & 1)) v[e] = 0xff800000u;
    }
    if (WEIGHTS && scores) {
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
    const bool need = (m_run != -INFINITY) && (m_new > m_run + 8.f);
    wait_pv();
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
        if (q4 == 1) half_done();
    }
    {
        float a0, a1;
        f2_unpack(f2_add(f2_add(lacc[0], lacc[1]), f2_add(lacc[2], lacc[3])), a0, a1);
        l_run += a0 + a1;
    }
    tmem_wait_st();
    tc_fence_before();
}

// A row's maximum once its tiles are done: -inf says that it saw nothing, which a row whose
// scores are all NaN (a sum that is not zero) did not.
__device__ __forceinline__ float row_max(float m_run, float l_run)
{
    return (m_run == -INFINITY && !(l_run == 0.f)) ? 0.f : m_run;
}

// The finished row (index `row` over all query rows), or its part of a cut unit's result:
// row rc of the slot.  Partial outputs lie four entries at a time, rows adjacent, so that
// the lanes' rows are written and read side by side.
template <int DV, bool WEIGHTS>
__device__ __forceinline__ void write_row(const CacheAttnParams &p, uint32_t o_addr, bool whole, bool row_ok,
                                          size_t row, int slot, int rc, float m_run, float l_run)
{
    const float inv = (l_run > 0.f) ? 1.f / l_run : 0.f;
    if (row_ok && !whole) p.ws_ml[(size_t)slot * p.rows_cap + rc] = make_float2(row_max(m_run, l_run), l_run);
    if (WEIGHTS && row_ok && whole) p.lse[row] = m_run + log2f(l_run);
    uint4 *dst16 = reinterpret_cast<uint4 *>(p.out + row * DV);
    uint4 *dst32 = reinterpret_cast<uint4 *>(p.ws_o + (size_t)slot * p.rows_cap * DV) + rc;
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
                dst32[(size_t)(8 * ch + q4) * p.rows_cap] = make_uint4(v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]);
        }
    }
}

}  // namespace
}  // namespace apex
