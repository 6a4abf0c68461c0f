// decode4.cu -- attention of one or a few new tokens over a cache held in 4 bits (layout:
// bits4.h), with a window and sinks.
//
// Work: as for bf16 caches (cache_attn.cuh): tiles of 128 keys of all (sequence, KV head,
// row group) units are dealt out in equal shares, cut units leave partial results.  A tile is
// 32 keys for each of a CTA's 4 warps; a warp has its own running maximum, sum and output, and
// its own ring of slices in shared memory, filled by its own asynchronous copies: warps wait
// for one another only where a unit ends.
//
// Mathematics: S^T = K Q^T and O^T += V^T P^T on mma.sync (keys and value entries as rows of
// A, the queries of a KV head as the 8 columns of B), fp16 with fp32 sums.  A product of an
// e2m1 value with its e4m3 scale is exact in fp16.  Queries go to fp16 scaled by a power of two
// for each row, exact but for entries below 2^-21 of the row's largest; the factor goes into the
// scores' scale.  Weights are taken relative to a reference 2^11 below the running
// maximum, as fp16 up to 2^15 is: those of 2^-25 of the largest keep 11 bits, and what is lost
// lies below 2^-36 of it.  The reference moves only when a score outgrows it, so a slice costs one
// vote and no exchange of maxima; past 2^20 it is the maximum itself (kLargeScore).
//
// Keys: lane 4g + t holds bytes 16t .. 16t + 15 of key g's row, 32 neighbouring entries, as the
// order of the sum over entries is free; queries are laid out alike.  Values: lane 4g + t holds
// entries 16g.. of keys 2t, 2t + 1, 2t + 8, 2t + 9; the halves of two keys' bytes are
// interleaved so that one conversion gives both keys' values of an entry, which is how the
// second product takes them.
//
// Bound: HBM, 0.5625 bytes an entry, and close behind it the issue of conversions: a step of 16
// keys takes some 290 instructions a warp, 64 of them conversions and 64 scales.  64 caches of 9001 to
// 32767 keys, 32/8 heads of 128 (1.54 GB): 251 us, 6.1 TB/s; with slices of 16 keys for 8 warps 279, and 303
// with addresses and masks made anew for each.  16 rows over 8 such caches (193 MB): 56 us, where the
// conversions are the same and the products twice as many.  One cache under a window of 1024: 6.7 us.
#include <math.h>

#include "bits4.cuh"
#include "bits4.h"
#include "cache_attn.cuh"

namespace apex {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlice = 32;  // keys of a warp's slice
constexpr int kStep = 16;   // keys of a step: the rows of one product
constexpr int kStages = 2;  // slices of a warp's ring
static_assert(kWarps * kSlice == kCacheTileKeys, "a tile is a slice for each warp");
constexpr float kHeadroom = 11.f;  // the reference of weights below the maximum, log2
constexpr float kSlack = 15.f;     // scores may lie this far above the reference

template <int DQK, int DV, int NT>
struct Cfg {
    static constexpr bool kWide = DQK >= 128;     // keys have a part of 128 entries
    static constexpr bool kNarrow = DQK % 128 != 0;  // and one of 64
    static constexpr int kStepsWide = kWide ? 8 : 0, kSteps = DQK / 16;
    static constexpr int kBlocks = DV / 16;  // 16-entry row blocks of O^T
    static constexpr int kRows = 8 * NT;
    // a slice: wide parts of the keys | narrow parts | values | key scales | value scales
    static constexpr int kKNarrow = kWide ? kSlice * 64 : 0;
    static constexpr int kV = kKNarrow + (kNarrow ? kSlice * 32 : 0);
    static constexpr int kKScale = kV + kSlice * DV / 2;
    static constexpr int kVScale = kKScale + kSlice * DQK / 16;
    static constexpr int kStage = kVScale + kSlice * DV / 16;
    static_assert(kStage % 16 == 0, "slices of 16-byte chunks");
    static constexpr int kRing = kWarps * kStages * kStage;
    // where a unit ends the ring holds the warps' outputs instead
    static constexpr int kMerge = kWarps * kRows * DV * 4;
    static constexpr int kMl = kRing > kMerge ? kRing : kMerge;  // [warps][rows] (reference, sum)
    static constexpr int kSched = kMl + kWarps * kRows * 8;
    static constexpr int kBytes = kSched + 64;
    static_assert(decode4_ctas(8 * NT) * (kBytes + 1024) <= 227 * 1024, "CTAs of an SM");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(  // not volatile: may move among the conversions
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where key i of a step lies among its value rows, and which of its 16-byte chunks comes first: the
// four keys of a load are neighbours, and at 128 entries the chunks of every other pair trade
// places, so that the load's words lie in all 32 banks.
__device__ __forceinline__ int value_slot(int i) { return ((i >> 1) & 3) + 4 * (i & 1) + (i & ~7); }
template <int DV>
__device__ __forceinline__ int value_chunk(int slot, int c)
{
    return DV == 128 ? c ^ (slot & 2) : c;
}

// A warp's copies of its slices, one tile after another.
template <typename C, int DQK, int DV>
struct Feed {
    const uint8_t *k, *v, *k_scale, *v_scale;  // of the next slice, where this lane's copies start
    int key, left, pre, gap;                   // its first key; tiles to go, those before the sinks' end, keys behind it
    uint32_t slot, first, last;                // ring

    __device__ __forceinline__ void start(const Decode4Params &p, const Frag &f, size_t kv, uint32_t ring)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        first = slot = ring;
        last = ring + kStages * C::kStage;
        left = f.n;
        gap = kCacheTileKeys * (f.s.tile0 - f.s.sink);
        pre = f.s.tile0 - f.first;  // below 1: the fragment has none of the sinks' tiles
        key = kCacheTileKeys * f.tile<true>(0) + kSlice * warp;
        const size_t row = kv * p.c.S_cap + key;
        // rows follow one another, so a slice is one run of bytes
        k = p.k + row * (DQK / 2) + 16 * lane;
        v = p.v + row * (DV / 2) + 16 * lane;
        k_scale = p.k_scale + row * (DQK / 16);
        v_scale = p.v_scale + row * (DV / 16);
    }
    // keys past the capacity are not copied: what their slots hold is masked
    template <bool WHOLE>
    __device__ __forceinline__ void copies(int room)
    {
        const int lane = threadIdx.x & 31;
        constexpr int kKChunks = DQK / 32, kVChunks = DV / 32;
#pragma unroll
        for (int i = 0; i < kSlice * kKChunks / 32; ++i) {
            const int id = lane + 32 * i, key = id / kKChunks, c = id % kKChunks;
            const uint32_t at = !C::kWide || !C::kNarrow ? 16 * id
                                : c < 4                  ? key * 64 + 16 * c
                                                         : C::kKNarrow + key * 32 + 16 * (c - 4);
            if (WHOLE || key < room) copy16(slot + at, k + 512 * i);
        }
#pragma unroll
        for (int i = 0; i < kSlice * kVChunks / 32; ++i) {
            const int id = lane + 32 * i, key = id / kVChunks, c = id % kVChunks, to = value_slot(key);
            if (WHOLE || key < room) copy16(slot + C::kV + to * (DV / 2) + 16 * value_chunk<DV>(to, c), v + 512 * i);
        }
        // scales: a word or two of a row at a time, as rows need not start on 16 bytes
        scales<DQK, WHOLE>(slot + C::kKScale, k_scale, room);
        scales<DV, WHOLE>(slot + C::kVScale, v_scale, room);
    }
    template <int D, bool WHOLE>
    static __device__ __forceinline__ void scales(uint32_t dst, const uint8_t *src, int room)
    {
        const int lane = threadIdx.x & 31;
        if (D == 128) {
            if (WHOLE || lane < room) copy8(dst + 8 * lane, src + 8 * lane);
        } else {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int id = lane + 32 * i;
                if (WHOLE || id / (D / 64) < room) copy4(dst + 4 * id, src + 4 * id);
            }
        }
    }
    __device__ __forceinline__ void skip(int keys)
    {
        key += keys;
        k += (long long)keys * (DQK / 2);
        v += (long long)keys * (DV / 2);
        k_scale += (long long)keys * (DQK / 16);
        v_scale += (long long)keys * (DV / 16);
    }
    __device__ __forceinline__ void next(int S_cap)
    {
        if (left > 0) {
            if (S_cap - key >= kSlice)
                copies<true>(kSlice);
            else
                copies<false>(S_cap - key);
            skip(kCacheTileKeys);
            if (--pre == 0) skip(gap);
            --left;
        }
        copies_commit();
        slot += C::kStage;
        if (slot == last) slot = first;
    }
};

__device__ __forceinline__ uint32_t splat_lo(uint32_t w) { return __byte_perm(w, 0, 0x1010); }
__device__ __forceinline__ uint32_t splat_hi(uint32_t w) { return __byte_perm(w, 0, 0x3232); }

// Four steps' rows of keys times queries: 16 entries (two words) of keys g and g + 8 of one scale
// each.
template <int NT>
__device__ __forceinline__ void key_steps(float (&s)[NT][4], uint32_t lo0, uint32_t lo1, uint32_t hi0, uint32_t hi1,
                                          uint32_t scale_lo, uint32_t scale_hi, const uint32_t (*q)[NT][2])
{
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t x[4], y[4];
        e2m1_bytes_to_f16x2(w ? lo1 : lo0, x);
        e2m1_bytes_to_f16x2(w ? hi1 : hi0, y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {mul_f16x2(x[2 * h], scale_lo), mul_f16x2(y[2 * h], scale_hi),
                                   mul_f16x2(x[2 * h + 1], scale_lo), mul_f16x2(y[2 * h + 1], scale_hi)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16_16816(s[n], a, q[2 * w + h][n][0], q[2 * w + h][n][1]);
        }
    }
}

template <int DQK, int DV, int NT>
__global__ void __launch_bounds__(kThreads, decode4_ctas(8 * NT)) decode4_kernel(const __grid_constant__ Decode4Params p)
{
    using C = Cfg<DQK, DV, NT>;
    const CacheAttnParams &pc = p.c;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float *merge = reinterpret_cast<float *>(smem);                // [warps][rows][DV]
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kMl);        // [warps][rows]
    Sched *sched = reinterpret_cast<Sched *>(smem + C::kSched);
    // launched as a programmatic dependent: inputs may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) make_sched<true>(pc, blockIdx.x, gridDim.x, sched);
    __syncthreads();

    Walk<true> walk(pc, *sched);
    Frag f;
    while (walk.next(pc, f)) {
        const size_t kv = (size_t)f.b * pc.H_kv + f.hk;
        if (threadIdx.x == 0 && f.head) pc.units[f.unit] = make_int2(blockIdx.x, f.last);
        Feed<C, DQK, DV> feed;
        feed.start(p, f, kv, smem_u32(smem) + warp * kStages * C::kStage);
#pragma unroll
        for (int j = 0; j < kStages - 1; ++j) feed.next(pc.S_cap);

        // ---- queries: column n of tile nt is row 8 nt + n of the group
        uint32_t q[C::kSteps][NT][2];
        float factor[NT][2];  // of the scores of columns 2t, 2t + 1, in log2 units
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rc = 8 * nt + g, r = f.group * pc.group + rc;
            const bool ok = rc < pc.rows_cap && r < pc.R;
            const uint16_t *row = p.q + (kv * pc.R + r) * DQK;
            uint32_t w[DQK / 8];  // the lane's entries: 32 of the wide part, 16 of the narrow one
#pragma unroll
            for (int i = 0; i < DQK / 32; ++i) {
                const int e = (C::kWide && i < 4) ? 32 * t + 8 * i : (C::kWide ? 128 : 0) + 16 * t + 8 * (i - (C::kWide ? 4 : 0));
                uint4 x = make_uint4(0, 0, 0, 0);
                if (ok) x = *reinterpret_cast<const uint4 *>(row + e);
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < DQK / 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // largest magnitude 2^(ex - 127) to under twice that: entries times 2^(131 - ex) are below 32
            const uint32_t ex = min(max(top >> 7, 5u), 254u);
            const float down = __uint_as_float((258u - ex) << 23), up = __uint_as_float((ex - 4u) << 23);
#pragma unroll
            for (int i = 0; i < DQK / 8; ++i)
                q[i >> 1][nt][i & 1] = pack_f16x2(bf16lo_to_f32(w[i]) * down, bf16hi_to_f32(w[i]) * down);
#pragma unroll
            for (int e = 0; e < 2; ++e) factor[nt][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + e));
        }
        const float kf = (p.k_factor ? p.k_factor[f.hk] : 1.f) * pc.scale_log2;
        const float vf = pc.v_factor ? pc.v_factor[f.hk] : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) factor[nt][e] = fmaxf(factor[nt][e] * kf, 1e-37f);  // not 0: masked scores stay -inf
        // keys that every row sees: [all_lo, all_hi]; that some row sees: [any_lo, any_hi] and the sinks
        const int m1 = f.s.len + pc.T - 1;
        const int all_lo = pc.window > 0 ? m1 - pc.window + 1 : 0, all_hi = min(f.s.len, pc.S_cap - 1);
        const int any_lo = pc.window > 0 ? f.s.len - pc.window + 1 : 0, any_hi = min(m1, pc.S_cap - 1);

        // weights are 2^(score - ref); a row that has seen nothing starts far below every score
        constexpr float kUnseen = -3e38f;
        float o[NT][C::kBlocks][4], ref[NT][2], sum[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < C::kBlocks; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
            ref[nt][0] = ref[nt][1] = kUnseen;
            sum[nt][0] = sum[nt][1] = 0.f;
        }
        bool large = false;  // some reference is: scores are rounded before they are compared with it

        constexpr int U = kSlice / kStep;  // steps whose scores are there together
        const uint8_t *at = smem + warp * kStages * C::kStage;
        int slice0 = kCacheTileKeys * f.tile<true>(0) + kSlice * warp, pre = f.s.tile0 - f.first;
        for (int j = 0; j < f.n; ++j) {
            __syncwarp();  // all lanes are done with the slot that is filled next
            feed.next(pc.S_cap);
            copies_wait<kStages - 1>();
            __syncwarp();

            // ---- scores of keys g, g + 8 (rows) and queries 2t, 2t + 1 (columns) of each step
            float s[U][NT][4];
            int key0[U];
            bool all[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r0 = kStep * u;  // first row of the slot
                key0[u] = slice0 + r0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
                if (C::kWide) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(at + (r0 + g) * 64 + 16 * t);
                    const uint4 b = *reinterpret_cast<const uint4 *>(at + (r0 + g + 8) * 64 + 16 * t);
                    const uint32_t sa = e4m3x2_to_f16x2(
                        *reinterpret_cast<const uint16_t *>(at + C::kKScale + (r0 + g) * (DQK / 16) + 2 * t));
                    const uint32_t sc = e4m3x2_to_f16x2(
                        *reinterpret_cast<const uint16_t *>(at + C::kKScale + (r0 + g + 8) * (DQK / 16) + 2 * t));
                    key_steps<NT>(s[u], a.x, a.y, b.x, b.y, splat_lo(sa), splat_lo(sc), &q[0]);
                    key_steps<NT>(s[u], a.z, a.w, b.z, b.w, splat_hi(sa), splat_hi(sc), &q[C::kWide ? 4 : 0]);
                }
                if (C::kNarrow) {
                    const uint2 a = *reinterpret_cast<const uint2 *>(at + C::kKNarrow + (r0 + g) * 32 + 8 * t);
                    const uint2 b = *reinterpret_cast<const uint2 *>(at + C::kKNarrow + (r0 + g + 8) * 32 + 8 * t);
                    const int block = (C::kWide ? 8 : 0) + t;
                    const uint32_t sa = e4m3x2_to_f16x2(at[C::kKScale + (r0 + g) * (DQK / 16) + block]);
                    const uint32_t sc = e4m3x2_to_f16x2(at[C::kKScale + (r0 + g + 8) * (DQK / 16) + block]);
                    key_steps<NT>(s[u], a.x, a.y, b.x, b.y, splat_lo(sa), splat_lo(sc), &q[C::kStepsWide]);
                }
                all[u] = key0[u] >= all_lo && key0[u] + kStep - 1 <= all_hi;
                if (!all[u]) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int rc = 8 * nt + 2 * t + e, r = f.group * pc.group + rc;
                            const int m = f.s.len + r % pc.T, hi = min(m, pc.S_cap - 1);
                            const int lo = pc.window > 0 ? m - pc.window + 1 : 0;
                            const bool none = rc >= pc.rows_cap || r >= pc.R;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int key = key0[u] + g + 8 * h;
                                if (none || key > hi || (key < lo && key >= pc.n_sink)) s[u][nt][e + 2 * h] = -INFINITY;
                            }
                        }
                }
            }
            float x[U][NT][4];  // scores above the reference
            float most = kUnseen;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[u][nt][e] = fmaf(s[u][nt][e], factor[nt][e & 1], -ref[nt][e & 1]);
                    most = fmax3(most, fmaxf(x[u][nt][0], x[u][nt][1]), fmaxf(x[u][nt][2], x[u][nt][3]));
                }
            if (__any_sync(0xffffffffu, large || most > kSlack)) {
                bool grown = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y[U][2], top = kUnseen;
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            y[u][0] = __fmul_rn(s[u][nt][e], factor[nt][e]);
                            y[u][1] = __fmul_rn(s[u][nt][e + 2], factor[nt][e]);
                            top = fmax3(top, y[u][0], y[u][1]);
                        }
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                        if (top - ref[nt][e] > kSlack) {
                            // a large one as it is: less the headroom it could be rounded to 16 below itself, and
                            // weights end at 2^16
                            const float now = top - (fabsf(top) > kLargeScore ? 0.f : kHeadroom);
                            const float keep = fast_exp2(ref[nt][e] - now);
                            ref[nt][e] = now;
                            sum[nt][e] *= keep;
#pragma unroll
                            for (int i = 0; i < C::kBlocks; ++i) {
                                o[nt][i][e] *= keep;
                                o[nt][i][e + 2] *= keep;
                            }
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            x[u][nt][e] = __fsub_rn(y[u][0], ref[nt][e]);
                            x[u][nt][e + 2] = __fsub_rn(y[u][1], ref[nt][e]);
                        }
                        grown |= fabsf(ref[nt][e]) > kLargeScore - kHeadroom && ref[nt][e] != kUnseen;
                    }
                large = __any_sync(0xffffffffu, grown);
            }
            uint32_t pb[U][NT][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float p0 = fast_exp2(x[u][nt][0]), p1 = fast_exp2(x[u][nt][1]);
                    const float p2 = fast_exp2(x[u][nt][2]), p3 = fast_exp2(x[u][nt][3]);
                    sum[nt][0] += p0 + p2;
                    sum[nt][1] += p1 + p3;
                    pb[u][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
                    pb[u][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
                }

            // ---- outputs: keys 2t, 2t + 1 and 2t + 8, 2t + 9 of the lane's entries
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r0 = kStep * u;
                uint32_t vs[2];
                const int block = DV == 128 ? g : g >> 1;
                const uint8_t *sv = at + C::kVScale + (r0 + 2 * t) * (DV / 16) + block;
                vs[0] = e4m3x2_to_f16x2(sv[0] | (uint32_t)sv[DV / 16] << 8);
                vs[1] = e4m3x2_to_f16x2(sv[8 * (DV / 16)] | (uint32_t)sv[9 * (DV / 16)] << 8);
                if (!all[u]) {  // values of keys that no row sees may be anything: codes are finite, scales not
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = key0[u] + 2 * t + 8 * h + e;
                            if (key > any_hi || (key < any_lo && key >= pc.n_sink)) vs[h] &= e ? 0x0000ffffu : 0xffff0000u;
                        }
                }
                constexpr int kWords = DV / 64;  // of a lane's entries of one key
                uint32_t v[4][kWords];           // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int slot = r0 + t + 4 * h;  // value_slot of the key
                    const uint8_t *row = at + C::kV + slot * (DV / 2);
                    if (DV == 128) {
                        const uint2 two =
                            *reinterpret_cast<const uint2 *>(row + 16 * value_chunk<DV>(t, g >> 1) + 8 * (g & 1));
                        v[h][0] = two.x;
                        v[h][kWords - 1] = two.y;
                    } else {
                        v[h][0] = *reinterpret_cast<const uint32_t *>(row + 4 * g);
                    }
                }
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    uint32_t even[2][4], odd[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a = v[2 * h][w], b = v[2 * h + 1][w];
                        e2m1_bytes_to_f16x2((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), even[h]);
                        e2m1_bytes_to_f16x2(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), odd[h]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a[4] = {mul_f16x2(even[0][i], vs[0]), mul_f16x2(odd[0][i], vs[0]),
                                               mul_f16x2(even[1][i], vs[1]), mul_f16x2(odd[1][i], vs[1])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][4 * w + i], a, pb[u][nt][0], pb[u][nt][1]);
                    }
                }
            }
            at = smem + (warp * kStages + (j + 1) % kStages) * C::kStage;
            slice0 += kCacheTileKeys;
            if (--pre == 0) slice0 += kCacheTileKeys * (f.s.tile0 - f.s.sink);
        }

        // ---- the warps' results become one
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = sum[nt][e];
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
                if (g == 0)
                    ml[warp * C::kRows + 8 * nt + 2 * t + e] = make_float2(ref[nt][e] == kUnseen ? row_max(-INFINITY, x) : ref[nt][e], x);
            }
        copies_wait<0>();
        __syncthreads();  // and every ring is done with
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rc = 8 * nt + 2 * t + e;
                if (rc >= pc.rows_cap) continue;
                float *to = merge + (warp * C::kRows + rc) * DV + (DV / 8) * g;
#pragma unroll
                for (int i = 0; i < C::kBlocks; i += 2)  // entries 2i .. 2i + 3 of the lane's
                    *reinterpret_cast<float4 *>(to + 2 * i) =
                        make_float4(o[nt][i][e], o[nt][i][e + 2], o[nt][i + 1][e], o[nt][i + 1][e + 2]);
            }
        __syncthreads();
        const int slot = 2 * blockIdx.x + (f.head ? 1 : 0);
        for (int i = threadIdx.x; i < pc.rows_cap * (DV / 4); i += kThreads) {
            const int rc = i / (DV / 4), c = i % (DV / 4), r = f.group * pc.group + rc;
            if (r >= pc.R) break;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * C::kRows + rc].x);
            float L = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 part = ml[w * C::kRows + rc];
                if (part.x == -INFINITY) continue;
                const float k = exp2f(part.x - top);
                const float4 y = *reinterpret_cast<const float4 *>(merge + (w * C::kRows + rc) * DV + 4 * c);
                L = fmaf(part.y, k, L);
                x.x = fmaf(y.x, k, x.x);
                x.y = fmaf(y.y, k, x.y);
                x.z = fmaf(y.z, k, x.z);
                x.w = fmaf(y.w, k, x.w);
            }
            // the values' factor comes last, when a row is whole: sums of weights up to 2^15 times values up to
            // 2688 would leave fp32 with the largest factors
            if (f.head && f.tail) {
                const float inv = L == 0.f ? 0.f : vf / L;
                *reinterpret_cast<uint2 *>(pc.out + (kv * pc.R + r) * DV + 4 * c) =
                    make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
            } else {
                if (c == 0) pc.ws_ml[(size_t)slot * pc.rows_cap + rc] = make_float2(top, L);
                reinterpret_cast<float4 *>(pc.ws_o + (size_t)slot * pc.rows_cap * DV)[(size_t)c * pc.rows_cap + rc] = x;
            }
        }
        __syncthreads();  // the rings are filled again
    }
}

template <int DQK, int DV, int NT>
cudaError_t launch_t(const Decode4Params &p, int grid, cudaStream_t stream)
{
    using C = Cfg<DQK, DV, NT>;
    static KernelSetup setup;
    const cudaError_t err = setup(decode4_kernel<DQK, DV, NT>, C::kBytes);
    if (err != cudaSuccess) return err;
    return launch_dependent(decode4_kernel<DQK, DV, NT>, grid, kThreads, C::kBytes, stream, p);
}

template <int NT>
cudaError_t launch_rows(const Decode4Params &p, int grid, cudaStream_t stream)
{
    if (p.c.d_qk == 64) return launch_t<64, 64, NT>(p, grid, stream);
    if (p.c.d_qk == 128) return launch_t<128, 128, NT>(p, grid, stream);
    return launch_t<192, 128, NT>(p, grid, stream);
}

}  // namespace

cudaError_t launch_decode4(Decode4Params &p, int sm_count, cudaStream_t stream)
{
    CacheAttnParams &c = p.c;
    const long long n_units = (long long)c.B * c.H_kv * c.n_groups;
    const int room = decode4_ctas(c.group) * std::min(sm_count, kCacheMaxCtas);
    int shares = decode4_shares(n_units, c.S_cap, room);
    // keys that a unit can reach: a window and the sinks bound them, the new rows and a tile's slack beside
    const int reach = c.window > 0 ? (int)std::min<long long>(c.S_cap, (long long)c.window + c.n_sink + c.drafts + 2 * kCacheTileKeys)
                                   : c.S_cap;
    c.whole = decode4_whole(n_units, reach, c.group);
    if (c.whole) shares = (int)std::min<long long>(shares, n_units);
    const cudaError_t err = c.group == 8    ? launch_rows<1>(p, shares, stream)
                            : c.group == 16 ? launch_rows<2>(p, shares, stream)
                                            : launch_decode4_wide(p, shares, stream);
    if (err != cudaSuccess || c.whole) return err;
    return launch_cache_join(c, shares, stream);
}

}  // namespace apex
