// decode4_wide.cu -- attention over a cache held in 4 bits for many query rows of a KV head
// (drafted tokens, wide groups): up to 128 rows share each key's conversion, and the products run
// on tcgen05.  Mathematics, format and roundings as in decode4.cu, schedule and partial results as
// in cache_attn.cuh.
//
// Warp roles: 0-3 softmax and epilogue (thread i owns row i = TMEM lane i; before a fragment's first
// tile it writes its query row to shared memory as fp16), 4-7 conversion of keys (thread i turns key
// i of a tile, from 64 bytes of codes and 8 of scales to a row of fp16 in the tiles' 128-byte
// swizzle; the next tile's bytes are under way meanwhile), 8-11 the same for values, 12 issues
// S = Q K^T and O += P V.  S has two buffers, so the product of the next tile runs under this tile's
// softmax.
//
// Bound: the softmax of a tile (0.9 us beside the conversions' instructions) and the products (0.6) in
// turn, 1.3 us a tile of 128 keys and SM whatever the rows; its bytes take 0.4.  8 caches of 9001 to
// 32768 keys, 8 KV heads of 128: 32 rows 92 us, 64 rows 93, 128 rows 100 (142 with the four warps of one
// warpgroup for the conversions), where groups of 16 rows take 56 each.
#include <math.h>

#include "bits4.cuh"
#include "bits4.h"
#include "cache_attn.cuh"

namespace apex {
namespace {

constexpr int kKeys = kCacheTileKeys;
constexpr int kBox = 128 * 128;  // [128 rows][64 fp16]
constexpr int kThreads = 16 * 32;
constexpr int kWarpK = 4, kWarpV = 8, kWarpMma = 12;
// registers of a thread at launch, and of each warpgroup's from then on
constexpr int kLaunchRegs = 128, kRegsSoftmax = 208, kRegsConvert = 104, kRegsMma = 96;
static_assert(128 * (kRegsSoftmax + 2 * kRegsConvert + kRegsMma) <= kThreads * kLaunchRegs, "register split");
constexpr float kBias = 7.f;  // weights are 2^7 times those relative to the running maximum, 2^15 at most

template <int DQK, int DV>
struct Cfg {
    static constexpr int kQTile = DQK / 64 * kBox, kKTile = kQTile, kVTile = DV / 64 * kBox;
    static constexpr int kStages = 2;
    static constexpr int kKOff = kQTile, kVOff = kKOff + kStages * kKTile, kBarOff = kVOff + kStages * kVTile;
    static constexpr int kBarQReady = 0, kBarQEmpty = 1, kBarKFull = 2, kBarKEmpty = 4, kBarVFull = 6, kBarVEmpty = 8;
    static constexpr int kBarSFull = 10, kBarPReady = 12, kBarPV = 14, kBarOEmpty = 15, kNumBars = 16;
    static constexpr int kSched = kBarOff + kNumBars * 8;
    static constexpr int kTmemSlot = kSched + 48;
    static constexpr int kSmemBytes = kTmemSlot + 16 + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    __device__ static constexpr uint32_t col_s(int s) { return 128u * s; }
    static constexpr uint32_t kColO = 256;
};

// Instruction descriptor as idesc_bf16_f32, with fp16 inputs (format 0 of A and B).
constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major)
{
    return idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));
}

// A packed row of D entries in registers, as it comes from memory.
template <int D>
struct PackedRow {
    uint4 w[D / 32];
    uint32_t s[D / 64];
    __device__ __forceinline__ void load(const uint8_t *bytes, const uint8_t *scales, size_t row, bool there)
    {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (there) w[i] = reinterpret_cast<const uint4 *>(bytes + row * (D / 2))[i];
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            s[i] = 0;
            if (there) s[i] = reinterpret_cast<const uint32_t *>(scales + row * (D / 16))[i];
        }
    }
    // to row r of the tile, boxes of 64 entries; a scale's value times codes is exact
    __device__ __forceinline__ void store(uint8_t *tile, int r) const
    {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t two = e4m3x2_to_f16x2(i & 1 ? s[i >> 1] >> 16 : s[i >> 1]);  // of 32 entries
            const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t scale = __byte_perm(two, 0, k < 2 ? 0x1010 : 0x3232);
                uint32_t v[4];
                e2m1_bytes_to_f16x2(words[k], v);
                const int c = 4 * i + k;
                *reinterpret_cast<uint4 *>(tile + (c >> 3) * kBox + swz128(r, c & 7)) =
                    make_uint4(mul_f16x2(v[0], scale), mul_f16x2(v[1], scale), mul_f16x2(v[2], scale), mul_f16x2(v[3], scale));
            }
        }
    }
};

template <int DQK, int DV>
__global__ void __launch_bounds__(kThreads, 1) decode4_wide_kernel(const __grid_constant__ Decode4Params p)
{
    using C = Cfg<DQK, DV>;
    const CacheAttnParams &pc = p.c;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sb + C::kBarOff + 8 * i; };
    const int live = min(4, (pc.rows_cap + 31) / 32);  // softmax warps that hold rows

    if (threadIdx.x == 0) {
        mbar_init(bar(C::kBarQReady), live);
        mbar_init(bar(C::kBarQEmpty), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(C::kBarKFull + s), 4);
            mbar_init(bar(C::kBarKEmpty + s), 1);
            mbar_init(bar(C::kBarVFull + s), 4);
            mbar_init(bar(C::kBarVEmpty + s), 1);
            mbar_init(bar(C::kBarSFull + s), 1);
            mbar_init(bar(C::kBarPReady + s), live);
        }
        mbar_init(bar(C::kBarPV), 1);
        mbar_init(bar(C::kBarOEmpty), live);
        fence_mbarrier_init();
    }
    if (warp == kWarpMma) tmem_alloc(sb + C::kTmemSlot, 512);
    // launched as a programmatic dependent: nothing in global memory is touched
    // before the stream's previous kernel is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Sched *sched = reinterpret_cast<Sched *>(smem + C::kSched);
    if (warp == kWarpK) make_sched<true>(pc, blockIdx.x, gridDim.x, sched);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kTmemSlot);

    Walk<true> walk(pc, *sched);
    Frag f;
    if (warp >= kWarpMma) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp >= kWarpK && warp < kWarpMma) {
        // ------------------------------------------------------------ conversion
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
        const int r = threadIdx.x & 127;  // row of the tile
        auto convert = [&](auto packed, bool values, const uint8_t *bytes, const uint8_t *scales, int off, int size,
                           int full, int empty) {
            int g = 0;  // tiles so far
            while (walk.next(pc, f)) {
                if (threadIdx.x == 32 * kWarpK && f.head) pc.units[f.unit] = make_int2(blockIdx.x, f.last);
                const size_t base = ((size_t)f.b * pc.H_kv + f.hk) * pc.S_cap;
                // of values, those of keys that some row sees: the others may be anything
                const int hi = values ? min(f.s.len + pc.T, pc.S_cap) : pc.S_cap;
                const int lo = values && pc.window > 0 ? f.s.len - pc.window + 1 : 0;
                auto there = [&](int key) { return key < hi && (key >= lo || key < pc.n_sink); };
                int key = kKeys * f.tile<true>(0) + r;
                packed.load(bytes, scales, base + key, there(key));
                for (int j = 0; j < f.n; ++j, ++g) {
                    const int st = g % C::kStages;
                    key = kKeys * f.tile<true>(min(j + 1, f.n - 1)) + r;
                    mbar_wait(bar(empty + st), ((g / C::kStages) & 1) ^ 1, p.c.wait);
                    packed.store(smem + off + st * size, r);
                    packed.load(bytes, scales, base + key, there(key));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(full + st));
                }
            }
        };
        if (warp < kWarpV)
            convert(PackedRow<DQK>(), false, p.k, p.k_scale, C::kKOff, C::kKTile, C::kBarKFull, C::kBarKEmpty);
        else
            convert(PackedRow<DV>(), true, p.v, p.v_scale, C::kVOff, C::kVTile, C::kBarVFull, C::kBarVEmpty);
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t idesc_qk = idesc_f16_f32(128, kKeys, false);
        constexpr uint32_t idesc_pv = idesc_f16_f32(128, DV, true);
        const bool one = elect_one();
        auto commit = [&](int i) {
            if (one) tc_commit(bar(i));
        };
        auto issue_qk = [&](int s, int ks) {
            const uint64_t da = smem_desc_sw128(sb, 16, 1024);
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
        auto issue_pv = [&](int s, int vs, bool acc) {
            const uint64_t dv = smem_desc_sw128(sb + C::kVOff + vs * C::kVTile, kBox, 1024);
            if (one) {
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i)
                    umma_ts(tmem + C::kColO, tmem + C::col_s(s) + 8 * i, dv + (uint64_t)(i * 2048 >> 4), idesc_pv,
                            (acc || i > 0) ? 1u : 0u);
            }
        };
        int g = 0;
        for (int fi = 0; walk.next(pc, f); ++fi) {
            mbar_wait(bar(C::kBarQReady), fi & 1, p.c.wait);
            mbar_wait(bar(C::kBarKFull + g % C::kStages), (g / C::kStages) & 1, p.c.wait);
            tc_fence_after();
            issue_qk(g & 1, g % C::kStages);
            commit(C::kBarKEmpty + g % C::kStages);
            if (f.n == 1) commit(C::kBarQEmpty);
            for (int j = 0; j < f.n; ++j, ++g) {
                const int ks = (g + 1) % C::kStages, vs = g % C::kStages;
                if (j + 1 < f.n) {
                    mbar_wait(bar(C::kBarKFull + ks), ((g + 1) / C::kStages) & 1, p.c.wait);
                    tc_fence_after();
                    issue_qk((g + 1) & 1, ks);
                    commit(C::kBarKEmpty + ks);
                    if (j + 2 == f.n) commit(C::kBarQEmpty);
                }
                mbar_wait(bar(C::kBarVFull + vs), (g / C::kStages) & 1, p.c.wait);
                mbar_wait(bar(C::kBarPReady + (g & 1)), (g >> 1) & 1, p.c.wait);
                if (j == 0) mbar_wait(bar(C::kBarOEmpty), (fi & 1) ^ 1, p.c.wait);
                tc_fence_after();
                issue_pv(g & 1, vs, j > 0);
                commit(C::kBarPV);
                commit(C::kBarVEmpty + vs);
            }
        }
    } else if (warp < kWarpK) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------------------ queries, softmax, epilogue
        const int i = threadIdx.x;  // row of the M tile == TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t o_addr = lane_base + C::kColO;
        int g = 0;
        for (int fi = 0; warp < live && walk.next(pc, f); ++fi) {
            const int r = f.group * pc.group + i;  // row of the KV head
            const bool row_ok = i < pc.rows_cap && r < pc.R;
            const size_t kv = (size_t)f.b * pc.H_kv + f.hk, row = kv * pc.R + r;

            // ---- the query row, relative to its largest entry, as fp16
            mbar_wait(bar(C::kBarQEmpty), (fi & 1) ^ 1, p.c.wait);
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + row * DQK);
            uint32_t top = 0;
#pragma unroll 8
            for (int c = 0; c < DQK / 8; ++c)
                if (row_ok) {
                    const uint4 x = src[c];
                    top = __vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
                    top = __vmaxu2(__vmaxu2(top, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
                }
            top = max(top & 0xffffu, top >> 16);
            // largest magnitude 2^(ex - 127) to under twice that: entries times 2^(131 - ex) are below 32
            const uint32_t ex = min(max(top >> 7, 5u), 254u);
            const float down = __uint_as_float((258u - ex) << 23), up = __uint_as_float((ex - 4u) << 23);
#pragma unroll 8
            for (int c = 0; c < DQK / 8; ++c) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (row_ok) x = src[c];
                uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack_f16x2(bf16lo_to_f32(w[e]) * down, bf16hi_to_f32(w[e]) * down);
                *reinterpret_cast<uint4 *>(smem + (c >> 3) * kBox + swz128(i, c & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarQReady));
            const float kf = p.k_factor ? p.k_factor[f.hk] : 1.f, vf = pc.v_factor ? pc.v_factor[f.hk] : 1.f;
            const float scale = fmaxf(up * kf * pc.scale_log2, 1e-37f);  // not 0: masked scores stay -inf

            const int m = f.s.len + r % pc.T;  // position
            const int key_hi = row_ok ? min(m, pc.S_cap - 1) : -1, key_lo = pc.window > 0 ? m - pc.window + 1 : 0;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < f.n; ++j, ++g) {
                const uint32_t s_addr = lane_base + C::col_s(g & 1);
                const int key0 = kKeys * f.tile<true>(j), lo = key_lo - key0, hi = key_hi - key0, sink = pc.n_sink - key0;
                mbar_wait(bar(C::kBarSFull + (g & 1)), (g >> 1) & 1, p.c.wait);
                tc_fence_after();
                uint32_t v[128];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    tmem_ld32(s_addr + 32 * ch, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * ch]));
                tmem_wait_ld();
                if (!__all_sync(0xffffffffu, (lo <= 0 || sink >= kKeys) && hi >= kKeys - 1)) {
                    if (sink > 0)
                        mask_row128_sink(v, lo, hi, sink);
                    else
                        mask_row128(v, lo, hi);
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
                const float m_new = fmaxf(m_run, mx * scale);
                const bool large = fabsf(m_new) > kLargeScore && m_new != -INFINITY;
                const bool need = (m_run != -INFINITY && m_new - m_run > 8.f) || large;
                // the last tile's product must be done before O is touched, and is waited for in every
                // tile, so that no phase of its barrier is skipped
                if (g > 0) mbar_wait(bar(C::kBarPV), (g - 1) & 1, p.c.wait);
                float factor = scale, base = 0.f;  // of the scores from here on, where they are large
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
                    if (__any_sync(0xffffffffu, large)) {
                        base = m_run == -INFINITY ? 0.f : m_run;
                        factor = 1.f;
#pragma unroll
                        for (int e = 0; e < 128; ++e)
                            v[e] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(v[e]), scale), base));
                    }
                } else if (m_run == -INFINITY) {
                    m_run = m_new;
                }
                const float m_use = kBias - (m_run == -INFINITY ? 0.f : m_run - base);
                const uint64_t SC = f2_pack(factor, factor), NM = f2_pack(m_use, m_use);
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
                        pk[e2] = pack_f16x2(p0, p1);  // the tensor cores take fp16; the sum keeps fp32
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
                if (lane == 0) mbar_arrive(bar(C::kBarPReady + (g & 1)));
            }

            // ---- the finished row, or this fragment's part of it
            mbar_wait(bar(C::kBarPV), (g - 1) & 1, p.c.wait);
            tc_fence_after();
            write_row<DV, false>(pc, o_addr, f.head && f.tail, row_ok, row, 2 * blockIdx.x + (f.head ? 1 : 0), i, m_run,
                                 l_run, vf);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarOEmpty));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DQK, int DV>
cudaError_t launch_t(const Decode4Params &p, int grid, cudaStream_t stream)
{
    using C = Cfg<DQK, DV>;
    static KernelSetup setup;
    const cudaError_t err = setup(decode4_wide_kernel<DQK, DV>, C::kSmemBytes, kLaunchRegs);
    if (err != cudaSuccess) return err;
    return launch_dependent(decode4_wide_kernel<DQK, DV>, grid, kThreads, C::kSmemBytes, stream, p);
}

}  // namespace

cudaError_t launch_decode4_wide(const Decode4Params &p, int grid, cudaStream_t stream)
{
    if (p.c.d_qk == 64) return launch_t<64, 64>(p, grid, stream);
    if (p.c.d_qk == 128) return launch_t<128, 128>(p, grid, stream);
    return launch_t<192, 128>(p, grid, stream);
}

}  // namespace apex
