// bits4.cu -- rows of keys and values into a cache held in 4 bits, and back.
//
// A thread has 16 neighbouring entries of a row, those of one scale: 32 bytes of bf16, 8 bytes of
// codes and a byte of scale, so nothing is exchanged between threads; it takes the same entries
// of a few rows of a (sequence, head), whose loads are in flight together.
//   scale = e4m3(max |x| / (6 factor)),  code = e2m1(x / (scale factor))
// both rounded to nearest, ties to even.  A quotient is a product with the reciprocal and one
// correction by its residual: an exact tie then comes out as exactly that, and a quotient that is
// no tie is further from one than this is off (x has 8 significant bits, the scale 4).
//
// Bound: HBM, 2.56 bytes an entry either way.  32767 tokens of 8 heads of 128 written and read back (344
// MB): 60 us, 32.5 and 27.6 (67 in blocks of 256 threads with two rows of a thread and more blocks, 84
// with 16 bytes of a row at a time, as half sectors go twice); writing is near the issue of its
// instructions as well.  One token for each of 16 sequences, both ways: 3.5 us.
#include <algorithm>

#include "bits4.cuh"
#include "bits4.h"
#include "device_common.cuh"

namespace apex {
namespace {

constexpr int kRows = 4;  // of a thread, whose loads are in flight together

// A block's rows: `per` at a time of head blockIdx.x of tensor blockIdx.z % 2 and sequence
// blockIdx.z / 2, and of those a grid's width behind.  Blocks of the same tokens run side by side, as
// projections leave the heads of a token beside one another.
struct Place {
    int mine, block, s;  // this thread's row of them, its 16 entries, its first row
    __device__ __forceinline__ Place(const Bits4Tensor &t)
    {
        mine = (threadIdx.x * t.inv_blocks) >> 16;  // threadIdx.x / (d / 16)
        block = threadIdx.x - mine * (t.d / kBits4Block);
        s = blockIdx.y * t.per * kRows + mine;
    }
};

// 16 entries, by what their addresses are multiples of: 32, 16 or 2 bytes.
__device__ __forceinline__ void load16(const uint16_t *src, int wide, uint32_t (&w)[8])
{
    if (wide == 32) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(src)
                     : "memory");
    } else if (wide == 16) {
        const uint4 a = reinterpret_cast<const uint4 *>(src)[0], b = reinterpret_cast<const uint4 *>(src)[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = src[2 * e] | (uint32_t)src[2 * e + 1] << 16;
    }
}

__device__ __forceinline__ void store16(uint16_t *dst, int wide, const uint32_t (&w)[8])
{
    if (wide == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else if (wide == 16) {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dst[2 * e] = (uint16_t)w[e];
            dst[2 * e + 1] = (uint16_t)(w[e] >> 16);
        }
    }
}

// Codes (8 bytes) and scale of 16 entries; f: the head's factor, six, sixth: 6 f and about 1 / (6 f).
__device__ __forceinline__ uint32_t quantise(const uint32_t (&w)[8], float f, float six, float sixth, uint2 &codes)
{
    uint32_t top = abs_bf16x2(w[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) top = max_nan_bf16x2(top, abs_bf16x2(w[e]));
    top = max(top & 0xffffu, top >> 16);  // magnitudes order as their bits do: infinity is 0x7f80, NaN above it
    codes = make_uint2(0, 0);
    if (top >= 0x7f80u) return 0x7f;  // 4 bits hold no infinity and no NaN: the whole block reads as NaN
    const float x0 = __uint_as_float(top << 16), y0 = x0 * sixth;
    float most = fmaf(fmaf(-y0, six, x0), sixth, y0);
    const bool plain = most < 448.f && six < 1e37f && six > 1e-37f;
    if (!plain) most = x0 / six;
    const uint32_t scale = f32_to_e4m3(most);
    const float step = f16x2_to_f32(e4m3x2_to_f16x2(scale)).x * f, inv = fast_reciprocal(step);
    float q[2][8];
    if (plain && inv < 1e38f) {
        // quotients are below 16, so nothing overflows
        const uint64_t inv2 = f2_pack(inv, inv), step2 = f2_pack(-step, -step);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint64_t x = f2_pack(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e])), y = f2_mul(x, inv2);
            f2_unpack(f2_fma(f2_fma(y, step2, x), inv2, y), q[e >> 2][2 * (e & 3)], q[e >> 2][2 * (e & 3) + 1]);
        }
    } else if (step > 0.f) {  // the scale at its end, or numbers past what the reciprocals hold: divide
        for (int e = 0; e < 8; ++e) {
            q[e >> 2][2 * (e & 3)] = bf16lo_to_f32(w[e]) / step;
            q[e >> 2][2 * (e & 3) + 1] = bf16hi_to_f32(w[e]) / step;
        }
    } else {
        return scale;  // a scale of zero
    }
    codes.x = f32x8_to_e2m1(q[0]);
    codes.y = f32x8_to_e2m1(q[1]);
    return scale;
}

__device__ __forceinline__ void append_rows(const Bits4Params &p, const Bits4Tensor &t, const Place &at, int b, int h)
{
    const long long to = (p.row0 ? (long long)p.row0[b] : 0) + at.s, row = ((long long)b * p.H + h) * p.S_cap + to;
    const uint16_t *src = t.x + b * t.x_b + h * t.x_h + at.s * t.x_s + kBits4Block * at.block;
    const long long x_step = t.per * t.x_s;
    uint8_t *bytes = t.bytes + row * (t.d / 2) + 8 * at.block, *scales = t.scales + row * (t.d / kBits4Block) + at.block;
    const float f = t.factor ? t.factor[h] : 1.f, six = 6.f * f, sixth = fast_reciprocal(six);
    uint32_t w[kRows][8];
    bool in[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k, src += x_step) {
        in[k] = at.s + k * t.per < p.S && to + k * t.per >= 0 && to + k * t.per < p.S_cap;
        if (in[k]) load16(src, t.wide, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        if (in[k]) {
            uint2 codes;
            const uint32_t scale = quantise(w[k], f, six, sixth, codes);
            *reinterpret_cast<uint2 *>(bytes) = codes;
            *scales = (uint8_t)scale;
        }
        bytes += t.per * (t.d / 2);
        scales += t.per * (t.d / kBits4Block);
    }
}

__global__ void __launch_bounds__(kBits4Threads, 6) append4_kernel(const __grid_constant__ Bits4Params p)
{
    // launched as a programmatic dependent: inputs may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Bits4Tensor t = p.t[blockIdx.z & 1];
    Place at(t);
    if (at.mine >= t.per) return;
    for (; at.s < p.S + at.mine; at.s += gridDim.y * t.per * kRows)
        for (int b = blockIdx.z >> 1; b < p.B; b += gridDim.z >> 1)
            for (int h = blockIdx.x; h < p.H; h += gridDim.x) append_rows(p, t, at, b, h);
}

__device__ __forceinline__ void unpack_rows(const Bits4Params &p, const Bits4Tensor &t, const Place &at, int b, int h)
{
    const long long from = (p.row0 ? (long long)p.row0[b] : 0) + at.s, row = ((long long)b * p.H + h) * p.S_cap + from;
    uint16_t *to = t.x + b * t.x_b + h * t.x_h + at.s * t.x_s + kBits4Block * at.block;
    const long long x_step = t.per * t.x_s;
    const uint8_t *bytes = t.bytes + row * (t.d / 2) + 8 * at.block, *scales = t.scales + row * (t.d / kBits4Block) + at.block;
    const float f = t.factor ? t.factor[h] : 1.f;
    const uint64_t f2 = f2_pack(f, f);
    uint2 c[kRows];
    uint32_t s[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        c[k] = make_uint2(0, 0);
        s[k] = 0;  // rows outside the cache read as zeros
        if (at.s + k * t.per < p.S && from + k * t.per >= 0 && from + k * t.per < p.S_cap) {
            c[k] = *reinterpret_cast<const uint2 *>(bytes);
            s[k] = *scales;
        }
        bytes += t.per * (t.d / 2);
        scales += t.per * (t.d / kBits4Block);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k, to += x_step) {
        if (at.s + k * t.per >= p.S) break;
        const uint32_t scale = __byte_perm(e4m3x2_to_f16x2(s[k]), 0, 0x1010);
        uint32_t v[2][4], w[8];
        e2m1_bytes_to_f16x2(c[k].x, v[0]);
        e2m1_bytes_to_f16x2(c[k].y, v[1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 x = f16x2_to_f32(mul_f16x2(v[e >> 2][e & 3], scale));  // exact
            float lo, hi;
            f2_unpack(f2_mul(f2_pack(x.x, x.y), f2), lo, hi);
            w[e] = pack_bf16x2(lo, hi);
        }
        store16(to, t.wide, w);
    }
}

__global__ void __launch_bounds__(kBits4Threads, 6) unpack4_kernel(const __grid_constant__ Bits4Params p)
{
    // launched as a programmatic dependent: inputs may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Bits4Tensor t = p.t[blockIdx.z & 1];
    Place at(t);
    if (at.mine >= t.per) return;
    for (; at.s < p.S + at.mine; at.s += gridDim.y * t.per * kRows)
        for (int b = blockIdx.z >> 1; b < p.B; b += gridDim.z >> 1)
            for (int h = blockIdx.x; h < p.H; h += gridDim.x) unpack_rows(p, t, at, b, h);
}

template <typename K>
cudaError_t launch(K kernel, Bits4Params &p, cudaStream_t stream)
{
    // threads for one row of each turn at least, and for no more rows than there are
    int threads = 32;
    for (Bits4Tensor &t : p.t) {
        const int blocks = t.d / kBits4Block;
        threads = std::max(threads, std::min(kBits4Threads, (p.S * blocks + 31) / 32 * 32));
        t.inv_blocks = (65535 + blocks) / blocks;
    }
    int least = kBits4Threads;
    for (Bits4Tensor &t : p.t) {
        t.per = threads / (t.d / kBits4Block);
        least = std::min(least, t.per);
    }
    const int per = least * kRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.H, std::min((p.S + per - 1) / per, 65535), 2 * std::min(p.B, 32767));
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_append4(Bits4Params &p, cudaStream_t stream) { return launch(append4_kernel, p, stream); }
cudaError_t launch_unpack4(Bits4Params &p, cudaStream_t stream) { return launch(unpack4_kernel, p, stream); }

}  // namespace apex
