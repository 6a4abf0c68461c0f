// bits4.cu -- rows of keys and values into a cache held in 4 bits, and back.
//
// A thread has 16 neighbouring entries, those of one scale: 32 bytes of bf16, 8 bytes of codes
// and a byte of scale, so nothing is exchanged between threads.
//   scale = e4m3(max |x| / (6 factor)),  code = e2m1(x / (scale factor))
// both rounded to nearest, ties to even.  The quotient is a product with the reciprocal and one
// correction by its residual: an exact tie then comes out as exactly that, and a quotient that is
// no tie is further from one than this is off (x has 8 significant bits, the scale 4).
//
// Bound: HBM, 2.56 bytes an entry either way.
#include "bits4.cuh"
#include "bits4.h"
#include "device_common.cuh"

namespace apex {
namespace {

// What thread `threadIdx.x` of a block works on: rows are (b, h, s) in that order.
struct Place {
    long long in, row;  // element of x, row of the cache
    int h, block;       // KV head, block of 16 entries within the row
    bool ok, there;     // a row of x; one inside the cache
    __device__ __forceinline__ Place(const Bits4Params &p, const Bits4Tensor &t)
    {
        const int blocks = t.d / kBits4Block, per = kBits4Threads / blocks;
        const int mine = threadIdx.x / blocks;
        const long long r = (long long)blockIdx.x * per + mine;
        ok = mine < per && r < (long long)p.B * p.H * p.S;
        const uint32_t rr = ok ? (uint32_t)r : 0u;  // below 2^31
        const uint32_t bh = rr / (uint32_t)p.S, s = rr - bh * (uint32_t)p.S, b = bh / (uint32_t)p.H;
        h = (int)(bh - b * (uint32_t)p.H);
        block = threadIdx.x - mine * blocks;
        const long long to = (p.row0 ? (long long)p.row0[b] : 0) + s;
        there = to >= 0 && to < p.S_cap;
        in = b * t.x_b + h * t.x_h + s * t.x_s + kBits4Block * block;
        row = (long long)bh * p.S_cap + to;
    }
};

__global__ void __launch_bounds__(kBits4Threads) append4_kernel(const __grid_constant__ Bits4Params p)
{
    // launched as a programmatic dependent: inputs may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Bits4Tensor &t = p.t[blockIdx.y];
    const Place at(p, t);
    if (!at.ok || !at.there) return;
    const uint16_t *src = t.x + at.in;
    uint32_t w[8];
    if (t.wide) {
        const uint4 a = reinterpret_cast<const uint4 *>(src)[0], b = reinterpret_cast<const uint4 *>(src)[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = src[2 * e] | (uint32_t)src[2 * e + 1] << 16;
    }
    // magnitudes order as their bits do: infinity is 0x7f80, NaN above it
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    const float f = t.factor ? t.factor[at.h] : 1.f;
    uint32_t scale = f32_to_e4m3(__uint_as_float(top << 16) / (6.f * f));
    uint32_t codes[2] = {0, 0};
    if (top >= 0x7f80u) {
        scale = 0x7f;  // 4 bits hold no infinity and no NaN: the whole block reads as NaN
    } else {
        const float step = f16x2_to_f32(e4m3x2_to_f16x2(scale)).x * f;
        const float inv = step > 0.f ? 1.f / step : 0.f;
        const bool far = !(inv <= 3e38f);  // a reciprocal past the largest number: divide
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = i ? bf16hi_to_f32(w[e]) : bf16lo_to_f32(w[e]);
                const float y = fminf(fmaxf(x * inv, -8.f), 8.f);
                q[i] = far ? x / step : fmaf(fmaf(-y, step, x), inv, y);
            }
            codes[e >> 2] |= f32x2_to_e2m1x2(q[0], q[1]) << (8 * (e & 3));
        }
    }
    *reinterpret_cast<uint2 *>(t.bytes + at.row * (t.d / 2) + 8 * at.block) = make_uint2(codes[0], codes[1]);
    t.scales[at.row * (t.d / kBits4Block) + at.block] = (uint8_t)scale;
}

__global__ void __launch_bounds__(kBits4Threads) unpack4_kernel(const __grid_constant__ Bits4Params p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Bits4Tensor &t = p.t[blockIdx.y];
    const Place at(p, t);
    if (!at.ok) return;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0;
    if (at.there) {  // rows outside the cache read as zeros
        const uint2 c = *reinterpret_cast<const uint2 *>(t.bytes + at.row * (t.d / 2) + 8 * at.block);
        const float s = f16x2_to_f32(e4m3x2_to_f16x2(t.scales[at.row * (t.d / kBits4Block) + at.block])).x;
        const float f = t.factor ? t.factor[at.h] : 1.f;
        uint32_t v[2][4];
        e2m1_bytes_to_f16x2(c.x, v[0]);
        e2m1_bytes_to_f16x2(c.y, v[1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 x = f16x2_to_f32(v[e >> 2][e & 3]);
            w[e] = pack_bf16x2(x.x * s * f, x.y * s * f);
        }
    }
    uint16_t *dst = t.x + at.in;
    if (t.wide) {
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

template <typename K>
cudaError_t launch(K kernel, const Bits4Params &p, cudaStream_t stream)
{
    const int d = p.t[0].d > p.t[1].d ? p.t[0].d : p.t[1].d;
    const long long per = kBits4Threads / (d / kBits4Block), rows = (long long)p.B * p.H * p.S;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + per - 1) / per), 2);
    cfg.blockDim = dim3(kBits4Threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_append4(const Bits4Params &p, cudaStream_t stream) { return launch(append4_kernel, p, stream); }
cudaError_t launch_unpack4(const Bits4Params &p, cudaStream_t stream) { return launch(unpack4_kernel, p, stream); }

}  // namespace apex
