// rope.cu -- rotary positions of query and key rows at given token positions
// (Part 1, §4.2-§4.4), interleaved or half layout, any part of the row, with an
// optional append of rotated keys and of values to cache rows.  How angles are made: rope.cuh.
//
// A thread owns one unit of a token's row and walks over heads, so the sines and
// cosines of the unit (4 or 8 pairs) are computed once per head group; a unit is
// one 16-byte chunk (interleaved), or the two 16-byte chunks whose elements pair up
// (half layout).  The bound is HBM: every row is read and written once.  8191 tokens of
// 128 + 8 heads of 192 entries (856 MB): 130 us, 6.6 TB/s; one token of 32 + 8 heads with its
// key and value appended: 2.4 us.
#include "device_common.cuh"
#include "rope.cuh"
#include "rope.h"

namespace apex {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads whose loads are in flight together

// (cos, sin) of pair i at position m
__device__ __forceinline__ void pair_angle(const RopeParams &p, int i, int m, float &c, float &s)
{
    turn_angle(p.turns[i], m, p.sign, c, s);
}

// Output row of token s of sequence b, or -1 when it is not written.
__device__ __forceinline__ long long out_row(const RopeParams &p, const RopeTensor &t, int b, int s)
{
    if (!t.append || !p.row0) return s;
    const long long r = (long long)p.row0[b] + s;
    return (r < 0 || r >= p.out_rows) ? -1 : r;
}

// Units of a row, 16 bytes wide: NC of the d_row / 8 chunks are rotated.
//   interleaved: unit u = chunk u; half: unit u < NP = d_rot / 16 is the chunk pair
//   (c0 + u, c0 + u + NP), the other units are the copied chunks in order.
template <bool HALF>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const __grid_constant__ RopeParams p)
{
    // launched as a programmatic dependent: inputs may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RopeGroup g = p.groups[blockIdx.y];
    const RopeTensor &t = p.t[g.tensor];
    const int c0 = p.rot_start >> 3, nrot = p.d_rot >> 3;
    const int np = HALF ? nrot >> 1 : nrot;  // units that rotate
    const int units = t.rotate ? (t.d_row >> 3) - (HALF ? np : 0) : t.d_row >> 3;
    const long long n = (long long)p.B * p.S * units;
    for (long long idx = (long long)blockIdx.x * kThreads + threadIdx.x; idx < n;
         idx += (long long)gridDim.x * kThreads) {
        const int u = (int)(idx % units);
        const int token = (int)(idx / units);
        const int b = token / p.S, s = token % p.S;
        const long long row = out_row(p, t, b, s);
        if (row < 0) continue;
        // chunk(s) of the unit
        int ca = u, cb = -1, pair = -1;
        if (t.rotate) {
            if (HALF) {
                if (u < np) {
                    ca = c0 + u;
                    cb = ca + np;
                    pair = 8 * u;
                } else {
                    ca = u - np;
                    if (ca >= c0) ca += nrot;
                }
            } else if (u >= c0 && u < c0 + nrot) {
                pair = 4 * (u - c0);
            }
        }
        const uint16_t *src = t.in + b * t.in_b + s * t.in_s + 8 * ca;
        uint16_t *dst = t.out + b * t.out_b + row * t.out_s + 8 * ca;
        constexpr int NA = HALF ? 8 : 4;
        float c[NA], sn[NA];
        if (pair >= 0) {
            const int m = p.positions[b * p.pos_stride + s];
#pragma unroll
            for (int e = 0; e < NA; ++e) pair_angle(p, pair + e, m, c[e], sn[e]);
        }
        const int h1 = g.h0 + g.n;
        for (int h = g.h0; h < h1; h += kBatch) {
            uint4 x[kBatch], y[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (h + k < h1) {
                    x[k] = *reinterpret_cast<const uint4 *>(src + (h + k) * t.in_h);
                    if (HALF && cb >= 0) y[k] = *reinterpret_cast<const uint4 *>(src + (h + k) * t.in_h + 8 * np);
                }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (h + k < h1) {
                    if (pair >= 0) {
                        uint32_t *xw = &x[k].x, *yw = &y[k].x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (HALF) {
                                float u0, u1, w0, w1;
                                rotate2(bf16lo_to_f32(xw[e]), bf16lo_to_f32(yw[e]), c[2 * e], sn[2 * e], u0, w0);
                                rotate2(bf16hi_to_f32(xw[e]), bf16hi_to_f32(yw[e]), c[(2 * e + 1) % NA],
                                        sn[(2 * e + 1) % NA], u1, w1);
                                xw[e] = pack_bf16x2(u0, u1);
                                yw[e] = pack_bf16x2(w0, w1);
                            } else {
                                float u0, w0;
                                rotate2(bf16lo_to_f32(xw[e]), bf16hi_to_f32(xw[e]), c[e], sn[e], u0, w0);
                                xw[e] = pack_bf16x2(u0, w0);
                            }
                        }
                    }
                    *reinterpret_cast<uint4 *>(dst + (h + k) * t.out_h) = x[k];
                    if (HALF && cb >= 0) *reinterpret_cast<uint4 *>(dst + (h + k) * t.out_h + 8 * np) = y[k];
                }
        }
    }
}

// The same for rows whose parts, strides or alignment do not fit 16-byte chunks: a
// thread owns one pair, or one copied entry, and reads and writes 2 bytes at a time
// (395 us on the 8191 tokens above, where the other kernel takes 130).
__global__ void __launch_bounds__(kThreads) rope_pairs_kernel(const __grid_constant__ RopeParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RopeGroup g = p.groups[blockIdx.y];
    const RopeTensor &t = p.t[g.tensor];
    const int pairs = p.d_rot / 2;
    const int units = t.rotate ? t.d_row - pairs : t.d_row;
    const long long n = (long long)p.B * p.S * units;
    for (long long idx = (long long)blockIdx.x * kThreads + threadIdx.x; idx < n;
         idx += (long long)gridDim.x * kThreads) {
        const int u = (int)(idx % units);
        const int token = (int)(idx / units);
        const int b = token / p.S, s = token % p.S;
        const long long row = out_row(p, t, b, s);
        if (row < 0) continue;
        const uint16_t *src = t.in + b * t.in_b + s * t.in_s;
        uint16_t *dst = t.out + b * t.out_b + row * t.out_s;
        if (t.rotate && u < pairs) {
            const int a = p.rot_start + (p.half ? u : 2 * u);
            const int d = a + (p.half ? pairs : 1);
            float c, sn;
            pair_angle(p, u, p.positions[b * p.pos_stride + s], c, sn);
            for (int h = g.h0; h < g.h0 + g.n; ++h) {
                float x, y;
                rotate2(bf16lo_to_f32(src[h * t.in_h + a]), bf16lo_to_f32(src[h * t.in_h + d]), c, sn, x, y);
                const uint32_t w = pack_bf16x2(x, y);
                dst[h * t.out_h + a] = (uint16_t)w;
                dst[h * t.out_h + d] = (uint16_t)(w >> 16);
            }
        } else {
            int a = u - (t.rotate ? pairs : 0);
            if (t.rotate && a >= p.rot_start) a += p.d_rot;
            for (int h = g.h0; h < g.h0 + g.n; ++h) dst[h * t.out_h + a] = src[h * t.in_h + a];
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int kind, int grid_x, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid_x, p.n_groups);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (kind == kRopeInterleaved) return cudaLaunchKernelEx(&cfg, rope_rows_kernel<false>, p);
    if (kind == kRopeHalf) return cudaLaunchKernelEx(&cfg, rope_rows_kernel<true>, p);
    return cudaLaunchKernelEx(&cfg, rope_pairs_kernel, p);
}

}  // namespace apex
