// norm_rope.cu -- RMS norm of query and key heads (Part 1, §3) and their rotary positions
// (Part 1, §4.2-§4.4) in one pass, and the gradient of both.
//
// With x a row of d entries, w its weights and R the rotation by the token's position:
//   rs = 1 / sqrt(mean(x^2) + eps),  u = x rs,  y = R (u w)
// and for the gradient dy of y
//   g = R^-1 dy,  dx = rs (g w - u mean(g w u)),  dw = sum over rows of g u.
// rs is made again from x: keeping it would save none of x's bytes.
//
// The bound is HBM: a row is read once (twice as many bytes for the gradient) and written once.
// A row belongs to 8, 16 or 32 neighbouring lanes with 16 bytes each, so its sums are a few
// shuffles, the other half of a pair (half layout) is one lane away, and nothing goes through
// shared memory.  A lane walks over the heads of its token: their loads are in flight
// together and share the sines.
//
// dw: a thread adds up its 8 columns over all rows that it meets, a block its threads' sums,
// and a second kernel the blocks' sums, in 64 bits: a fixed order, so equal inputs give equal
// bits.
#include "device_common.cuh"
#include "norm_rope.h"
#include "rope.cuh"

namespace apex {
namespace {

constexpr int kBatch = 4;      // heads whose loads are in flight together
constexpr int kGradBatch = 2;  // of the gradient, with two rows each

__device__ __forceinline__ long long out_row(const NormRopeParams &p, const NormTensor &t, int b, int s)
{
    if (!t.append || !p.row0) return s;
    const long long r = (long long)p.row0[b] + s;
    return (r < 0 || r >= p.out_rows) ? -1 : r;
}

__device__ __forceinline__ float weight_at(const NormTensor &t, int h, int e)
{
    if (!t.weight) return 1.f;
    const size_t i = (size_t)h * t.weight_h + e;
    return t.weight_f32 ? static_cast<const float *>(t.weight)[i]
                        : bf16lo_to_f32(static_cast<const uint16_t *>(t.weight)[i]);
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16lo_to_f32(w[e]);
        f[2 * e + 1] = bf16hi_to_f32(w[e]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

template <int L>
__device__ __forceinline__ float sum_lanes(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ uint4 shfl4(const uint4 &v, int lane)
{
    return make_uint4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                      __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
}

// What a lane does with its chunk of 8 entries: which pairs they belong to and where the
// other halves of the pairs are.
template <int L, bool HALF>
struct Chunk {
    int at;       // its index in the row
    bool mine;    // inside the row
    bool turned;  // inside the part that turns
    bool second;  // half layout: holds the second entries of its pairs
    int pair;     // first pair
    int other;    // lane (and chunk, below) of the pairs' other entries
    int other_at;
    __device__ __forceinline__ Chunk(const NormRopeParams &p, const NormTensor &t)
    {
        const int lane = threadIdx.x & 31;
        at = lane % L;
        mine = at < (t.d_row >> 3);
        const int c0 = p.rot_start >> 3, n = p.d_rot >> 3, in = at - c0;
        turned = t.norm && in >= 0 && in < n;
        second = HALF && turned && in >= n / 2;
        pair = HALF ? 8 * (second ? in - n / 2 : in) : 4 * in;
        other_at = (HALF && turned) ? (second ? at - n / 2 : at + n / 2) : at;
        other = lane - at + other_at;
    }
    // entries a (own) and o (the other halves', half layout) turned by (c, s)
    __device__ __forceinline__ void turn(float (&a)[8], const float (&o)[8], const float *c, const float *s) const
    {
        if (HALF) {
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = second ? fmaf(o[e], s[e], a[e] * c[e]) : fmaf(a[e], c[e], -o[e] * s[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) rotate2(a[2 * e], a[2 * e + 1], c[e], s[e], a[2 * e], a[2 * e + 1]);
        }
    }
};

__device__ __forceinline__ const NormTensor &tensor_of(const NormRopeParams &p, int &group)
{
    int i = 0;
    group = blockIdx.y;
    while (group >= p.t[i].n_groups) group -= p.t[i++].n_groups;
    return p.t[i];
}

template <int L, bool HALF>
__global__ void __launch_bounds__(kNormThreads) norm_rows_kernel(const __grid_constant__ NormRopeParams p)
{
    // launched as a programmatic dependent: inputs may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kRows = kNormThreads / L, kWarpRows = 32 / L, NA = HALF ? 8 : 4;
    int group;
    const NormTensor &t = tensor_of(p, group);
    const int h0 = group * p.per, h1 = min(h0 + p.per, t.n_heads);
    const Chunk<L, HALF> ch(p, t);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float w[8], wo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = wo[e] = 1.f;
    auto load_weights = [&](int h) {
        if (!t.norm || !t.weight || !ch.mine) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = weight_at(t, h, 8 * ch.at + e);
            if (HALF) wo[e] = weight_at(t, h, 8 * ch.other_at + e);
        }
    };
    if (t.weight_h == 0) load_weights(0);
    const int tokens = p.B * p.S;  // below 2^31
    // the warp's rows together: every lane takes part in the shuffles
    for (long long base = (long long)blockIdx.x * kRows + warp * kWarpRows; base < tokens;
         base += (long long)gridDim.x * kRows) {
        const long long token = base + lane / L;
        const bool real = token < tokens;
        const int b = real ? (int)(token / p.S) : 0, s = real ? (int)(token % p.S) : 0;
        const long long row = out_row(p, t, b, s);
        const bool ok = real && ch.mine && row >= 0;
        const uint16_t *src = t.x + b * t.x_b + s * t.x_s + 8 * ch.at;
        uint16_t *dst = t.out + b * t.out_b + row * t.out_s + 8 * ch.at;
        float c[NA], sn[NA];
        if (ch.turned) {
            const int m = p.positions[b * p.pos_stride + s];
#pragma unroll
            for (int e = 0; e < NA; ++e) turn_angle(p.turns[ch.pair + e], m, p.sign, c[e], sn[e]);
        }
        for (int h = h0; h < h1; h += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                x[k] = make_uint4(0, 0, 0, 0);
                if (ok && h + k < h1) x[k] = *reinterpret_cast<const uint4 *>(src + (h + k) * t.x_h);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (h + k >= h1) break;
                if (t.norm) {
                    float a[8], o[8];
                    unpack8(x[k], a);
                    if (HALF) unpack8(shfl4(x[k], ch.other), o);
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], ss);
                    const float rs = rsqrtf(fmaf(sum_lanes<L>(ss), t.inv_d, p.eps));
                    if (t.weight_h != 0) load_weights(h + k);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        a[e] *= rs * w[e];
                        if (HALF) o[e] *= rs * wo[e];
                    }
                    if (ch.turned) ch.turn(a, o, c, sn);
                    x[k] = pack8(a);
                }
                if (ok) *reinterpret_cast<uint4 *>(dst + (h + k) * t.out_h) = x[k];
            }
        }
    }
}

template <int L, bool HALF>
__global__ void __launch_bounds__(kNormThreads, 3) norm_grad_rows_kernel(const __grid_constant__ NormRopeParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kRows = kNormThreads / L, kWarpRows = 32 / L, NA = HALF ? 8 : 4;
    __shared__ float sums[kRows][8 * L];
    int group;
    const NormTensor &t = tensor_of(p, group);
    const int h0 = group * p.per, h1 = min(h0 + p.per, t.n_heads);
    const Chunk<L, HALF> ch(p, t);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float w[8], dw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        dw[e] = 0.f;
        // with weights for each head a block has one head
        w[e] = ch.mine ? weight_at(t, h0, 8 * ch.at + e) : 0.f;
    }
    const int tokens = p.B * p.S;
    for (long long base = (long long)blockIdx.x * kRows + warp * kWarpRows; base < tokens;
         base += (long long)gridDim.x * kRows) {
        const long long token = base + lane / L;
        const bool real = token < tokens, ok = real && ch.mine;
        const int b = real ? (int)(token / p.S) : 0, s = real ? (int)(token % p.S) : 0;
        const uint16_t *src = t.x + b * t.x_b + s * t.x_s + 8 * ch.at;
        const uint16_t *grad = t.dy + b * t.dy_b + s * t.dy_s + 8 * ch.at;
        uint16_t *dst = t.out + b * t.out_b + s * t.out_s + 8 * ch.at;
        float c[NA], sn[NA];
        if (ch.turned) {
            const int m = p.positions[b * p.pos_stride + s];
#pragma unroll
            for (int e = 0; e < NA; ++e) turn_angle(p.turns[ch.pair + e], m, p.sign, c[e], sn[e]);
        }
        for (int h = h0; h < h1; h += kGradBatch) {
            uint4 x[kGradBatch], y[kGradBatch];
#pragma unroll
            for (int k = 0; k < kGradBatch; ++k) {
                x[k] = y[k] = make_uint4(0, 0, 0, 0);
                if (ok && h + k < h1) {
                    x[k] = *reinterpret_cast<const uint4 *>(src + (h + k) * t.x_h);
                    y[k] = *reinterpret_cast<const uint4 *>(grad + (h + k) * t.dy_h);
                }
            }
#pragma unroll
            for (int k = 0; k < kGradBatch; ++k) {
                if (h + k >= h1) break;
                float a[8], g[8], o[8];
                unpack8(x[k], a);
                unpack8(y[k], g);
                if (HALF) unpack8(shfl4(y[k], ch.other), o);
                if (ch.turned) ch.turn(g, o, c, sn);
                float ss = 0.f, gx = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(a[e], a[e], ss);
                    gx = fmaf(g[e] * w[e], a[e], gx);
                }
                ss = sum_lanes<L>(ss);
                gx = sum_lanes<L>(gx);
                const float rs = rsqrtf(fmaf(ss, t.inv_d, p.eps));
                const float mean = gx * rs * t.inv_d;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = a[e] * rs;
                    dw[e] = fmaf(g[e], u, dw[e]);
                    a[e] = rs * fmaf(-u, mean, g[e] * w[e]);
                }
                if (ok) *reinterpret_cast<uint4 *>(dst + (h + k) * t.out_h) = pack8(a);
            }
        }
    }
    if (!t.dweight) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[threadIdx.x / L][8 * (threadIdx.x % L) + e] = dw[e];
    __syncthreads();
    float *to = t.partial + ((size_t)group * gridDim.x + blockIdx.x) * t.d_row;
    for (int e = threadIdx.x; e < t.d_row; e += kNormThreads) {
        float x = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) x += sums[r][e];
        to[e] = x;
    }
}

// Rows whose parts, strides or alignment do not fit 16-byte chunks, or that are wider than
// 256 entries: a warp has a row, and its lanes go over the pairs and the other entries, 2 bytes
// at a time.  Unit u of a row is its pair u, or past the pairs a copied entry.
struct Unit {
    int a, b;  // entries; b = -1: one that does not turn
    __device__ __forceinline__ Unit(const NormRopeParams &p, int u, bool half)
    {
        const int pairs = p.d_rot / 2;
        if (u < pairs) {
            a = p.rot_start + (half ? u : 2 * u);
            b = a + (half ? pairs : 1);
        } else {
            a = u - pairs;
            if (a >= p.rot_start) a += p.d_rot;
            b = -1;
        }
    }
};

__global__ void __launch_bounds__(kNormThreads) norm_pairs_kernel(const __grid_constant__ NormRopeParams p, bool half)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int group;
    const NormTensor &t = tensor_of(p, group);
    const int h0 = group * p.per, h1 = min(h0 + p.per, t.n_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kNormThreads / 32;
    const int tokens = p.B * p.S;
    for (long long token = (long long)blockIdx.x * warps + warp; token < tokens; token += (long long)gridDim.x * warps) {
        const int b = (int)(token / p.S), s = (int)(token % p.S);
        const long long row = out_row(p, t, b, s);
        if (row < 0) continue;
        const int m = p.d_rot ? p.positions[b * p.pos_stride + s] : 0;
        for (int h = h0; h < h1; ++h) {
            const uint16_t *src = t.x + b * t.x_b + s * t.x_s + h * t.x_h;
            uint16_t *dst = t.out + b * t.out_b + row * t.out_s + h * t.out_h;
            if (!t.norm) {
                for (int e = lane; e < t.d_row; e += 32) dst[e] = src[e];
                continue;
            }
            float ss = 0.f;
            for (int e = lane; e < t.d_row; e += 32) {
                const float x = bf16lo_to_f32(src[e]);
                ss = fmaf(x, x, ss);
            }
            const float rs = rsqrtf(fmaf(sum_lanes<32>(ss), t.inv_d, p.eps));
            for (int u = lane; u < t.d_row - p.d_rot / 2; u += 32) {
                const Unit at(p, u, half);
                float x = bf16lo_to_f32(src[at.a]) * rs * weight_at(t, h, at.a);
                if (at.b >= 0) {
                    float y = bf16lo_to_f32(src[at.b]) * rs * weight_at(t, h, at.b), c, sn;
                    turn_angle(p.turns[u], m, p.sign, c, sn);
                    rotate2(x, y, c, sn, x, y);
                    dst[at.b] = (uint16_t)pack_bf16x2(y, 0.f);
                }
                dst[at.a] = (uint16_t)pack_bf16x2(x, 0.f);
            }
        }
    }
}

__global__ void __launch_bounds__(kNormThreads) norm_grad_pairs_kernel(const __grid_constant__ NormRopeParams p, bool half)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ float acc[];  // [warps][d_row]
    int group;
    const NormTensor &t = tensor_of(p, group);
    const int h0 = group * p.per, h1 = min(h0 + p.per, t.n_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kNormThreads / 32;
    const int tokens = p.B * p.S;
    float *dw = acc + warp * t.d_row;  // an entry always belongs to the same lane
    const int units = t.d_row - p.d_rot / 2;
    for (int u = lane; u < units; u += 32) {
        const Unit at(p, u, half);
        dw[at.a] = 0.f;
        if (at.b >= 0) dw[at.b] = 0.f;
    }
    for (long long token = (long long)blockIdx.x * warps + warp; token < tokens; token += (long long)gridDim.x * warps) {
        const int b = (int)(token / p.S), s = (int)(token % p.S);
        const int m = p.d_rot ? p.positions[b * p.pos_stride + s] : 0;
        for (int h = h0; h < h1; ++h) {
            const uint16_t *src = t.x + b * t.x_b + s * t.x_s + h * t.x_h;
            const uint16_t *grad = t.dy + b * t.dy_b + s * t.dy_s + h * t.dy_h;
            uint16_t *dst = t.out + b * t.out_b + s * t.out_s + h * t.out_h;
            // the unit's entries of x and of the gradient turned back
            auto load = [&](int u, const Unit &at, float &x0, float &x1, float &g0, float &g1) {
                x0 = bf16lo_to_f32(src[at.a]);
                g0 = bf16lo_to_f32(grad[at.a]);
                x1 = g1 = 0.f;
                if (at.b >= 0) {
                    float c, sn;
                    x1 = bf16lo_to_f32(src[at.b]);
                    g1 = bf16lo_to_f32(grad[at.b]);
                    turn_angle(p.turns[u], m, p.sign, c, sn);
                    rotate2(g0, g1, c, sn, g0, g1);
                }
            };
            float ss = 0.f, gx = 0.f;
            for (int u = lane; u < units; u += 32) {
                const Unit at(p, u, half);
                float x0, x1, g0, g1;
                load(u, at, x0, x1, g0, g1);
                ss = fmaf(x0, x0, fmaf(x1, x1, ss));
                gx = fmaf(g0 * weight_at(t, h, at.a), x0, gx);
                if (at.b >= 0) gx = fmaf(g1 * weight_at(t, h, at.b), x1, gx);
            }
            const float rs = rsqrtf(fmaf(sum_lanes<32>(ss), t.inv_d, p.eps));
            const float mean = sum_lanes<32>(gx) * rs * t.inv_d;
            for (int u = lane; u < units; u += 32) {
                const Unit at(p, u, half);
                float x0, x1, g0, g1;
                load(u, at, x0, x1, g0, g1);
                const float u0 = x0 * rs, u1 = x1 * rs;
                dw[at.a] = fmaf(g0, u0, dw[at.a]);
                dst[at.a] = (uint16_t)pack_bf16x2(rs * fmaf(-u0, mean, g0 * weight_at(t, h, at.a)), 0.f);
                if (at.b >= 0) {
                    dw[at.b] = fmaf(g1, u1, dw[at.b]);
                    dst[at.b] = (uint16_t)pack_bf16x2(rs * fmaf(-u1, mean, g1 * weight_at(t, h, at.b)), 0.f);
                }
            }
        }
    }
    if (!t.dweight) return;
    __syncthreads();
    float *to = t.partial + ((size_t)group * gridDim.x + blockIdx.x) * t.d_row;
    for (int e = threadIdx.x; e < t.d_row; e += kNormThreads) {
        float x = 0.f;
        for (int r = 0; r < warps; ++r) x += acc[r * t.d_row + e];
        to[e] = x;
    }
}

// Weights' gradients: a block adds up 8 columns of the partial sums of a tensor (of a head of
// it, with weights for each head); blocks in the grid's z, heads in its y.
__global__ void __launch_bounds__(kNormThreads) norm_weights_kernel(const __grid_constant__ NormRopeParams p, int blocks)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ double sums[32][8];
    const NormTensor &t = p.t[blockIdx.z];
    const int e = 8 * blockIdx.x + threadIdx.x % 8, r0 = threadIdx.x / 8;
    const bool heads = t.weight_h != 0;
    if (!t.dweight || (int)blockIdx.y >= (heads ? t.n_heads : 1)) return;  // whole blocks
    const int rows = heads ? blocks : t.n_groups * blocks;
    const float *from = t.partial + (heads ? (size_t)blockIdx.y * blocks * t.d_row : 0) + e;
    double x = 0.;
    if (e < t.d_row) {
#pragma unroll 4
        for (int r = r0; r < rows; r += 32) x += from[(size_t)r * t.d_row];
    }
    sums[r0][threadIdx.x % 8] = x;
    __syncthreads();
    if (r0 == 0 && e < t.d_row) {
        for (int r = 1; r < 32; ++r) x += sums[r][threadIdx.x];
        t.dweight[(heads ? (size_t)blockIdx.y * t.d_row : 0) + e] = (float)x;
    }
}

template <typename K, typename... A>
cudaError_t launch_grid(K kernel, dim3 grid, int smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kNormThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, bool half, int lanes, int grid_x, int grid_y,
                             cudaStream_t stream)
{
    const dim3 grid(grid_x, grid_y);
    if (lanes == 8)
        return half ? launch_grid(norm_rows_kernel<8, true>, grid, 0, stream, p)
                    : launch_grid(norm_rows_kernel<8, false>, grid, 0, stream, p);
    if (lanes == 16)
        return half ? launch_grid(norm_rows_kernel<16, true>, grid, 0, stream, p)
                    : launch_grid(norm_rows_kernel<16, false>, grid, 0, stream, p);
    if (lanes == 32)
        return half ? launch_grid(norm_rows_kernel<32, true>, grid, 0, stream, p)
                    : launch_grid(norm_rows_kernel<32, false>, grid, 0, stream, p);
    return launch_grid(norm_pairs_kernel, grid, 0, stream, p, half);
}

cudaError_t launch_norm_rope_grad(const NormRopeParams &p, bool half, int lanes, int grid_x, int grid_y,
                                  cudaStream_t stream)
{
    const dim3 grid(grid_x, grid_y);
    int width = 0, heads = 1;
    bool weights = false;
    for (int i = 0; i < p.n_tensors; ++i) {
        width = std::max(width, p.t[i].d_row);
        weights = weights || p.t[i].dweight;
        if (p.t[i].weight_h != 0) heads = std::max(heads, p.t[i].n_heads);
    }
    cudaError_t err;
    if (lanes == 8)
        err = half ? launch_grid(norm_grad_rows_kernel<8, true>, grid, 0, stream, p)
                   : launch_grid(norm_grad_rows_kernel<8, false>, grid, 0, stream, p);
    else if (lanes == 16)
        err = half ? launch_grid(norm_grad_rows_kernel<16, true>, grid, 0, stream, p)
                   : launch_grid(norm_grad_rows_kernel<16, false>, grid, 0, stream, p);
    else if (lanes == 32)
        err = half ? launch_grid(norm_grad_rows_kernel<32, true>, grid, 0, stream, p)
                   : launch_grid(norm_grad_rows_kernel<32, false>, grid, 0, stream, p);
    else
        err = launch_grid(norm_grad_pairs_kernel, grid, kNormThreads / 32 * width * (int)sizeof(float), stream, p, half);
    if (err != cudaSuccess || !weights) return err;
    return launch_grid(norm_weights_kernel, dim3((width + 7) / 8, heads, p.n_tensors), 0, stream, p, grid_x);
}

}  // namespace apex
