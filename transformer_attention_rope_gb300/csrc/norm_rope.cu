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
// A row belongs to 4, 8, 16 or 32 neighbouring lanes.  A lane holds two 16-byte chunks, chosen so
// that it has both entries of its 8 pairs: pairs need no exchange, sums a few shuffles.  A block
// has a tile of neighbouring tokens and a slice of one tensor's heads; it makes the tile's sines
// once, in shared memory (c = 1, s = 0 where nothing turns, so that every pair goes the same way),
// and a lane takes them, times the weights, once for its heads of a token.  Pairs are worked on
// two at a time, as packed fp32.
//
// dw: a thread adds up its 16 columns over all rows that it meets, a block its threads' sums,
// and a second kernel the blocks' sums, to 64 bits: a fixed order, so equal inputs give equal
// bits.  With weights for each head a thread has one head.
//
// Measured: 8191 tokens of 128 + 8 heads of 128, half layout (570 MB): 91.5 us, 6.2 TB/s (97 with two
// rows of a lane in flight and 24 warps an SM in place of four and 20, 109 to 124 with rows by
// asynchronous copies as the gradient has them, 195 with a chunk a lane and the pairs' other halves
// exchanged); one token of 32 + 8 heads with its key and value appended: 3.0 us; the gradient of 16384
// tokens of 32 + 8 heads (503 MB): 96 us, 5.2 TB/s, with two rows in shared memory on their way (111 with
// one in registers, 125 with three copied beside three blocks an SM), where the issue of some 320
// instructions for a row of four warps a scheduler is behind it; of 1026 tokens with weights for each
// head: 17 us, 5 of them the second kernel.
#include "cache_attn.cuh"
#include "device_common.cuh"
#include "norm_rope.h"
#include "rope.cuh"

namespace apex {
namespace {

constexpr int kStages = 3;  // a lane's rows of a gradient in shared memory: one worked on, the others on their way
constexpr int kPart = 16 * kNormThreads;  // a chunk of each lane

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

__device__ __forceinline__ float sum2(uint64_t x)
{
    float lo, hi;
    f2_unpack(x, lo, hi);
    return lo + hi;
}

template <int L>
__device__ __forceinline__ float sum_lanes(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Number of a block's tensor, and its group of heads and its number within the group.
__device__ __forceinline__ int tensor_of(const NormRopeParams &p, int &group, int &block)
{
    int i = 0;
    block = blockIdx.x;
    while (block >= p.t[i].n_groups * p.t[i].blocks) {
        block -= p.t[i].n_groups * p.t[i].blocks;
        ++i;
    }
    group = block / p.t[i].blocks;
    block -= group * p.t[i].blocks;
    return i;
}

// The two chunks of 8 entries that lane u of a row holds (-1: none).  Half layout: those whose
// entries pair up; of the others, and of interleaved rows all, one of each half, so that
// neighbouring lanes' accesses are neighbours (side by side in a lane they went as half sectors: the
// gradient of 16384 tokens of 64 + 8 heads, 64 of 128 entries turned, interleaved, 158 us and 245).
template <bool HALF>
__device__ __forceinline__ void chunks_of(const NormRopeParams &p, int d_row, bool turns, int u, int &a, int &b)
{
    const int n = d_row >> 3, c0 = p.rot_start >> 3, nrot = HALF && turns ? p.d_rot >> 3 : 0, np = nrot >> 1;
    if (u < np) {
        a = c0 + u;
        b = a + np;
        return;
    }
    const int rest = n - nrot, lanes = (rest + 1) >> 1;
    a = u - np;
    b = a + lanes;
    if (a >= lanes) a = -1;
    if (b >= rest) b = -1;
    if (nrot > 0) {  // past the turned part
        if (a >= c0) a += nrot;
        if (b >= c0) b += nrot;
    }
}

// Two chunks as pairs of fp32: A the first entries of the lane's pairs, B the second ones.
template <bool HALF>
__device__ __forceinline__ void unpack(const uint4 &x, const uint4 &y, uint64_t (&A)[4], uint64_t (&B)[4])
{
    const uint32_t v[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (HALF) {
            A[e] = f2_pack(bf16lo_to_f32(v[e]), bf16hi_to_f32(v[e]));
            B[e] = f2_pack(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
        } else {
            const uint32_t lo = e < 2 ? v[2 * e] : w[2 * e - 4], hi = e < 2 ? v[2 * e + 1] : w[2 * e - 3];
            A[e] = f2_pack(bf16lo_to_f32(lo), bf16lo_to_f32(hi));
            B[e] = f2_pack(bf16hi_to_f32(lo), bf16hi_to_f32(hi));
        }
    }
}

template <bool HALF>
__device__ __forceinline__ void pack(const uint64_t (&A)[4], const uint64_t (&B)[4], uint4 &x, uint4 &y)
{
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a0, a1, b0, b1;
        f2_unpack(A[e], a0, a1);
        f2_unpack(B[e], b0, b1);
        if (HALF) {
            v[e] = pack_bf16x2(a0, a1);
            v[4 + e] = pack_bf16x2(b0, b1);
        } else {
            v[2 * e] = pack_bf16x2(a0, b0);
            v[2 * e + 1] = pack_bf16x2(a1, b1);
        }
    }
    x = make_uint4(v[0], v[1], v[2], v[3]);
    y = make_uint4(v[4], v[5], v[6], v[7]);
}

// Where a lane stands: its chunks of a row, and its slot's place among the rows of a tile.  `wide`
// slots beside one another share the heads of a token, per_token each; the others have further
// tokens.
template <int L, bool HALF>
struct Lane {
    int u, a, b;  // number in the row, entries where its chunks start (-1: none)
    int wide, deep, h0, t0, per_token;
    __device__ __forceinline__ Lane(const NormRopeParams &p, const NormTensor &t, int heads)
    {
        const int slot = threadIdx.x / L;
        u = threadIdx.x % L;
        chunks_of<HALF>(p, t.d_row, t.norm, u, a, b);
        a *= 8, b *= 8;
        wide = min((heads + t.batch - 1) / t.batch, kNormThreads / L);
        deep = kNormThreads / L / wide;
        h0 = slot % wide;
        t0 = slot / wide;
        if (t0 >= deep) t0 = kNormThreads / L;  // a slot that is left over: past every tile
        per_token = (heads + wide - 1) / wide;
    }
    // address of the lane's first chunk: of its second where there is none, which is not used then
    template <typename T>
    __device__ __forceinline__ T *at(T *row) const
    {
        return row + max(a, 0);
    }
    __device__ __forceinline__ int apart() const { return b - a; }
};

// Weight of the first or second entry of pair e of the chunks at entries a and b, for head h.
template <bool HALF>
__device__ __forceinline__ float pair_weight(const NormTensor &t, int h, int a, int b, int e, bool second)
{
    const int at = HALF ? (second ? b : a) + e : (e < 4 ? a : b) + 2 * (e & 3) + second;
    const bool there = HALF ? (second ? b : a) >= 0 : (e < 4 ? a : b) >= 0;
    return there ? weight_at(t, h, at) : 0.f;
}

// Sines of a tile's tokens and the weights that all heads share, as the lanes' pairs lie:
// [four pairs][lane][4].
template <int L>
struct Shared {
    float c[kNormThreads / L][2][L][4], s[kNormThreads / L][2][L][4], ns[kNormThreads / L][2][L][4];  // a tile has a token for each slot at most
    float wa[kNormHeads / L][2][L][4], wb[kNormHeads / L][2][L][4];  // of the group's heads, or of all

    static __device__ __forceinline__ void get(const float (&from)[2][L][4], int u, uint64_t (&x)[4])
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(from[h][u]);
            x[2 * h] = v.x;
            x[2 * h + 1] = v.y;
        }
    }
    // weights of the group's heads, or those that all share, by the block
    template <bool HALF>
    __device__ __forceinline__ void weights(const NormRopeParams &p, const NormTensor &t, int first, int heads)
    {
        const int n = t.weight_h == 0 ? 1 : heads;
        for (int i = threadIdx.x; i < n * 8 * L; i += kNormThreads) {
            const int h = i / (8 * L), u = i / 8 % L, e = i % 8;
            int a, b;
            chunks_of<HALF>(p, t.d_row, true, u, a, b);
            wa[h][e >> 2][u][e & 3] = pair_weight<HALF>(t, first + h, 8 * a, 8 * b, e, false);
            wb[h][e >> 2][u][e & 3] = pair_weight<HALF>(t, first + h, 8 * a, 8 * b, e, true);
        }
    }
    // sines of tokens s0 .. s0 + n - 1 of sequence b, by the block
    template <bool HALF>
    __device__ __forceinline__ void turn(const NormRopeParams &p, const NormTensor &t, int b, int s0, int n)
    {
#pragma unroll 2
        for (int i = threadIdx.x; i < n * 8 * L; i += kNormThreads) {
            const int k = i / (8 * L), u = i / 8 % L, e = i % 8;
            int ca, cb;
            chunks_of<HALF>(p, t.d_row, true, u, ca, cb);
            // entry that the pair starts with
            const int x = HALF ? 8 * ca + e : 8 * (e < 4 ? ca : cb) + 2 * (e & 3), in = x - p.rot_start;
            float cos = 1.f, sin = 0.f;
            if (ca >= 0 && (HALF ? u < p.d_rot >> 4 : (e < 4 || cb >= 0) && in >= 0 && in < p.d_rot))
                turn_angle(p.turns[HALF ? in : in >> 1], p.positions[b * p.pos_stride + s0 + k], p.sign, cos, sin);
            c[k][e >> 2][u][e & 3] = cos;
            s[k][e >> 2][u][e & 3] = sin;
            ns[k][e >> 2][u][e & 3] = -sin;
        }
    }
};

template <int L, bool HALF>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) norm_rows_kernel(const __grid_constant__ NormRopeParams p)
{
    // launched as a programmatic dependent: inputs may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ Shared<L> sh;
    int group, block;
    const NormTensor t = p.t[tensor_of(p, group, block)];
    const int first = group * t.per, heads = min(t.per, t.n_heads - first);
    const Lane<L, HALF> my(p, t, heads);
    const bool shared = t.weight_h == 0;
    if (t.norm) sh.template weights<HALF>(p, t, first, heads);
    const long long x_step = my.wide * t.x_h, out_step = my.wide * t.out_h;
    for (int tile = block; tile < p.B * t.tiles; tile += t.blocks) {  // below 2^31
        const int b = tile / t.tiles, s0 = tile % t.tiles * t.tile, n = min(t.tile, p.S - s0);
        const bool moved = t.append && p.row0;
        const long long row0 = (moved ? p.row0[b] : 0) + (long long)s0, rows = moved ? p.out_rows : p.S;
        const uint16_t *src = my.at(t.x + b * t.x_b + (s0 + my.t0) * t.x_s + (first + my.h0) * t.x_h);
        uint16_t *dst = my.at(t.out + b * t.out_b + (row0 + my.t0) * t.out_s + (first + my.h0) * t.out_h);
        bool made = !t.norm;
        for (int tok = my.t0, i = 0; i < n; i += my.deep, tok += my.deep, src += my.deep * t.x_s, dst += my.deep * t.out_s) {
            const bool in = my.a >= 0 && tok < n, two = my.b >= 0, out = in && row0 + tok >= 0 && row0 + tok < rows;
            const uint16_t *from = src;
            uint16_t *to = dst;
            // u = a ca + b nsb, w = a sa + b cb: sines, times the weights that all heads share
            uint64_t ca[4], sa[4], cb[4], nsb[4];
            for (int h = my.h0, j = 0; j < my.per_token; j += kNormBatch) {
                uint4 x[kNormBatch], y[kNormBatch];
#pragma unroll
                for (int k = 0; k < kNormBatch; ++k, from += x_step) {
                    x[k] = y[k] = make_uint4(0, 0, 0, 0);
                    if (in && h + k * my.wide < heads) {
                        x[k] = *reinterpret_cast<const uint4 *>(from);
                        if (two) y[k] = *reinterpret_cast<const uint4 *>(from + my.apart());
                    }
                }
                if (!made) {          // while the first rows are on the way
                    __syncthreads();  // the last tile's sines are done with
                    sh.template turn<HALF>(p, t, b, s0, n);
                    __syncthreads();
                    made = true;
                }
                if (t.norm && j == 0) {
                    Shared<L>::get(sh.c[min(tok, n - 1)], my.u, ca);
                    Shared<L>::get(sh.s[min(tok, n - 1)], my.u, sa);
                    Shared<L>::get(sh.c[min(tok, n - 1)], my.u, cb);
                    Shared<L>::get(sh.ns[min(tok, n - 1)], my.u, nsb);
                    if (shared) {
                        uint64_t wa[4], wb[4];
                        Shared<L>::get(sh.wa[0], my.u, wa);
                        Shared<L>::get(sh.wb[0], my.u, wb);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            ca[e] = f2_mul(wa[e], ca[e]);
                            sa[e] = f2_mul(wa[e], sa[e]);
                            cb[e] = f2_mul(wb[e], cb[e]);
                            nsb[e] = f2_mul(wb[e], nsb[e]);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < kNormBatch; ++k, h += my.wide, to += out_step) {
                    if (j + k >= my.per_token) break;
                    if (t.norm) {
                        uint64_t A[4], B[4];
                        unpack<HALF>(x[k], y[k], A, B);
                        uint64_t s2 = 0, s3 = 0;  // +0
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s2 = f2_fma(A[e], A[e], s2);
                            s3 = f2_fma(B[e], B[e], s3);
                        }
                        const float rs = rsqrtf(fmaf(sum_lanes<L>(sum2(f2_add(s2, s3))), t.inv_d, p.eps));
                        const uint64_t rs2 = f2_pack(rs, rs);
                        if (!shared) {  // weights of the head's own
                            uint64_t wa[4], wb[4];
                            Shared<L>::get(sh.wa[min(h, heads - 1)], my.u, wa);
                            Shared<L>::get(sh.wb[min(h, heads - 1)], my.u, wb);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                A[e] = f2_mul(A[e], wa[e]);
                                B[e] = f2_mul(B[e], wb[e]);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint64_t u = f2_fma(B[e], nsb[e], f2_mul(A[e], ca[e]));
                            B[e] = f2_mul(f2_fma(A[e], sa[e], f2_mul(B[e], cb[e])), rs2);
                            A[e] = f2_mul(u, rs2);
                        }
                        pack<HALF>(A, B, x[k], y[k]);
                    }
                    if (out && h < heads) {
                        *reinterpret_cast<uint4 *>(to) = x[k];
                        if (two) *reinterpret_cast<uint4 *>(to + my.apart()) = y[k];
                    }
                }
            }
        }
    }
}

// A block of a gradient has an equal part of all tokens of its tensor's sequences, in tiles of neighbours.
struct Span {
    int at, end;  // next token, over all sequences
    __device__ __forceinline__ Span(const NormRopeParams &p, const NormTensor &t, int block)
        : at((int)((long long)p.B * p.S * block / t.blocks)), end((int)((long long)p.B * p.S * (block + 1) / t.blocks))
    {
    }
    // the next tile: its sequence, first token, and number of tokens (0: none left)
    __device__ __forceinline__ int next(const NormRopeParams &p, const NormTensor &t, int &b, int &s0)
    {
        b = at / p.S;
        s0 = at - b * p.S;
        const int n = min(t.tile, min(p.S - s0, end - at));
        at += n;
        return n;
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint4 shared16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// A lane's rows, one after another over the heads of a token, the tokens of a tile and the tiles of
// a block, and their gradients, copied to its own ring: those that follow are under way while one is
// worked on.
template <int L, bool HALF>
struct Feed {
    static constexpr int kStage = 4 * kPart, kBytes = kStages * kStage;
    const uint16_t *x, *dy;
    long long x_step, dy_step, x_wrap, dy_wrap;  // to the next head, and from the last to the next token's first
    Span span;
    int n, tok, j, h;  // the row to copy next
    uint32_t first, slot, next;
    __device__ __forceinline__ Feed(const NormRopeParams &p, const NormTensor &t, const Lane<L, HALF> &my, int block,
                                    uint32_t ring)
        : x_step(my.wide * t.x_h), dy_step(my.wide * t.dy_h), x_wrap(my.deep * t.x_s - my.per_token * x_step),
          dy_wrap(my.deep * t.dy_s - my.per_token * dy_step), span(p, t, block), first(ring + 16 * threadIdx.x),
          slot(first), next(first)
    {
    }
    static __device__ __forceinline__ void turn(uint32_t &at, uint32_t first)
    {
        at += kStage;
        if (at == first + kBytes) at = first;
    }
    __device__ __forceinline__ void tile(const NormRopeParams &p, const NormTensor &t, const Lane<L, HALF> &my, int head0)
    {
        int b, s0;
        n = span.next(p, t, b, s0);
        j = 0;
        h = my.h0;
        tok = my.t0;
        if (n == 0) return;
        x = my.at(t.x + b * t.x_b + (s0 + tok) * t.x_s + (head0 + h) * t.x_h);
        dy = my.at(t.dy + b * t.dy_b + (s0 + tok) * t.dy_s + (head0 + h) * t.dy_h);
    }
    // zeros where there is no row
    __device__ __forceinline__ void load(const NormRopeParams &p, const NormTensor &t, const Lane<L, HALF> &my, int head0,
                                         int heads)
    {
        const bool in = my.a >= 0 && tok < n && h < heads, two = in && my.b >= 0;
        copy16(next, in ? x : t.x, in);
        copy16(next + kPart, two ? x + my.apart() : t.x, two);
        copy16(next + 2 * kPart, in ? dy : t.x, in);
        copy16(next + 3 * kPart, two ? dy + my.apart() : t.x, two);
        asm volatile("cp.async.commit_group;" ::: "memory");
        turn(next, first);
        x += x_step;
        dy += dy_step;
        h += my.wide;
        if (++j < my.per_token) return;
        j = 0;
        h = my.h0;
        tok += my.deep;
        x += x_wrap;
        dy += dy_wrap;
        if (tok - my.t0 >= n && n > 0) tile(p, t, my, head0);  // the same for all slots
    }
    __device__ __forceinline__ void start(const NormRopeParams &p, const NormTensor &t, const Lane<L, HALF> &my, int head0,
                                          int heads)
    {
        tile(p, t, my, head0);
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) load(p, t, my, head0, heads);
    }
    // the next row, in the order of the copies; the one before it is overwritten
    __device__ __forceinline__ void take(const NormRopeParams &p, const NormTensor &t, const Lane<L, HALF> &my, int head0,
                                         int heads, uint4 (&v)[4])
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = shared16(slot + i * kPart);
        turn(slot, first);
        load(p, t, my, head0, heads);
    }
};

template <int L, bool HALF>
__global__ void __launch_bounds__(kNormThreads, kNormGradCtas) norm_grad_rows_kernel(const __grid_constant__ NormRopeParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ union {
        Shared<L> t;
        float sums[kNormThreads / L][16 * L];  // of each slot
    } sh;
    int group, block;
    const NormTensor t = p.t[tensor_of(p, group, block)];
    const int first = group * t.per, heads = min(t.per, t.n_heads - first);
    const Lane<L, HALF> my(p, t, heads);
    uint64_t da[4] = {0, 0, 0, 0}, db[4] = {0, 0, 0, 0};
    const long long out_step = my.wide * t.out_h;
    extern __shared__ __align__(16) uint8_t ring[];
    Feed<L, HALF> feed(p, t, my, block, smem_u32(ring));
    feed.start(p, t, my, first, heads);
    // with weights for each head a slot has one head
    sh.t.template weights<HALF>(p, t, first, heads);
    const int w = t.weight_h == 0 ? 0 : my.h0;
    Span span(p, t, block);
    int b, s0;
    while (const int n = span.next(p, t, b, s0)) {
        uint16_t *dst = my.at(t.out + b * t.out_b + (s0 + my.t0) * t.out_s + (first + my.h0) * t.out_h);
        __syncthreads();  // the last tile's sines are done with
        sh.t.template turn<HALF>(p, t, b, s0, n);
        __syncthreads();
        for (int tok = my.t0, i = 0; i < n; i += my.deep, tok += my.deep, dst += my.deep * t.out_s) {
            uint16_t *to = dst;
            for (int h = my.h0, j = 0; j < my.per_token; ++j, h += my.wide, to += out_step) {
                const bool real = tok < n && h < heads;
                uint64_t A[4], B[4], G[4], H[4];
                uint4 v[4];
                feed.take(p, t, my, first, heads, v);
                unpack<HALF>(v[0], v[1], A, B);
                unpack<HALF>(v[2], v[3], G, H);
                uint64_t c[4], s[4], ns[4], s2 = 0, s3 = 0, d2 = 0, d3 = 0;  // +0
                Shared<L>::get(sh.t.c[min(tok, n - 1)], my.u, c);
                Shared<L>::get(sh.t.s[min(tok, n - 1)], my.u, s);
                Shared<L>::get(sh.t.ns[min(tok, n - 1)], my.u, ns);
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // the gradient turned back
                    const uint64_t g = f2_fma(H[e], ns[e], f2_mul(G[e], c[e]));
                    H[e] = f2_fma(G[e], s[e], f2_mul(H[e], c[e]));
                    G[e] = g;
                    s2 = f2_fma(A[e], A[e], s2);
                    s3 = f2_fma(B[e], B[e], s3);
                }
                Shared<L>::get(sh.t.wa[w], my.u, c);
                Shared<L>::get(sh.t.wb[w], my.u, s);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d2 = f2_fma(f2_mul(G[e], c[e]), A[e], d2);
                    d3 = f2_fma(f2_mul(H[e], s[e]), B[e], d3);
                }
                const float all = sum_lanes<L>(sum2(f2_add(s2, s3))), dot = sum_lanes<L>(sum2(f2_add(d2, d3)));
                const float rs = real ? rsqrtf(fmaf(all, t.inv_d, p.eps)) : 0.f;  // no row adds to the weights' sums
                const float back = -(dot * rs * t.inv_d) * rs * rs;  // dx = rs g w - x rs^2 mean(g w u)
                const uint64_t rs2 = f2_pack(rs, rs), back2 = f2_pack(back, back);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    G[e] = f2_mul(G[e], rs2);
                    H[e] = f2_mul(H[e], rs2);
                    da[e] = f2_fma(G[e], A[e], da[e]);
                    db[e] = f2_fma(H[e], B[e], db[e]);
                    A[e] = f2_fma(A[e], back2, f2_mul(G[e], c[e]));
                    B[e] = f2_fma(B[e], back2, f2_mul(H[e], s[e]));
                }
                uint4 o0, o1;
                pack<HALF>(A, B, o0, o1);
                if (real && my.a >= 0) {
                    *reinterpret_cast<uint4 *>(to) = o0;
                    if (my.b >= 0) *reinterpret_cast<uint4 *>(to + my.apart()) = o1;
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!t.dweight) return;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float4 *to = reinterpret_cast<float4 *>(&sh.sums[threadIdx.x / L][16 * my.u + 4 * e]);
        float4 v;
        f2_unpack(da[e], v.x, v.y);
        f2_unpack(db[e], v.z, v.w);
        *to = v;
    }
    __syncthreads();
    // the slots of a head, or all of them, in order
    const bool each = t.weight_h != 0;
    for (int i = threadIdx.x; i < (each ? heads : 1) * 16 * L; i += kNormThreads) {
        // pairs 2q, 2q + 1: first entries, then second ones
        const int h = i / (16 * L), at = i % (16 * L), u = at / 16, q = at % 16 / 4, second = at % 4 / 2, e = 2 * q + at % 2;
        int a, b;
        chunks_of<HALF>(p, t.d_row, true, u, a, b);
        const int chunk = HALF ? (second ? b : a) : e < 4 ? a : b;
        if (chunk < 0) continue;
        float x = 0.f;
        if (each)
            for (int r = 0; r < my.deep; ++r) x += sh.sums[r * my.wide + h][at];
        else
#pragma unroll
            for (int r = 0; r < kNormThreads / L; ++r) x += sh.sums[r][at];
        float *to = t.partial + ((size_t)(each ? first + h : group) * t.blocks + block) * t.d_row;
        to[8 * chunk + (HALF ? e : 2 * (e & 3) + second)] = x;
    }
}

// Rows whose parts, strides or alignment do not fit 16-byte chunks, or that are wider than
// 512 entries: a warp has a row, and its lanes go over the pairs and the other entries, 2 bytes
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

// Cosines and sines of a token's pairs, once for the heads that a warp goes over (16384 tokens of 81 + 8
// heads of 100: 497 us and 782, the gradient, with more blocks, 1030 and 2082).
__device__ __forceinline__ void sines_of(const NormRopeParams &p, int m, float2 *turn)
{
    for (int u = threadIdx.x & 31; u < p.d_rot / 2; u += 32) turn_angle(p.turns[u], m, p.sign, turn[u].x, turn[u].y);
}

__global__ void __launch_bounds__(kNormThreads) norm_pairs_kernel(const __grid_constant__ NormRopeParams p, bool half)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int group, block;
    const NormTensor &t = p.t[tensor_of(p, group, block)];
    const int h0 = group * t.per, h1 = min(h0 + t.per, t.n_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kNormThreads / 32;
    const int tokens = p.B * p.S;
    extern __shared__ float2 sines[];  // [warps][pairs] of the warp's token; a lane's own alone
    float2 *turn = sines + warp * (p.d_rot / 2);
    for (long long token = (long long)block * warps + warp; token < tokens; token += (long long)t.blocks * warps) {
        const int b = (int)(token / p.S), s = (int)(token % p.S);
        const long long row = out_row(p, t, b, s);
        if (row < 0) continue;
        if (t.norm) sines_of(p, p.positions[b * p.pos_stride + s], turn);
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
                    float y = bf16lo_to_f32(src[at.b]) * rs * weight_at(t, h, at.b);
                    rotate2(x, y, turn[u].x, turn[u].y, x, y);
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
    extern __shared__ float2 sines[];  // [warps][pairs] of the warp's token, a lane's own alone; then sums
    float *acc = reinterpret_cast<float *>(sines + kNormThreads / 32 * (p.d_rot / 2));  // [warps][d_row]
    int group, block;
    const NormTensor &t = p.t[tensor_of(p, group, block)];
    const int h0 = group * t.per, h1 = min(h0 + t.per, t.n_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kNormThreads / 32;
    const int tokens = p.B * p.S;
    float *dw = acc + warp * t.d_row;  // an entry always belongs to the same lane
    float2 *turn = sines + warp * (p.d_rot / 2);
    const int units = t.d_row - p.d_rot / 2;
    for (int u = lane; u < units; u += 32) {
        const Unit at(p, u, half);
        dw[at.a] = 0.f;
        if (at.b >= 0) dw[at.b] = 0.f;
    }
    for (long long token = (long long)block * warps + warp; token < tokens; token += (long long)t.blocks * warps) {
        const int b = (int)(token / p.S), s = (int)(token % p.S);
        sines_of(p, p.positions[b * p.pos_stride + s], turn);
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
                    x1 = bf16lo_to_f32(src[at.b]);
                    g1 = bf16lo_to_f32(grad[at.b]);
                    rotate2(g0, g1, turn[u].x, turn[u].y, g0, g1);
                }
            };
            float ss = 0.f, gx = 0.f;
#pragma unroll 4
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
#pragma unroll 4
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
    float *to = t.partial + ((size_t)group * t.blocks + block) * t.d_row;
    for (int e = threadIdx.x; e < t.d_row; e += kNormThreads) {
        float x = 0.f;
        for (int r = 0; r < warps; ++r) x += acc[r * t.d_row + e];
        to[e] = x;
    }
}

// Weights' gradients: a block adds up 8 columns of the partial sums of a tensor (of a head of
// it, with weights for each head); blocks in the grid's z, heads in its y.  A thread's sum is held as
// two fp32, what rounding took from the first in the second: 64-bit additions are slow here, and come
// last.
__global__ void __launch_bounds__(kNormSumThreads) norm_weights_kernel(const __grid_constant__ NormRopeParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ double sums[kNormSumThreads / 32][8];
    const NormTensor &t = p.t[blockIdx.z];
    const int lane = threadIdx.x & 31, e = 8 * blockIdx.x + lane % 8, r0 = threadIdx.x / 8;
    const bool heads = t.weight_h != 0;
    if (!t.dweight || (int)blockIdx.y >= (heads ? t.n_heads : 1)) return;  // whole blocks
    const int rows = heads ? t.blocks : t.n_groups * t.blocks;
    const float *from = t.partial + (heads ? (size_t)blockIdx.y * t.blocks * t.d_row : 0) + e;
    float hi = 0.f, lo = 0.f;
    if (e < t.d_row) {
#pragma unroll 8
        for (int r = r0; r < rows; r += kNormSumThreads / 8) {
            const float x = from[(size_t)r * t.d_row], sum = hi + x, back = sum - hi;
            lo += (hi - (sum - back)) + (x - back);
            hi = sum;
        }
    }
    double x = (double)hi + lo;
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    x += __shfl_xor_sync(0xffffffffu, x, 16);
    if (lane < 8) sums[threadIdx.x / 32][lane] = x;
    __syncthreads();
    if (threadIdx.x < 8 && e < t.d_row) {
        for (int r = 1; r < kNormSumThreads / 32; ++r) x += sums[r][lane];
        t.dweight[(heads ? (size_t)blockIdx.y * t.d_row : 0) + e] = (float)x;
    }
}

template <typename K, typename... A>
cudaError_t launch_grid(K kernel, dim3 grid, int threads, int smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

unsigned grid_of(const NormRopeParams &p)
{
    unsigned n = 0;
    for (int i = 0; i < p.n_tensors; ++i) n += (unsigned)p.t[i].n_groups * p.t[i].blocks;
    return n;
}

}  // namespace

namespace {

template <int L>
cudaError_t launch_rows(const NormRopeParams &p, bool half, bool grad, cudaStream_t stream)
{
    const dim3 grid(grid_of(p));
    if (!grad)
        return half ? launch_grid(norm_rows_kernel<L, true>, grid, kNormThreads, 0, stream, p)
                    : launch_grid(norm_rows_kernel<L, false>, grid, kNormThreads, 0, stream, p);
    constexpr int ring = Feed<L, false>::kBytes;
    static KernelSetup setup[2];
    const auto kernel = half ? norm_grad_rows_kernel<L, true> : norm_grad_rows_kernel<L, false>;
    const cudaError_t err = setup[half](kernel, ring);
    return err != cudaSuccess ? err : launch_grid(kernel, grid, kNormThreads, ring, stream, p);
}

cudaError_t launch_lanes(const NormRopeParams &p, bool half, bool grad, int lanes, cudaStream_t stream)
{
    return lanes == 4    ? launch_rows<4>(p, half, grad, stream)
           : lanes == 8  ? launch_rows<8>(p, half, grad, stream)
           : lanes == 16 ? launch_rows<16>(p, half, grad, stream)
                         : launch_rows<32>(p, half, grad, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, bool half, int lanes, cudaStream_t stream)
{
    return lanes ? launch_lanes(p, half, false, lanes, stream)
                 : launch_grid(norm_pairs_kernel, dim3(grid_of(p)), kNormThreads,
                               kNormThreads / 32 * (p.d_rot / 2) * (int)sizeof(float2), stream, p, half);
}

cudaError_t launch_norm_rope_grad(const NormRopeParams &p, bool half, int lanes, cudaStream_t stream)
{
    int width = 0, heads = 1;
    bool weights = false;
    for (int i = 0; i < p.n_tensors; ++i) {
        width = std::max(width, p.t[i].d_row);
        weights = weights || p.t[i].dweight;
        if (p.t[i].weight_h != 0) heads = std::max(heads, p.t[i].n_heads);
    }
    const cudaError_t err =
        lanes ? launch_lanes(p, half, true, lanes, stream)
              : launch_grid(norm_grad_pairs_kernel, dim3(grid_of(p)), kNormThreads,
                            kNormThreads / 32 * (p.d_rot + width) * (int)sizeof(float), stream, p, half);
    if (err != cudaSuccess || !weights) return err;
    return launch_grid(norm_weights_kernel, dim3((width + 7) / 8, heads, p.n_tensors), kNormSumThreads, 0, stream, p);
}

}  // namespace apex
