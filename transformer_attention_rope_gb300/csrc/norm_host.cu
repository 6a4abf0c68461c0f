// norm_host.cu -- entry points of include/apex_attn.h that norm and turn heads in one pass,
// and their gradient: argument checks and launches.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "norm_rope.h"
#include "rope_host.h"

namespace apex {
namespace {

// Entries of bf16 or fp32 as 2-byte elements.
RowSet flat_rows(const void *at, size_t bytes)
{
    return RowSet{(__int128)(reinterpret_cast<uintptr_t>(at) / 2), {0, 0, 0}, {1, 1, 1}, (int)(bytes / 2)};
}

RowSet rows_of(const void *at, long long b, long long h, long long s, int B, int H, int S, int d)
{
    return RowSet{(__int128)(reinterpret_cast<uintptr_t>(at) / 2), {b, h, s}, {B, H, S}, d};
}

bool same_rows(const RowSet &a, const RowSet &b)
{
    bool same = a.at == b.at;
    for (int i = 0; i < 3; ++i) same = same && (a.stride[i] == b.stride[i] || a.count[i] == 1);
    return same;
}

bool tensor_ok(const apex_norm_tensor *t, bool grad)
{
    if (!t->x || !t->out || t->n_heads <= 0 || t->d_row <= 0) return false;
    if (!aligned(t->x, 2) || !aligned(t->out, 2)) return false;
    if (t->weight_f32 < 0 || t->weight_f32 > 1) return false;
    if (t->weight && !aligned(t->weight, t->weight_f32 ? 4 : 2)) return false;
    if (!grad) return true;
    return t->dy && aligned(t->dy, 2) && (!t->dweight || aligned(t->dweight, 4));
}

size_t weight_count(const apex_norm_tensor &t) { return (size_t)t.d_row * (t.weight_per_head ? t.n_heads : 1); }

// An output shares no element with an input or another output, but for rows worked on in
// place: a row's lanes have read it before one of them writes (not with row0, which may shift
// rows).
bool outputs_apart(const apex_norm_tensor *const (&t)[3], bool grad, int B, int S, bool row0, int out_rows)
{
    struct Set {
        RowSet r;
        int of;  // tensor
        bool own;  // rows that its output may be
    };
    Set in[9], out[6];
    int ni = 0, no = 0;
    for (int i = 0; i < 3; ++i) {
        if (!t[i]) continue;
        const apex_norm_tensor &a = *t[i];
        const bool moved = row0 && i > 0;
        in[ni++] = Set{rows_of(a.x, a.x_b, a.x_h, a.x_s, B, a.n_heads, S, a.d_row), i, !moved};
        if (grad) in[ni++] = Set{rows_of(a.dy, a.dy_b, a.dy_h, a.dy_s, B, a.n_heads, S, a.d_row), i, true};
        if (a.weight) in[ni++] = Set{flat_rows(a.weight, weight_count(a) * (a.weight_f32 ? 4 : 2)), i, false};
        out[no++] = Set{rows_of(a.out, a.out_b, a.out_h, a.out_s, B, a.n_heads, moved ? out_rows : S, a.d_row), i, true};
        if (grad && a.dweight) out[no++] = Set{flat_rows(a.dweight, weight_count(a) * 4), i, false};
    }
    for (int i = 0; i < no; ++i) {
        if (out[i].own && share_elements(out[i].r, out[i].r)) return false;
        for (int k = 0; k < i; ++k)
            if (share_elements(out[i].r, out[k].r)) return false;
        for (int k = 0; k < ni; ++k) {
            const bool in_place = out[i].own && in[k].own && out[i].of == in[k].of && same_rows(out[i].r, in[k].r);
            if (!in_place && share_elements(out[i].r, in[k].r)) return false;
        }
    }
    return true;
}

// Whether 16-byte chunks fit the rows; a lane then holds two.
bool rows_of_16_bytes(const apex_norm_tensor &t, bool grad)
{
    long long strides = t.x_b | t.x_h | t.x_s | t.out_b | t.out_h | t.out_s;
    if (grad) strides |= t.dy_b | t.dy_h | t.dy_s;
    return aligned16(t.x) && aligned16(t.out) && (!grad || aligned16(t.dy)) && t.d_row % 8 == 0 && strides % 8 == 0 &&
           t.d_row <= kNormFastRow;
}

struct Plan {
    NormRopeParams p;
    bool half;
    int lanes;   // of a row; 0: 2 bytes at a time
    int heads;   // of all tensors
    int sm_count;
    int slots;   // rows that a block works on at once
};

// Checks and parameters shared by the pass and its gradient; t: q, k, v.
apex_status make_plan(const apex_norm_tensor *const (&t)[3], bool grad, int B, int S, const int *positions,
                      long long pos_stride, const int *row0, int out_rows, const apex_rope_options *opt, float eps,
                      Plan *plan)
{
    if (!opt || !positions || !t[0]) return APEX_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(row0, 4)) return APEX_ERR_INVALID_ARG;
    if (B <= 0 || S <= 0 || pos_stride < 0 || (row0 && out_rows <= 0)) return APEX_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !isfinite(eps)) return APEX_ERR_INVALID_ARG;
    if (opt->layout != APEX_ROPE_INTERLEAVED && opt->layout != APEX_ROPE_HALF) return APEX_ERR_INVALID_ARG;
    if (opt->rot_start < 0 || opt->d_rot < 0 || opt->d_rot % 2 != 0) return APEX_ERR_INVALID_ARG;
    apex_attn_options fo;
    memset(&fo, 0, sizeof fo);
    fo.rope_base = opt->rope_base;
    fo.yarn_scale = opt->yarn_scale;
    fo.yarn_beta_fast = opt->yarn_beta_fast;
    fo.yarn_beta_slow = opt->yarn_beta_slow;
    RopeFreq f;
    if (!freq_of(fo, &f)) return APEX_ERR_INVALID_ARG;
    const float linear = opt->linear_scale == 0.f ? 1.f : opt->linear_scale;
    if (!(linear > 0.f) || !isfinite(linear)) return APEX_ERR_INVALID_ARG;
    int d_rot = opt->d_rot;
    for (int i = 0; i < 3; ++i) {
        if (!t[i]) continue;
        if (!tensor_ok(t[i], grad)) return APEX_ERR_INVALID_ARG;
        if (i == 2) continue;
        const int room = t[i]->d_row - opt->rot_start;
        if (d_rot == 0) d_rot = room;  // the whole row from rot_start on
        if (d_rot <= 0 || d_rot > room || d_rot % 2 != 0) return APEX_ERR_INVALID_ARG;
        if (opt->d_rot == 0 && d_rot != room) return APEX_ERR_INVALID_ARG;  // q and k disagree
    }
    if (B > kMaxSeq || S > kMaxSeq || (long long)B * S >= (1ll << 31)) return APEX_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (t[i] && (t[i]->d_row > 1024 || t[i]->n_heads > 16384)) return APEX_ERR_UNSUPPORTED;
    if (d_rot > 2 * kRopeMaxPairs) return APEX_ERR_UNSUPPORTED;
    if (!outputs_apart(t, grad, B, S, row0 != nullptr, out_rows)) return APEX_ERR_INVALID_ARG;

    NormRopeParams &p = plan->p;
    memset(&p, 0, sizeof p);
    plan->half = opt->layout == APEX_ROPE_HALF;
    bool wide = opt->rot_start % 8 == 0 && (plan->half ? d_rot / 2 : d_rot) % 8 == 0;
    int width = 0;
    plan->heads = 0;
    for (int i = 0; i < 3; ++i) {
        if (!t[i]) continue;
        const apex_norm_tensor &a = *t[i];
        NormTensor &n = p.t[p.n_tensors++];
        n.x = static_cast<const uint16_t *>(a.x);
        n.dy = static_cast<const uint16_t *>(a.dy);
        n.out = static_cast<uint16_t *>(a.out);
        n.x_b = a.x_b, n.x_h = a.x_h, n.x_s = a.x_s;
        n.dy_b = a.dy_b, n.dy_h = a.dy_h, n.dy_s = a.dy_s;
        n.out_b = a.out_b, n.out_h = a.out_h, n.out_s = a.out_s;
        n.weight = a.weight;
        n.weight_f32 = a.weight_f32;
        n.weight_h = a.weight_per_head ? a.d_row : 0;
        n.n_heads = a.n_heads;
        n.d_row = a.d_row;
        n.norm = i != 2;
        n.append = i != 0;
        n.inv_d = (float)(1.0 / a.d_row);
        n.dweight = grad ? a.dweight : nullptr;
        wide = wide && rows_of_16_bytes(a, grad);
        plan->heads += a.n_heads;
        width = std::max(width, a.d_row);
    }
    plan->lanes = !wide ? 0 : width <= 64 ? 4 : width <= 128 ? 8 : width <= 256 ? 16 : 32;
    plan->slots = kNormThreads / (wide ? plan->lanes : 32);
    p.positions = positions;
    p.pos_stride = pos_stride;
    p.row0 = row0;
    p.out_rows = out_rows;
    p.B = B;
    p.S = S;
    p.rot_start = opt->rot_start;
    p.d_rot = d_rot;
    p.eps = eps;
    p.sign = grad ? -1.f : 1.f;
    if (!turns_of(f, linear, d_rot, p.turns)) return APEX_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&plan->sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return APEX_ERR_CUDA;
    return APEX_OK;
}

// Cuts the work for rows that go 16 bytes at a time, into `blocks` (group, tile)s if there is so
// much.  A block makes the sines of its tile for all heads of its group, and so has `rows` rows for each
// of its slots, of as many heads and then tokens as there are; a slot takes up to kNormBatch heads of a token,
// whose loads are in flight together (a gradient's slot two, one by one from its ring).  Where that leaves SMs
// without blocks, a block has fewer rows, and at last one for each slot.  Weights of each head's own are
// held for `most` heads of a block; a gradient's slot has one head then, whose sums it makes.
void cut_rows(Plan &plan, int rows, bool grad, int most, long long blocks)
{
    NormRopeParams &p = plan.p;
    for (;; rows /= 2) {
        long long n = 0;
        for (int i = 0; i < p.n_tensors; ++i) {
            NormTensor &t = p.t[i];
            const int room = std::max(1, rows) * plan.slots;
            t.per = std::min(t.n_heads, room);
            t.batch = rows == 0 ? 1 : grad ? 2 : std::min(kNormBatch, rows);
            if (t.weight_h != 0) {
                t.per = std::min(t.per, most);
                if (grad) t.batch = 1;
            }
            t.n_groups = (t.n_heads + t.per - 1) / t.per;
            t.tile = std::max(1, std::min({plan.slots, room / t.per, p.S}));
            t.tiles = (p.S + t.tile - 1) / t.tile;
            n += (long long)t.n_groups * p.B * t.tiles;
        }
        if (n >= blocks || rows == 0) return;
    }
}

// The same for rows that go 2 bytes at a time: a token for each warp, head after head.
void cut_tokens(Plan &plan, int per)
{
    for (int i = 0; i < plan.p.n_tensors; ++i) {
        NormTensor &t = plan.p.t[i];
        t.per = per;
        t.n_groups = (t.n_heads + per - 1) / per;
    }
}

}  // namespace
}  // namespace apex

using namespace apex;

extern "C" {

apex_status apex_attn_norm_rope(const apex_norm_tensor *q, const apex_norm_tensor *k, const apex_rope_tensor *v, int B,
                                int S, const int *positions, long long pos_stride, const int *row0, int out_rows,
                                const apex_rope_options *opt, float eps, apex_stream_t stream)
{
    apex_norm_tensor rows;
    memset(&rows, 0, sizeof rows);
    if (v) {
        rows.x = v->in;
        rows.out = v->out;
        rows.n_heads = v->n_heads;
        rows.d_row = v->d_row;
        rows.x_b = v->in_b, rows.x_h = v->in_h, rows.x_s = v->in_s;
        rows.out_b = v->out_b, rows.out_h = v->out_h, rows.out_s = v->out_s;
    }
    const apex_norm_tensor *t[3] = {q, k, v ? &rows : nullptr};
    Plan plan;
    const apex_status s = make_plan(t, false, B, S, positions, pos_stride, row0, out_rows, opt, eps, &plan);
    if (s != APEX_OK) return s;
    NormRopeParams &p = plan.p;
    if (plan.lanes) {
        // 3.5 blocks an SM of the 5 that run at once: 1026 tokens of 32 + 8 heads 6.4 us (8.5 with 2 asked
        // for), 1000 of 128 + 8 10.5 us (14.4 with 4, which makes it a wave and a half)
        cut_rows(plan, 16, false, kNormHeads / plan.lanes, 7 * plan.sm_count / 2);
        // a tile for each block; with weights for each head, which a block fetches first, and tiles for
        // three waves or more, as many blocks as run at once (8191 tokens of 128 + 8 heads 124 us, 136 with a
        // tile each; 4096 of 32 + 8, just a wave, 24.5 and 22.2)
        const long long wave = kNormCtas * plan.sm_count;
        long long n = 0;
        for (int i = 0; i < p.n_tensors; ++i) n += (long long)p.t[i].n_groups * B * p.t[i].tiles;
        for (int i = 0; i < p.n_tensors; ++i) {
            NormTensor &a = p.t[i];
            const long long room = a.weight_h && n >= 3 * wave ? wave * a.n_heads / plan.heads / a.n_groups : 1 << 16;
            a.blocks = (int)std::max(1ll, std::min((long long)B * a.tiles, room));
        }
    } else {
        // up to 8 heads with four blocks an SM
        const long long bx = ((long long)B * S + plan.slots - 1) / plan.slots;
        const long long share = (bx * plan.heads + 4 * plan.sm_count - 1) / (4 * plan.sm_count);
        cut_tokens(plan, (int)std::min<long long>(8, share));
        for (int i = 0; i < p.n_tensors; ++i) p.t[i].blocks = (int)std::min<long long>(bx, 1 << 16);
    }
    if (launch_norm_rope(p, plan.half, plan.lanes, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return APEX_ERR_CUDA;
    return APEX_OK;
}

size_t apex_attn_norm_rope_grad_workspace_bytes(int H_q, int H_kv, int d_q, int d_k)
{
    if (H_q <= 0 || H_kv < 0 || d_q <= 0 || d_k < 0 || H_q > 16384 || H_kv > 16384 || d_q > 1024 || d_k > 1024) return 0;
    return ((size_t)kNormGradBlocks * kNormGradHeads + H_q + H_kv) * std::max(d_q, d_k) * sizeof(float);
}

apex_status apex_attn_norm_rope_grad(const apex_norm_tensor *q, const apex_norm_tensor *k, int B, int S,
                                     const int *positions, long long pos_stride, const apex_rope_options *opt, float eps,
                                     void *workspace, size_t workspace_bytes, apex_stream_t stream)
{
    const apex_norm_tensor *t[3] = {q, k, nullptr};
    if (!q || !workspace || !aligned16(workspace)) return APEX_ERR_INVALID_ARG;
    if (workspace_bytes < apex_attn_norm_rope_grad_workspace_bytes(q->n_heads, k ? k->n_heads : 0, q->d_row,
                                                                   k ? k->d_row : 0))
        return APEX_ERR_INVALID_ARG;
    Plan plan;
    const apex_status s = make_plan(t, true, B, S, positions, pos_stride, nullptr, 0, opt, eps, &plan);
    if (s != APEX_OK) return s;
    NormRopeParams &p = plan.p;
    // as many blocks as run at once (2 bytes at a time: as there may be)
    const int room = std::min(kNormGradBlocks, (plan.lanes ? kNormGradCtas : 16) * plan.sm_count);
    if (plan.lanes) {
        cut_rows(plan, 8, true, std::min({kNormGradHeads, plan.slots, kNormHeads / plan.lanes}), room);
    } else {
        // with weights for each head a block has one head, whose sums it makes
        cut_tokens(plan, 8);
        for (int i = 0; i < p.n_tensors; ++i)
            if (p.t[i].weight_h != 0) p.t[i].n_groups = p.t[i].n_heads, p.t[i].per = 1;
    }
    // blocks in proportion to the heads, so that a block's sums are of many rows and all end together:
    // room at most in all, or one for each group
    float *partial = static_cast<float *>(workspace);
    for (int i = 0; i < p.n_tensors; ++i) {
        NormTensor &a = p.t[i];
        const long long most = plan.lanes ? (long long)B * a.tiles : ((long long)B * S + plan.slots - 1) / plan.slots;
        const long long share = (long long)room * a.n_heads / plan.heads / a.n_groups;
        a.blocks = (int)std::max(1ll, std::min(most, share));
        a.partial = partial;
        partial += (size_t)(a.weight_h != 0 ? a.n_heads : a.n_groups) * a.blocks * a.d_row;
    }
    if (launch_norm_rope_grad(p, plan.half, plan.lanes, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return APEX_ERR_CUDA;
    return APEX_OK;
}

}  // extern "C"
