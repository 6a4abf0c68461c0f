// cache_host.cu -- entry points of include/apex_attn.h that work on caches of
// rotated keys: argument checks, workspace layout and launches.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "cache_attn.h"
#include "evict.h"
#include "host_common.h"
#include "rope_host.h"

namespace apex {
namespace {

// ----------------------------------------------------------------- rope

// theta_i / 2 pi as 0.64 fixed-point fractions of a turn.  The last few parameter
// sets are kept, as the tables of the other entry points are: 64 pow() calls take
// longer than launching a small rotation.
struct TurnSet {
    RopeFreq f;
    float linear;
    int d_rot;  // 0: empty
    uint64_t turns[kRopeMaxPairs];
};

}  // namespace

bool turns_of(const RopeFreq &f, float linear, int d_rot, uint64_t *out)
{
    static std::mutex mu;
    static TurnSet sets[8];
    static int next = 0;
    std::unique_lock<std::mutex> lk(mu, std::defer_lock);
    try {
        lk.lock();
    } catch (...) {
        return false;  // no exception passes a C entry point
    }
    for (const TurnSet &t : sets)
        if (t.d_rot == d_rot && t.f == f && t.linear == linear) {
            memcpy(out, t.turns, sizeof(uint64_t) * (d_rot / 2));
            return true;
        }
    TurnSet &t = sets[next];
    next = (next + 1) % 8;
    t.f = f;
    t.linear = linear;
    t.d_rot = d_rot;
    for (int i = 0; i < d_rot / 2; ++i) {
        // whole turns per position do not change the angle
        const double turn = fmod(rope_frequency(i, d_rot, f) / linear / 6.283185307179586476925, 1.0);
        t.turns[i] = (uint64_t)ldexp(turn, 64);
    }
    memcpy(out, t.turns, sizeof(uint64_t) * (d_rot / 2));
    return true;
}

namespace {

// The span of stride * x over the counts, from its least (negative strides) to its largest.
void span_of(const RowSet &r, __int128 *lo, __int128 *hi)
{
    *lo = r.at;
    *hi = r.at + r.d - 1;
    for (int i = 0; i < 3; ++i) (r.stride[i] < 0 ? *lo : *hi) += (__int128)r.stride[i] * (r.count[i] - 1);
}

// Whether two sets of rows share an element (b == &a: whether two rows of a do).  That is a
// sum of strides times bounded integers, the differences of the rows' indices, that falls
// into the rows' lengths: searched from the largest stride down, where sums of the smaller
// strides leave one or two candidates each in any layout of nested dimensions.  Layouts
// that would take long to tell count as sharing.
struct RowSearch {
    struct Term {
        __int128 stride, lo, hi;  // stride > 0, times an integer of [lo, hi]
    } t[6];
    __int128 least[7], most[7];  // sums of the terms from i on
    int n = 0, left = 4096;
    bool self;
    void add(__int128 stride, __int128 lo, __int128 hi)
    {
        if (stride < 0)
            t[n++] = Term{-stride, -hi, -lo};
        else
            t[n++] = Term{stride, lo, hi};
    }
    static __int128 floor_div(__int128 a, __int128 b) { return a / b - (a % b < 0 ? 1 : 0); }
    bool search(int i, __int128 lo, __int128 hi, bool moved)  // a sum of the terms from i on in [lo, hi]
    {
        if (i == n) return lo <= 0 && hi >= 0 && (moved || !self);
        const __int128 from = std::max(t[i].lo, -floor_div(-(lo - most[i + 1]), t[i].stride));
        const __int128 to = std::min(t[i].hi, floor_div(hi - least[i + 1], t[i].stride));
        for (__int128 x = from; x <= to; ++x) {
            if (--left < 0) return true;
            if (search(i + 1, lo - x * t[i].stride, hi - x * t[i].stride, moved || x != 0)) return true;
        }
        return false;
    }
};

// Whether every dimension steps over all that the smaller ones reach: no element comes twice.
bool nested(const RowSet &r)
{
    int by[3] = {0, 1, 2};
    auto step = [&](int i) -> __int128 { return r.stride[i] < 0 ? -(__int128)r.stride[i] : r.stride[i]; };
    std::sort(by, by + 3, [&](int x, int y) { return step(x) < step(y); });
    __int128 reach = r.d;
    for (int i : by) {
        if (r.count[i] == 1) continue;
        if (step(i) < reach) return false;
        reach = step(i) * (r.count[i] - 1) + reach;
    }
    return true;
}

}  // namespace

bool share_elements(const RowSet &a, const RowSet &b)
{
    RowSearch r;
    r.self = &a == &b;
    if (r.self && nested(a)) return false;
    __int128 a0, a1, b0, b1;
    span_of(a, &a0, &a1);
    span_of(b, &b0, &b1);
    if (a1 < b0 || b1 < a0) return false;
    for (int i = 0; i < 3; ++i) {
        const bool one = a.stride[i] == b.stride[i];
        if (r.self && a.stride[i] == 0 && a.count[i] > 1) return true;
        if (a.stride[i] != 0 && (one ? a.count[i] + b.count[i] > 2 : a.count[i] > 1))
            r.add(a.stride[i], one ? 1 - b.count[i] : 0, a.count[i] - 1);
        if (!one && b.stride[i] != 0 && b.count[i] > 1) r.add(b.stride[i], 1 - b.count[i], 0);
    }
    std::sort(r.t, r.t + r.n, [](const RowSearch::Term &x, const RowSearch::Term &y) { return x.stride > y.stride; });
    r.least[r.n] = r.most[r.n] = 0;
    for (int i = r.n - 1; i >= 0; --i) {
        r.least[i] = r.least[i + 1] + r.t[i].stride * r.t[i].lo;
        r.most[i] = r.most[i + 1] + r.t[i].stride * r.t[i].hi;
    }
    const __int128 apart = b.at - a.at;
    return r.search(0, apart - (a.d - 1), apart + b.d - 1, false);
}

namespace {

bool rope_tensor_ok(const apex_rope_tensor *t)
{
    return t->in && t->out && t->n_heads > 0 && t->d_row > 0 && aligned(t->in, 2) && aligned(t->out, 2);
}

// Whether the tensors' outputs may be written while other threads still read or write: an
// output shares no element with an input or another output, but for a tensor turned in
// place (a thread reads the pairs that it writes; not with row0, which may shift rows).
bool outputs_apart(const apex_rope_tensor *const (&t)[3], int B, int S, bool row0, int out_rows)
{
    RowSet in[3], out[3];
    for (int i = 0; i < 3; ++i) {
        if (!t[i]) continue;
        in[i] = RowSet{(__int128)(reinterpret_cast<uintptr_t>(t[i]->in) / 2), {t[i]->in_b, t[i]->in_h, t[i]->in_s},
                       {B, t[i]->n_heads, S}, t[i]->d_row};
        out[i] = RowSet{(__int128)(reinterpret_cast<uintptr_t>(t[i]->out) / 2),
                        {t[i]->out_b, t[i]->out_h, t[i]->out_s},
                        {B, t[i]->n_heads, row0 && i > 0 ? out_rows : S}, t[i]->d_row};
    }
    for (int i = 0; i < 3; ++i) {
        if (!t[i]) continue;
        if (share_elements(out[i], out[i])) return false;
        for (int k = 0; k < 3; ++k) {
            if (!t[k]) continue;
            if (k < i && share_elements(out[i], out[k])) return false;
            bool in_place = k == i && in[i].at == out[i].at && !(row0 && i > 0);
            for (int d = 0; d < 3; ++d)
                in_place = in_place && (in[i].stride[d] == out[i].stride[d] || in[i].count[d] == 1);
            if (!in_place && share_elements(out[i], in[k])) return false;
        }
    }
    return true;
}

bool rows_of_16_bytes(const apex_rope_tensor *t)
{
    const long long strides = t->in_b | t->in_h | t->in_s | t->out_b | t->out_h | t->out_s;
    return aligned16(t->in) && aligned16(t->out) && t->d_row % 8 == 0 && strides % 8 == 0;
}

}  // namespace
}  // namespace apex

using namespace apex;

extern "C" {

apex_status apex_attn_rope(const apex_rope_tensor *q, const apex_rope_tensor *k, const apex_rope_tensor *v, int B,
                           int S, const int *positions, long long pos_stride, const int *row0, int out_rows,
                           const apex_rope_options *opt, apex_stream_t stream)
{
    if (!opt || !positions || (!q && !k && !v)) return APEX_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || (row0 && !aligned(row0, 4))) return APEX_ERR_INVALID_ARG;
    if (B <= 0 || S <= 0 || pos_stride < 0 || (row0 && out_rows <= 0)) return APEX_ERR_INVALID_ARG;
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
    if (B > kMaxSeq || S > kMaxSeq || (long long)B * S >= (1ll << 31)) return APEX_ERR_UNSUPPORTED;

    const apex_rope_tensor *in[3] = {q, k, v};
    int d_rot = opt->d_rot;
    for (int i = 0; i < 3; ++i) {
        if (!in[i]) continue;
        if (!rope_tensor_ok(in[i])) return APEX_ERR_INVALID_ARG;
        if (i == 2) continue;
        const int room = in[i]->d_row - opt->rot_start;
        if (d_rot == 0) d_rot = room;  // the whole row from rot_start on
        if (d_rot <= 0 || d_rot > room || d_rot % 2 != 0) return APEX_ERR_INVALID_ARG;
        if (opt->d_rot == 0 && d_rot != room) return APEX_ERR_INVALID_ARG;  // q and k disagree
    }
    for (int i = 0; i < 3; ++i)
        if (in[i] && (in[i]->d_row > 1024 || in[i]->n_heads > (1 << 20))) return APEX_ERR_UNSUPPORTED;
    if (d_rot > 2 * kRopeMaxPairs) return APEX_ERR_UNSUPPORTED;
    if (!outputs_apart(in, B, S, row0 != nullptr, out_rows)) return APEX_ERR_INVALID_ARG;
    const bool turns = q || k;
    if (d_rot == 0) d_rot = 2;  // values alone: nothing turns, and no frequency is used

    RopeParams p;
    memset(&p, 0, sizeof p);
    const bool half = opt->layout == APEX_ROPE_HALF;
    bool wide = !turns || (opt->rot_start % 8 == 0 && (half ? d_rot / 2 : d_rot) % 8 == 0);
    int heads = 0, nt = 0, width = 0;
    for (int i = 0; i < 3; ++i) {
        if (!in[i]) continue;
        RopeTensor &t = p.t[nt++];
        t = RopeTensor{static_cast<const uint16_t *>(in[i]->in), static_cast<uint16_t *>(in[i]->out),
                       in[i]->in_b, in[i]->in_h, in[i]->in_s, in[i]->out_b, in[i]->out_h, in[i]->out_s,
                       in[i]->d_row, i != 2, i != 0};
        wide = wide && rows_of_16_bytes(in[i]);
        heads += in[i]->n_heads;
        width = std::max(width, in[i]->d_row);
    }
    p.positions = positions;
    p.pos_stride = pos_stride;
    p.row0 = row0;
    p.out_rows = out_rows;
    p.B = B;
    p.S = S;
    p.rot_start = opt->rot_start;
    p.d_rot = d_rot;
    p.half = half;
    p.sign = opt->inverse ? -1.f : 1.f;
    if (!turns_of(f, linear, d_rot, p.turns)) return APEX_ERR_CUDA;

    int sm_count = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return APEX_ERR_CUDA;
    // Heads per group: a thread's heads share the sines of a unit, but with few tokens blocks
    // for the SMs are what there is to gain from fewer.  16 bytes at a time: up to 4 heads,
    // whose loads are in flight together, as far as a block for every SM goes, and 8 beyond
    // (32 + 8 + 8 heads of 128, interleaved, with 1 / 2 / 4 / 8 heads: one token 2.2 / 2.2 / 2.2 /
    // 2.7 us, 32 tokens 2.4 / 2.5 / 2.7 / 3.2, 64 tokens 3.2 / 2.5 / 2.7 / 3.2, 8 x 16 tokens
    // 3.7 / 3.2 / 2.7 / 3.2, 256 tokens 5.6 / 4.0 / 3.6 / 3.3 (half layout 4.2 / 3.6 / 3.2 / 4.1), 2048
    // tokens 29 / 16 / 10 / 8; 8191 tokens of 136 heads of 192: 4 heads 149, 8 heads 130).  2 bytes
    // at a time, head after head: up to 8 with four blocks an SM (the same: one token 1.9 / 2.1 /
    // 2.5 / 3.2, 64 tokens 3.9 / 2.9 / 3.0 / 3.5, 128 tokens 5.7 / 4.1 / 3.5 / 3.9, 256 tokens 9.6 / 6.2 /
    // 4.9 / 4.5).
    const long long units = (long long)B * S * (wide ? width / 8 : width);
    const long long bx = (units + kRopeThreads - 1) / kRopeThreads;
    const long long room = wide ? sm_count : 4ll * sm_count, share = (bx * heads + room - 1) / room;
    int per = share >= 8 ? 8 : (int)std::min<long long>(wide ? 4 : 8, share);
    auto groups = [&](int n) {  // n heads each
        int sum = 0;
        for (int i = 0; i < 3; ++i)
            if (in[i]) sum += (in[i]->n_heads + n - 1) / n;
        return sum;
    };
    per = std::max(per, heads / kRopeMaxGroups);
    while (groups(per) > kRopeMaxGroups) ++per;
    for (int i = 0, k = 0; i < 3; ++i) {
        if (!in[i]) continue;
        for (int h = 0; h < in[i]->n_heads; h += per)
            p.groups[p.n_groups++] = RopeGroup{k, h, std::min(per, in[i]->n_heads - h)};
        ++k;
    }
    const int kind = !wide ? kRopePairs : half ? kRopeHalf : kRopeInterleaved;
    const int grid_x = (int)std::min<long long>(bx, 1 << 20);
    if (launch_rope(p, kind, grid_x, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return APEX_ERR_CUDA;
    return APEX_OK;
}

// ----------------------------------------------------------------- eviction

size_t apex_attn_evict_workspace_bytes(int B, int H_kv, int S_cap, int budget)
{
    if (B <= 0 || H_kv <= 0 || S_cap <= 0 || budget <= 0 || S_cap > kMaxSeq) return 0;
    if ((long long)B * H_kv > (1 << 24)) return 0;
    return evict_workspace(B * H_kv, S_cap, budget).bytes;
}

apex_status apex_attn_evict(void *k_cache, void *v_cache, int B, int H_kv, int S_cap, int d_k, int d_v,
                            const float *acc, const int *positions, const int *lens, const int *next_pos, int budget,
                            int n_sink, int n_recent, float *acc_out, int *positions_out, int *lens_out,
                            void *workspace, size_t workspace_bytes, apex_stream_t stream)
{
    if (!k_cache || !v_cache || !acc || !lens || !acc_out || !positions_out || !lens_out || !workspace)
        return APEX_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(acc) || !aligned16(positions) || !aligned(lens, 4) ||
        !aligned(next_pos, 4) || !aligned16(acc_out) || !aligned16(positions_out) || !aligned(lens_out, 4) ||
        !aligned16(workspace))
        return APEX_ERR_INVALID_ARG;
    if (B <= 0 || H_kv <= 0 || S_cap <= 0 || d_k <= 0 || d_v <= 0) return APEX_ERR_INVALID_ARG;
    if (budget <= 0 || n_sink < 0 || n_recent < 0 || (long long)n_sink + n_recent > budget) return APEX_ERR_INVALID_ARG;
    if (S_cap > kMaxSeq || (long long)B * H_kv > (1 << 24)) return APEX_ERR_UNSUPPORTED;
    // every CTA reads its inputs while others already write: no output may lie on an input
    const size_t row_bytes = (size_t)B * H_kv * S_cap * 4, seq_bytes = (size_t)B * 4;
    auto same_rows = [&](const void *a, const void *b) { return overlap(a, row_bytes, b, row_bytes); };
    if (same_rows(acc_out, acc) || same_rows(positions_out, positions) || same_rows(acc_out, positions) ||
        same_rows(positions_out, acc) || same_rows(acc_out, positions_out) ||
        overlap(lens_out, seq_bytes, lens, seq_bytes) || overlap(lens_out, seq_bytes, next_pos, seq_bytes))
        return APEX_ERR_INVALID_ARG;
    if (d_k % 8 != 0 || d_v % 8 != 0 || d_k > 1024 || d_v > 1024) return APEX_ERR_UNSUPPORTED;
    const EvictWorkspace w = evict_workspace(B * H_kv, S_cap, budget);
    if (workspace_bytes < w.bytes) return APEX_ERR_INVALID_ARG;
    EvictParams p;
    memset(&p, 0, sizeof p);
    p.k = static_cast<uint4 *>(k_cache);
    p.v = static_cast<uint4 *>(v_cache);
    p.ck = d_k / 8;
    p.cv = d_v / 8;
    p.acc = acc;
    p.positions = positions;
    p.lens = lens;
    p.next_pos = next_pos ? next_pos : lens;
    p.newest = positions && !next_pos;
    p.acc_out = acc_out;
    p.positions_out = positions_out;
    p.lens_out = lens_out;
    p.holes = reinterpret_cast<int *>(workspace);
    p.sources = reinterpret_cast<int *>(static_cast<char *>(workspace) + w.sources);
    p.cap = w.cap;
    p.B = B;
    p.H_kv = H_kv;
    p.S_cap = S_cap;
    p.budget = budget;
    p.n_sink = n_sink;
    p.n_recent = n_recent;
    int sm_count = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return APEX_ERR_CUDA;
    if (launch_evict(p, sm_count, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return APEX_ERR_CUDA;
    return APEX_OK;
}

// ----------------------------------------------------------------- attention over a cache of rotated keys

static apex_status check_cache_attn(int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v)
{
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || T <= 0 || S_cap <= 0 || d_qk <= 0 || d_v <= 0) return APEX_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return APEX_ERR_INVALID_ARG;
    if (T > kTreeMaxDrafts || S_cap > kMaxSeq || B > 65536) return APEX_ERR_UNSUPPORTED;
    if (!((d_qk == 64 && d_v == 64) || (d_qk == 128 && d_v == 128) || (d_qk == 192 && d_v == 128)))
        return APEX_ERR_UNSUPPORTED;
    if (!supported_group(H_q / H_kv)) return APEX_ERR_UNSUPPORTED;
    if ((long long)B * H_q > (1 << 24) || (long long)B * H_kv * (long long)S_cap > (1ll << 40))
        return APEX_ERR_UNSUPPORTED;
    return APEX_OK;
}

static apex_status cache_attn(const void *q, const void *k_cache, const void *v_cache, void *out, int B, int H_q,
                              int H_kv, int T, int S_cap, int d_qk, int d_v, const int *lens,
                              const uint64_t *tree_mask, long long mask_stride, const int *positions, int window,
                              int n_sink, float *acc, bool weights, float scale, void *workspace, size_t workspace_bytes,
                              apex_stream_t stream)
{
    if (!q || !k_cache || !v_cache || !out || !lens || !workspace || (weights && !acc)) return APEX_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
        !aligned(lens, 4) || !aligned(tree_mask, 8) || !aligned(positions, 4) || !aligned(acc, 4))
        return APEX_ERR_INVALID_ARG;
    if (!isfinite(scale) || scale < 0.f || mask_stride < 0 || n_sink < 0) return APEX_ERR_INVALID_ARG;
    apex_status s = check_cache_attn(B, H_q, H_kv, T, S_cap, d_qk, d_v);
    if (s != APEX_OK) return s;
    // a CTA writes its rows while others still read theirs
    const size_t rows = (size_t)B * H_q * T, keys = (size_t)B * H_kv * S_cap;
    if (overlap(out, 2 * rows * d_v, q, 2 * rows * d_qk) || overlap(out, 2 * rows * d_v, k_cache, 2 * keys * d_qk) ||
        overlap(out, 2 * rows * d_v, v_cache, 2 * keys * d_v) || (acc && overlap(out, 2 * rows * d_v, acc, 4 * keys)))
        return APEX_ERR_INVALID_ARG;
    const CacheAttnWorkspace w = cache_attn_workspace(B, H_q, H_kv, T, S_cap, d_v, weights);
    if (workspace_bytes < w.bytes) return APEX_ERR_INVALID_ARG;
    DeviceScope dev;
    if (dev.status != APEX_OK) return dev.status;
    if (cache_attn_pairs(H_q / H_kv * T, d_v) && dev.sm_count < 2) return APEX_ERR_UNSUPPORTED;
    CacheAttnLaunch L;
    memset(&L, 0, sizeof L);
    CacheAttnParams &p = L.p;
    p.out = static_cast<uint16_t *>(out);
    p.B = B;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.G = H_q / H_kv;
    p.T = T;
    p.S_cap = S_cap;
    p.d_qk = d_qk;
    p.d_v = d_v;
    p.lens = lens;
    p.tree_mask = tree_mask;
    p.mask_stride = mask_stride;
    p.positions = positions;
    p.window = window > 0 ? window : 0;
    p.n_sink = window > 0 ? n_sink : 0;  // without a window every key stays visible; drafts may stand past S_cap
    p.drafts = weights ? 0 : T;
    p.acc = acc;
    p.scale_log2 = (float)(1.4426950408889634 * (scale == 0.f ? 1.0 / sqrt((double)d_qk) : (double)scale));
    p.wait = dev.wait;
    cache_attn_bind(p, w, workspace);
    if (!make_map(&L.tm_q, q, d_qk, p.R, B * H_kv, 128, 1) || !make_map(&L.tm_k, k_cache, d_qk, S_cap, B * H_kv, cache_attn_pairs(p.R, d_v) ? 64 : 128, 1) ||
        !make_map(&L.tm_v, v_cache, d_v, S_cap, B * H_kv, 128, 1))
        return APEX_ERR_CUDA;
    if (launch_cache_attn(L, dev.sm_count, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return APEX_ERR_CUDA;
    return APEX_OK;
}

size_t apex_attn_tree_workspace_bytes(int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v)
{
    if (check_cache_attn(B, H_q, H_kv, T, S_cap, d_qk, d_v) != APEX_OK) return 0;
    return cache_attn_workspace(B, H_q, H_kv, T, S_cap, d_v, false).bytes;
}

size_t apex_attn_decode_weights_workspace_bytes(int B, int H_q, int H_kv, int S_cap, int d_qk, int d_v)
{
    if (check_cache_attn(B, H_q, H_kv, 1, S_cap, d_qk, d_v) != APEX_OK) return 0;
    return cache_attn_workspace(B, H_q, H_kv, 1, S_cap, d_v, true).bytes;
}

apex_status apex_attn_tree_decode(const void *q, const void *k_cache, const void *v_cache, void *out, int B, int H_q,
                                  int H_kv, int T, int S_cap, int d_qk, int d_v, const int *lens,
                                  const uint64_t *tree_mask, long long mask_stride, const int *positions, int window,
                                  float scale, void *workspace, size_t workspace_bytes, apex_stream_t stream)
{
    return cache_attn(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens, tree_mask, mask_stride,
                      positions, window, 0, nullptr, false, scale, workspace, workspace_bytes, stream);
}

apex_status apex_attn_sink_tree_decode(const void *q, const void *k_cache, const void *v_cache, void *out, int B,
                                       int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v, const int *lens,
                                       const uint64_t *tree_mask, long long mask_stride, const int *positions,
                                       int window, int n_sink, float scale, void *workspace, size_t workspace_bytes,
                                       apex_stream_t stream)
{
    return cache_attn(q, k_cache, v_cache, out, B, H_q, H_kv, T, S_cap, d_qk, d_v, lens, tree_mask, mask_stride,
                      positions, window, n_sink, nullptr, false, scale, workspace, workspace_bytes, stream);
}

apex_status apex_attn_decode_weights(const void *q, const void *k_cache, const void *v_cache, void *out, int B,
                                     int H_q, int H_kv, int S_cap, int d_qk, int d_v, const int *lens, float *acc,
                                     float scale, void *workspace, size_t workspace_bytes, apex_stream_t stream)
{
    return cache_attn(q, k_cache, v_cache, out, B, H_q, H_kv, 1, S_cap, d_qk, d_v, lens, nullptr, 0, nullptr, 0, 0, acc,
                      true, scale, workspace, workspace_bytes, stream);
}

}  // extern "C"
