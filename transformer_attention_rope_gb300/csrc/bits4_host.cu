// bits4_host.cu -- entry points of include/apex_attn.h that work on caches held in 4 bits:
// argument checks, workspace layout and launches.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "bits4.h"
#include "rope_host.h"

namespace apex {
namespace {

size_t cache_bytes(int B, int H, int S_cap, int d) { return (size_t)B * H * S_cap * (d / 2); }
size_t scale_bytes(int B, int H, int S_cap, int d) { return (size_t)B * H * S_cap * (d / kBits4Block); }

// `bytes` at an address as 2-byte elements, in rows of about 2^30 that end with the last of them: equal
// steps, each row as long as what the steps leave.
RowSet bytes_of(const void *at, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(at);
    const long long first = (long long)(a / 2), n = (long long)((a + bytes + 1) / 2) - first;
    const long long count = (n >> 30) + 1, step = n / count;
    return RowSet{(__int128)first, {0, 0, step}, {1, 1, (int)count}, (int)(n - (count - 1) * step)};
}

// Rows of bf16 in and packed rows out (append), or the other way round (unpack).
apex_status move_rows(const apex_bits4_tensor *const (&t)[2], bool append, int B, int H, int S, int S_cap,
                      const int *row0, apex_stream_t stream)
{
    if (!t[0] || !t[1]) return APEX_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || S <= 0 || S_cap <= 0 || !aligned(row0, 4)) return APEX_ERR_INVALID_ARG;
    for (const apex_bits4_tensor *a : t) {
        if (!a->rows || !a->bytes || !a->scales || !aligned(a->rows, 2) || !aligned16(a->bytes) || !aligned16(a->scales) ||
            !aligned(a->factor, 4) || a->d <= 0)
            return APEX_ERR_INVALID_ARG;
        if (a->d % kBits4Block != 0 || a->d > kBits4MaxRow) return APEX_ERR_UNSUPPORTED;
    }
    if (B > kMaxSeq || S > kMaxSeq || S_cap > kMaxSeq || H > (1 << 20) || (__int128)B * H * S >= (1ll << 31) ||
        (__int128)B * H * S_cap > (1ll << 40))
        return APEX_ERR_UNSUPPORTED;
    // an output lies on no input and on no other output
    RowSet rows[2];
    const void *packed[4];
    size_t size[4];
    for (int i = 0; i < 2; ++i) {
        rows[i] = RowSet{(__int128)(reinterpret_cast<uintptr_t>(t[i]->rows) / 2), {t[i]->b, t[i]->h, t[i]->s}, {B, H, S}, t[i]->d};
        packed[2 * i] = t[i]->bytes;
        size[2 * i] = cache_bytes(B, H, S_cap, t[i]->d);
        packed[2 * i + 1] = t[i]->scales;
        size[2 * i + 1] = scale_bytes(B, H, S_cap, t[i]->d);
    }
    for (int i = 0; i < 4; ++i) {
        const RowSet held = bytes_of(packed[i], size[i]);
        for (int k = 0; k < 2; ++k)
            if (share_elements(held, rows[k])) return APEX_ERR_INVALID_ARG;
        for (int k = 0; append && k < i; ++k)
            if (overlap(packed[i], size[i], packed[k], size[k])) return APEX_ERR_INVALID_ARG;
    }
    if (!append && (share_elements(rows[0], rows[0]) || share_elements(rows[1], rows[1]) || share_elements(rows[0], rows[1])))
        return APEX_ERR_INVALID_ARG;
    Bits4Params p;
    memset(&p, 0, sizeof p);
    for (int i = 0; i < 2; ++i) {
        const apex_bits4_tensor &a = *t[i];
        const long long strides = a.b | a.h | a.s;
        p.t[i] = Bits4Tensor{static_cast<uint16_t *>(a.rows), a.b, a.h, a.s, static_cast<uint8_t *>(a.bytes),
                             static_cast<uint8_t *>(a.scales), a.factor, a.d,
                             aligned(a.rows, 32) && strides % 16 == 0  ? 32
                             : aligned16(a.rows) && strides % 8 == 0 ? 16
                                                                     : 2,
                             0, 0};
    }
    p.row0 = row0;
    p.B = B;
    p.H = H;
    p.S = S;
    p.S_cap = S_cap;
    const cudaStream_t at = reinterpret_cast<cudaStream_t>(stream);
    if ((append ? launch_append4(p, at) : launch_unpack4(p, at)) != cudaSuccess) return APEX_ERR_CUDA;
    return APEX_OK;
}

apex_status check_decode4(int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v)
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

}  // namespace
}  // namespace apex

using namespace apex;

extern "C" {

apex_status apex_attn_append4(const apex_bits4_tensor *k, const apex_bits4_tensor *v, int B, int H_kv, int S, int S_cap,
                              const int *row0, apex_stream_t stream)
{
    const apex_bits4_tensor *t[2] = {k, v};
    return move_rows(t, true, B, H_kv, S, S_cap, row0, stream);
}

apex_status apex_attn_unpack4(const apex_bits4_tensor *k, const apex_bits4_tensor *v, int B, int H_kv, int S, int S_cap,
                              const int *row0, apex_stream_t stream)
{
    const apex_bits4_tensor *t[2] = {k, v};
    return move_rows(t, false, B, H_kv, S, S_cap, row0, stream);
}

size_t apex_attn_decode4_workspace_bytes(int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v)
{
    if (check_decode4(B, H_q, H_kv, T, S_cap, d_qk, d_v) != APEX_OK) return 0;
    return decode4_workspace(B, H_q, H_kv, T, S_cap, d_v).bytes;
}

apex_status apex_attn_decode4(const void *q, const void *k4, const void *k_scale, const void *v4, const void *v_scale,
                              void *out, int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v, const int *lens,
                              int window, int n_sink, const float *k_factor, const float *v_factor, float scale,
                              void *workspace, size_t workspace_bytes, apex_stream_t stream)
{
    if (!q || !k4 || !k_scale || !v4 || !v_scale || !out || !lens || !workspace) return APEX_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k4) || !aligned16(k_scale) || !aligned16(v4) || !aligned16(v_scale) ||
        !aligned16(out) || !aligned16(workspace) || !aligned(lens, 4) || !aligned(k_factor, 4) || !aligned(v_factor, 4))
        return APEX_ERR_INVALID_ARG;
    if (!isfinite(scale) || scale < 0.f || n_sink < 0) return APEX_ERR_INVALID_ARG;
    apex_status s = check_decode4(B, H_q, H_kv, T, S_cap, d_qk, d_v);
    if (s != APEX_OK) return s;
    // a CTA writes its rows while others still read theirs
    const size_t rows = (size_t)B * H_q * T;
    if (overlap(out, 2 * rows * d_v, q, 2 * rows * d_qk) ||
        overlap(out, 2 * rows * d_v, k4, cache_bytes(B, H_kv, S_cap, d_qk)) ||
        overlap(out, 2 * rows * d_v, v4, cache_bytes(B, H_kv, S_cap, d_v)) ||
        overlap(out, 2 * rows * d_v, k_scale, scale_bytes(B, H_kv, S_cap, d_qk)) ||
        overlap(out, 2 * rows * d_v, v_scale, scale_bytes(B, H_kv, S_cap, d_v)) ||
        overlap(out, 2 * rows * d_v, lens, (size_t)B * 4) || overlap(out, 2 * rows * d_v, k_factor, (size_t)H_kv * 4) ||
        overlap(out, 2 * rows * d_v, v_factor, (size_t)H_kv * 4))
        return APEX_ERR_INVALID_ARG;
    const Decode4Workspace w = decode4_workspace(B, H_q, H_kv, T, S_cap, d_v);
    if (workspace_bytes < w.bytes) return APEX_ERR_INVALID_ARG;
    DeviceScope dev;
    if (dev.status != APEX_OK) return dev.status;
    Decode4Params p;
    memset(&p, 0, sizeof p);
    CacheAttnParams &c = p.c;
    c.out = static_cast<uint16_t *>(out);
    c.B = B;
    c.H_q = H_q;
    c.H_kv = H_kv;
    c.G = H_q / H_kv;
    c.T = T;
    c.S_cap = S_cap;
    c.d_qk = d_qk;
    c.d_v = d_v;
    c.lens = lens;
    c.window = window > 0 ? window : 0;
    c.n_sink = window > 0 ? n_sink : 0;  // without a window every key stays visible
    c.drafts = T;
    c.scale_log2 = (float)(1.4426950408889634 * (scale == 0.f ? 1.0 / sqrt((double)d_qk) : (double)scale));
    c.R = c.G * T;
    c.group = decode4_group(c.R);
    c.n_groups = w.n_groups;
    c.rows_cap = w.rows_cap;
    char *base = static_cast<char *>(workspace);
    c.ws_o = reinterpret_cast<float *>(base);
    c.ws_ml = reinterpret_cast<float2 *>(base + w.ml);
    c.units = reinterpret_cast<int2 *>(base + w.units);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint8_t *>(k4);
    p.v = static_cast<const uint8_t *>(v4);
    p.k_scale = static_cast<const uint8_t *>(k_scale);
    p.v_scale = static_cast<const uint8_t *>(v_scale);
    p.k_factor = k_factor;
    c.v_factor = v_factor;
    c.wait = dev.wait;
    if (launch_decode4(p, dev.sm_count, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return APEX_ERR_CUDA;
    return APEX_OK;
}

}  // extern "C"
