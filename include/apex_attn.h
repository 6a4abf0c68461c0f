/*
 * apex_attn.h -- C ABI of the GB300 (sm_103a) APEX-1 attention block.
 *
 * The block computes, for every batch b, query head h and query row r
 * (APEX-1 Mathematical Reference, Part 1 §4 and Part 2 §6, §8, §10):
 *
 *   m      = q_pos0 + r                       position of the query row
 *   g      = floor(h / G),  G = H_q / H_kv    KV head shared by the group
 *                                             (Part 2 §8.2; §8.4 example)
 *   q'     = RoPE(q[b,h,r], m)                interleaved pairs (2i, 2i+1)
 *   k'_j   = RoPE(k[b,g,j], j)                rotated by angle pos*theta_i,
 *                                             theta_i = base^(-2i/d_h)
 *                                             (Part 1 §4.2-§4.4)
 *   out    = sum_j softmax_j(<q', k'_j> / sqrt(d_h)) v[b,g,j]
 *            over the keys j visible from m   (Part 2 §6.2)
 *   visible(m, j) <=> j <= m  and  (window <= 0  or  m - j < window)
 *                                             (Part 2 §10.2)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Tensors are dense, row-major, bf16 (raw 16-bit patterns), in device
 *   memory, with the 4-D attention layout [B, H, S, d_h] (Part 1 §1 "Tensor
 *   Shape Convention").  Every pointer must be 16-byte aligned.
 * - The caller owns every buffer it passes, scratch included: the decode's
 *   split partials and the prefill's rotated keys live in workspaces the caller
 *   passes (sizes from the *_workspace_bytes functions).  The library owns only
 *   a per-device cache of RoPE cos/sin tables (fp32, built in double precision
 *   on the host), allocated on first use and grown on demand.  A call that has to build or
 *   grow that table allocates device memory and synchronises the device;
 *   apex_attn_rope_reserve() builds it ahead of time.
 * - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *   stream) and returns before it finishes.  Calls are thread-compatible:
 *   concurrent calls on one device serialise on an internal lock while they
 *   enqueue.
 * - Supported: d_h in {64, 128}; H_q % H_kv == 0 with G = H_q / H_kv in
 *   {1, 2, 4, 8, 16}; 1 <= S <= 2^24; q_pos0 >= 0 and q_pos0 + S_q <= S_k, so
 *   that every query row sees at least its own key.
 * - Arguments are validated before anything is launched: a rejected call
 *   launches nothing and returns APEX_ERR_INVALID_ARG (bad value) or
 *   APEX_ERR_UNSUPPORTED (valid but outside the supported set).  A CUDA
 *   failure while enqueuing returns APEX_ERR_CUDA; the CUDA error state is left
 *   as the runtime reports it.  No entry point prints, traps or exits.
 * - Every wait inside the kernels is bounded in time.  A wait that gives up
 *   records a code in a per-device status word and lets the kernel finish
 *   (with unspecified output); apex_attn_device_status() reads and clears it.
 */
#ifndef APEX_ATTN_H
#define APEX_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum apex_status {
    APEX_OK = 0,
    APEX_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, bad size or position */
    APEX_ERR_UNSUPPORTED = 2,  /* valid arguments outside the supported set     */
    APEX_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed             */
    APEX_ERR_NO_MEMORY = 4,    /* the RoPE table could not be allocated          */
    APEX_ERR_DEVICE_TIMEOUT = 5 /* a kernel's bounded wait gave up (see below)   */
} apex_status;

/* Opaque CUDA stream handle (same object as cudaStream_t / CUstream). */
typedef struct CUstream_st *apex_stream_t;

/*
 * Prefill: attention of S_q query rows against S_k keys.
 *
 *   q   [B, H_q,  S_q, d_h]  bf16, read      (query row r sits at q_pos0 + r)
 *   k   [B, H_kv, S_k, d_h]  bf16, read      (raw keys: RoPE is applied here,
 *   v   [B, H_kv, S_k, d_h]  bf16, read       key j at position j)
 *   out [B, H_q,  S_q, d_h]  bf16, written   (must not overlap q, k or v)
 *   window     <= 0: causal only; > 0: key j visible iff 0 <= m - j < window
 *   rope_base  RoPE base b of theta_i = b^(-2i/d_h) (10000 on the pages);
 *              must be finite and > 0
 *
 * Cites: Part 2 §6.2 (SDPA), §8.2 (GQA), §10.2 (mask); Part 1 §4 (RoPE).
 * Errors: see the conventions above.  Result: softmax in fp32 with exp2; Q, K
 * are rotated in fp32 and rounded to bf16 for the tensor cores, as is P.
 */
apex_status apex_attn_fwd(const void *q, const void *k, const void *v, void *out,
                          int B, int H_q, int H_kv, int S_q, int S_k, int d_h,
                          int window, int q_pos0, float rope_base, apex_stream_t stream);

/*
 * Options of the _ex entry points.  Zero-initialise the struct and set what is
 * needed: all zeros is the plain block with rope_base 10000.
 */
typedef struct apex_attn_options {
    int window;           /* <= 0: causal only; > 0: sliding window W            */
    int q_pos;            /* fwd: position of query row 0; decode: the query's   */
    float rope_base;      /* RoPE base b of theta_i = b^(-2i/d_h); 0 means 10000 */
    float yarn_scale;     /* YaRN factor s (Part 1 §5); <= 1: no YaRN            */
    float yarn_beta_fast; /* wavelength below which a pair is unscaled; 0: 32    */
    float yarn_beta_slow; /* beta_slow * s: wavelength above which theta/s; 0: 1 */
    int prefix_len;       /* P > 0: positions [0, P) attend to each other
                             bidirectionally (Part 2 §11.1); 0 <= P <= S_k       */
    int keys_prerotated;  /* non-zero: k / k_cache already hold RoPE(k_j, j)     */
} apex_attn_options;

/*
 * YaRN (Part 1 §5.3-§5.5), when yarn_scale > 1: with the wavelength
 * lambda_i = 2 pi / theta_i, pairs with lambda_i < beta_fast keep theta_i,
 * pairs with lambda_i > beta_slow * s use theta_i / s, the others use
 * theta_i / (t s + 1 - t), t = clamp((lambda_i / beta_slow - 1) / (s - 1), 0, 1);
 * the scores are multiplied by 0.1 ln(s) + 1.
 * Prefix (Part 2 §11.1), when prefix_len = P > 0: a query at m < P sees the keys
 * j < P and nothing else; queries at m >= P follow the causal/window rule.
 */

/*
 * Prefill with options: as apex_attn_fwd, with window, q_pos0 (= opt->q_pos)
 * and rope_base taken from *opt.  opt may not be NULL.
 */
apex_status apex_attn_fwd_ex(const void *q, const void *k, const void *v, void *out,
                             int B, int H_q, int H_kv, int S_q, int S_k, int d_h,
                             const apex_attn_options *opt, apex_stream_t stream);

/*
 * Bytes of caller-provided device workspace apex_attn_fwd_ws will use for this
 * call (same arguments): one rotated copy of the keys, B * H_kv * S_k * d_h bf16
 * values, when the library's cost model rotates the keys before the prefill;
 * 0 when it would not (then no workspace is needed), when opt->keys_prerotated
 * is set, and when the arguments are invalid.  Host-only, no CUDA call.
 */
size_t apex_attn_fwd_workspace_bytes(int B, int H_q, int H_kv, int S_q, int S_k, int d_h,
                                     const apex_attn_options *opt);

/*
 * Prefill with options and a workspace: the same result as apex_attn_fwd_ex
 * (same arguments, layouts, masks and rounding up to the order of fp32 sums),
 * computed faster on long or wide problems.  The pages rotate every key by its
 * position (Part 1 §4.2-§4.5); the prefill rotates each 128-key tile in shared
 * memory once for every work item that reaches it, which on long windows or
 * wide head groups means tens of times.  Given a workspace, the library may
 * instead rotate the keys once, RoPE(k_j, j) in bf16 as apex_attn_rope_keys
 * computes it, into the workspace and run the prefill on those (it does so when
 * its cost model -- key-tile visits against one read and write of K -- says
 * that is faster; otherwise the workspace is left untouched).
 *
 *   workspace, workspace_bytes: NULL (then this is apex_attn_fwd_ex), or device
 *     memory of at least apex_attn_fwd_workspace_bytes(...) bytes for the same
 *     arguments, 16-byte aligned, owned by the caller, not overlapping q, k, v
 *     or out, not read before written; a smaller or misaligned workspace gives
 *     APEX_ERR_INVALID_ARG before any launch.
 *   The pass is a second kernel on `stream` before the prefill; with
 *   opt->keys_prerotated no pass runs.
 * Errors as for apex_attn_fwd_ex.
 */
apex_status apex_attn_fwd_ws(const void *q, const void *k, const void *v, void *out,
                             int B, int H_q, int H_kv, int S_q, int S_k, int d_h,
                             const apex_attn_options *opt, void *workspace, size_t workspace_bytes,
                             apex_stream_t stream);

/*
 * Prefill of multi-head latent attention with decoupled RoPE (Part 2 §9.3):
 * query and key rows are [content | rope part], the rope part alone is
 * rotated, and values keep the content length.
 *
 *   q   [B, H_q,  S_q, d_h + d_r] bf16, read     (row: q_content | q_rope)
 *   k   [B, H_kv, S_k, d_h + d_r] bf16, read     (row: k_content | k_rope)
 *   v   [B, H_kv, S_k, d_h]       bf16, read
 *   out [B, H_q,  S_q, d_h]       bf16, written  (must not overlap q, k or v)
 *
 * The rope part is rotated as a d_r-dimensional RoPE vector (pairs numbered
 * from its start, theta_i = b^(-2i/d_r), with the options' YaRN rule); the
 * content part is used as it is.  Scores are the dot products of the whole
 * rows divided by sqrt(d_h + d_r) (times the YaRN temperature).  With
 * opt->keys_prerotated the rope part of k is taken as already rotated.  All
 * other options and the masks are those of apex_attn_fwd_ex.
 * Supported: d_h = 128, d_r = 64 (else APEX_ERR_UNSUPPORTED); d_r must be
 * even and > 0 (else APEX_ERR_INVALID_ARG); H_q / H_kv as for apex_attn_fwd.
 * Runs on pairs of CTAs (a thread-block cluster of 2).
 */
apex_status apex_attn_mla_fwd(const void *q, const void *k, const void *v, void *out,
                              int B, int H_q, int H_kv, int S_q, int S_k, int d_h, int d_r,
                              const apex_attn_options *opt, apex_stream_t stream);

/*
 * Bytes of caller-provided device workspace apex_attn_mla_fwd_ws will use for
 * this call (same arguments): one copy of the key rows with the rope part
 * rotated, B * H_kv * S_k * (d_h + d_r) bf16 values, when the library's cost
 * model rotates the keys before the prefill; 0 when it would not, when
 * opt->keys_prerotated is set, and when the arguments are invalid or
 * unsupported.  Host-only, no CUDA call.
 */
size_t apex_attn_mla_fwd_workspace_bytes(int B, int H_q, int H_kv, int S_q, int S_k, int d_h, int d_r,
                                         const apex_attn_options *opt);

/*
 * Decoupled-RoPE prefill with a workspace: the same result as apex_attn_mla_fwd
 * (up to the order of fp32 sums), with the rope part of every key row rotated
 * once into the workspace beforehand (as apex_attn_mla_rope_keys computes it;
 * the content part copied) when the cost model says that is faster than
 * rotating it in every work item that visits the key tile.  workspace and
 * workspace_bytes as for apex_attn_fwd_ws, sized by
 * apex_attn_mla_fwd_workspace_bytes(...); NULL makes this apex_attn_mla_fwd.
 * Errors as for apex_attn_mla_fwd, plus APEX_ERR_INVALID_ARG for a smaller or
 * misaligned workspace (before any launch).
 */
apex_status apex_attn_mla_fwd_ws(const void *q, const void *k, const void *v, void *out,
                                 int B, int H_q, int H_kv, int S_q, int S_k, int d_h, int d_r,
                                 const apex_attn_options *opt, void *workspace, size_t workspace_bytes,
                                 apex_stream_t stream);

/*
 * Prefill under a sliding window whose first tokens stay visible (sinks):
 *   visible(m, j) <=> j <= m  and  (m - j < opt->window  or  j < n_sink)
 * and for everything else apex_attn_fwd_ws (d_r = 0) or apex_attn_mla_fwd_ws (d_r > 0:
 * q and k rows of d_h + d_r entries): layouts, options (a query inside a prefix sees the
 * prefix alone), workspaces, supported sizes and errors.  n_sink >= 0; 0, or no window, is
 * the call without sinks.  A work item visits the key tiles of its window and those of the
 * sinks, whatever lies between.  As for the calls without, k and v hold no infinities or NaN, at
 * masked keys either: a weight of 0 does not hide them.
 */
apex_status apex_attn_sink_fwd(const void *q, const void *k, const void *v, void *out,
                               int B, int H_q, int H_kv, int S_q, int S_k, int d_h, int d_r, int n_sink,
                               const apex_attn_options *opt, void *workspace, size_t workspace_bytes,
                               apex_stream_t stream);

/* Bytes of workspace apex_attn_sink_fwd will use, as apex_attn_fwd_workspace_bytes.  Host-only. */
size_t apex_attn_sink_fwd_workspace_bytes(int B, int H_q, int H_kv, int S_q, int S_k, int d_h, int d_r, int n_sink,
                                          const apex_attn_options *opt);

/*
 * Decode under the same rule: apex_attn_decode_ex (d_r = 0) or apex_attn_mla_decode (d_r > 0)
 * with the first n_sink keys visible behind opt->window; workspace as for them, and caches without
 * infinities or NaN.
 */
apex_status apex_attn_sink_decode(const void *q, const void *k_cache, const void *v_cache, void *out,
                                  int B, int H_q, int H_kv, int S_k, int d_h, int d_r, int n_sink,
                                  const apex_attn_options *opt, void *workspace, size_t workspace_bytes,
                                  apex_stream_t stream);

/*
 * Decode with options: as apex_attn_decode, with window, q_pos and rope_base
 * taken from *opt.  With a prefix and q_pos < P the query sees keys [0, P).
 * The workspace size is apex_attn_decode_workspace_bytes(...) as for
 * apex_attn_decode.
 */
apex_status apex_attn_decode_ex(const void *q, const void *k_cache, const void *v_cache, void *out,
                                int B, int H_q, int H_kv, int S_k, int d_h,
                                const apex_attn_options *opt, void *workspace,
                                size_t workspace_bytes, apex_stream_t stream);

/*
 * Diagnostic (the pages have no counterpart): launches one CTA whose bounded
 * mbarrier wait -- the wait every kernel of this library uses -- can never
 * complete.  After timeout_ms (1..5000, else APEX_ERR_INVALID_ARG) the wait
 * gives up, records its code in the per-device status word and the kernel
 * returns; apex_attn_device_status() then reports APEX_ERR_DEVICE_TIMEOUT
 * (and clears it) and the context stays usable.  Asynchronous on `stream`.
 */
apex_status apex_attn_selftest_wait_timeout(int timeout_ms, apex_stream_t stream);

/*
 * Decode of multi-head latent attention with decoupled RoPE (Part 2 §9.3):
 * one query per sequence against a cache of [content | rope part] keys.
 *
 *   q       [B, H_q,  1,   d_h + d_r] bf16, read   (the query sits at opt->q_pos)
 *   k_cache [B, H_kv, S_k, d_h + d_r] bf16, read   (key j at position j)
 *   v_cache [B, H_kv, S_k, d_h]       bf16, read
 *   out     [B, H_q,  1,   d_h]       bf16, written
 *   workspace: at least apex_attn_decode_workspace_bytes(B, H_q, H_kv, S_k, d_h)
 *           bytes (d_h: the value row length), 16-byte aligned.
 *
 * Rotation, scores and options as for apex_attn_mla_fwd; the result equals
 * apex_attn_mla_fwd with S_q = 1 and q_pos0 = q_pos (up to the order of fp32
 * sums).  Supported: d_h = 128, d_r = 64.
 */
apex_status apex_attn_mla_decode(const void *q, const void *k_cache, const void *v_cache, void *out,
                                 int B, int H_q, int H_kv, int S_k, int d_h, int d_r,
                                 const apex_attn_options *opt, void *workspace, size_t workspace_bytes,
                                 apex_stream_t stream);

/*
 * Rotate keys for a pre-rotated KV cache (Part 1 §4.2-§4.4, with the options'
 * rope_base / YaRN): for each of n_heads heads h and each s < n_pos,
 *   k_out[h * out_head_stride + s * d_h + :] = RoPE(k_in[h * in_head_stride + s * d_h + :], pos0 + s)
 * in bf16 (fp32 arithmetic).  Strides are in elements; with
 * out_head_stride = S_cache * d_h and k_out pointing at row pos0 of a cache,
 * this appends freshly projected keys to that cache.  k_out may equal k_in
 * (same strides) for an in-place rotation; otherwise the ranges must not
 * overlap.  Only window/prefix-independent fields of *opt are used.
 */
apex_status apex_attn_rope_keys(const void *k_in, void *k_out, int n_heads, int n_pos, int d_h, int pos0,
                                long long in_head_stride, long long out_head_stride,
                                const apex_attn_options *opt, apex_stream_t stream);

/*
 * The same for decoupled-RoPE key rows [content (d_h) | rope part (d_r)]
 * (Part 2 §9.3): for each head h and s < n_pos the row at
 * k_in[h * in_head_stride + s * (d_h + d_r)] goes to k_out with its content
 * part copied and its rope part rotated as a d_r-dimensional RoPE vector at
 * position pos0 + s (pairs numbered from the rope part's start,
 * theta_i = b^(-2i/d_r), the options' YaRN rule) -- the keys
 * apex_attn_mla_fwd / apex_attn_mla_decode take with opt->keys_prerotated.
 * Strides in elements (at least n_pos * (d_h + d_r), multiples of 8), overlap
 * rules as for apex_attn_rope_keys.  Supported: d_h = 128, d_r = 64 (else
 * APEX_ERR_UNSUPPORTED); d_r must be even and > 0 (else APEX_ERR_INVALID_ARG).
 */
apex_status apex_attn_mla_rope_keys(const void *k_in, void *k_out, int n_heads, int n_pos, int d_h, int d_r,
                                    int pos0, long long in_head_stride, long long out_head_stride,
                                    const apex_attn_options *opt, apex_stream_t stream);

/*
 * Bytes of caller-provided device workspace apex_attn_decode needs for these
 * sizes (the split-KV partial results).  Returns 0 when the sizes are invalid.
 * The same sizes with any window / q_pos never need more.
 */
size_t apex_attn_decode_workspace_bytes(int B, int H_q, int H_kv, int S_k, int d_h);

/*
 * Decode: one query per sequence against a bf16 KV cache.
 *
 *   q       [B, H_q,  1,   d_h] bf16, read   (the query sits at position q_pos)
 *   k_cache [B, H_kv, S_k, d_h] bf16, read   (raw keys, key j at position j)
 *   v_cache [B, H_kv, S_k, d_h] bf16, read
 *   out     [B, H_q,  1,   d_h] bf16, written
 *   q_pos   0 <= q_pos < S_k; keys j > q_pos are masked (causal)
 *   window  as for apex_attn_fwd
 *   workspace, workspace_bytes: device scratch of at least
 *           apex_attn_decode_workspace_bytes(B, H_q, H_kv, S_k, d_h) bytes,
 *           16-byte aligned, owned by the caller, not read before written.
 *
 * The result equals apex_attn_fwd with S_q = 1 and q_pos0 = q_pos (up to the
 * order of fp32 sums).  The KV range is split across CTAs; each split writes
 * a partial (max, sum, unnormalised output) and a log-sum-exp combine kernel
 * merges them (Part 2 §6.2: softmax is invariant to the shift by the max).
 * Cites: Part 2 §6.2, §7.4 (KV cache), §8.2, §10.2; Part 1 §4.
 */
apex_status apex_attn_decode(const void *q, const void *k_cache, const void *v_cache, void *out,
                             int B, int H_q, int H_kv, int S_k, int d_h, int window, int q_pos,
                             float rope_base, void *workspace, size_t workspace_bytes,
                             apex_stream_t stream);

/*
 * Decode that allocates nothing, for callers that cannot allocate device
 * memory when they call: an engine whose device memory is all handed out by
 * its own pool at start-up (a cudaMalloc would fail, fragment the pool or
 * synchronise the device), a plugin interface with a fixed signature and no
 * workspace slot, or a latency-critical loop that cannot afford an
 * allocation's synchronisation.  The APEX-1 pages have no counterpart of this
 * entry point; it computes exactly what apex_attn_decode computes.
 *
 *   Arguments, layouts and results: as apex_attn_decode, without workspace.
 *   Scratch: split-KV partials live in a 16 MiB file-scope device array and
 *     the RoPE table in a 16 MiB one (positions < 32768); every GPU that loads
 *     the library holds these 32 MiB until the process exits.  Nothing in them
 *     has to start at zero: each call writes every partial it reads.
 *   Limits (APEX_ERR_UNSUPPORTED beyond them): S_k <= 32768, d_h in {64, 128},
 *     G in {1, 2, 4, 8, 16}, and B * H_q * (4 * d_h + 8) <= 16 MiB (one split);
 *     larger B * H_q only lowers the number of KV splits the scratch allows.
 *   Set-up: the first call on a device (and the first call with a new
 *     (d_h, rope_base) pair) looks up the arrays' device addresses, builds the
 *     RoPE table on `stream` and synchronises that stream; make that call before
 *     capturing any CUDA graph.
 *   Concurrency: all calls on a device share the arrays, so calls that may
 *     overlap on the GPU (different streams without ordering between them) race
 *     and must not be issued.  Kernel waits are bounded as on the other entry
 *     points (APEX_ATTN_WAIT_TIMEOUT_MS, 2 s by default), but a wait that times
 *     out is not recorded (there is no status word without allocation); the
 *     output is then unspecified.  If the table build fails (APEX_ERR_CUDA),
 *     the next call rebuilds it.
 */
apex_status apex_attn_decode_noalloc(const void *q, const void *k_cache, const void *v_cache, void *out,
                                     int B, int H_q, int H_kv, int S_k, int d_h, int window, int q_pos,
                                     float rope_base, apex_stream_t stream);

/*
 * Build (or grow) the RoPE cos/sin table of the current device so that
 * positions [0, max_pos) are covered for this (d_h, rope_base).  Synchronous.
 * Calling it before capturing a CUDA graph keeps the captured calls free of
 * allocations.  Part 1 §4.7 (cos/sin cache computed once, reused).
 */
apex_status apex_attn_rope_reserve(int max_pos, int d_h, float rope_base);

/* ======================================================================
 * Operators over a cache of rotated keys.
 *
 * The entry points below work on caches whose keys were rotated before they
 * were stored ("pre-rotated": apex_attn_rope_keys or apex_attn_rope), so a
 * cache row need not sit at the index of its position.  Lengths, positions and
 * masks are device arrays and may change between replays of a captured graph;
 * nothing is read back to the host.  Supported row lengths of the attention
 * entry points: (d_qk, d_v) = (64, 64), (128, 128) or, for decoupled rows
 * [content | rope part], (192, 128).  None of them allocates device memory
 * once the device's first call of the library has been made.
 * ====================================================================== */

/* Pair layouts of apex_attn_rope. */
enum {
    APEX_ROPE_INTERLEAVED = 0, /* pairs (2i, 2i+1): the layout of every other entry point */
    APEX_ROPE_HALF = 1         /* pairs (i, i + d_rot/2)                                  */
};

/* Options of apex_attn_rope; all zeros: interleaved, the whole row, base 10000. */
typedef struct apex_rope_options {
    int layout;           /* APEX_ROPE_INTERLEAVED or APEX_ROPE_HALF                     */
    int rot_start;        /* first rotated entry of a row                                */
    int d_rot;            /* rotated entries (even); 0: all from rot_start on            */
    int inverse;          /* non-zero: rotate by -angle (the gradient of the rotation)   */
    float rope_base;      /* base b of theta_i = b^(-2i/d_rot); 0 means 10000            */
    float linear_scale;   /* positions divided by this (> 0); 0 means 1                  */
    float yarn_scale;     /* YaRN factor s as in apex_attn_options; <= 1: none           */
    float yarn_beta_fast; /* 0: 32                                                       */
    float yarn_beta_slow; /* 0: 1                                                        */
} apex_rope_options;

/* One tensor of apex_attn_rope: rows of consecutive entries at in + b * in_b +
 * h * in_h + s * in_s (strides in elements, any order), written to out likewise.
 * out may be in with the same strides (of k and v only without row0).  Otherwise no
 * out may share an element with any in or other out of the call, the rows up to
 * out_rows counted whole with row0, nor hold an element twice.  Views that interleave in
 * one buffer do not; strides that no nesting of dimensions gives may take too long to tell,
 * and are refused then. */
typedef struct apex_rope_tensor {
    const void *in;
    void *out;
    int n_heads;
    int d_row; /* entries per row */
    long long in_b, in_h, in_s;
    long long out_b, out_h, out_s;
} apex_rope_tensor;

/*
 * Rotary positions: rows of q and k turned by their tokens' positions, and v
 * copied beside them.  For every token (b, s) at m = positions[b * pos_stride + s]
 * and every pair (x, y) of a row's rotated part, i = 0 .. d_rot/2 - 1,
 *   (x, y) -> (x cos(m theta_i) - y sin(m theta_i), x sin(m theta_i) + y cos(m theta_i))
 * (Part 1 §4.2-§4.4; YaRN's theta_i of Part 1 §5.3-§5.4), in fp32, rounded once to
 * bf16; the other entries are copied.  Positions are any int32, negative ones
 * included: the angle is reduced exactly, in 64-bit fractions of a turn, so no
 * table is read or grown.
 *
 *   q, k, v     tensors (either may be NULL, not all three); q and k need
 *               rot_start + d_rot <= d_row; v's rows are copied unchanged
 *   positions   [B, S] int32, device (pos_stride elements between sequences, 0: shared)
 *   row0        NULL, or [B] int32, device: token s of k and of v is written at
 *               row row0[b] + s of out (instead of s), e.g. appended to a cache;
 *               rows outside [0, out_rows) are not written
 *   out_rows    rows of k's and v's out (with row0)
 *
 * 1 <= B, S <= 2^24 with B * S < 2^31, d_row <= 1024, d_rot <= 512.  Any strides
 * and element alignment are taken; 16-byte aligned rows with d_rot (half layout:
 * d_rot / 2), rot_start and d_row multiples of 8 run 16 bytes at a time.
 * The YaRN temperature (0.1 ln s + 1) is not applied: it belongs to the scores'
 * scale.
 */
apex_status apex_attn_rope(const apex_rope_tensor *q, const apex_rope_tensor *k, const apex_rope_tensor *v, int B,
                           int S, const int *positions, long long pos_stride, const int *row0, int out_rows,
                           const apex_rope_options *opt, apex_stream_t stream);

/* One tensor of apex_attn_norm_rope or of its gradient: rows of consecutive bf16 entries at
 * x + b * x_b + h * x_h + s * x_s (strides in elements, any order), the result at out
 * likewise.  For the gradient dy is that of the result and out receives x's. */
typedef struct apex_norm_tensor {
    const void *x;
    const void *dy;      /* gradient only                                                    */
    void *out;
    const void *weight;  /* [d_row], or [n_heads][d_row]; NULL: ones                         */
    float *dweight;      /* gradient only: the weights' gradient, shaped as they; NULL: none */
    int n_heads, d_row;
    int weight_f32;      /* weights are fp32 (0: bf16)                                       */
    int weight_per_head; /* non-zero: [n_heads][d_row]                                       */
    long long x_b, x_h, x_s;
    long long dy_b, dy_h, dy_s;
    long long out_b, out_h, out_s;
} apex_norm_tensor;

/*
 * RMS norm of every query and key head (Part 1 §3) and its rotary position in one pass, with
 * v copied beside them.  For a row x of d = d_row entries at position m
 *   y = R_m (x / sqrt(mean(x^2) + eps) * weight)
 * with R_m the rotation of apex_attn_rope (the whole row is normed, the part that *opt names is
 * turned), in fp32, rounded once to bf16.  Positions, row0, out_rows, layouts and limits are
 * those of apex_attn_rope; opt->inverse is not used.  q may not be NULL, k and v may be.  The sum of
 * squares is fp32 too: a row whose sum passes 2^128 comes out as zeros, and under an eps of 0 one whose
 * sum is below 2^-126 loses precision, a row of zeros giving NaN.
 *
 * An out may be its own x with the same strides (of k and v only without row0); otherwise no
 * out may share an element with any x, weight or other out, nor hold one twice.
 * d_row <= 1024, n_heads <= 16384, d_rot <= 512; eps >= 0 and finite.  16-byte aligned rows of
 * up to 512 entries with d_rot (half layout: d_rot / 2), rot_start and d_row multiples of 8 run
 * 16 bytes at a time.
 */
apex_status apex_attn_norm_rope(const apex_norm_tensor *q, const apex_norm_tensor *k, const apex_rope_tensor *v, int B,
                                int S, const int *positions, long long pos_stride, const int *row0, int out_rows,
                                const apex_rope_options *opt, float eps, apex_stream_t stream);

/*
 * Gradients of apex_attn_norm_rope.  With u = x / sqrt(mean(x^2) + eps) and g = R_m^-1 dy
 *   dx      = (g * weight - u * mean(g * weight * u)) / sqrt(mean(x^2) + eps)   to out, bf16
 *   dweight = sum of g * u over all rows (of the head, with weights for each), fp32
 * The sums are made in a fixed order: equal inputs give equal bits.  An out may be its own x
 * or dy with the same strides.
 *   workspace at least apex_attn_norm_rope_grad_workspace_bytes(...) bytes, 16-byte aligned,
 *             owned by the caller, not read before written; calls that may run at the same
 *             time need one each
 */
apex_status apex_attn_norm_rope_grad(const apex_norm_tensor *q, const apex_norm_tensor *k, int B, int S,
                                     const int *positions, long long pos_stride, const apex_rope_options *opt,
                                     float eps, void *workspace, size_t workspace_bytes, apex_stream_t stream);

/* Bytes of workspace apex_attn_norm_rope_grad needs (H_kv, d_k: 0 without k); 0 when the sizes are invalid.
 * Host-only. */
size_t apex_attn_norm_rope_grad_workspace_bytes(int H_q, int H_kv, int d_q, int d_k);

/*
 * Attention of a tree of T drafted tokens per sequence over a cache: every
 * drafted token sees the sequence's cached keys and its own ancestors among the
 * drafts, whose keys and values already sit behind them in the cache.
 *
 *   q         [B, H_q,  T,     d_qk] bf16, read   (rotated)
 *   k_cache   [B, H_kv, S_cap, d_qk] bf16, read   (rotated; rows lens[b] + u: the drafts)
 *   v_cache   [B, H_kv, S_cap, d_v]  bf16, read
 *   out       [B, H_q,  T,     d_v]  bf16, written (must not overlap q or the caches)
 *   lens      [B] int32, device: cached keys before the drafts (taken as
 *             clamped to [0, S_cap]; rows at or past S_cap are not visible)
 *   tree_mask NULL (draft t sees the drafts u <= t), or uint64, device: bit u of
 *             tree_mask[b * mask_stride + t] set <=> draft t sees draft u
 *             (mask_stride 0: one tree for the batch)
 *   positions NULL (draft t at lens[b] + t), or [B, T] int32, device; used with a
 *             window only; a position below lens[b] counts as lens[b]
 *   window    <= 0: none; > 0: cached key j is at position j, draft u at its own,
 *             and a key is seen only if (position of t) - (its position) < window; not
 *             for caches whose rows are elsewhere (after apex_attn_evict, or appended
 *             by apex_attn_rope at rows that are not their positions)
 *   scale     factor of the scores, > 0; 0: 1 / sqrt(d_qk)
 *   workspace at least apex_attn_tree_workspace_bytes(...) bytes, 16-byte aligned,
 *             owned by the caller, not read before written; calls that may run at
 *             the same time need one each
 *
 * 1 <= T <= 64, 1 <= B <= 65536; G = H_q / H_kv as for the other entry points.  A
 * row that sees no key gives zeros.  Cache rows that no draft of the sequence
 * sees (past the drafts, before every window, masked in the whole tree) may hold
 * anything, infinities and NaN included; the values of the others must be finite.
 * Softmax statistics and sums are fp32; the weights are rounded to bf16 for the
 * tensor cores.
 */
apex_status apex_attn_tree_decode(const void *q, const void *k_cache, const void *v_cache, void *out, int B, int H_q,
                                  int H_kv, int T, int S_cap, int d_qk, int d_v, const int *lens,
                                  const uint64_t *tree_mask, long long mask_stride, const int *positions, int window,
                                  float scale, void *workspace, size_t workspace_bytes, apex_stream_t stream);

/*
 * The same under a window whose first n_sink positions stay visible (sinks): with a window > 0 a
 * key is also seen if its position is below n_sink (>= 0).  Workspace as for
 * apex_attn_tree_decode.
 */
apex_status apex_attn_sink_tree_decode(const void *q, const void *k_cache, const void *v_cache, void *out, int B,
                                       int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v, const int *lens,
                                       const uint64_t *tree_mask, long long mask_stride, const int *positions,
                                       int window, int n_sink, float scale, void *workspace, size_t workspace_bytes,
                                       apex_stream_t stream);

/* Bytes of workspace apex_attn_tree_decode needs; 0 when the sizes are invalid.  Host-only. */
size_t apex_attn_tree_workspace_bytes(int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v);

/*
 * Decode (one query per sequence) over a cache of rotated keys that also adds
 * each cached row's attention weight to a running sum:
 *   out[b,h]      = sum_j p[b,h,j] v[b,g,j],   p = softmax over j < lens[b]
 *   acc[b,g,j]   += sum of p[b,h,j] over the G query heads h of KV head g, j < lens[b]
 *
 *   q       [B, H_q,  1,     d_qk] bf16, read (rotated)
 *   k_cache [B, H_kv, S_cap, d_qk] bf16, v_cache [B, H_kv, S_cap, d_v] bf16, read
 *   out     [B, H_q,  1,     d_v]  bf16, written (must not overlap q, the caches or acc)
 *   lens    [B] int32, device (taken as clamped to [0, S_cap]); 0 gives zeros
 *   acc     [B, H_kv, S_cap] fp32, read and written up to lens[b]; rows behind stay
 *   scale   as for apex_attn_tree_decode
 *   workspace at least apex_attn_decode_weights_workspace_bytes(...) bytes, as above
 *
 * Cache rows at or past lens[b] may hold anything.  The sums are made in a fixed
 * order: equal inputs give equal bits.  Statistics, sums and what is added to acc are
 * fp32; the weights are rounded to bf16 for out alone, on the tensor cores.  Most of
 * the workspace holds the scores, 4 bytes for every query head and row of capacity.
 */
apex_status apex_attn_decode_weights(const void *q, const void *k_cache, const void *v_cache, void *out, int B,
                                     int H_q, int H_kv, int S_cap, int d_qk, int d_v, const int *lens, float *acc,
                                     float scale, void *workspace, size_t workspace_bytes, apex_stream_t stream);

/* Bytes of workspace apex_attn_decode_weights needs; 0 when the sizes are invalid.  Host-only. */
size_t apex_attn_decode_weights_workspace_bytes(int B, int H_q, int H_kv, int S_cap, int d_qk, int d_v);

/*
 * Cut every (sequence, KV head) of a cache down to `budget` rows, by position and
 * accumulated attention weight.  Of the rows j < lens[b] it keeps those at
 * positions < n_sink or >= next_pos[b] - n_recent first and then those with the
 * largest acc (ties, and more such positions than the budget: the lowest row; NaN
 * counts as the least weight).  Kept rows below `budget` stay where they are;
 * kept rows at or past it move, in ascending order, into the freed rows below it,
 * in ascending order: attention over rotated keys does not depend on the order of
 * the rows, and so only rows that must move do.  A sequence of lens[b] <= budget
 * keeps everything in place.
 *
 *   k_cache [B, H_kv, S_cap, d_k], v_cache [B, H_kv, S_cap, d_v] bf16, moved in place;
 *           rows at or past min(lens[b], budget) are left as they were
 *   acc, positions      [B, H_kv, S_cap] fp32 / int32, read; positions NULL: row j is
 *                       at position j
 *   acc_out, positions_out  the same shapes, written whole, in the new row order, with
 *                       0 and -1 from row min(lens[b], budget) on; must not overlap
 *                       acc, positions
 *   lens, next_pos      [B] int32; next_pos NULL: lens, or one past the largest of the
 *                       head's positions where that is more (a cache that was cut before)
 *   lens_out            [B] int32, written: min(lens[b], budget); not lens, not next_pos
 *   budget >= 1, n_sink, n_recent >= 0, n_sink + n_recent <= budget
 *   workspace           at least apex_attn_evict_workspace_bytes(...) bytes, as above
 *
 * d_k and d_v: multiples of 8 up to 1024.
 */
apex_status apex_attn_evict(void *k_cache, void *v_cache, int B, int H_kv, int S_cap, int d_k, int d_v,
                            const float *acc, const int *positions, const int *lens, const int *next_pos, int budget,
                            int n_sink, int n_recent, float *acc_out, int *positions_out, int *lens_out,
                            void *workspace, size_t workspace_bytes, apex_stream_t stream);

/* Bytes of workspace apex_attn_evict needs; 0 when the sizes are invalid.  Host-only. */
size_t apex_attn_evict_workspace_bytes(int B, int H_kv, int S_cap, int budget);

/* ======================================================================
 * Caches held in 4 bits.
 *
 * A packed row of d entries is d / 2 bytes of e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives; entry 2i in the low half of byte i) and d / 16 e4m3 scales, one for 16
 * neighbouring entries.  An entry stands for value * scale * factor, where factor is an fp32
 * number of the KV head that the caller chooses (> 0 and finite, best a power of two; no array:
 * 1): e4m3 scales lose precision below 2^-6 and end at 448, so a head's factor should be near
 * its largest entry / 1000.  Packed tensors are dense, [B, H_kv, S_cap, d / 2] and
 * [B, H_kv, S_cap, d / 16] bytes, 16-byte aligned.
 * ====================================================================== */

/* One tensor of apex_attn_append4 and apex_attn_unpack4. */
typedef struct apex_bits4_tensor {
    void *rows;          /* bf16 rows at rows + i_b * b + i_h * h + i_s * s (strides in elements); read by
                            apex_attn_append4, written by apex_attn_unpack4                              */
    void *bytes;         /* [B, H_kv, S_cap, d / 2]                                                      */
    void *scales;        /* [B, H_kv, S_cap, d / 16]                                                     */
    const float *factor; /* [H_kv], device, or NULL: 1                                                   */
    long long b, h, s;
    int d;               /* entries of a row: a multiple of 16 up to 512                                 */
} apex_bits4_tensor;

/*
 * Append keys and values to a 4-bit cache: row s < S of sequence b goes to row row0[b] + s
 * (row0 NULL: s); rows outside [0, S_cap) are dropped, the others of the cache untouched.  For
 * each 16 entries x
 *   scale = e4m3(max |x| / (6 factor)),  value = e2m1(x / (scale * factor))
 * rounded to nearest, ties to even, to at most 448 and 6 (with a factor that is no power of two
 * a quotient within 2^-22 of a tie may go either way); a scale of 0 gives zeros.  16 entries that
 * hold an infinity or a NaN read as NaN.  The packed tensors share no byte with the rows or with
 * one another.  B * H_kv * S < 2^31.
 */
apex_status apex_attn_append4(const apex_bits4_tensor *k, const apex_bits4_tensor *v, int B, int H_kv, int S, int S_cap,
                              const int *row0, apex_stream_t stream);

/*
 * The same rows back as bf16, rounded once (exact for factors that are powers of two); rows
 * outside [0, S_cap) give zeros.  The rows share no element with the packed tensors or with one
 * another.
 */
apex_status apex_attn_unpack4(const apex_bits4_tensor *k, const apex_bits4_tensor *v, int B, int H_kv, int S, int S_cap,
                              const int *row0, apex_stream_t stream);

/*
 * Attention of T new tokens per sequence over a 4-bit cache that holds their own rows too:
 *   m        = lens[b] + t                    position of token t, and its row of the cache
 *   out      = sum_j softmax_j(scale <q, k_j>) v_j   over the rows j < S_cap visible from m:
 *   visible(m, j) <=> j <= m and (window <= 0 or m - j < window or j < n_sink)
 *
 *   q         [B, H_q, T, d_qk] bf16, read (rotated)
 *   k4, k_scale, v4, v_scale  packed tensors, read; keys rotated before they were packed
 *   out       [B, H_q, T, d_v] bf16, written (must not overlap an input)
 *   lens      [B] int32, device: rows before the new tokens' (taken as clamped to [0, S_cap])
 *   n_sink    first rows that stay visible behind a window (>= 0)
 *   k_factor, v_factor  [H_kv], device, or NULL: 1
 *   scale     factor of the scores, > 0; 0: 1 / sqrt(d_qk)
 *   workspace at least apex_attn_decode4_workspace_bytes(...) bytes, 16-byte aligned, owned by
 *             the caller, not read before written; calls that may run at the same time need
 *             one each
 *
 * Row lengths, groups and limits as for apex_attn_tree_decode (1 <= T <= 64).  A row that sees no
 * key gives zeros.  Cache rows that no token of the sequence sees may hold anything; the values of
 * the others and the scores, in fp32, must be finite, and factors from 2^-90 to 2^90.  Queries are
 * held in fp16 relative to their row's largest entry, where entries below 2^-21 of it lose precision;
 * scores, statistics and sums are fp32, weights are rounded to fp16 for the tensor cores, where those
 * below 2^-36 of the largest (with more than 16 rows G * T: 2^-32) vanish.  Equal inputs give equal bits.
 */
apex_status apex_attn_decode4(const void *q, const void *k4, const void *k_scale, const void *v4, const void *v_scale,
                              void *out, int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v, const int *lens,
                              int window, int n_sink, const float *k_factor, const float *v_factor, float scale,
                              void *workspace, size_t workspace_bytes, apex_stream_t stream);

/* Bytes of workspace apex_attn_decode4 needs; 0 when the sizes are invalid.  Host-only. */
size_t apex_attn_decode4_workspace_bytes(int B, int H_q, int H_kv, int T, int S_cap, int d_qk, int d_v);

/*
 * Read and clear the current device's status word, after synchronising the
 * device.  APEX_OK when no kernel recorded a problem since the last call;
 * APEX_ERR_DEVICE_TIMEOUT when a bounded wait gave up; APEX_ERR_CUDA when the
 * synchronisation itself failed.
 */
apex_status apex_attn_device_status(void);

/* Static, human-readable name of a status code (never NULL). */
const char *apex_attn_status_string(apex_status s);

#ifdef __cplusplus
}
#endif

#endif /* APEX_ATTN_H */
