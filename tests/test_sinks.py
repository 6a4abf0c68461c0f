"""Prefill, decode and drafted trees under a window whose first tokens stay visible, against plain 64-bit
attention.

Tolerances (u = 2^-8: half a step of bf16, relative to the value): the rotated queries and keys are
rounded to bf16, each by u relative, so a score moves by at most e = (2 u + u^2) scale sum |q k| over
the worst signs; the sum of d such roundings of either sign stays below 6 standard deviations of u / sqrt(3)
each (a row's largest over n keys: 6 covers n = 2^20), which is what is counted:
  e = 6 (2 u / sqrt 3) scale sqrt(sum (q k)^2) + d 2^-24 scale sum |q k|;
numerators and denominators of the weights move by e: 2 e A, A = sum p |v|, in the sum.  Weights are rounded
to bf16: u A; the result: u |out|; exp2 and sums in fp32: 2^-13 A.  Trees take rotated rows: there
e = d 2^-24 scale sum |q k|.
"""
import math

import pytest
import torch

import transformer_attention_rope_gb300 as apex

U = 2.0 ** -8


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _turn(x, pos, d_r, yarn=1.0):
    """Rows with their last d_r entries turned, interleaved pairs, 64 bits."""
    x = x.double()
    theta = []
    for i in range(d_r // 2):
        th = 10000.0 ** (-2.0 * i / d_r)
        if yarn > 1.0:
            lam = 2 * math.pi / th
            t = min(1.0, max(0.0, (lam - 1.0) / (yarn - 1.0)))
            th = th if lam < 32.0 else th / yarn if lam > yarn else th / (t * yarn + 1 - t)
        theta.append(th)
    ang = pos.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device=x.device)
    y = x.clone()
    a = x.shape[-1] - d_r + 2 * torch.arange(d_r // 2, device=x.device)
    y[..., a] = x[..., a] * ang.cos() - x[..., a + 1] * ang.sin()
    y[..., a + 1] = x[..., a] * ang.sin() + x[..., a + 1] * ang.cos()
    return y


def _ref(q, k, v, q0, window, n_sink, d_r=0, prefix=0, yarn=1.0, turned=False):
    """(out, tolerance)"""
    B, Hq, S, d = q.shape
    Hkv, Sk = k.shape[1:3]
    G = Hq // Hkv
    dev = q.device
    d_rot = d_r or d
    scale = (0.1 * math.log(yarn) + 1 if yarn > 1 else 1) / math.sqrt(d)
    m = q0 + torch.arange(S, device=dev)
    j = torch.arange(Sk, device=dev)
    seen = (j <= m[:, None]) & ((m[:, None] - j < window) | (j < n_sink)) if window > 0 else j <= m[:, None]
    if prefix:
        seen = torch.where((m < prefix)[:, None], j < prefix, seen)
    out = torch.zeros(*q.shape[:3], v.shape[-1], dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    for b in range(B):
        for h in range(Hkv):
            kk = k[b, h].double() if turned else _turn(k[b, h], j, d_rot, yarn)
            vv = v[b, h].double()
            for i in range(h * G, (h + 1) * G):
                x = _turn(q[b, i], m, d_rot, yarn)
                s = (x @ kk.T * scale).masked_fill(~seen, -math.inf)
                p = torch.softmax(s, -1)
                o, A = p @ vv, p @ vv.abs()
                e = 12 * U / math.sqrt(3) * scale * ((x * x) @ (kk * kk).T).sqrt() + d * 2.0 ** -24 * scale * (x.abs() @ kk.abs().T)
                e = e.masked_fill(~seen, 0).amax(-1, keepdim=True)
                out[b, i] = o
                tol[b, i] = U * o.abs() + A * (U + 2 * e + 2.0 ** -13)
    return out, tol


def _close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert torch.isfinite(err).all()
    assert (err <= tol).all(), float((err - tol).max())


def _inputs(dev, seed, B, Hq, Hkv, S, Sk, d, d_r=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    return f(B, Hq, S, d + d_r), f(B, Hkv, Sk, d + d_r), f(B, Hkv, Sk, d)


FWD = [  # B, Hq, Hkv, S, Sk, d, d_r, window, sinks
    (1, 4, 2, 128, 128, 64, 0, 16, 4),
    (1, 4, 2, 700, 700, 64, 0, 100, 1),
    (2, 8, 8, 513, 700, 64, 0, 64, 130),
    (1, 8, 2, 1000, 1000, 128, 0, 128, 4),
    (1, 8, 2, 1000, 1300, 128, 0, 200, 128),
    (2, 16, 1, 300, 1500, 128, 0, 257, 300),
    (1, 2, 2, 1100, 1100, 128, 0, 1, 1),
    (1, 4, 4, 1, 1000, 128, 0, 17, 64),
    (1, 32, 4, 600, 900, 128, 64, 100, 4),
    (1, 4, 2, 500, 500, 128, 64, 33, 200),
    (1, 4, 2, 300, 300, 128, 0, 299, 5000),       # every key is a sink
    (1, 4, 2, 700, 700, 128, 0, 650, 3),          # sinks within the window's reach for most rows
]


@pytest.mark.gpu
@pytest.mark.parametrize("workspace", [None, False])
@pytest.mark.parametrize("B,Hq,Hkv,S,Sk,d,d_r,window,sinks", FWD)
def test_prefill_matches_the_formula(B, Hq, Hkv, S, Sk, d, d_r, window, sinks, workspace):
    dev = _gpu()
    q, k, v = _inputs(dev, S + Sk, B, Hq, Hkv, S, Sk, d, d_r)
    how = dict(window=window, n_sink=sinks, q_pos0=Sk - S, workspace=workspace)
    got = apex.mla_fwd(q, k, v, d_r, **how) if d_r else apex.fwd(q, k, v, **how)
    _close(got, *_ref(q, k, v, Sk - S, window, sinks, d_r))
    assert apex.apex_attn_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_r", [(64, 0), (128, 0), (128, 64)])
def test_keys_rotated_once(d, d_r):
    """The pass that rotates the keys beforehand, and keys that the caller rotated."""
    dev = _gpu()
    q, k, v = _inputs(dev, 3, 1, 8, 1, 700, 700, d, d_r)
    call = (lambda *a, **o: apex.mla_fwd(*a, d_r, **o)) if d_r else apex.fwd
    need = apex.apex_attn_sink_fwd_workspace_bytes
    ref = _ref(q, k, v, 0, 90, 10, d_r)
    turned = apex.mla_rope_keys(k, d_r) if d_r else apex.rope_keys(k)
    _close(call(q, turned, v, window=90, n_sink=10, keys_prerotated=True), *ref)
    # long enough for the cost model to choose the pass
    q, k, v = _inputs(dev, 4, 1, 16, 1, 6000, 6000, d, d_r)
    opt = apex.Options(window=3000)
    n = need(1, 16, 1, 6000, 6000, d, d_r, 5, opt)
    got = call(q, k, v, window=3000, n_sink=5)
    raw = call(q, k, v, window=3000, n_sink=5, workspace=False)
    assert n in (0, k.numel() * 2)
    assert (got.float() - raw.float()).abs().max() <= 2 * U * raw.float().abs().max()


@pytest.mark.gpu
def test_without_a_window_or_sinks_it_is_the_plain_call():
    dev = _gpu()
    for d, d_r in ((64, 0), (128, 0), (128, 64)):
        q, k, v = _inputs(dev, 5, 2, 8, 2, 400, 400, d, d_r)
        call = (lambda *a, **o: apex.mla_fwd(*a, d_r, **o)) if d_r else apex.fwd
        one = (lambda *a, **o: apex.mla_decode(*a, 399, d_r, **o)) if d_r else (lambda *a, **o: apex.decode(*a, 399, **o))
        q1 = q[:, :, -1:].contiguous()
        assert torch.equal(call(q, k, v, n_sink=7), call(q, k, v))
        assert torch.equal(call(q, k, v, window=50, n_sink=0), call(q, k, v, window=50))
        assert torch.equal(one(q1, k, v, n_sink=7), one(q1, k, v))
        # a window that reaches everything, and one that the sinks fill up
        want, tol = _ref(q, k, v, 0, 0, 0, d_r)
        _close(call(q, k, v, window=400, n_sink=7), want, tol)
        _close(call(q, k, v, window=1, n_sink=400), want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_r", [(64, 0), (128, 0), (128, 64)])
def test_prefix_and_yarn(d, d_r):
    dev = _gpu()
    q, k, v = _inputs(dev, 6, 1, 8, 2, 600, 600, d, d_r)
    call = (lambda *a, **o: apex.mla_fwd(*a, d_r, **o)) if d_r else apex.fwd
    got = call(q, k, v, window=70, n_sink=150, prefix_len=40, yarn_scale=16.0)
    _close(got, *_ref(q, k, v, 0, 70, 150, d_r, prefix=40, yarn=16.0))


DECODE = [  # B, Hq, Hkv, Sk, q_pos, d, d_r, window, sinks
    (1, 4, 2, 1, 0, 64, 0, 16, 4),
    (3, 8, 8, 700, 699, 64, 0, 100, 1),
    (2, 32, 8, 3000, 2999, 128, 0, 1024, 4),
    (2, 32, 8, 3000, 1500, 128, 0, 64, 200),
    (1, 16, 1, 5000, 4990, 128, 0, 1, 64),
    (2, 8, 2, 1000, 130, 128, 0, 128, 4),
    (2, 8, 2, 1000, 999, 128, 64, 100, 65),
    (1, 4, 2, 900, 899, 128, 0, 300, 900),
]


@pytest.mark.gpu
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Sk,at,d,d_r,window,sinks", DECODE)
def test_decode_matches_the_formula(B, Hq, Hkv, Sk, at, d, d_r, window, sinks, turned):
    dev = _gpu()
    q, k, v = _inputs(dev, Sk + at, B, Hq, Hkv, 1, Sk, d, d_r)
    if turned:
        k = apex.mla_rope_keys(k, d_r) if d_r else apex.rope_keys(k)
    how = dict(window=window, n_sink=sinks, keys_prerotated=turned)
    got = apex.mla_decode(q, k, v, at, d_r, **how) if d_r else apex.decode(q, k, v, at, **how)
    ref = _ref(q, k, v, at, window, sinks, d_r, turned=turned)
    err = (got.double() - ref[0]).abs()
    assert (err <= ref[1]).all(), float((err - ref[1]).max())


TREES = [  # Hq, Hkv, T, dk, dv, cap, lens, window, sinks
    (4, 2, 1, 64, 64, 300, [299, 5, 0], 16, 4),
    (32, 8, 1, 128, 128, 1500, [1400, 300, 60], 128, 4),
    (32, 8, 4, 128, 128, 1500, [1400, 130, 3], 1, 1),
    (8, 2, 6, 192, 128, 900, [890, 255], 70, 300),
    (16, 1, 12, 128, 128, 1300, [1288, 700, 2], 100, 130),   # CTA pairs, one M tile
    (16, 1, 40, 128, 128, 2000, [1960, 20], 300, 5),         # two
    (16, 1, 20, 192, 128, 900, [880, 500], 129, 64),
    (16, 1, 12, 64, 64, 1000, [988, 400], 33, 140),          # two M tiles on one CTA
    (8, 1, 64, 64, 64, 700, [636, 10], 20, 3),
]


@pytest.mark.gpu
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Hq,Hkv,T,dk,dv,cap,lens,window,sinks", TREES)
def test_drafts_match_the_formula(Hq, Hkv, T, dk, dv, cap, lens, window, sinks, tree):
    dev = _gpu()
    g = torch.Generator(device=dev)
    g.manual_seed(cap + T)
    B, G = len(lens), Hq // Hkv
    q, k, v = (torch.randn(B, h, n, d, generator=g, device=dev).to(torch.bfloat16)
               for h, n, d in ((Hq, T, dk), (Hkv, cap, dk), (Hkv, cap, dv)))
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    mask = pos = None
    words = [(1 << (t + 1)) - 1 for t in range(T)]
    depth = list(range(T))
    if tree:  # every draft but the first hangs on one a little before it
        for t in range(1, T):
            p = max(0, t - 1 - t % 3)
            words[t], depth[t] = words[p] | (1 << t), depth[p] + 1
        mask = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device=dev)
        pos = ln[:, None] + torch.tensor(depth, dtype=torch.int32, device=dev)
    # rows that nobody sees may hold anything
    j = torch.arange(cap, device=dev)
    seen = torch.zeros(B, T, cap, dtype=torch.bool, device=dev)
    for b, n in enumerate(lens):
        at = j.clone()
        at[n:n + T] = n + torch.tensor(depth, device=dev)[:cap - n]
        for t in range(T):
            m = n + depth[t]
            draft = torch.zeros(cap, dtype=torch.bool, device=dev)
            for u in range(min(T, cap - n)):
                draft[n + u] = bool((words[t] >> u) & 1)
            seen[b, t] = ((j < n) | draft) & ((m - at < window) | (at < sinks))
        hidden = ~seen[b].any(0)
        k[b, :, hidden] = float("nan")
        v[b, :, hidden] = float("inf")
    got = apex.tree_decode(q, k, v, ln, tree_mask=mask, positions=pos, window=window, n_sink=sinks)
    scale = 1 / math.sqrt(dk)
    for b in range(B):
        for h in range(Hq):
            x, kk, vv = q[b, h].double(), k[b, h // G].double().nan_to_num(0.0), v[b, h // G].double().nan_to_num(0.0, 0.0, 0.0)
            s = (x @ kk.T * scale).masked_fill(~seen[b], -math.inf)
            p = torch.softmax(s, -1).nan_to_num(0.0)
            o, A = p @ vv, p @ vv.abs()
            e = (dk * 2.0 ** -24 * scale * (x.abs() @ kk.abs().T)).masked_fill(~seen[b], 0).amax(-1, keepdim=True)
            err = (got[b, h].double() - o).abs()
            assert torch.isfinite(err).all()
            assert (err <= U * o.abs() + A * (U + 2 * e + 2.0 ** -13)).all()
    assert apex.apex_attn_device_status() == 0


@pytest.mark.gpu
def test_drafts_without_a_window_are_the_plain_call():
    dev = _gpu()
    q, k, v = _inputs(dev, 11, 2, 8, 2, 5, 600, 128)
    ln = torch.tensor([590, 77], dtype=torch.int32, device=dev)
    assert torch.equal(apex.tree_decode(q, k, v, ln, n_sink=9), apex.tree_decode(q, k, v, ln))
    # a window that sinks fill up
    assert torch.equal(apex.tree_decode(q, k, v, ln, window=1, n_sink=600), apex.tree_decode(q, k, v, ln))
    with pytest.raises(ValueError):
        apex.tree_decode(q, k, v, ln, window=8, n_sink=-1)


@pytest.mark.gpu
def test_prompt_then_tokens():
    """Chunks of a prompt and then single tokens give the rows of one call over all."""
    dev = _gpu()
    S, window, sinks = 700, 150, 6
    q, k, v = _inputs(dev, 8, 2, 8, 2, S, S, 128)
    ref, tol = _ref(q, k, v, 0, window, sinks)
    _close(apex.fwd(q, k, v, window=window, n_sink=sinks), ref, tol)
    for lo, hi in ((0, 300), (300, 301), (301, 650)):
        got = apex.fwd(q[:, :, lo:hi].contiguous(), k[:, :, :hi].contiguous(), v[:, :, :hi].contiguous(), window=window,
                       n_sink=sinks, q_pos0=lo)
        assert ((got.double() - ref[:, :, lo:hi]).abs() <= tol[:, :, lo:hi]).all()
    for at in (650, 651, 699):
        got = apex.decode(q[:, :, at:at + 1].contiguous(), k, v, at, window=window, n_sink=sinks)
        assert ((got.double() - ref[:, :, at:at + 1]).abs() <= tol[:, :, at:at + 1]).all()


@pytest.mark.gpu
def test_captured_and_replayed():
    dev = _gpu()
    q, k, v = _inputs(dev, 9, 1, 8, 2, 600, 600, 128)
    q1 = q[:, :, -1:].contiguous()
    ws = torch.empty(apex.decode_workspace_bytes(1, 8, 2, 600, 128), dtype=torch.uint8, device=dev)

    def calls():
        return (apex.fwd(q, k, v, window=100, n_sink=4, workspace=False),
                apex.decode(q1, k, v, 599, window=100, n_sink=4, workspace=ws))

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for _ in range(2):
        for x in (q, k, v, q1):
            x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, calls()))


# ------------------------------------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    try:
        return apex.load_library()
    except RuntimeError:
        pytest.skip("library not built")


P = 1 << 20  # an aligned address that a refused call never touches
BAD, UNSUPPORTED = 1, 2

REFUSED = [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(q=P + 2), BAD),
    (dict(out=P + 8), BAD), (dict(n_sink=-1), BAD), (dict(d_r=-64), BAD), (dict(d_r=63), BAD),
    (dict(d_r=32), UNSUPPORTED), (dict(d=64, d_r=64), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(H_kv=3), BAD),
    (dict(B=0), BAD), (dict(opt=dict(rope_base=-1.0)), BAD),
]


@pytest.mark.parametrize("o,code", REFUSED + [(dict(ws=P + 8), BAD), (dict(S=0), BAD), (dict(S=65), BAD),
                                              (dict(opt=dict(prefix_len=65)), BAD), (dict(opt=dict(q_pos=-1)), BAD)])
def test_prefill_refuses(lib, o, code):
    a = dict(q=P, k=P, v=P, out=2 * P, B=1, H_q=8, H_kv=2, S=64, Sk=64, d=128, d_r=0, n_sink=4, ws=None, n=0, opt={})
    a.update(o)
    opt = apex.Options(**dict(dict(window=16), **a["opt"]))
    assert apex.apex_attn_sink_fwd(a["q"], a["k"], a["v"], a["out"], a["B"], a["H_q"], a["H_kv"], a["S"], a["Sk"], a["d"],
                                   a["d_r"], a["n_sink"], opt, a["ws"], a["n"], None) == code
    assert apex.apex_attn_sink_fwd(P, P, P, 2 * P, 1, 8, 2, 64, 64, 128, 0, 4, None, None, 0, None) == BAD


@pytest.mark.parametrize("o,code", REFUSED + [(dict(ws=None), BAD), (dict(ws=P + 8), BAD), (dict(n=15), BAD),
                                              (dict(opt=dict(q_pos=64)), BAD), (dict(opt=dict(q_pos=-1)), BAD)])
def test_decode_refuses(lib, o, code):
    a = dict(q=P, k=P, v=P, out=2 * P, B=1, H_q=8, H_kv=2, Sk=64, d=128, d_r=0, n_sink=4, ws=P, n=1 << 40, opt={})
    a.update(o)
    opt = apex.Options(**dict(dict(window=16), **a["opt"]))
    assert apex.apex_attn_sink_decode(a["q"], a["k"], a["v"], a["out"], a["B"], a["H_q"], a["H_kv"], a["Sk"], a["d"],
                                      a["d_r"], a["n_sink"], opt, a["ws"], a["n"], None) == code


def test_drafts_refuse(lib):
    call = lambda n_sink, window, q=P: apex.apex_attn_sink_tree_decode(  # noqa: E731
        q, P, P, 8 * P, 1, 8, 2, 4, 64, 128, 128, P, None, 0, None, window, n_sink, 0.0, P, 1 << 40, None)
    assert call(-1, 16) == BAD and call(-1, 0) == BAD and call(4, 16, None) == BAD


def test_workspace_bytes(lib):
    opt, plain = apex.Options(window=4096), apex.apex_attn_fwd_workspace_bytes
    sized = apex.apex_attn_sink_fwd_workspace_bytes
    assert sized(1, 32, 8, 65536, 65536, 128, 0, 64, opt) == plain(1, 32, 8, 65536, 65536, 128, opt) > 0
    assert sized(1, 32, 8, 65536, 65536, 128, 0, -1, opt) == 0 and sized(1, 32, 8, 64, 64, 128, 0, 4, None) == 0
    assert sized(1, 32, 8, 64, 65, 128, -64, 4, opt) == 0 and sized(1, 32, 8, 64, 64, 64, 64, 4, opt) == 0


@pytest.mark.gpu
def test_conveniences_refuse():
    dev = _gpu()
    q, k, v = _inputs(dev, 10, 1, 4, 2, 64, 64, 128)
    for bad in (lambda: apex.fwd(q, k, v, window=8, n_sink=-1), lambda: apex.decode(q[:, :, :1].contiguous(), k, v, 63, window=8, n_sink=-2)):
        with pytest.raises(ValueError):
            bad()
    # tensors that do not belong together: nothing is launched
    k1, k2, long = k[:, :1].contiguous(), torch.cat([k, k]), torch.cat([k, k], dim=2)
    one = q[:, :, :1].contiguous()
    for bad in ((q, k1, v), (q, k, k1), (q, k2, v), (q, k, k2), (q, long, v), (q, k, v[..., :64].contiguous())):
        with pytest.raises(ValueError):
            apex.fwd(*bad, window=8, n_sink=2)
        with pytest.raises(ValueError):
            apex.decode(one, *bad[1:], 63, window=8, n_sink=2)
    with pytest.raises(ValueError):
        apex.fwd(q, k, v, window=8, n_sink=2, out=torch.empty_like(k))
    with pytest.raises(ValueError):
        apex.decode(one, k, v, 63, window=8, n_sink=2, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(apex.ApexError):
        apex.decode(one, k, v, 63, window=8, n_sink=2, workspace=torch.empty(16, dtype=torch.uint8, device=dev))


@pytest.mark.gpu
def test_a_window_past_32_bits_is_none():
    dev = _gpu()
    q, k, v = _inputs(dev, 11, 1, 4, 2, 300, 300, 128)
    wide = 2 ** 32 + 5
    assert torch.equal(apex.fwd(q, k, v, window=wide, n_sink=3), apex.fwd(q, k, v, window=300, n_sink=3))
    one = q[:, :, -1:].contiguous()
    assert torch.equal(apex.decode(one, k, v, 299, window=wide, n_sink=3), apex.decode(one, k, v, 299))


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_r", [(128, 0), (128, 64)])
def test_on_another_stream(d, d_r):
    """Inputs made on a stream that the call is given, with the allocator busy on both."""
    dev = _gpu()
    S, window, sinks = 1200, 300, 4
    made = _inputs(dev, 12, 1, 16, 2, S, S, d, d_r)
    ref, tol = _ref(*made, 0, window, sinks, d_r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            q, k, v = (x.clone() for x in made)
            q1 = q[:, :, -1:].contiguous()
        if d_r:
            out = apex.mla_fwd(q, k, v, d_r, window=window, n_sink=sinks, stream=side)
            one = apex.mla_decode(q1, k, v, S - 1, d_r, window=window, n_sink=sinks, stream=side)
        else:
            out = apex.fwd(q, k, v, window=window, n_sink=sinks, stream=side)
            one = apex.decode(q1, k, v, S - 1, window=window, n_sink=sinks, stream=side)
        junk = [torch.full((1 << 22,), float("nan"), device=dev) for _ in range(4)]  # over memory that is free
        side.synchronize()
        _close(out, ref, tol)
        assert ((one.double() - ref[:, :, -1:]).abs() <= tol[:, :, -1:]).all()
        del junk


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_r,S", [(128, 0, 2100), (128, 64, 2100), (128, 64, 6000)])
def test_a_workspace_of_the_callers(d, d_r, S):
    """Keys rotated once into a caller's workspace of the bytes that are asked for, in a captured call."""
    dev = _gpu()
    B, Hq, Hkv, window, sinks = 1, 32, 2, 700, 4
    q, k, v = _inputs(dev, 14, B, Hq, Hkv, S, S, d, d_r)
    if d_r:
        need = apex.mla_fwd_workspace_bytes(B, Hq, Hkv, S, S, d, d_r, window=window, n_sink=sinks)
        call = lambda ws: apex.mla_fwd(q, k, v, d_r, window=window, n_sink=sinks, workspace=ws)  # noqa: E731
    else:
        need = apex.fwd_workspace_bytes(B, Hq, Hkv, S, S, d, window=window, n_sink=sinks)
        call = lambda ws: apex.fwd(q, k, v, window=window, n_sink=sinks, workspace=ws)  # noqa: E731
    # short prompts of decoupled rows are cheaper without the pass
    assert need == (0 if d_r and S < 3000 else B * Hkv * S * (d + d_r) * 2)
    assert apex.fwd_workspace_bytes(B, Hq, Hkv, S, S, d, window=0, n_sink=sinks) == \
        apex.fwd_workspace_bytes(B, Hq, Hkv, S, S, d)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev) if need else False
    ref, tol = _ref(q, k, v, 0, window, sinks, d_r)
    _close(call(ws), ref, tol)
    if need:
        with pytest.raises(apex.ApexError):
            call(ws[:-16])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(ws)
    k.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call(None))


@pytest.mark.gpu
def test_sinks_and_drafts_past_the_capacity():
    """Drafts stand at positions of any size; those below n_sink stay visible, whatever rows the cache has."""
    dev = _gpu()
    T, cap, window = 5, 200, 4
    q, k, v = _inputs(dev, 15, 2, 8, 2, T, cap, 128)
    ln = torch.tensor([0, 150], dtype=torch.int32, device=dev)
    at = torch.tensor([1000, 1010, 1020, 1021, 1 << 25], dtype=torch.int32)
    for sinks in (3, 190, 1010, 1021, 2 ** 25, 2 ** 31 - 1, 2 ** 40):
        got = apex.tree_decode(q, k, v, ln, positions=at.expand(2, T).contiguous().to(dev), window=window, n_sink=sinks)
        for b, n in enumerate(ln.tolist()):
            pos = torch.cat([torch.arange(n), at.long()]).to(dev)  # of the rows: cached ones, drafts
            m = at.long().to(dev)[:, None]
            row = torch.arange(n + T, device=dev)
            seen = (row <= n + torch.arange(T, device=dev)[:, None]) & ((m - pos < window) | (pos < sinks))
            for h in range(8):
                x, kk, vv = q[b, h].double(), k[b, h // 4, :n + T].double(), v[b, h // 4, :n + T].double()
                s = (x @ kk.T / math.sqrt(128)).masked_fill(~seen, -math.inf)
                p = torch.softmax(s, -1)
                e = (2.0 ** -17 / math.sqrt(128) * (x.abs() @ kk.abs().T)).masked_fill(~seen, 0).amax(-1, keepdim=True)
                o, A = p @ vv, p @ vv.abs()
                err = (got[b, h].double() - o).abs()
                assert (err <= U * o.abs() + A * (U + 2 * e + 2.0 ** -13)).all(), sinks


@pytest.mark.gpu
def test_without_sinks_a_window_past_32_bits_is_none_too():
    dev = _gpu()
    for d, d_r in ((128, 0), (128, 64)):
        q, k, v = _inputs(dev, 16, 1, 4, 2, 300, 300, d, d_r)
        one = q[:, :, -1:].contiguous()
        call = (lambda **o: apex.mla_fwd(q, k, v, d_r, **o)) if d_r else lambda **o: apex.fwd(q, k, v, **o)
        dec = (lambda **o: apex.mla_decode(one, k, v, 299, d_r, **o)) if d_r else lambda **o: apex.decode(one, k, v, 299, **o)
        for window in (2 ** 32 + 5, 2 ** 31, 5 - 2 ** 32, -1):
            for f in (call, dec):
                assert torch.equal(f(window=window), f()), window
                assert torch.equal(f(window=window, n_sink=3), f()), window
        with pytest.raises(ValueError):
            call(q_pos0=2 ** 32)
        with pytest.raises(ValueError):
            call(prefix_len=2 ** 32, window=8, n_sink=2)
    with pytest.raises(ValueError):
        apex.decode(one[..., :128].contiguous(), k[..., :128].contiguous(), v, 2 ** 32 + 5)
    with pytest.raises(ValueError):
        apex.rope_keys(v, pos0=2 ** 32)


def test_integers_past_32_bits_are_refused(lib):
    with pytest.raises(ValueError):
        apex.fwd_workspace_bytes(1, 16, 1, 6000, 6000, 128, q_pos0=2 ** 32)
    with pytest.raises(ValueError):
        apex.mla_fwd_workspace_bytes(1, 16, 1, 6000, 6000, 128, 64, prefix_len=2 ** 32, window=100, n_sink=3)
    for window in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 5 - 2 ** 32):
        assert apex.fwd_workspace_bytes(1, 16, 1, 6000, 6000, 128, window=window) == \
            apex.fwd_workspace_bytes(1, 16, 1, 6000, 6000, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_r", [(128, 0), (128, 64)])
@pytest.mark.parametrize("sinks", [0, 4])
def test_a_call_on_another_stream_keeps_off_the_current_ones_memory(d, d_r, sinks):
    """Outputs and workspaces of a call that waits on its stream: what the current stream allocates and writes
    meanwhile stays as it is, and so do they."""
    dev = _gpu()
    S, window = 6000, 3000
    q, k, v = _inputs(dev, 17, 1, 16, 1, S, S, d, d_r)
    q1 = q[:, :, -1:].contiguous()
    how = dict(window=window, n_sink=sinks)

    def calls(**at):
        if d_r:
            return [apex.mla_fwd(q, k, v, d_r, **how, **at), apex.mla_decode(q1, k, v, S - 1, d_r, **how, **at),
                    apex.mla_rope_keys(k, d_r, **at)]
        return [apex.fwd(q, k, v, **how, **at), apex.decode(q1, k, v, S - 1, **how, **at), apex.rope_keys(k, **at)]
    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    got = calls(stream=side)
    junk = [torch.full((n,), 7, dtype=torch.uint8, device=dev) for n in (k.numel() * 2, 1 << 20, 1 << 21, 1 << 22) for _ in "ab"]
    side.synchronize()
    assert all(bool((x == 7).all()) for x in junk)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [0, 2])
def test_tensors_that_do_not_belong_together_are_refused(sinks):
    """Nothing is launched; without sinks as with them."""
    dev = _gpu()
    how = dict(window=8, n_sink=sinks)
    for d, d_r in ((128, 0), (128, 64)):
        q, k, v = _inputs(dev, 18, 2, 4, 2, 64, 64, d, d_r)
        one = q[:, :, :1].contiguous()
        fwd = (lambda *a, **o: apex.mla_fwd(*a, d_r, **how, **o)) if d_r else lambda *a, **o: apex.fwd(*a, **how, **o)
        dec = (lambda q, k, v, **o: apex.mla_decode(q, k, v, 63, d_r, **how, **o)) if d_r else \
            lambda q, k, v, **o: apex.decode(q, k, v, 63, **how, **o)
        k1, v1, k_long, v_long = k[:, :1].contiguous(), v[:, :1].contiguous(), torch.cat([k, k], 2), torch.cat([v, v], 2)
        for bad in ((k1, v), (k, v1), (k[:1], v), (k, v[:1]), (k_long, v), (k, v_long), (k, v[..., :64].contiguous()),
                    (k[..., :64].contiguous(), v)):
            with pytest.raises(ValueError):
                fwd(q, *bad)
            with pytest.raises(ValueError):
                dec(one, *bad)
        with pytest.raises(ValueError):
            fwd(q, k, v, out=torch.empty_like(v))
        with pytest.raises(ValueError):
            dec(one, k, v, out=torch.empty(2, 4, 1, 64, dtype=torch.bfloat16, device=dev))
        for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, 2, dtype=torch.uint8, device=dev)[:, 0]):
            with pytest.raises(ValueError):
                dec(one, k, v, workspace=ws)
            if not sinks:
                with pytest.raises(ValueError):
                    fwd(q, k, v, workspace=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_r,Hq,Hkv,S,window", [(64, 0, 32, 2, 2100, 700), (128, 0, 32, 2, 2100, 700), (128, 64, 16, 1, 6000, 3000)])
def test_the_pass_that_rotates_keys_matches_the_formula(d, d_r, Hq, Hkv, S, window):
    """Sizes at which the pass runs, with it and without."""
    dev = _gpu()
    sinks = 5
    assert apex.apex_attn_sink_fwd_workspace_bytes(1, Hq, Hkv, S, S, d, d_r, sinks, apex.Options(window=window)) == \
        Hkv * S * (d + d_r) * 2
    q, k, v = _inputs(dev, 19, 1, Hq, Hkv, S, S, d, d_r)
    ref = _ref(q, k, v, 0, window, sinks, d_r)
    for ws in (None, False):
        how = dict(window=window, n_sink=sinks, workspace=ws)
        _close(apex.mla_fwd(q, k, v, d_r, **how) if d_r else apex.fwd(q, k, v, **how), *ref)
