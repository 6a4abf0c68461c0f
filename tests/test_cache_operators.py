"""Operators over caches of rotated keys -- rope, tree_decode, decode_weights, evict --
against plain 64-bit implementations, at the sizes and masks where they can go wrong.

Tolerances (u = 2^-8: half a step of bf16, relative to the value; fp32 half a step 2^-24):
  rope     one rounding to bf16, u |y|; the angle is off by under 2^-24 half turns and each
           sine and cosine by a few 2^-24, so both products together by (|x| + |y|) 2^-21.
  out      the weights are rounded to bf16, so the sum moves by at most u A, A = sum p |v|; the
           result is rounded, u |out|.  A score is a sum of d products of bf16 values, exact in
           fp32 but for d additions: off by at most e = d 2^-24 sum |q k| scale, and scaled once
           more; a weight's numerator and denominator move by e^(2e), 2 e A in the sum.  exp2 and the
           sums of weights in fp32 (blocks of 128 keys added one after another): 2^-13 A at
           most for the lengths here.
  acc      the same without roundings to bf16: w (2 e + 2^-13) and two additions, 2^-23 |acc|.
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


def _gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _normal(g, dev, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=dev) * scale).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------- rope
def _theta(d_rot, base=10000.0, linear=1.0, yarn=1.0, fast=32.0, slow=1.0):
    out = []
    for i in range(d_rot // 2):
        th = base ** (-2.0 * i / d_rot)
        if yarn > 1.0:
            lam = 2.0 * math.pi / th
            if lam > slow * yarn:
                div = yarn
            else:
                t = min(1.0, max(0.0, (lam / slow - 1.0) / (yarn - 1.0)))
                div = t * yarn + 1.0 - t
            th = th if lam < fast else th / div
        out.append(th / linear)
    return torch.tensor(out, dtype=torch.float64)


def _rope_ref(x, positions, half=False, rot_start=0, d_rot=None, inverse=False, **freq):
    """x [B,H,S,d] -> (rotated, bound on what fp32 loses) in 64 bits; positions [B,S]."""
    d_rot = x.shape[-1] - rot_start if d_rot is None else d_rot
    x = x.double().cpu()
    ang = positions.double().cpu()[:, None, :, None] * _theta(d_rot, **freq)
    if inverse:
        ang = -ang
    n = d_rot // 2
    a = rot_start + torch.arange(n) * (1 if half else 2)
    b = a + (n if half else 1)
    y, slack = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * ang.cos() - x[..., b] * ang.sin()
    y[..., b] = x[..., a] * ang.sin() + x[..., b] * ang.cos()
    slack[..., a] = slack[..., b] = (x[..., a].abs() + x[..., b].abs()) * 2.0 ** -21
    return y, slack


def _rope_close(got, ref, slack):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(err).all()
    assert (err <= U * ref.abs() + slack).all(), float((err - U * ref.abs() - slack).max())


ROPE = [  # B, S, Hq, Hkv, d, options
    (1, 1, 4, 2, 64, {}),
    (3, 7, 8, 8, 128, dict(half=True)),
    (2, 33, 5, 1, 192, dict(rot_start=128, d_rot=64)),
    (2, 5, 16, 2, 128, dict(d_rot=32, half=True, base=500000.0)),
    (1, 300, 64, 8, 128, dict(linear=4.0)),
    (2, 9, 3, 1, 80, dict(d_rot=20, half=True)),         # halves of ten: pair by pair
    (2, 9, 3, 1, 66, dict(rot_start=6, d_rot=18)),       # nothing on 16 bytes
    (1, 4, 2, 2, 8, {}),
    (2, 40, 8, 2, 128, dict(yarn=32.0)),
    (2, 40, 8, 2, 128, dict(yarn=16.0, fast=8.0, slow=2.0, half=True)),
    (1, 3, 40, 40, 256, dict(half=True)),
    (1, 2, 200, 100, 64, {}),                            # more heads than head groups
    (1, 3, 2, 1, 1024, dict(d_rot=512, half=True, rot_start=256)),  # the widest row
    (2, 2, 1, 1, 1024, dict(d_rot=510)),
]


def _rope_call(dev, q, k, positions, o, **more):
    names = dict(base="rope_base", linear="linear_scale", yarn="yarn_scale", fast="yarn_beta_fast",
                 slow="yarn_beta_slow")
    how = {names.get(n, n): x for n, x in o.items() if n != "half"}
    return apex.rope(q, k, positions=positions, layout="half" if o.get("half") else "interleaved", **how, **more)


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hkv,d,o", ROPE)
def test_rope_matches_the_formula(B, S, Hq, Hkv, d, o, inverse):
    dev = _gpu()
    g = _gen(dev, 10 * S + d)
    q, k = _normal(g, dev, B, Hq, S, d), _normal(g, dev, B, Hkv, S, d)
    pos = torch.randint(0, 5000, (B, S), generator=g, device=dev, dtype=torch.int32)
    got = _rope_call(dev, q, k, pos, o, inverse=inverse)
    for x, y in zip((q, k), got):
        _rope_close(y, *_rope_ref(x, pos, inverse=inverse, **o))


@pytest.mark.gpu
@pytest.mark.parametrize("half", [False, True])
def test_rope_positions_far_negative_and_shared(half):
    dev = _gpu()
    g = _gen(dev, 3)
    q = _normal(g, dev, 2, 4, 6, 128)
    lay = "half" if half else "interleaved"
    pos = torch.tensor([0, -1, 131071, 2 ** 24 - 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev)
    got = apex.rope(q, positions=pos, layout=lay)
    # theta carries 2^-53 of its value: the angle of position 2^31 is off by up to 2^-22
    ref, slack = _rope_ref(q, pos[None].expand(2, 6), half=half)
    far = pos.double().abs().cpu()[None, None, :, None] * 2.0 ** -52
    _rope_close(got, ref, slack * (1 + far * 2.0 ** 21))


@pytest.mark.gpu
@pytest.mark.parametrize("half", [False, True])
def test_rope_strides_and_in_place(half):
    dev = _gpu()
    g = _gen(dev, 4)
    lay = "half" if half else "interleaved"
    B, S, H, d = 2, 19, 6, 128
    pos = torch.randint(0, 999, (B, S), generator=g, device=dev, dtype=torch.int32)
    x = _normal(g, dev, B, S, H, d)
    ref, slack = _rope_ref(x.transpose(1, 2), pos, half=half)
    _rope_close(apex.rope(x.transpose(1, 2), positions=pos, layout=lay), ref, slack)
    # from one fused projection [B, S, (H + 2) d + 1], whose rows are not on 16 bytes
    fused = torch.zeros(B, S, (H + 2) * d + 1, dtype=torch.bfloat16, device=dev)
    view = fused[..., d + 1:d + 1 + H * d].view(B, S, H, d).transpose(1, 2)
    view.copy_(x.transpose(1, 2))
    before = fused.clone()
    apex.rope(view, positions=pos, layout=lay, q_out=view)  # in place
    _rope_close(view, ref, slack)
    keep = torch.ones_like(fused, dtype=torch.bool)
    keep[..., d + 1:d + 1 + H * d] = False
    assert torch.equal(fused[keep], before[keep])
    y = x.clone()
    apex.rope(y.transpose(1, 2), positions=pos, layout=lay, q_out=y.transpose(1, 2))
    _rope_close(y.transpose(1, 2), ref, slack)


@pytest.mark.gpu
def test_rope_appends_to_a_cache():
    dev = _gpu()
    g = _gen(dev, 5)
    B, S, Hq, Hkv, cap = 4, 5, 8, 2, 40
    q, k, v = _normal(g, dev, B, Hq, S, 192), _normal(g, dev, B, Hkv, S, 192), _normal(g, dev, B, Hkv, S, 128)
    kc, vc = _normal(g, dev, B, Hkv, cap, 192), _normal(g, dev, B, Hkv, cap, 128)
    row0 = [0, 17, cap - 2, -3]  # the third loses its tail, the fourth its head
    pos = torch.randint(0, 9999, (B, S), generator=g, device=dev, dtype=torch.int32)
    kr, sl = _rope_ref(k, pos, rot_start=128, d_rot=64)
    want_k, want_v, slack = kc.double().cpu(), vc.double().cpu(), torch.zeros(B, Hkv, cap, 192, dtype=torch.float64)
    for b in range(B):
        for s in range(S):
            r = row0[b] + s
            if 0 <= r < cap:
                want_k[b, :, r], slack[b, :, r], want_v[b, :, r] = kr[b, :, s], sl[b, :, s], v[b, :, s].double().cpu()
    qo, ko, vo = apex.rope(q, k, v, positions=pos, rot_start=128, d_rot=64, k_out=kc, v_out=vc,
                           row0=torch.tensor(row0, dtype=torch.int32, device=dev))
    assert ko is kc and vo is vc
    _rope_close(qo, *_rope_ref(q, pos, rot_start=128, d_rot=64))
    _rope_close(kc, want_k, slack)
    assert torch.equal(vc.double().cpu(), want_v)


@pytest.mark.gpu
def test_rope_gradient_is_the_inverse():
    """<rope(x), g> = <x, rope^-1(g)>, and differences of the formula along a direction."""
    dev = _gpu()
    g = _gen(dev, 6)
    x, up = _normal(g, dev, 1, 2, 9, 64), _normal(g, dev, 1, 2, 9, 64)
    pos = torch.arange(9, dtype=torch.int32, device=dev)[None] * 37
    grad = apex.rope(up, positions=pos, layout="half", inverse=True).double().cpu()
    y, _ = _rope_ref(x, pos, half=True)
    for trial in range(3):
        way = torch.randn(x.shape, generator=torch.Generator().manual_seed(trial), dtype=torch.float64)
        moved, _ = _rope_ref((x.double().cpu() + way), pos, half=True)  # linear: a whole step is exact
        diff = ((moved - y) * up.double().cpu()).sum()
        # every entry of grad is rounded once
        assert abs(diff - (grad * way).sum()) <= (U * grad.abs() * way.abs()).sum() * 1.01


@pytest.mark.gpu
def test_rope_agrees_with_the_rotation_of_cached_keys():
    dev = _gpu()
    g = _gen(dev, 7)
    for d, d_r in ((64, 0), (128, 0), (192, 64)):
        k = _normal(g, dev, 2, 3, 50, d)
        pos = 1000 + torch.arange(50, dtype=torch.int32, device=dev)
        if d_r:
            a = apex.mla_rope_keys(k, d_r, pos0=1000, yarn_scale=8.0)
            b = apex.rope(k, positions=pos, rot_start=d - d_r, yarn_scale=8.0)
        else:
            a, b = apex.rope_keys(k, pos0=1000, yarn_scale=8.0), apex.rope(k, positions=pos, yarn_scale=8.0)
        # each is within u of the formula
        assert ((a.double() - b.double()).abs() <= 2 * U * b.double().abs() + 1e-5).all()


# ------------------------------------------------------------------------------------------------- attention
def _attn_ref(q, k, v, lens, drafts, mask=None, positions=None, window=0, scale=None):
    """out, its bound, and per (b, h_kv) the weights summed over heads with their bound; one sequence at a time."""
    B, Hq, T, d = q.shape
    Hkv, cap = k.shape[1:3]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(B, Hq, T, v.shape[-1], dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    w = torch.zeros(B, Hkv, cap, dtype=torch.float64, device=q.device)
    wtol = torch.zeros_like(w)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        m = min(n + (T if drafts else 0), cap)
        seen = torch.zeros(T, m, dtype=torch.bool)
        for t in range(T):
            seen[t, :n] = True
            word = (1 << (t + 1)) - 1 if mask is None else int(mask[t] if mask.dim() == 1 else mask[b, t])
            at_t = max(int(positions[b, t]), n) if positions is not None else n + t
            if window > 0:
                seen[t, :max(0, min(n, at_t - window + 1))] = False
            for u in range(m - n):
                at_u = max(int(positions[b, u]), n) if positions is not None else n + u
                seen[t, n + u] = bool((word >> u) & 1) and (window <= 0 or at_t - at_u < window)
        seen = seen.to(q.device)
        used = seen.any(0)
        for h in range(Hkv):
            qq = q[b, h * G:(h + 1) * G].double().reshape(G * T, d)
            kk = torch.where(used[:, None], k[b, h, :m].double(), 0.0)
            vv = torch.where(used[:, None], v[b, h, :m].double(), 0.0)
            x = (qq @ kk.T * scale).reshape(G, T, m)
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(-1, keepdim=True) if m else x.sum(-1, keepdim=True)
            p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
            p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
            size = (qq.abs() @ kk.abs().T * abs(scale)).reshape(G, T, m).masked_fill(~seen, 0.0)
            e = (size.amax(-1, keepdim=True) if m else size.sum(-1, keepdim=True)) * (d + 2) * 2.0 ** -24
            o, A = p @ vv, p @ vv.abs()
            out[b, h * G:(h + 1) * G] = o
            tol[b, h * G:(h + 1) * G] = U * (A * (1 + U) + o.abs()) + (2 * e + 2.0 ** -13) * A
            w[b, h, :m] = p.sum((0, 1))
            wtol[b, h, :m] = (p * (2 * e + 2.0 ** -13)).sum((0, 1))
    return out, tol, w, wtol


def _close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert torch.isfinite(err).all()
    assert (err <= tol).all(), "off by %.3g where %.3g may be" % (float((err - tol).max()), float(tol.max()))


def _tree(g, B, T, lens):
    """A random tree per sequence: ancestor masks (the draft itself among them) and positions."""
    up = torch.randint(1, 7, (B, T), generator=torch.Generator().manual_seed(g)).tolist()
    mask, pos = [], []
    for b in range(B):
        mm, dd = [], []
        for t in range(T):
            p = t - up[b][t]
            mm.append((1 << t) | (mm[p] if p >= 0 else 0))
            dd.append(dd[p] + 1 if p >= 0 else 0)
        mask.append([m - (1 << 64) if m >> 63 else m for m in mm])
        pos.append([lens[b] + x for x in dd])
    return torch.tensor(mask, dtype=torch.int64), torch.tensor(pos, dtype=torch.int32)


ATTN = [  # Hq, Hkv, T, d_qk, d_v, S_cap, lens, window
    (2, 2, 1, 64, 64, 1, [0], 0),
    (4, 2, 5, 64, 64, 160, [128, 0, 1], 0),
    (8, 8, 1, 128, 128, 130, [129, 127, 128], 0),
    (8, 2, 7, 128, 128, 700, [0, 1, 63, 127, 500, 693], 0),
    (16, 1, 8, 64, 64, 333, [256, 325], 0),              # 128 rows: one whole tile
    (16, 1, 9, 128, 128, 400, [255, 391], 0),            # 144 rows
    (32, 2, 16, 128, 128, 600, [300, 584], 0),           # 256 rows
    (16, 1, 33, 128, 128, 300, [200, 267], 0),           # 528 rows, odd
    (16, 1, 64, 64, 64, 1000, [936, 129], 0),            # 1024 rows, a full tree
    (4, 1, 64, 128, 128, 200, [136], 0),
    (8, 2, 3, 192, 128, 515, [512, 100, 0], 0),
    (32, 2, 13, 192, 128, 900, [887, 600], 0),           # 208 rows, decoupled
    (8, 2, 6, 128, 128, 2000, [1500, 1994, 3], 100),
    (8, 2, 20, 64, 64, 1100, [1080, 4], 3),              # a window smaller than the tree is deep
    (4, 4, 4, 128, 128, 5000, [4996, 2500], 1024),
    (16, 1, 40, 192, 128, 600, [128, 560], 130),
    (32, 8, 2, 128, 128, 9000, [8998], 0),
]


def _attn_inputs(dev, seed, Hq, Hkv, T, dk, dv, cap, lens, q_scale=1.5):
    g = _gen(dev, seed)
    B = len(lens)
    q = _normal(g, dev, B, Hq, T, dk, scale=q_scale)
    k, v = _normal(g, dev, B, Hkv, cap, dk), _normal(g, dev, B, Hkv, cap, dv)
    return q, k, v, torch.tensor(lens, dtype=torch.int32, device=dev)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,T,dk,dv,cap,lens,window", ATTN)
def test_tree_decode_matches_the_formula(Hq, Hkv, T, dk, dv, cap, lens, window):
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, T + cap, Hq, Hkv, T, dk, dv, cap, lens)
    mask, pos = _tree(T, len(lens), T, lens)
    for b, n in enumerate(lens):  # rows behind the drafts, and before every window, hold garbage
        k[b, :, n + T:], v[b, :, n + T:] = float("nan"), float("inf")
        if window and n + T > 1:
            first = max(0, n - window + 1)
            k[b, :, :first], v[b, :, :first] = float("inf"), float("nan")
    got = apex.tree_decode(q, k, v, ln, tree_mask=mask.to(dev), positions=pos.to(dev), window=window)
    ref, tol, _, _ = _attn_ref(q, k, v, lens, True, mask, pos, window)
    _close(got, ref, tol)
    assert apex.apex_attn_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 2, 50])
def test_tree_decode_defaults_are_a_chain(window):
    """Without masks and positions the drafts follow one another: the rows of a causal prefill."""
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 1, 8, 2, 6, 128, 128, 306, [300, 17])
    got = apex.tree_decode(q, k, v, ln, window=window)
    ref, tol, _, _ = _attn_ref(q, k, v, [300, 17], True, window=window)
    _close(got, ref, tol)
    chain = torch.tensor([(1 << (t + 1)) - 1 for t in range(6)], dtype=torch.int64, device=dev)
    assert torch.equal(got, apex.tree_decode(q, k, v, ln, tree_mask=chain, window=window))


@pytest.mark.gpu
def test_tree_decode_masks_that_leave_nothing_and_padded_drafts():
    dev = _gpu()
    lens, T = [0, 0, 200], 8
    q, k, v, ln = _attn_inputs(dev, 2, 8, 2, T, 128, 128, 256, lens)
    # sequence 0: nothing visible to drafts 3.. ; 1: no draft sees anything; 2: five real drafts
    mask = torch.tensor([[1, 3, 7, 0, 0, 0, 0, 0], [0] * 8, [1, 3, 5, 11, 19, 0, 0, 0]], dtype=torch.int64)
    for b, real in ((0, 3), (1, 0), (2, 5)):
        k[b, :, lens[b] + real:], v[b, :, lens[b] + real:] = float("nan"), float("nan")
    got = apex.tree_decode(q, k, v, ln, tree_mask=mask.to(dev))
    ref, tol, _, _ = _attn_ref(q, k, v, lens, True, mask)
    _close(got, ref, tol)
    assert (got[0, :, 3:] == 0).all() and (got[1] == 0).all()


@pytest.mark.gpu
def test_tree_decode_lengths_out_of_range_and_past_the_capacity():
    dev = _gpu()
    lens = [-5, 90, 97, 2 ** 31 - 1]  # drafts 90..97 of 96 rows: two are cut off; all rows seen past it
    q, k, v, ln = _attn_inputs(dev, 3, 4, 2, 8, 64, 64, 96, lens)
    got = apex.tree_decode(q, k, v, ln)
    ref, tol, _, _ = _attn_ref(q, k, v, lens, True)
    _close(got, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_tree_decode_scale(scale):
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 4, 8, 2, 4, 128, 128, 700, [650, 300])
    got = apex.tree_decode(q, k, v, ln, scale=scale)
    ref, tol, _, _ = _attn_ref(q, k, v, [650, 300], True, scale=scale)
    _close(got, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,T,dk,dv", [(8, 2, 4, 64, 64), (16, 1, 20, 64, 64), (8, 2, 4, 128, 128),
                                            (16, 1, 10, 128, 128), (16, 1, 40, 128, 128), (16, 1, 33, 192, 128)])
def test_tree_decode_rising_scores(Hq, Hkv, T, dk, dv):
    """Scores that keep rising along the keys: the running maximum is raised in every tile."""
    dev = _gpu()
    n = 1500
    q, k, v, ln = _attn_inputs(dev, 5, Hq, Hkv, T, dk, dv, n + T, [n])
    q[..., 0], k[..., 0] = 8.0, torch.linspace(-60, 60, n + T, device=dev).to(torch.bfloat16)
    got = apex.tree_decode(q, k, v, ln)
    ref, tol, _, _ = _attn_ref(q, k, v, [n], True)
    _close(got, ref, tol)
    k[..., 0] = -k[..., 0]
    ref, tol, _, _ = _attn_ref(q, k, v, [n], True)
    _close(apex.tree_decode(q, k, v, ln), ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,T,d,cap", [(33, 4, 2, 3, 64, 300), (70, 8, 2, 5, 128, 700), (300, 4, 1, 1, 64, 140),
                                              (40, 16, 1, 17, 128, 400), (1, 8, 8, 4, 128, 40000)])
def test_many_and_long_sequences(B, Hq, Hkv, T, d, cap):
    """More sequences than a warp's lanes hold, shares that end in the middle of units, one long sequence."""
    dev = _gpu()
    lens = torch.randint(0, cap - T + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    lens[-1] = cap - T
    q, k, v, ln = _attn_inputs(dev, B, Hq, Hkv, T, d, d, cap, lens)
    mask, _ = _tree(B, B, T, lens)
    ref, tol, _, _ = _attn_ref(q, k, v, lens, True, mask)
    _close(apex.tree_decode(q, k, v, ln, tree_mask=mask.to(dev)), ref, tol)
    q1 = q[:, :, :1].contiguous()
    acc = torch.zeros(B, Hkv, cap, device=dev)
    ref, tol, w, wtol = _attn_ref(q1, k, v, lens, False)
    _close(apex.decode_weights(q1, k, v, ln, acc), ref, tol)
    _close(acc, w, wtol + 2.0 ** -23 * w)


@pytest.mark.gpu
def test_thousands_of_short_sequences():
    dev = _gpu()
    B, T, cap = 5000, 2, 5
    lens = torch.randint(0, cap - T + 1, (B,), generator=torch.Generator().manual_seed(4)).to(torch.int32).to(dev)
    g = _gen(dev, 70)
    q, k, v = _normal(g, dev, B, 2, T, 64), _normal(g, dev, B, 1, cap, 64), _normal(g, dev, B, 1, cap, 64)
    got = apex.tree_decode(q, k, v, lens)
    some = [0, 1, 77, 2499, 4095, 4096, 4998, 4999]
    ref, tol, _, _ = _attn_ref(q[some], k[some], v[some], lens[some].tolist(), True)
    _close(got[some], ref, tol)
    one = torch.arange(cap, device=dev) < (lens + T)[:, None]  # every row of a unit sums its weights to one
    ones = torch.where(one[:, None, :, None], 1.0, float("nan")).to(torch.bfloat16).expand(B, 1, cap, 64).contiguous()
    out = apex.tree_decode(q, k, ones, lens)
    assert ((out.float() - 1).abs() <= 2 * U).all()
    acc = torch.rand(B, 1, cap, generator=g, device=dev)
    a, p, n = apex.evict(k, v, acc, lens + T, 3)
    assert torch.equal(n, (lens + T).clamp(max=3))
    kept = torch.where(one, acc[:, 0], -1.0).sort(-1, descending=True).values[:, :3].clamp(min=0).sort(-1).values
    assert torch.equal(a[:, 0, :3].sort(-1).values, kept) and (a[:, 0, 3:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,T,d", [(4, 3, 128), (16, 12, 128), (16, 40, 128), (16, 12, 64)])
def test_a_query_that_is_not_finite_stays_alone(Hq, T, d):
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 80, Hq, 1, T, d, d, 800, [700])
    q[0, 1, 1, 5] = float("nan")
    got = apex.tree_decode(q, k, v, ln)
    assert torch.isnan(got[0, 1, 1]).all()
    q[0, 1, 1, 5] = 0.0
    ref, tol, _, _ = _attn_ref(q, k, v, [700], True)
    got[0, 1, 1] = ref[0, 1, 1].to(torch.bfloat16)
    _close(got, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(40))
def test_random_configurations(seed):
    """Seeded draws over head groups, rows, lengths, windows and trees, on every kernel."""
    dev = _gpu()
    r = torch.Generator().manual_seed(1000 + seed)

    def pick(*xs):
        return xs[int(torch.randint(0, len(xs), (1,), generator=r))]

    def log(lo, hi):
        return int(round(math.exp(math.log(lo) + float(torch.rand(1, generator=r)) * (math.log(hi) - math.log(lo)))))

    G, Hkv, B, T = pick(1, 2, 4, 8, 16), pick(1, 2, 3), pick(1, 2, 5), log(1, 64)
    dk, dv = pick((64, 64), (128, 128), (192, 128))
    cap = T + log(1, 3000)
    lens = torch.randint(0, cap - T + 1, (B,), generator=r).tolist()
    window = pick(0, 0, log(1, 1000))
    q, k, v, ln = _attn_inputs(dev, seed, G * Hkv, Hkv, T, dk, dv, cap, lens)
    mask, pos = _tree(seed, B, T, lens)
    if pick(0, 1):  # some drafts see nothing of the tree, not even themselves
        mask[:, ::3] = 0
    ref, tol, _, _ = _attn_ref(q, k, v, lens, True, mask, pos, window)
    got = apex.tree_decode(q, k, v, ln, tree_mask=mask.to(dev), positions=pos.to(dev), window=window)
    _close(got, ref, tol)
    assert apex.apex_attn_device_status() == 0


WEIGHTS = [  # Hq, Hkv, d_qk, d_v, S_cap, lens
    (1, 1, 64, 64, 1, [1]),
    (4, 2, 64, 64, 300, [0, 1, 127, 128, 129, 300]),
    (8, 8, 128, 128, 1000, [999, 500]),
    (32, 8, 128, 128, 1001, [1001]),
    (16, 1, 128, 128, 5000, [4097, 64]),
    (16, 8, 128, 128, 600, [600] * 5),
    (32, 2, 192, 128, 777, [777, 400, 5]),
    (8, 2, 192, 128, 130, [130]),
    (64, 8, 64, 64, 20000, [20000, 333]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,dk,dv,cap,lens", WEIGHTS)
def test_decode_weights_matches_the_formula(Hq, Hkv, dk, dv, cap, lens):
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, cap, Hq, Hkv, 1, dk, dv, cap, lens)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")
    acc0 = torch.rand(len(lens), Hkv, cap, generator=_gen(dev, 1), device=dev)
    acc = acc0.clone()
    got = apex.decode_weights(q, k, v, ln, acc)
    ref, tol, w, wtol = _attn_ref(q, k, v, lens, False)
    _close(got, ref, tol)
    want = acc0.double() + w
    _close(acc, want, wtol + 2.0 ** -23 * want)
    for b, n in enumerate(lens):
        assert torch.equal(acc[b, :, n:], acc0[b, :, n:])
    # the sums are made in a fixed order
    acc2 = acc0.clone()
    assert torch.equal(got, apex.decode_weights(q, k, v, ln, acc2)) and torch.equal(acc, acc2)
    assert apex.apex_attn_device_status() == 0


@pytest.mark.gpu
def test_decode_weights_peaked_and_scaled():
    dev = _gpu()
    n = 900
    q, k, v, ln = _attn_inputs(dev, 9, 8, 2, 1, 128, 128, n, [n], q_scale=8.0)
    acc = torch.zeros(1, 2, n, device=dev)
    got = apex.decode_weights(q, k, v, ln, acc, scale=0.3)
    ref, tol, w, wtol = _attn_ref(q, k, v, [n], False, scale=0.3)
    _close(got, ref, tol)
    _close(acc, w, wtol + 2.0 ** -23 * w + 2.0 ** -126)


@pytest.mark.gpu
def test_decode_weights_equals_tree_of_one_and_decode():
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 10, 32, 8, 1, 128, 128, 1200, [1200, 1200])
    got = apex.decode_weights(q, k, v, ln, torch.zeros(2, 8, 1200, device=dev))
    tree = apex.tree_decode(q, k, v, ln - 1)
    ref, tol, _, _ = _attn_ref(q, k, v, [1200, 1200], False)
    _close(got, ref, tol)
    _close(tree, ref, tol)
    qr = apex.rope(q, positions=torch.full((2, 1), 1199, dtype=torch.int32, device=dev))
    dec = apex.decode(q, k, v, 1199, keys_prerotated=True)
    _close(apex.decode_weights(qr, k, v, ln, torch.zeros(2, 8, 1200, device=dev)).float() - dec.float() + ref.float(),
           ref, 3 * tol)


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_r,window,yarn", [(64, 0, 0, 1.0), (128, 0, 100, 1.0), (128, 0, 0, 16.0), (128, 64, 0, 1.0)])
def test_rope_and_tree_are_the_causal_block(d, d_r, window, yarn):
    """Queries and keys rotated by rope, a chain of drafts over them: the last rows of the block's
    prefill by the oracle, at the block's tolerance (Q and K rounded after the rotation)."""
    import oracle
    from transformer_attention_rope_gb300 import inputs
    dev = _gpu()
    B, Hq, Hkv, S, T = 2, 8, 2, 400, 12
    q, k, v = inputs.make_qkv(B, Hq, Hkv, T, S, d, 77, **({"d_r": d_r} if d_r else {}))
    how = dict(rot_start=d, d_rot=d_r) if d_r else {}
    at = torch.arange(S, dtype=torch.int32, device=dev)
    qr = apex.rope(q.to(dev), positions=at[S - T:], yarn_scale=yarn, **how)
    kr = apex.rope(k.to(dev), positions=at, yarn_scale=yarn, **how)
    scale = (0.1 * math.log(yarn) + 1.0) / math.sqrt(d + d_r) if yarn > 1 else None
    got = apex.tree_decode(qr, kr, v.to(dev), torch.full((B,), S - T, dtype=torch.int32, device=dev), window=window,
                           scale=scale)
    if d_r:
        ref = oracle.mla_attn(q, k, v, d_r, window=window, q_pos0=S - T)
    else:
        ref = oracle.attn(q, k, v, window=window, q_pos0=S - T, **({"yarn_s": yarn} if yarn > 1 else {}))
    e = (got.double().cpu() - torch.as_tensor(ref)).abs()
    assert e.max() <= 2e-2 and e.mean() <= 2e-3, (float(e.max()), float(e.mean()))


# ------------------------------------------------------------------------------------------------- eviction
def _evict_ref(k, v, acc, lens, budget, n_sink, n_recent, positions, next_pos):
    k, v, acc = k.cpu().clone(), v.cpu().clone(), acc.cpu().double()
    B, H, cap = acc.shape
    a_out, p_out = torch.zeros(B, H, cap, dtype=torch.float64), torch.full((B, H, cap), -1, dtype=torch.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        nxt = int(next_pos[b]) if next_pos is not None else int(lens[b])
        for h in range(H):
            pos = positions[b, h].tolist() if positions is not None else list(range(cap))
            must = [pos[j] < n_sink or pos[j] >= nxt - n_recent for j in range(n)]
            a = acc[b, h].tolist()
            rank = sorted(range(n), key=lambda j: (0 if must[j] else 1, 0 if must[j] else
                                                   math.inf if a[j] != a[j] else -a[j], 0 if must[j] else
                                                   int(a[j] != a[j]), j))
            kept = sorted(rank[:budget])
            rows = {j: j for j in kept if j < budget}
            holes = [j for j in range(min(n, budget)) if j not in rows]
            for hole, j in zip(holes, [j for j in kept if j >= budget]):
                k[b, h, hole], v[b, h, hole], rows[hole] = k[b, h, j], v[b, h, j], j
            for to, j in rows.items():
                a_out[b, h, to], p_out[b, h, to] = a[j], pos[j]
    return k, v, a_out, p_out, [min(min(max(int(n), 0), cap), budget) for n in lens]


def _evict_check(dev, k, v, acc, lens, budget, n_sink, n_recent, positions=None, next_pos=None):
    want = _evict_ref(k, v, acc, lens, budget, n_sink, n_recent, positions, next_pos)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    a, p, n = apex.evict(k, v, acc, ln, budget, n_sink=n_sink, n_recent=n_recent, positions=positions,
                         next_pos=torch.tensor(next_pos, dtype=torch.int32, device=dev) if next_pos else None)
    assert n.tolist() == want[4]
    assert torch.equal(p.cpu(), want[3])
    assert torch.equal(torch.nan_to_num(a.double().cpu(), nan=-7.0), torch.nan_to_num(want[2], nan=-7.0))
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    return a, p, n


EVICT = [  # H, d_k, d_v, S_cap, lens, budget, n_sink, n_recent
    (1, 64, 64, 1, [1, 0], 1, 0, 0),
    (2, 128, 128, 40, [40, 33, 32, 31, 0], 32, 4, 8),
    (2, 128, 128, 500, [500, 499, 260], 250, 4, 100),
    (1, 192, 128, 5000, [5000, 4097], 513, 4, 64),       # two CTAs a row set
    (2, 64, 64, 9001, [9001, 4500], 1000, 0, 1000),      # nothing but the newest
    (1, 8, 8, 40000, [40000], 3000, 7, 0),               # eight CTAs
    (1, 8, 8, 400000, [399999], 100000, 3, 9000),        # more rows than shared memory holds
    (3, 128, 128, 600, [-4, 600, 9999], 599, 0, 0),      # one row goes
    (1, 128, 128, 300, [300], 1, 1, 0),
    (1, 128, 128, 64, [64], 100, 4, 4),                  # budget past the capacity
]


@pytest.mark.gpu
@pytest.mark.parametrize("aged", [False, True])
@pytest.mark.parametrize("H,dk,dv,cap,lens,budget,sink,recent", EVICT)
def test_evict_matches_a_plain_one(H, dk, dv, cap, lens, budget, sink, recent, aged):
    dev = _gpu()
    g = _gen(dev, cap + budget)
    B = len(lens)
    k, v = _normal(g, dev, B, H, cap, dk), _normal(g, dev, B, H, cap, dv)
    acc = torch.exp(torch.randn(B, H, cap, generator=g, device=dev))
    pos = nxt = None
    if aged:  # rows in any order, with gaps
        pos = (torch.rand(B, H, cap, generator=g, device=dev).argsort(-1) * 3).to(torch.int32).contiguous()
        nxt = [3 * cap] * B
    _evict_check(dev, k, v, acc, lens, budget, sink, recent, pos, nxt)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [200, 9000])
def test_evict_ties_and_odd_weights(cap):
    dev = _gpu()
    g = _gen(dev, 11)
    k, v = _normal(g, dev, 2, 2, cap, 64), _normal(g, dev, 2, 2, cap, 64)
    # few distinct weights, all equal in one head, and NaN, infinities, both zeros, negatives
    acc = torch.randint(0, 3, (2, 2, cap), generator=g, device=dev).float()
    acc[0, 1] = 0.5
    odd = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1.0, 1e-42, 3.0], device=dev)
    acc[1, 1] = odd[torch.randint(0, 8, (cap,), generator=g, device=dev)]
    for budget in (3, cap // 2, cap - 1):
        _evict_check(dev, k, v, acc, [cap, cap - 1], budget, 1, 2)


@pytest.mark.gpu
def test_evict_more_forced_rows_than_budget():
    """Equal positions can force more rows than the budget: the lowest of them stay."""
    dev = _gpu()
    g = _gen(dev, 12)
    k, v = _normal(g, dev, 1, 2, 100, 64), _normal(g, dev, 1, 2, 100, 64)
    acc = torch.rand(1, 2, 100, generator=g, device=dev)
    _evict_check(dev, k, v, acc, [100], 20, 5, 0, torch.zeros(1, 2, 100, dtype=torch.int32, device=dev), [7])


@pytest.mark.gpu
def test_evict_again():
    """A second cut with the first one's outputs as inputs."""
    dev = _gpu()
    g = _gen(dev, 13)
    k, v = _normal(g, dev, 2, 2, 700, 128), _normal(g, dev, 2, 2, 700, 128)
    acc = torch.rand(2, 2, 700, generator=g, device=dev)
    ln = torch.tensor([700, 650], dtype=torch.int32, device=dev)
    nxt = ln.clone()
    want = _evict_ref(k, v, acc, [700, 650], 300, 4, 50, None, None)
    a, p, n = apex.evict(k, v, acc, ln, 300, n_sink=4, n_recent=50)
    assert n.tolist() == [300, 300] and ln.tolist() == [700, 650]
    want = _evict_ref(want[0], want[1], want[2], [300, 300], 120, 4, 50, want[3], nxt.tolist())
    n2 = torch.empty_like(n)
    a, p, out = apex.evict(k, v, a, n, 120, n_sink=4, n_recent=50, positions=p, next_pos=nxt, lens_out=n2)
    assert out is n2 and n2.tolist() == [120, 120]
    assert torch.equal(p.cpu(), want[3]) and torch.equal(a.double().cpu(), want[2])
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    """One sequence of the longest cache, 2 heads of 2^24 rows of 64: entries past 2^31."""
    dev = _gpu()
    if torch.cuda.mem_get_info(dev)[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    cap, T, H = 1 << 24, 3, 2
    n = cap - T - 2
    g = _gen(dev, 60)
    kc, vc = (torch.full((1, H, cap, 64), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    seen = 500
    kc[:, :, n - seen:n], vc[:, :, n - seen:n] = _normal(g, dev, 1, H, seen, 64), _normal(g, dev, 1, H, seen, 64)
    q, k, v = _normal(g, dev, 1, 4, T, 64), _normal(g, dev, 1, H, T, 64), _normal(g, dev, 1, H, T, 64)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    at = (lens[:, None] + torch.arange(T, device=dev, dtype=torch.int32)).contiguous()
    qr, _, _ = apex.rope(q, k, v, positions=at, k_out=kc, v_out=vc, row0=lens)
    _rope_close(kc[:, :, n:n + T], *_rope_ref(k, at))
    assert torch.equal(vc[:, :, n:n + T], v) and torch.isnan(vc[:, :, n + T:].float()).all()
    got = apex.tree_decode(qr, kc, vc, lens, window=seen)
    # the same rows as a short cache: a window of `seen` counts positions alike
    lo = n - seen
    ref, tol, _, _ = _attn_ref(qr, kc[:, :, lo:n + T], vc[:, :, lo:n + T], [seen], True, window=seen)
    _close(got, ref, tol)
    # keep eight rows, the heaviest at the end of the cache
    acc = torch.zeros(1, H, cap, device=dev)
    acc[:, :, n - 5:n] = 1.0 + torch.arange(5, device=dev)
    last_k, last_v = kc[:, :, n - 5:n].clone(), vc[:, :, n - 5:n].clone()
    a, p, m = apex.evict(kc, vc, acc, lens, 8, n_sink=3)
    assert m.tolist() == [8]
    assert p[..., :8].tolist() == [[[0, 1, 2] + list(range(n - 5, n))] * H] and (p[..., 8:] == -1).all()
    assert torch.equal(a[..., :8].cpu(), torch.tensor([0.0] * 3 + [1, 2, 3, 4, 5]).expand(1, H, 8))
    assert torch.equal(kc[:, :, 3:8], last_k) and torch.equal(vc[:, :, 3:8], last_v)
    # every weight of a row of equal keys is 1 / n
    kc[:, :, :n] = 0
    vc[:, :, :n] = 0
    vc[:, :, n - 1] = 1.0
    acc.zero_()
    out = apex.decode_weights(qr[:, :, :1].contiguous(), kc, vc, lens, acc)
    assert ((acc[..., :n].double() - 2.0 / n).abs() <= 2.0 / n * 2.0 ** -11).all() and (acc[..., n:] == 0).all()
    assert ((out.double() - 1.0 / n).abs() <= 1.0 / n * 2 * U).all()


# ------------------------------------------------------------------------------------------------- together
def _served(dev, seed, dk, dv, layout):
    """A bounded cache served for a few steps, each checked against the formulas on the same inputs."""
    g = _gen(dev, seed)
    B, Hq, Hkv, cap, budget, T = 2, 8, 2, 420, 256, 5
    rot = dict(layout=layout, rot_start=dk - 64 if dk != dv else 0)
    lens = torch.tensor([300, 270], dtype=torch.int32, device=dev)
    nxt = lens.clone()
    kc, vc = _normal(g, dev, B, Hkv, cap, dk), _normal(g, dev, B, Hkv, cap, dv)
    acc = torch.zeros(B, Hkv, cap, device=dev)
    pos = torch.arange(cap, dtype=torch.int32, device=dev).expand(B, Hkv, cap).contiguous()
    for step in range(4):
        # drafts
        q, k, v = (_normal(g, dev, B, T, h, d).transpose(1, 2) for h, d in ((Hq, dk), (Hkv, dk), (Hkv, dv)))
        mask, depth = _tree(step, B, T, [0, 0])
        at = (nxt[:, None] + depth.to(dev)).contiguous()
        qr, _, _ = apex.rope(q, k, v, positions=at, k_out=kc, v_out=vc, row0=lens, **rot)
        o = dict(half=layout == "half", rot_start=rot["rot_start"])
        _rope_close(qr, *_rope_ref(q, at, **o))
        got = apex.tree_decode(qr, kc, vc, lens, tree_mask=mask.to(dev))
        _close(got, *_attn_ref(qr, kc, vc, lens.tolist(), True, mask)[:2])
        # the first draft is accepted; the next token is decoded with its weights gathered
        for b in range(B):
            pos[b, :, int(lens[b])] = int(nxt[b])
        lens, nxt = lens + 1, nxt + 1
        q1 = apex.rope(_normal(g, dev, B, Hq, 1, dk), positions=(nxt - 1)[:, None].contiguous(), **rot)
        before = acc.double()
        got = apex.decode_weights(q1, kc, vc, lens, acc)
        ref, tol, w, wtol = _attn_ref(q1, kc, vc, lens.tolist(), False)
        _close(got, ref, tol)
        _close(acc, before + w, wtol + 2.0 ** -23 * (before + w))
        if step % 2 == 0:
            k0, v0, n0 = kc.clone(), vc.clone(), lens.tolist()
            want = _evict_ref(kc, vc, acc, n0, budget, 4, 64, pos, nxt.tolist())
            acc, pos, lens = apex.evict(kc, vc, acc, lens, budget, n_sink=4, n_recent=64, positions=pos, next_pos=nxt)
            assert torch.equal(pos.cpu(), want[3]) and torch.equal(kc.cpu(), want[0]) and lens.tolist() == want[4]
    assert apex.apex_attn_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv,layout", [(64, 64, "half"), (128, 128, "interleaved"), (192, 128, "interleaved")])
def test_a_bounded_cache_served(dk, dv, layout):
    _served(_gpu(), dk, dk, dv, layout)


@pytest.mark.gpu
def test_captured_and_replayed_with_new_lengths():
    """All four operators in one graph on a stream of their own; replays follow lengths, positions and data."""
    dev = _gpu()
    B, Hq, Hkv, T, d, cap, budget = 2, 16, 4, 6, 128, 900, 400
    g = _gen(dev, 21)
    q, k, v = (_normal(g, dev, B, h, T, d) for h in (Hq, Hkv, Hkv))
    kc, vc = _normal(g, dev, B, Hkv, cap, d), _normal(g, dev, B, Hkv, cap, d)
    lens = torch.tensor([500, 10], dtype=torch.int32, device=dev)
    at = torch.zeros(B, T, dtype=torch.int32, device=dev)
    acc = torch.rand(B, Hkv, cap, generator=g, device=dev)
    bufs = {n: torch.empty(x, dtype=torch.uint8, device=dev) for n, x in (
        ("tree", apex.tree_workspace_bytes(B, Hq, Hkv, T, cap, d)),
        ("weights", apex.decode_weights_workspace_bytes(B, Hq, Hkv, cap, d)),
        ("evict", apex.evict_workspace_bytes(B, Hkv, cap, budget)))}

    def calls():
        qr, _, _ = apex.rope(q, k, v, positions=at, k_out=kc, v_out=vc, row0=lens)
        tree = apex.tree_decode(qr, kc, vc, lens, window=300, workspace=bufs["tree"])
        one = apex.decode_weights(qr[:, :, :1].contiguous(), kc, vc, lens, acc, workspace=bufs["weights"])
        return (qr, tree, one) + apex.evict(kc, vc, acc, lens, budget, n_sink=2, n_recent=30,
                                            workspace=bufs["evict"])

    first = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for a, b in ((890, 401), (400, 0), (1, 777)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        at.copy_(lens[:, None] + torch.arange(T, device=dev, dtype=torch.int32))
        for x in (q, k, v, kc, vc):
            x.normal_()
        acc.uniform_()
        state = [x.clone() for x in (kc, vc, acc)]
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs] + [kc.clone(), vc.clone(), acc.clone()]
        for x, y in zip((kc, vc, acc), state):
            x.copy_(y)
        want = list(calls()) + [kc, vc, acc]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert len(first) == len(outs) and apex.apex_attn_device_status() == 0


@pytest.mark.gpu
def test_two_streams_with_their_own_workspaces():
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 30, 32, 8, 8, 128, 128, 3000, [2990, 1000, 5])
    want = apex.tree_decode(q, k, v, ln)
    accs = [torch.zeros(3, 8, 3000, device=dev) for _ in range(3)]
    q1 = q[:, :, :1].contiguous()
    one = apex.decode_weights(q1, k, v, ln, accs[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for i in range(6):
        s = streams[i % 2]
        got.append((apex.tree_decode(q, k, v, ln, stream=s), apex.decode_weights(q1, k, v, ln, accs[i % 2], stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) and torch.equal(o, one) for t, o in got)
    assert torch.equal(accs[0], accs[1])


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["rope", "tree", "weights", "evict"])
def test_memory_freed_on_the_current_stream_is_not_written_from_another(op):
    """A block freed while its stream still has a write to it ahead goes to that stream's next
    tensor only: a call on another stream takes its output and workspace elsewhere."""
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 31, 8, 2, 1, 128, 128, 600, [600, 20])
    acc, pos = torch.rand(2, 2, 600, device=dev), torch.zeros(2, 1, dtype=torch.int32, device=dev)
    s = torch.cuda.Stream(dev)
    own = [(acc.clone(), k.clone(), v.clone()) for _ in range(2)]  # what calls change

    def call(stream):
        a, kc, vc = own.pop()
        if op == "rope":
            return apex.rope(q, positions=pos, stream=stream)
        if op == "tree":
            return apex.tree_decode(q, k, v, ln, stream=stream)
        if op == "weights":
            return apex.decode_weights(q, k, v, ln, a, stream=stream)
        return apex.evict(kc, vc, a, ln, 500, stream=stream)[0]

    want = call(None)
    sizes = [want.numel() * want.element_size(), apex.tree_workspace_bytes(2, 8, 2, 1, 600, 128),
             apex.decode_weights_workspace_bytes(2, 8, 2, 600, 128), apex.evict_workspace_bytes(2, 2, 600, 500)]
    torch.cuda.synchronize()
    torch.cuda._sleep(int(1e8))
    late = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) for n in sizes for _ in range(4)]
    taken = {t.data_ptr() for t in late}
    del late
    got = call(s)
    assert got.data_ptr() not in taken
    s.synchronize()
    held = got.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(held, want)


@pytest.mark.gpu
def test_outputs_and_workspaces_stay_within_their_bounds():
    dev = _gpu()
    pad = 4096

    def guarded(n_bytes):
        buf = torch.full((n_bytes + 2 * pad,), 0xA5, dtype=torch.uint8, device=dev)
        return buf, buf[pad:pad + n_bytes]

    def clean(buf, n):
        return bool((buf[:pad] == 0xA5).all()) and bool((buf[pad + n:] == 0xA5).all())

    for Hq, Hkv, T, dk, dv, cap, lens, window in ATTN[1:12:2]:
        q, k, v, ln = _attn_inputs(dev, 40, Hq, Hkv, T, dk, dv, cap, lens)
        B = len(lens)
        n = B * Hq * T * dv * 2
        obuf, o = guarded(n)
        need = apex.tree_workspace_bytes(B, Hq, Hkv, T, cap, dk, dv)
        wbuf, w = guarded(need)
        apex.tree_decode(q, k, v, ln, out=o.view(torch.bfloat16).view(B, Hq, T, dv), workspace=w)
        assert clean(obuf, n) and clean(wbuf, need)
        need = apex.decode_weights_workspace_bytes(B, Hq, Hkv, cap, dk, dv)
        wbuf, w = guarded(need)
        abuf, a = guarded(B * Hkv * cap * 4)
        apex.decode_weights(q[:, :, :1].contiguous(), k, v, ln, a.view(torch.float32).view(B, Hkv, cap), workspace=w)
        assert clean(wbuf, need) and clean(abuf, B * Hkv * cap * 4)
        budget = max(1, cap // 3)
        need = apex.evict_workspace_bytes(B, Hkv, cap, budget)
        wbuf, w = guarded(need)
        apex.evict(k, v, torch.rand(B, Hkv, cap, device=dev), ln, budget, workspace=w)
        assert clean(wbuf, need)


# ------------------------------------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    try:
        return apex.load_library()
    except RuntimeError:
        pytest.skip("library not built")


P = 1 << 20  # an aligned address that a refused call never touches
BAD, UNSUPPORTED = 1, 2


def _tensor(**o):
    f = dict(in_=P, out=2 * P, n_heads=4, d_row=128, in_b=512, in_h=128, in_s=512, out_b=512, out_h=128, out_s=512)
    f.update(o)
    return apex.RopeTensor(*[f[n] for n, _ in apex.RopeTensor._fields_])


@pytest.mark.parametrize("tensor,opt,args,code", [
    (dict(in_=None), {}, {}, BAD), (dict(out=None), {}, {}, BAD), (dict(in_=P + 1), {}, {}, BAD),
    (dict(n_heads=0), {}, {}, BAD), (dict(d_row=-8), {}, {}, BAD), (dict(d_row=2048), {}, {}, UNSUPPORTED),
    ({}, dict(layout=2), {}, BAD), ({}, dict(d_rot=3), {}, BAD), ({}, dict(d_rot=130), {}, BAD),
    ({}, dict(rot_start=128), {}, BAD), ({}, dict(rot_start=-2), {}, BAD), ({}, dict(rot_start=64, d_rot=66), {}, BAD),
    ({}, dict(rope_base=-1.0), {}, BAD), ({}, dict(rope_base=float("inf")), {}, BAD),
    ({}, dict(linear_scale=-2.0), {}, BAD), ({}, dict(linear_scale=float("nan")), {}, BAD),
    ({}, dict(yarn_scale=float("nan")), {}, BAD), ({}, dict(yarn_scale=2.0, yarn_beta_fast=-1.0), {}, BAD),
    ({}, {}, dict(B=0), BAD), ({}, {}, dict(S=-1), BAD), ({}, {}, dict(positions=None), BAD),
    ({}, {}, dict(positions=P + 2), BAD), ({}, {}, dict(row0=P), BAD), ({}, {}, dict(pos_stride=-1), BAD),
    ({}, {}, dict(B=1 << 16, S=1 << 16), UNSUPPORTED), (dict(d_row=1024), dict(d_rot=1024), {}, UNSUPPORTED),
])
def test_rope_refuses(lib, tensor, opt, args, code):
    a = dict(B=1, S=1, positions=P, pos_stride=1, row0=None, out_rows=0)
    a.update(args)
    o = apex.RopeOptions(**opt)
    t = _tensor(**tensor)
    for k in (None, t):
        assert apex.apex_attn_rope(t, k, None, a["B"], a["S"], a["positions"], a["pos_stride"], a["row0"],
                                   a["out_rows"], o, None) == code
    assert apex.apex_attn_rope(None, None, None, 1, 1, P, 1, None, 0, o, None) == BAD
    assert apex.apex_attn_rope(t, None, None, 1, 1, P, 1, None, 0, None, None) == BAD


def test_rope_refuses_rows_that_disagree(lib):
    """With d_rot 0 the whole row turns, which rows of different lengths cannot share."""
    assert apex.apex_attn_rope(_tensor(), _tensor(d_row=64), None, 1, 1, P, 1, None, 0, apex.RopeOptions(), None) == BAD


ATTN_ARGS = dict(q=P, k=P, v=P, out=8 * P, B=1, H_q=8, H_kv=2, T=4, S_cap=64, d_qk=128, d_v=128, lens=P, mask=None,
                 stride=0, positions=None, window=0, scale=0.0, ws=P, n=1 << 40)


@pytest.mark.parametrize("o,code", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(lens=None), BAD),
    (dict(ws=None), BAD), (dict(q=P + 2), BAD), (dict(k=P + 8), BAD), (dict(out=P + 8), BAD), (dict(ws=P + 8), BAD),
    (dict(lens=P + 1), BAD), (dict(mask=P + 4), BAD), (dict(positions=P + 2), BAD), (dict(stride=-1), BAD),
    (dict(B=0), BAD), (dict(H_q=0), BAD), (dict(H_kv=3), BAD), (dict(T=0), BAD), (dict(S_cap=0), BAD),
    (dict(d_qk=0), BAD), (dict(T=65), UNSUPPORTED), (dict(S_cap=(1 << 24) + 1), UNSUPPORTED),
    (dict(B=65537), UNSUPPORTED), (dict(d_qk=64), UNSUPPORTED), (dict(d_qk=192, d_v=192), UNSUPPORTED),
    (dict(H_q=6), UNSUPPORTED), (dict(H_q=64), UNSUPPORTED), (dict(scale=float("inf")), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=-0.3), BAD), (dict(n=15), BAD),
    # outputs (8192 bytes) on the queries, on the keys (32768 bytes), on the values
    (dict(q=8 * P), BAD), (dict(q=8 * P + 8176), BAD), (dict(k=8 * P - 32752), BAD), (dict(v=8 * P + 16), BAD),
])
def test_tree_decode_refuses(lib, o, code):
    a = dict(ATTN_ARGS)
    a.update(o)
    assert apex.apex_attn_tree_decode(a["q"], a["k"], a["v"], a["out"], a["B"], a["H_q"], a["H_kv"], a["T"],
                                      a["S_cap"], a["d_qk"], a["d_v"], a["lens"], a["mask"], a["stride"],
                                      a["positions"], a["window"], a["scale"], a["ws"], a["n"], None) == code
    sizes = [a[n] for n in ("B", "H_q", "H_kv", "T", "S_cap", "d_qk", "d_v")]
    bad_sizes = any(n in o for n in ("B", "H_q", "H_kv", "T", "S_cap", "d_qk", "d_v"))
    assert (apex.tree_workspace_bytes(*sizes) == 0) == bad_sizes


@pytest.mark.parametrize("o,code", [
    (dict(acc=None), BAD), (dict(acc=P + 2), BAD), (dict(q=None), BAD), (dict(lens=None), BAD), (dict(B=0), BAD),
    (dict(H_kv=3), BAD), (dict(d_v=64), UNSUPPORTED), (dict(H_q=10), UNSUPPORTED), (dict(n=15), BAD),
    (dict(scale=float("-inf")), BAD), (dict(q=8 * P - 2032), BAD), (dict(acc=8 * P - 508), BAD),
])
def test_decode_weights_refuses(lib, o, code):
    a = dict(ATTN_ARGS, acc=P)
    a.update(o)
    assert apex.apex_attn_decode_weights(a["q"], a["k"], a["v"], a["out"], a["B"], a["H_q"], a["H_kv"], a["S_cap"],
                                         a["d_qk"], a["d_v"], a["lens"], a["acc"], a["scale"], a["ws"], a["n"],
                                         None) == code


EVICT_ARGS = dict(k=P, v=P, B=1, H=2, cap=64, dk=128, dv=128, acc=P, pos=None, lens=P, nxt=None, budget=16, sink=0,
                  recent=0, acc_out=2 * P, pos_out=4 * P, lens_out=2 * P, ws=P, n=1 << 40)


@pytest.mark.parametrize("o,code", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(acc=None), BAD), (dict(lens=None), BAD), (dict(acc_out=None), BAD),
    (dict(pos_out=None), BAD), (dict(lens_out=None), BAD), (dict(ws=None), BAD), (dict(k=P + 8), BAD),
    (dict(pos=P + 4), BAD), (dict(lens=P + 2), BAD), (dict(nxt=P + 2), BAD), (dict(acc_out=P), BAD),
    (dict(acc_out=P + 496), BAD), (dict(pos=2 * P), BAD), (dict(pos=4 * P - 16), BAD), (dict(pos_out=2 * P), BAD), (dict(lens_out=P), BAD), (dict(nxt=2 * P), BAD), (dict(B=0), BAD), (dict(H=-1), BAD), (dict(cap=0), BAD), (dict(budget=0), BAD),
    (dict(sink=-1), BAD), (dict(recent=-1), BAD), (dict(sink=10, recent=7), BAD), (dict(dk=0), BAD),
    (dict(dk=100), UNSUPPORTED), (dict(dv=2048), UNSUPPORTED), (dict(cap=(1 << 24) + 1), UNSUPPORTED),
    (dict(n=15), BAD),
])
def test_evict_refuses(lib, o, code):
    a = dict(EVICT_ARGS)
    a.update(o)
    assert apex.apex_attn_evict(a["k"], a["v"], a["B"], a["H"], a["cap"], a["dk"], a["dv"], a["acc"], a["pos"],
                                a["lens"], a["nxt"], a["budget"], a["sink"], a["recent"], a["acc_out"], a["pos_out"],
                                a["lens_out"], a["ws"], a["n"], None) == code


def test_conveniences_refuse_cpu_tensors_and_wrong_shapes(lib):
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        apex.rope(x, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        apex.rope(x, positions=torch.zeros(3, dtype=torch.int32), layout="neox")
    with pytest.raises(TypeError):
        apex.tree_decode(x, x, x, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        apex.decode_weights(x, x, x, torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 3))
    with pytest.raises(TypeError):
        apex.evict(x, x, torch.zeros(1, 2, 3), torch.zeros(1, dtype=torch.int32), 2)


@pytest.mark.gpu
def test_conveniences_refuse_what_does_not_fit():
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 50, 8, 2, 4, 128, 128, 64, [32, 40])
    pos = torch.zeros(2, 4, dtype=torch.int32, device=dev)
    for bad in (lambda: apex.tree_decode(q, k, v, ln.long()), lambda: apex.tree_decode(q, k, v, ln.cpu())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: apex.tree_decode(q, k, v, ln[:1]), lambda: apex.tree_decode(q, k[:, :, :60], v, ln),
                lambda: apex.tree_decode(q, k, v, ln, positions=pos[:, :3]),
                lambda: apex.tree_decode(q, k, v[..., :64].contiguous()[:1], ln),
                lambda: apex.decode_weights(q, k, v, ln, torch.zeros(2, 2, 64, device=dev)),
                lambda: apex.rope(q, positions=pos[:1]), lambda: apex.rope(q, v=v, positions=pos),
                lambda: apex.rope(q, k[:, :, :4], positions=pos, row0=ln), lambda: apex.rope(q, positions=pos, d_rot=0),
                lambda: apex.rope(q, positions=pos, q_out=q[:, :, :3]),
                lambda: apex.rope(q, positions=pos, q_out=q[:, :1].expand(2, 8, 4, 128)),
                lambda: apex.evict(k, v, torch.zeros(2, 2, 63, device=dev), ln, 8)):
        with pytest.raises(ValueError):
            bad()
    ws = torch.empty(16, dtype=torch.uint8, device=dev)
    with pytest.raises(apex.ApexError):
        apex.tree_decode(q, k, v, ln, workspace=ws[8:])
