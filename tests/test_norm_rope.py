"""norm_rope and norm_rope_grad against plain 64-bit implementations.

Tolerances (u = 2^-8: half a step of bf16, relative to the value; fp32 half a step 2^-24).  A row's
sum of squares has d positive terms, so it is off by at most d 2^-24 of itself, and rs = 1 / sqrt by
half of that and what rsqrtf loses (2 units: 2^-22): r = d 2^-25 + 2^-20 covers it with the products'
roundings.  Angles: both products of a pair together by (|a| + |b|) 2^-21.
  y    one rounding, u |y|; r + 2^-21 of the pair's normed entries together.
  dx   = rs (c - v m), c = g w, v = x rs, m = mean(c v): one rounding, u |dx|; c by 2^-20 of the
       pair's gradients times |w|, v by r, m by 2 r of mean(|c v|) and what c's errors add, all of
       it times rs.
  dw   = sum of g v over n rows: terms by 2^-20 of the pair's gradients times |v| and r of
       themselves; a thread adds at most n / 8 of them after one another, a block 32 and then in
       64 bits: (n / 8 + 32) 2^-24 of the sum of magnitudes.
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


def _theta(d_rot, base=10000.0, linear=1.0, yarn=1.0):
    out = []
    for i in range(d_rot // 2):
        th = base ** (-2.0 * i / d_rot)
        if yarn > 1.0:
            lam = 2.0 * math.pi / th
            t = min(1.0, max(0.0, (lam - 1.0) / (yarn - 1.0)))
            div = yarn if lam > yarn else t * yarn + 1.0 - t
            th = th if lam < 32.0 else th / div
        out.append(th / linear)
    return torch.tensor(out, dtype=torch.float64)


def _pairs(d, half=False, rot_start=0, d_rot=None, **freq):
    d_rot = d - rot_start if d_rot is None else d_rot
    n = d_rot // 2
    a = rot_start + torch.arange(n) * (1 if half else 2)
    return a, a + (n if half else 1), _theta(d_rot, **freq)


def _turn(x, positions, sign, half=False, rot_start=0, d_rot=None, **freq):
    """(turned rows, sum of the magnitudes of each entry's pair) in 64 bits."""
    a, b, theta = _pairs(x.shape[-1], half, rot_start, d_rot, **freq)
    ang = sign * positions.double().cpu()[:, None, :, None] * theta
    y, mag = x.clone(), x.abs()
    y[..., a] = x[..., a] * ang.cos() - x[..., b] * ang.sin()
    y[..., b] = x[..., a] * ang.sin() + x[..., b] * ang.cos()
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def _weight(w, H, d):
    if w is None:
        return torch.ones(1, d, dtype=torch.float64)
    return w.double().cpu() if w.dim() == 2 else w.double().cpu()[None]


def _norm_ref(x, w, positions, eps, o):
    """(y, slack)"""
    x = x.double().cpu()
    d = x.shape[-1]
    rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y, mag = _turn(x * rs * _weight(w, x.shape[1], d)[None, :, None], positions, 1.0, **o)
    return y, mag * (d * 2.0 ** -25 + 2.0 ** -20 + 2.0 ** -21)


def _grad_ref(dy, x, w, positions, eps, o):
    """(dx, slack, dw [H, d], slack) with dw for each head"""
    x, dy = x.double().cpu(), dy.double().cpu()
    d, n = x.shape[-1], x.shape[0] * x.shape[2]
    wt = _weight(w, x.shape[1], d)[None, :, None]
    r = d * 2.0 ** -25 + 2.0 ** -20
    rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    g, mag = _turn(dy, positions, -1.0, **o)
    v, c = x * rs, g * wt
    ec = mag * wt.abs() * 2.0 ** -20
    m, am = (c * v).mean(-1, keepdim=True), (c * v).abs().mean(-1, keepdim=True)
    em = 2 * r * am + (ec * v.abs()).mean(-1, keepdim=True)
    dx = rs * (c - v * m)
    slack = rs * (ec + 2 * r * c.abs() + v.abs() * em + 2 * r * v.abs() * m.abs())
    terms = (g * v).abs().sum(dim=(0, 2))
    dw = (g * v).sum(dim=(0, 2))
    return dx, slack, dw, (mag * v.abs()).sum(dim=(0, 2)) * 2.0 ** -20 + terms * r, terms, n


def _close(got, ref, tol, what=""):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(err).all(), what
    assert (err <= tol).all(), (what, float((err - tol).max()))


CASES = [  # B, S, Hq, Hkv, d, options, weights
    (1, 1, 4, 2, 64, {}, "bf16"),
    (3, 7, 8, 8, 128, dict(half=True), "bf16"),
    (2, 33, 5, 1, 192, dict(rot_start=128, d_rot=64), "fp32"),
    (2, 33, 5, 1, 192, dict(rot_start=128, d_rot=64, half=True), "heads"),
    (2, 5, 16, 2, 128, dict(d_rot=32, half=True, base=500000.0), "heads"),
    (1, 300, 64, 8, 128, dict(linear=4.0), "fp32"),
    (2, 17, 3, 1, 80, dict(half=True), "bf16"),                # 10 lanes of 16
    (2, 17, 3, 1, 80, dict(d_rot=48), "bf16"),
    (2, 9, 3, 1, 80, dict(d_rot=20, half=True), "fp32"),       # halves of ten: 2 bytes at a time
    (2, 9, 3, 1, 66, dict(rot_start=6, d_rot=18), "heads"),
    (1, 4, 2, 2, 8, {}, "bf16"),
    (2, 40, 8, 2, 128, dict(yarn=32.0), "none"),
    (1, 3, 40, 40, 256, dict(half=True), "bf16"),
    (1, 2, 200, 100, 64, {}, "heads"),
    (1, 3, 2, 1, 1024, dict(d_rot=512, half=True, rot_start=256), "bf16"),  # the widest row
    (2, 700, 6, 3, 64, dict(half=True), "bf16"),
    (1, 1500, 32, 8, 128, dict(half=True), "bf16"),
    (2, 45, 9, 3, 512, dict(half=True, d_rot=256), "heads"),   # 32 lanes a row
    (1, 90, 20, 5, 384, dict(rot_start=128, d_rot=256), "heads"),
    (2, 300, 12, 5, 72, dict(half=True, d_rot=64, rot_start=8), "heads"),  # an odd number of chunks
    (2, 300, 12, 5, 72, dict(d_rot=8, rot_start=64), "fp32"),
]


def _inputs(dev, B, S, Hq, Hkv, d, weights, seed):
    g = _gen(dev, seed)
    q = _normal(g, dev, B, Hq, S, d) * torch.exp(torch.randn(1, Hq, 1, 1, generator=g, device=dev)).to(torch.bfloat16)
    k = _normal(g, dev, B, Hkv, S, d, scale=0.1)
    pos = torch.randint(0, 5000, (B, S), generator=g, device=dev, dtype=torch.int32)
    ws = []
    for H in (Hq, Hkv):
        w = 1 + 0.3 * torch.randn(*((H, d) if weights == "heads" else (d,)), generator=g, device=dev)
        ws.append(None if weights == "none" else w if weights == "fp32" else w.to(torch.bfloat16))
    return g, q, k, pos, ws


def _options(o):
    names = dict(base="rope_base", linear="linear_scale", yarn="yarn_scale")
    how = {names.get(n, n): x for n, x in o.items() if n != "half"}
    return dict(layout="half" if o.get("half") else "interleaved", **how)


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,Hq,Hkv,d,o,weights", CASES)
def test_norm_rope_matches_the_formula(B, S, Hq, Hkv, d, o, weights):
    dev = _gpu()
    _, q, k, pos, (qw, kw) = _inputs(dev, B, S, Hq, Hkv, d, weights, 10 * S + d)
    got = apex.norm_rope(q, k, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5, **_options(o))
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        ref, slack = _norm_ref(x, w, pos, 1e-5, o)
        _close(y, ref, U * ref.abs() + slack)
    alone = apex.norm_rope(q, positions=pos, q_weight=qw, eps=1e-5, **_options(o))
    assert torch.equal(alone, got[0])


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,Hq,Hkv,d,o,weights", CASES)
def test_norm_rope_grad_matches_the_formula(B, S, Hq, Hkv, d, o, weights):
    dev = _gpu()
    g, q, k, pos, (qw, kw) = _inputs(dev, B, S, Hq, Hkv, d, weights, 20 * S + d)
    dq, dk = _normal(g, dev, B, Hq, S, d), _normal(g, dev, B, Hkv, S, d, scale=3.0)
    how = dict(positions=pos, q_weight=qw, eps=1e-5, **_options(o))
    gq, gk, gqw, gkw = apex.norm_rope_grad(dq, q, dk, k, k_weight=kw, **how)
    for x, w, dy, dx, dw in ((q, qw, dq, gq, gqw), (k, kw, dk, gk, gkw)):
        ref, slack, rw, ew, terms, n = _grad_ref(dy, x, w, pos, 1e-5, o)
        _close(dx, ref, U * ref.abs() + slack, "dx")
        if w is None:
            assert dw is None
            continue
        assert dw.dtype == torch.float32 and dw.shape == w.shape
        if w.dim() == 1:
            rw, ew, terms, n = rw.sum(0), ew.sum(0), terms.sum(0), n * x.shape[1]
        _close(dw, rw, ew + terms * (n / 8 + 32) * 2.0 ** -24, "dw")
    again = apex.norm_rope_grad(dq, q, dk, k, k_weight=kw, **how)
    assert all(a is b or torch.equal(a, b) for a, b in zip(again, (gq, gk, gqw, gkw)))
    one = apex.norm_rope_grad(dq, q, **how)
    assert torch.equal(one[0], gq)


@pytest.mark.gpu
def test_gradients_agree_with_differences():
    """The change of sum(dy * y) along random directions, from the 64-bit formula."""
    dev = _gpu()
    g, q, _, pos, (w, _) = _inputs(dev, 2, 19, 4, 2, 128, "fp32", 3)
    dy = _normal(g, dev, 2, 4, 19, 128)
    o = dict(half=True, d_rot=64, rot_start=32)
    dx, dw = apex.norm_rope_grad(dy, q, positions=pos, q_weight=w, eps=1e-6, **_options(o))
    _, slack, _, ew, terms, n = _grad_ref(dy, q, w, pos, 1e-6, o)
    x0, w0, d64 = q.double().cpu(), w.double().cpu(), dy.double().cpu()

    def loss(x, wt):
        return (_norm_ref(x, wt, pos, 1e-6, o)[0] * d64).sum()

    for seed in range(4):
        r = torch.Generator().manual_seed(seed)
        vx, vw = torch.randn(x0.shape, generator=r, dtype=torch.float64), torch.randn(128, generator=r, dtype=torch.float64)
        h = 1e-5  # the difference is off by h^2 of the third derivative: far below the roundings
        along = (loss(x0 + h * vx, w0) - loss(x0 - h * vx, w0)) / (2 * h)
        tol = ((U * dx.double().cpu().abs() * (1 + U) + slack) * vx.abs()).sum() + 1e-5
        assert (along - (dx.double().cpu() * vx).sum()).abs() <= tol
        along = (loss(x0, w0 + h * vw) - loss(x0, w0 - h * vw)) / (2 * h)
        tol = ((ew.sum(0) + terms.sum(0) * (n * 4 / 8 + 32) * 2.0 ** -24) * vw.abs()).sum() + 1e-5
        assert (along - (dw.double().cpu() * vw).sum()).abs() <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("half", [False, True])
def test_strides_in_place_and_unaligned_rows(half):
    dev = _gpu()
    o = dict(half=half)
    g, q, k, pos, (qw, kw) = _inputs(dev, 2, 21, 6, 2, 64, "bf16", 5)
    want = apex.norm_rope(q, k, positions=pos, q_weight=qw, k_weight=kw, **_options(o))
    # as one projection leaves them: [B, S, Hq + 2 Hkv, d], worked on in place
    both = torch.cat([q, k, k], dim=1).transpose(1, 2).contiguous()
    vq, vk = both[:, :, :6].transpose(1, 2), both[:, :, 6:8].transpose(1, 2)
    got = apex.norm_rope(vq, vk, positions=pos, q_weight=qw, k_weight=kw, q_out=vq, k_out=vk, **_options(o))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].data_ptr() == both.data_ptr()
    assert torch.equal(both[:, :, 8:].transpose(1, 2), k)
    # rows that start on odd elements: the kernels that go 2 bytes at a time
    odd = torch.zeros(2, 6, 21, 67, dtype=torch.bfloat16, device=dev)[..., 1:65]
    odd.copy_(q)
    y = apex.norm_rope(odd, positions=pos, q_weight=qw, **_options(o))
    ref, slack = _norm_ref(q, qw, pos, 1e-6, o)
    _close(y, ref, U * ref.abs() + slack)
    dy = _normal(g, dev, 2, 6, 21, 64)
    dx, dw = apex.norm_rope_grad(dy, odd, positions=pos, q_weight=qw, **_options(o))
    rx, sx, rw, ew, terms, n = _grad_ref(dy, q, qw, pos, 1e-6, o)
    _close(dx, rx, U * rx.abs() + sx)
    _close(dw, rw.sum(0), ew.sum(0) + terms.sum(0) * (6 * n / 8 + 32) * 2.0 ** -24)
    # gradients over their own gradients or inputs
    base = apex.norm_rope_grad(dy, q, positions=pos, q_weight=qw, **_options(o))
    over, inp = dy.clone(), q.clone()
    a = apex.norm_rope_grad(over, q, positions=pos, q_weight=qw, q_out=over, **_options(o))
    b = apex.norm_rope_grad(dy, inp, positions=pos, q_weight=qw, q_out=inp, **_options(o))
    assert torch.equal(over, base[0]) and torch.equal(inp, base[0])
    assert torch.equal(a[1], base[1]) and torch.equal(b[1], base[1])
    over = odd.clone().contiguous()
    a = apex.norm_rope_grad(dy, odd, positions=pos, q_weight=qw, q_out=odd, **_options(o))
    assert torch.equal(odd, dx) and torch.equal(a[1], dw)


@pytest.mark.gpu
def test_broadcast_gradients_and_inputs():
    """Gradients and inputs of stride 0 (a summed loss, heads that share rows)."""
    dev = _gpu()
    _, q, k, pos, (qw, _) = _inputs(dev, 2, 9, 4, 1, 128, "bf16", 6)
    dy = torch.full((1,), 0.5, dtype=torch.bfloat16, device=dev).repeat(128).expand(2, 4, 9, 128)
    a = apex.norm_rope_grad(dy, q, positions=pos, q_weight=qw)
    b = apex.norm_rope_grad(dy.contiguous(), q, positions=pos, q_weight=qw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = k.expand(2, 4, 9, 128)
    assert torch.equal(apex.norm_rope(wide, positions=pos), apex.norm_rope(wide.contiguous(), positions=pos))


@pytest.mark.gpu
def test_odd_values():
    """Rows of zeros, of one entry, and rows that hold an infinity or a NaN: alone in what they give."""
    dev = _gpu()
    _, q, _, pos, (qw, _) = _inputs(dev, 1, 8, 2, 1, 128, "bf16", 7)
    want = apex.norm_rope(q, positions=pos, q_weight=qw)
    x = q.clone()
    x[0, 0, 1] = 0
    x[0, 0, 2] = 0
    x[0, 0, 2, 5] = 3.0
    x[0, 0, 3, 7] = float("nan")
    x[0, 0, 5, 7] = float("inf")
    y = apex.norm_rope(x, positions=pos, q_weight=qw)
    assert (y[0, 0, 1] == 0).all() and torch.isnan(y[0, 0, 3]).all() and torch.isnan(y[0, 0, 5]).any()
    ref, slack = _norm_ref(x[:, :, 2:3], qw, pos[:, 2:3], 1e-6, {})
    _close(y[:, :, 2:3], ref, U * ref.abs() + slack)
    keep = [0, 4, 6, 7]
    assert torch.equal(y[0, 0, keep], want[0, 0, keep]) and torch.equal(y[0, 1], want[0, 1])
    dx, _ = apex.norm_rope_grad(want, x, positions=pos, q_weight=qw)
    assert torch.isfinite(dx[0, 0, [0, 1, 2, 4, 6, 7]].float()).all() and torch.isfinite(dx[0, 1].float()).all()
    # a row of zeros and eps: rs = 1000, mean(c v) = 0
    ref, slack, *_ = _grad_ref(want[:, :, 1:2], x[:, :, 1:2], qw, pos[:, 1:2], 1e-6, {})
    _close(dx[:, :, 1:2], ref, U * ref.abs() + slack)


@pytest.mark.gpu
def test_appends_to_a_cache():
    dev = _gpu()
    g, q, k, pos, (qw, kw) = _inputs(dev, 4, 5, 8, 2, 128, "bf16", 8)
    v = _normal(g, dev, 4, 2, 5, 64)
    kc, vc = _normal(g, dev, 4, 2, 50, 128), _normal(g, dev, 4, 2, 50, 64)
    k0, v0 = kc.clone(), vc.clone()
    row0 = torch.tensor([0, 47, -2, 20], dtype=torch.int32, device=dev)
    plain = apex.norm_rope(q, k, v, positions=pos, q_weight=qw, k_weight=kw)
    assert torch.equal(plain[2], v)
    got = apex.norm_rope(q, k, v, positions=pos, q_weight=qw, k_weight=kw, k_out=kc, v_out=vc, row0=row0)
    assert torch.equal(got[0], plain[0]) and got[1] is kc and got[2] is vc
    for b, r in enumerate(row0.tolist()):
        for s in range(5):
            if 0 <= r + s < 50:
                k0[b, :, r + s] = plain[1][b, :, s]
                v0[b, :, r + s] = v[b, :, s]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


@pytest.mark.gpu
def test_is_the_norm_then_rope():
    """The two passes agree up to the rounding in between: u of the pair's entries, and u of the result."""
    dev = _gpu()
    _, q, _, pos, (qw, _) = _inputs(dev, 2, 60, 8, 2, 128, "fp32", 9)
    x = q.double()
    n = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * qw.double()).to(torch.bfloat16)
    one, two = apex.norm_rope(q, positions=pos, q_weight=qw).double(), apex.rope(n, positions=pos).double()
    mag = n.double().abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(2, 8, 60, 64, 2).flatten(-2)
    assert ((one - two).abs() <= U * (one.abs() + two.abs()) + mag * (U + 2.0 ** -18)).all()


@pytest.mark.gpu
def test_captured_and_replayed():
    dev = _gpu()
    g, q, k, pos, (qw, kw) = _inputs(dev, 2, 37, 8, 2, 128, "bf16", 11)
    dq, dk = _normal(g, dev, 2, 8, 37, 128), _normal(g, dev, 2, 2, 37, 128)
    ws = torch.empty(apex.norm_rope_grad_workspace_bytes(8, 2, 128), dtype=torch.uint8, device=dev)

    def calls():
        y = apex.norm_rope(q, k, positions=pos, q_weight=qw, k_weight=kw, layout="half")
        return y + apex.norm_rope_grad(dq, q, dk, k, positions=pos, q_weight=qw, k_weight=kw, layout="half",
                                       workspace=ws)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for i in range(3):
        for x in (q, k, dq, dk, qw, kw):
            x.normal_()
        pos.add_(100 * i)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, calls()))


@pytest.mark.gpu
def test_other_streams():
    dev = _gpu()
    g, q, k, pos, (qw, kw) = _inputs(dev, 2, 200, 8, 2, 128, "bf16", 12)
    dq, dk = _normal(g, dev, 2, 8, 200, 128), _normal(g, dev, 2, 2, 200, 128)
    how = dict(positions=pos, q_weight=qw, k_weight=kw)
    want = apex.norm_rope(q, k, **how) + apex.norm_rope_grad(dq, q, dk, k, **how)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = [apex.norm_rope(q, k, stream=streams[i % 2], **how) +
           apex.norm_rope_grad(dq, q, dk, k, stream=streams[i % 2], **how) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x in got for a, b in zip(x, want))


@pytest.mark.gpu
def test_outputs_and_workspaces_stay_within_their_bounds():
    dev = _gpu()
    pad = 4096
    for B, S, Hq, Hkv, d, o, weights in CASES:
        g, q, k, pos, (qw, kw) = _inputs(dev, B, S, Hq, Hkv, d, weights, 13)
        need = apex.norm_rope_grad_workspace_bytes(Hq, Hkv, d)
        buf = torch.full((need + 2 * pad,), 0xA5, dtype=torch.uint8, device=dev)
        apex.norm_rope_grad(q, q, k, k, positions=pos, q_weight=qw, k_weight=kw, workspace=buf[pad:pad + need],
                            **_options(o))
        assert (buf[:pad] == 0xA5).all() and (buf[pad + need:] == 0xA5).all()


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
    f = dict(x=P, dy=3 * P, out=2 * P, weight=4 * P, dweight=5 * P, n_heads=4, d_row=128, weight_f32=0,
             weight_per_head=0, x_b=512, x_h=128, x_s=512, dy_b=512, dy_h=128, dy_s=512, out_b=512, out_h=128, out_s=512)
    f.update(o)
    return apex.NormTensor(*[f[n] for n, _ in apex.NormTensor._fields_])


BOTH = [
    (dict(x=None), {}, {}, BAD), (dict(out=None), {}, {}, BAD), (dict(x=P + 1), {}, {}, BAD),
    (dict(out=2 * P + 1), {}, {}, BAD), (dict(weight=4 * P + 1), {}, {}, BAD),
    (dict(weight=4 * P + 2, weight_f32=1), {}, {}, BAD), (dict(weight_f32=2), {}, {}, BAD),
    (dict(n_heads=0), {}, {}, BAD), (dict(d_row=-8), {}, {}, BAD), (dict(d_row=2048), dict(d_rot=64), {}, UNSUPPORTED),
    (dict(n_heads=16385), {}, {}, UNSUPPORTED),
    ({}, dict(layout=2), {}, BAD), ({}, dict(d_rot=3), {}, BAD), ({}, dict(d_rot=130), {}, BAD),
    ({}, dict(rot_start=128), {}, BAD), ({}, dict(rot_start=-2), {}, BAD), ({}, dict(rope_base=-1.0), {}, BAD),
    ({}, dict(linear_scale=float("nan")), {}, BAD), ({}, dict(yarn_scale=float("nan")), {}, BAD),
    ({}, {}, dict(B=0), BAD), ({}, {}, dict(S=-1), BAD), ({}, {}, dict(positions=None), BAD),
    ({}, {}, dict(positions=P + 2), BAD), ({}, {}, dict(pos_stride=-1), BAD), ({}, {}, dict(eps=-1e-6), BAD),
    ({}, {}, dict(eps=float("nan")), BAD), ({}, {}, dict(eps=float("inf")), BAD),
    ({}, {}, dict(B=1 << 16, S=1 << 16), UNSUPPORTED),
    (dict(out=P + 256), {}, {}, BAD), (dict(out=P, out_h=64), {}, {}, BAD),  # shifted rows, rows on one another
    (dict(weight=2 * P + 8), {}, {}, BAD),                                    # the result on the weights
]


@pytest.mark.parametrize("tensor,opt,args,code", BOTH + [({}, {}, dict(row0=P), BAD), ({}, {}, dict(row0=P + 1, rows=4), BAD)])
def test_norm_rope_refuses(lib, tensor, opt, args, code):
    a = dict(B=1, S=1, positions=P, pos_stride=1, row0=None, rows=0, eps=1e-6)
    a.update(args)
    t, o = _tensor(**tensor), apex.RopeOptions(**opt)
    for k in (None, _tensor(x=8 * P, out=9 * P)):
        assert apex.apex_attn_norm_rope(t, k, None, a["B"], a["S"], a["positions"], a["pos_stride"], a["row0"],
                                        a["rows"], o, a["eps"], None) == code
    assert apex.apex_attn_norm_rope(None, t, None, 1, 1, P, 1, None, 0, o, 1e-6, None) == BAD
    assert apex.apex_attn_norm_rope(t, None, None, 1, 1, P, 1, None, 0, None, 1e-6, None) == BAD


@pytest.mark.parametrize("tensor,opt,args,code", BOTH + [
    (dict(dy=None), {}, {}, BAD), (dict(dy=3 * P + 1), {}, {}, BAD), (dict(dweight=5 * P + 2), {}, {}, BAD),
    (dict(out=3 * P + 256), {}, {}, BAD), (dict(dweight=P), {}, {}, BAD), (dict(dweight=2 * P), {}, {}, BAD),
    (dict(dweight=4 * P), {}, {}, BAD), ({}, {}, dict(ws=None), BAD), ({}, {}, dict(ws=P + 8), BAD),
    ({}, {}, dict(n=1024 * 128 * 4 - 1), BAD),
])
def test_norm_rope_grad_refuses(lib, tensor, opt, args, code):
    a = dict(B=1, S=1, positions=P, pos_stride=1, eps=1e-6, ws=P, n=1 << 40)
    a.update(args)
    o = apex.RopeOptions(**opt)
    for k in (None, _tensor(x=8 * P, out=9 * P, dweight=10 * P)):
        assert apex.apex_attn_norm_rope_grad(_tensor(**tensor), k, a["B"], a["S"], a["positions"], a["pos_stride"], o,
                                             a["eps"], a["ws"], a["n"], None) == code


def test_rows_that_disagree_and_outputs_of_two_tensors(lib):
    o = apex.RopeOptions()
    call = lambda q, k: apex.apex_attn_norm_rope(q, k, None, 1, 1, P, 1, None, 0, o, 1e-6, None)  # noqa: E731
    assert call(_tensor(), _tensor(x=8 * P, out=9 * P, d_row=64)) == BAD
    assert call(_tensor(), _tensor(x=8 * P)) == BAD      # both results at 2 P
    assert call(_tensor(), _tensor(x=2 * P, out=9 * P)) == BAD
    grad = lambda q, k: apex.apex_attn_norm_rope_grad(q, k, 1, 1, P, 1, o, 1e-6, P, 1 << 40, None)  # noqa: E731
    assert grad(_tensor(), _tensor(x=8 * P, out=9 * P)) == BAD  # both weights' gradients at 5 P


@pytest.mark.parametrize("H_q,H_kv,d_q,d_k,bad", [(4, 2, 64, 64, False), (1, 0, 1024, 0, False), (0, 1, 64, 64, True),
                                                  (4, -1, 64, 64, True), (4, 2, 2048, 64, True), (20000, 2, 64, 64, True)])
def test_workspace_bytes(lib, H_q, H_kv, d_q, d_k, bad):
    assert (apex.norm_rope_grad_workspace_bytes(H_q, H_kv, d_q, d_k) == 0) == bad


def test_conveniences_refuse_cpu_tensors(lib):
    x, pos = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        apex.norm_rope(x, positions=pos)
    with pytest.raises(TypeError):
        apex.norm_rope_grad(x, x, positions=pos)
    with pytest.raises(ValueError):
        apex.norm_rope_grad(x, x, x, positions=pos)


@pytest.mark.gpu
def test_conveniences_refuse_what_does_not_fit():
    dev = _gpu()
    _, q, k, pos, (qw, kw) = _inputs(dev, 2, 4, 8, 2, 128, "bf16", 14)
    for bad in (lambda: apex.norm_rope(q, positions=pos.long()), lambda: apex.norm_rope(q, positions=pos, q_weight=qw.half()),
                lambda: apex.norm_rope(q, positions=pos, q_weight=qw.cpu()), lambda: apex.norm_rope(q.float(), positions=pos),
                lambda: apex.norm_rope_grad(q.float(), q, positions=pos)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: apex.norm_rope(q, positions=pos[:1]), lambda: apex.norm_rope(q, positions=pos, q_weight=qw[:64]),
                lambda: apex.norm_rope(q, positions=pos, q_weight=qw.expand(2, 128)),
                lambda: apex.norm_rope(q, positions=pos, k_weight=qw), lambda: apex.norm_rope(q, v=k, positions=pos),
                lambda: apex.norm_rope(q, k, positions=pos, row0=pos[:, 0].contiguous()),
                lambda: apex.norm_rope(q, positions=pos, layout="neox"), lambda: apex.norm_rope(q, positions=pos, d_rot=0),
                lambda: apex.norm_rope_grad(q[:, :4], q, positions=pos), lambda: apex.norm_rope_grad(q, q, k, positions=pos),
                lambda: apex.norm_rope_grad(q, q, positions=pos, q_out=q[:, :4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(apex.ApexError):
        apex.norm_rope(q, positions=pos, eps=-1.0)
    with pytest.raises(apex.ApexError):
        apex.norm_rope_grad(q, q, positions=pos, workspace=torch.empty(16, dtype=torch.uint8, device=dev))


# ------------------------------------------------------------------------------------------------- many tokens
@pytest.mark.gpu
@pytest.mark.parametrize("half,each", [(True, True), (False, True), (True, False)])
def test_many_tokens_are_their_parts(half, each):
    """Blocks that go over several tiles, over the ends of sequences: rows as those of a call over a part of
    the tokens, bit for bit, and sums of weights as those of the parts."""
    dev = _gpu()
    g = _gen(dev, 31)
    B, S, H, d, part = 3, 6301, 16, 128, 997
    q, k = _normal(g, dev, B, S, H, d).transpose(1, 2), _normal(g, dev, B, S, H, d).transpose(1, 2)
    dq, dk = _normal(g, dev, B, H, S, d), _normal(g, dev, B, H, S, d)
    w = [1 + 0.1 * torch.randn(*((H, d) if each else (d,)), generator=g, device=dev) for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (B, S), generator=g, device=dev, dtype=torch.int32)
    how = dict(q_weight=w[0], k_weight=w[1], layout="half" if half else "interleaved")
    whole = apex.norm_rope(q, k, positions=pos, **how)
    gq, gk, gqw, gkw = apex.norm_rope_grad(dq, q, dk, k, positions=pos, **how)
    sums = [torch.zeros_like(x, dtype=torch.float64) for x in (gqw, gkw)]
    sizes = [torch.zeros_like(x) for x in sums]
    for lo in range(0, S, part):
        at = slice(lo, lo + part)
        p = pos[:, at].contiguous()
        a = [x[:, :, at] for x in (q, k, dq, dk)]
        rows = apex.norm_rope(a[0], a[1], positions=p, **how)
        assert torch.equal(rows[0], whole[0][:, :, at]) and torch.equal(rows[1], whole[1][:, :, at])
        grads = apex.norm_rope_grad(a[2], a[0], a[3], a[1], positions=p, **how)
        assert torch.equal(grads[0], gq[:, :, at]) and torch.equal(grads[1], gk[:, :, at])
        for i in range(2):
            sums[i] += grads[2 + i].double()
            # magnitudes of the terms: a turned gradient's entry is at most its pair's, a normed one at most sqrt(d)
            x = a[i].float()
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True))
            y = a[2 + i].float()
            far = (y.unflatten(-1, (2, -1)) if half else y.unflatten(-1, (-1, 2))).norm(dim=-2 if half else -1)
            far = torch.cat([far, far], -1) if half else far.repeat_interleave(2, -1)
            sizes[i] += (far * x.abs()).double().sum((0, 2) if each else (0, 1, 2))
    # both ways sums of the same fp32 terms: threads' runs of at most n / 8 + 32 terms, as above, twice
    n = B * S * (1 if each else H)
    for got, ref, size in zip((gqw, gkw), sums, sizes):
        assert ((got.double() - ref).abs() <= 2 * (n / 8 + 32) * 2.0 ** -24 * size).all()


@pytest.mark.gpu
@pytest.mark.parametrize("half,weights", [(True, "bf16"), (False, "heads")])
def test_batches_of_single_tokens(half, weights):
    """More sequences of a token than blocks run at once, appended to caches of their own rows."""
    dev = _gpu()
    B, Hq, Hkv, d, cap = 1100, 24, 6, 128, 5
    g, q, k, pos, (qw, kw) = _inputs(dev, B, 1, Hq, Hkv, d, weights, 41)
    v = _normal(g, dev, B, Hkv, 1, d)
    row0 = torch.randint(-1, cap + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    kc, vc = (torch.full((B, Hkv, cap, d), 3.0, dtype=torch.bfloat16, device=dev) for _ in "kv")
    o = dict(half=half)
    got = apex.norm_rope(q, k, v, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5, k_out=kc, v_out=vc, row0=row0, **_options(o))
    ref, slack = _norm_ref(q, qw, pos, 1e-5, o)
    _close(got[0], ref, U * ref.abs() + slack)
    rk, sk = _norm_ref(k, kw, pos, 1e-5, o)
    rows = torch.arange(cap)[None] == row0.cpu()[:, None]
    keep = ~rows[:, None, :, None]
    ref = torch.where(keep, torch.full((1,), 3.0, dtype=torch.float64), rk)
    _close(kc, ref, torch.where(keep, torch.zeros(1, dtype=torch.float64), U * rk.abs() + sk))
    assert torch.equal(vc.cpu(), torch.where(keep, torch.full((1,), 3.0, dtype=torch.bfloat16), v.cpu()))
    dq, dk = _normal(g, dev, B, Hq, 1, d), _normal(g, dev, B, Hkv, 1, d)
    grads = apex.norm_rope_grad(dq, q, dk, k, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5, **_options(o))
    for x, w, dy, dx, dw in ((q, qw, dq, grads[0], grads[2]), (k, kw, dk, grads[1], grads[3])):
        ref, slack, rw, ew, terms, n = _grad_ref(dy, x, w, pos, 1e-5, o)
        _close(dx, ref, U * ref.abs() + slack, "dx")
        if w.dim() == 1:
            rw, ew, terms, n = rw.sum(0), ew.sum(0), terms.sum(0), n * x.shape[1]
        _close(dw, rw, ew + terms * (n / 8 + 32) * 2.0 ** -24, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["fp32", "heads"])
def test_many_rows_two_bytes_at_a_time(weights):
    """More tokens than warps: the pass past 2^18 of them, the gradient past its 1024 blocks of four."""
    dev = _gpu()
    o = dict(half=True, rot_start=2, d_rot=14)
    for B, S, Hq, Hkv, grad in ((2, 150001, 1, 1, False), (3, 3333, 5, 2, True)):
        d = 18
        g, q, k, pos, (qw, kw) = _inputs(dev, B, S, Hq, Hkv, d, weights, S)
        got = apex.norm_rope(q, k, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5, **_options(o))
        for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
            ref, slack = _norm_ref(x, w, pos, 1e-5, o)
            _close(y, ref, U * ref.abs() + slack)
        if not grad:
            continue
        dq, dk = _normal(g, dev, B, Hq, S, d), _normal(g, dev, B, Hkv, S, d)
        grads = apex.norm_rope_grad(dq, q, dk, k, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5, **_options(o))
        for x, w, dy, dx, dw in ((q, qw, dq, grads[0], grads[2]), (k, kw, dk, grads[1], grads[3])):
            ref, slack, rw, ew, terms, n = _grad_ref(dy, x, w, pos, 1e-5, o)
            _close(dx, ref, U * ref.abs() + slack, "dx")
            if w.dim() == 1:
                rw, ew, terms, n = rw.sum(0), ew.sum(0), terms.sum(0), n * x.shape[1]
            _close(dw, rw, ew + terms * (n / 8 + 32) * 2.0 ** -24, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 126])  # 16 bytes and 2 bytes at a time
def test_rows_past_32_bit_offsets(d):
    """Entries past 2^31 of a tensor, its output, a cache and the gradients: as a call over those tokens alone."""
    dev = _gpu()
    g = _gen(dev, 51)
    H, S, n = 64, 280000, 37  # 2.3e9 entries
    try:
        q = torch.empty(1, H, S, d, dtype=torch.bfloat16, device=dev)
        dq, out, cache = (torch.empty_like(q) for _ in range(3))
    except torch.OutOfMemoryError:
        pytest.skip("needs 20 GB")
    for x in (q, dq):
        for h in range(H):
            x[0, h].normal_(generator=g)
    pos = torch.arange(S, dtype=torch.int32, device=dev)
    w = torch.ones(d, dtype=torch.bfloat16, device=dev)
    last = slice(S - n, S)
    apex.norm_rope(q, positions=pos, q_weight=w, q_out=out)
    few = apex.norm_rope(q[:, :, last], positions=pos[last], q_weight=w)
    assert torch.equal(out[:, :, last], few)
    # appended behind, at rows of a cache whose last heads lie past 2^31
    row0 = torch.full((1,), S - n, dtype=torch.int32, device=dev)
    apex.norm_rope(q[:, :1, last], q[:, :, last], positions=pos[last], k_weight=w, k_out=cache, row0=row0)
    assert torch.equal(cache[:, :, last], few)
    apex.norm_rope_grad(dq, q, positions=pos, q_weight=w, q_out=out)
    few, _ = apex.norm_rope_grad(dq[:, :, last], q[:, :, last], positions=pos[last], q_weight=w)
    assert torch.equal(out[:, :, last], few)
