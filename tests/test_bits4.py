"""Caches held in 4 bits -- append4, unpack4, decode4 -- against plain 64-bit implementations.

Codes and scales are compared bit for bit: they follow from comparisons that 64 bits decide
exactly (a quotient is no nearer to a tie than 2^-16 of itself unless it is one, for inputs of 8
and scales of 4 significant bits and factors that are powers of two; for other factors quotients
within 2^-22 of a tie go either way, and are compared as values only).

Tolerances of decode4 (u = 2^-8: half a step of bf16, relative to the value; fp16 2^-11, fp32 2^-24):
  a weight is rounded to fp16 after its sum was made: 2^-11 A, A = sum p |v|, and weights 2^-25 below
  the largest lose up to 2^-36 of it each: n 2^-36 max|v|; the result is rounded, u |out|.  Values
  and keys are exact.  A query entry is exact in fp16 but for what lies 2^-18 below its row's largest q:
  off by up to 2^-29 of that.  A score is d products added in fp32: off by at most
  e = scale (d 2^-24 sum |q k| + 2^-29 max|q| sum |k|), and scaled twice more, 2^-23 |score|: the
  weights' numerators and denominators move by that, 2 e A in the sum.  exp2 and the sums of weights
  in fp32 (16 keys a warp one after another): 2^-13 A at most for the lengths here.
"""
import math

import pytest
import torch

import transformer_attention_rope_gb300 as apex

U = 2.0 ** -8
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


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


def _cache(dev, B, H, cap, d, fill=None, g=None):
    """Packed tensors: zeros, a byte everywhere, or random bytes."""
    out = []
    for n in (d // 2, d // 16):
        if g is not None:
            x = torch.randint(0, 256, (B, H, cap, n), generator=g, device=dev, dtype=torch.uint8)
        else:
            x = torch.full((B, H, cap, n), fill or 0, dtype=torch.uint8, device=dev)
        out.append(x)
    return out[0], out[1].view(torch.float8_e4m3fn)


def _bits(scale):
    return scale.view(torch.uint8)


def _pack_ref(x, factor, ties=None):
    """(codes [..., d] 0..7, scale bytes, values) of x [B, H, S, d], 64 bits; ties: a list that gets
    the mask of quotients that fp32 cannot tell from a tie (None: there are none)."""
    f = torch.ones(x.shape[1], dtype=torch.float64) if factor is None else factor.double().cpu()
    f = f[:, None, None, None]
    b = x.double().cpu().unflatten(-1, (-1, 16))
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    b = torch.where(bad, torch.zeros_like(b), b)
    top = (b.abs().amax(-1, keepdim=True) / (6 * f)).clamp(max=448.0)
    s8 = top.float().to(torch.float8_e4m3fn)
    step = s8.double() * f
    q = torch.where(step > 0, b.abs() / torch.where(step > 0, step, 1.0), torch.zeros_like(b))
    code = torch.zeros_like(q, dtype=torch.int64)
    near = torch.zeros_like(q, dtype=torch.bool)
    for mid, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (q >= mid) if up else (q > mid)
        off = (q / mid - 1).abs()
        near |= (off > 0) & (off <= 2.0 ** -21)
    assert ties is not None or not near.any()
    if ties is not None:
        ties.append(near.flatten(-2))
    mag = torch.tensor(VALUES, dtype=torch.float64)[code]
    val = torch.where(torch.signbit(x.cpu().unflatten(-1, (-1, 16))), -mag, mag) * step
    val = torch.where(bad, torch.full_like(val, float("nan")), val)
    code = torch.where(bad, torch.zeros_like(code), code)
    bytes_ = torch.where(bad, torch.tensor(0x7F, dtype=torch.uint8), s8.view(torch.uint8)).squeeze(-1)
    return code.flatten(-2), bytes_, val.flatten(-2)


def _codes(x4):
    """Magnitude codes [..., d] of packed bytes (the sign of a zero is not compared)."""
    x4 = x4.cpu().long()
    return torch.stack([x4 & 15, x4 >> 4], dim=-1).flatten(-2) & 7


def _values(x4, scale, factor):
    """What packed rows stand for, 64 bits."""
    x4 = x4.cpu().long()
    c = torch.stack([x4 & 15, x4 >> 4], dim=-1).flatten(-2)
    table = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64)
    v = table[c] * scale.cpu().float().double().repeat_interleave(16, dim=-1)
    return v if factor is None else v * factor.double().cpu()[:, None, None]


# ------------------------------------------------------------------------------------------------- rows
ROWS = [  # B, H, S, d_k, d_v, cap, factors
    (1, 1, 1, 64, 64, 1, False),
    (2, 8, 1, 128, 128, 33, True),
    (3, 2, 17, 192, 128, 40, True),
    (1, 4, 300, 128, 128, 300, False),
    (2, 3, 9, 16, 512, 9, True),
    (2, 3, 9, 48, 80, 11, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,S,dk,dv,cap,factors", ROWS)
def test_append_and_unpack(B, H, S, dk, dv, cap, factors):
    dev = _gpu()
    g = _gen(dev, S + dk)
    k, v = _normal(g, dev, B, H, S, dk), _normal(g, dev, B, H, S, dv, scale=0.02)
    fk = 2.0 ** -torch.arange(H, device=dev, dtype=torch.float32) if factors else None
    fv = torch.full((H,), 2.0 ** -9, device=dev) if factors else None
    k4, ks = _cache(dev, B, H, cap, dk, g=g)
    v4, vs = _cache(dev, B, H, cap, dv, g=g)
    before = [x.clone() for x in (k4, _bits(ks), v4, _bits(vs))]
    row0 = torch.randint(0, cap - S + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    apex.append4(k, v, k4, ks, v4, vs, row0=row0, k_factor=fk, v_factor=fv)
    ko, vo = apex.unpack4(k4, ks, v4, vs, row0=row0, n_rows=S, k_factor=fk, v_factor=fv)
    for x, x4, s, f, out, i in ((k, k4, ks, fk, ko, 0), (v, v4, vs, fv, vo, 2)):
        code, sb, val = _pack_ref(x, f)
        for b, r in enumerate(row0.tolist()):
            assert torch.equal(_codes(x4[b, :, r:r + S]), code[b])
            assert torch.equal(_bits(s)[b, :, r:r + S].cpu(), sb[b])
            before[i][b, :, r:r + S] = x4[b, :, r:r + S]
            before[i + 1][b, :, r:r + S] = _bits(s)[b, :, r:r + S]
        assert torch.equal(before[i], x4) and torch.equal(before[i + 1], _bits(s))  # the other rows stay
        assert torch.equal(out.double().cpu(), val)


@pytest.mark.gpu
def test_any_factor():
    """Factors that are no powers of two: codes still the nearest, values rounded once to bf16."""
    dev = _gpu()
    g = _gen(dev, 2)
    k = _normal(g, dev, 1, 2, 40, 64)
    f = torch.tensor([0.0123, 7.7], device=dev)
    k4, ks = _cache(dev, 1, 2, 40, 64)
    v4, vs = _cache(dev, 1, 2, 40, 64)
    apex.append4(k, k, k4, ks, v4, vs, k_factor=f, v_factor=f)
    ties = []
    code, sb, val = _pack_ref(k, f, ties)
    clear = ~ties[0]
    assert torch.equal(_codes(k4)[clear], code[clear]) and torch.equal(_bits(ks).cpu(), sb)
    assert clear.double().mean() > 0.9 and ((_codes(k4) - code).abs() <= 1).all()
    ko, _ = apex.unpack4(k4, ks, v4, vs, k_factor=f, v_factor=f)
    # value * scale is exact, the product with the factor off by 2^-24 before the one rounding
    val = _values(k4, ks, f)
    assert ((ko.double().cpu() - val).abs() <= (U + 2.0 ** -22) * val.abs()).all()


@pytest.mark.gpu
def test_ties_extremes_and_values_that_are_not_finite():
    dev = _gpu()
    x = torch.zeros(1, 1, 12, 64, dtype=torch.float64)
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    for r, s in enumerate((1.0, 0.25, 1.75, 448.0, 2.0 ** -6, 2.0 ** -9)):
        x[0, 0, r, :16] = torch.tensor([6.0] + mids + [-m for m in mids] + [-6.0], dtype=torch.float64) * s
    x[0, 0, 6, 0] = 3e38          # past what 448 * 6 holds
    x[0, 0, 7, :2] = torch.tensor([1e-30, -1e-38])  # a scale of zero
    x[0, 0, 8, 3] = float("inf")
    x[0, 0, 9, 20] = float("nan")
    x[0, 0, 10, 16:32] = -0.0
    k = x.to(torch.bfloat16).to(dev)
    k4, ks = _cache(dev, 1, 1, 12, 64, fill=0xFF)
    v4, vs = _cache(dev, 1, 1, 12, 64, fill=0xFF)
    apex.append4(k, k, k4, ks, v4, vs)
    code, sb, val = _pack_ref(k, None)
    assert torch.equal(_codes(k4), code) and torch.equal(_bits(ks).cpu(), sb)
    ko, vo = apex.unpack4(k4, ks, v4, vs)
    assert torch.equal(torch.isnan(ko.cpu()), torch.isnan(val)) and torch.isnan(val).sum() == 32
    assert torch.equal(ko.double().cpu().nan_to_num(0.0), val.nan_to_num(0.0)) and torch.equal(k4, v4)
    assert float(ko[0, 0, 6, 0]) == 2688.0


@pytest.mark.gpu
def test_reciprocals_past_the_largest_number():
    """scale * factor below 2^-126: the quotient is divided out."""
    dev = _gpu()
    k = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=dev)
    k[..., :8] = torch.tensor([6.0, 3.0, -1.5, 0.5, 4.0, 2.0, 1.0, -6.0]) * 2.0 ** -125
    f = torch.tensor([2.0 ** -119], device=dev)  # scale 2^-6
    k4, ks = _cache(dev, 1, 1, 1, 64)
    v4, vs = _cache(dev, 1, 1, 1, 64)
    apex.append4(k, k, k4, ks, v4, vs, k_factor=f)
    assert _codes(k4)[0, 0, 0, :8].tolist() == [7, 5, 3, 1, 6, 4, 2, 7]
    assert float(ks.float()[0, 0, 0, 0]) == 2.0 ** -6


@pytest.mark.gpu
def test_rows_outside_and_strides():
    dev = _gpu()
    g = _gen(dev, 4)
    B, H, S, d, cap = 4, 2, 6, 128, 20
    k, v = _normal(g, dev, B, H, S, d), _normal(g, dev, B, H, S, d)
    k4, ks = _cache(dev, B, H, cap, d, g=g)
    v4, vs = _cache(dev, B, H, cap, d, g=g)
    want = [x.clone() for x in (k4, _bits(ks), v4, _bits(vs))]
    full = [_cache(dev, B, H, S, d) for _ in range(2)]
    apex.append4(k, v, *full[0], *full[1])
    row0 = torch.tensor([-3, 17, 100, 5], dtype=torch.int32, device=dev)
    # as one projection leaves them: [B, S, 2 H, d]
    both = torch.cat([k, v], dim=1).transpose(1, 2).contiguous()
    apex.append4(both[:, :, :H].transpose(1, 2), both[:, :, H:].transpose(1, 2), k4, ks, v4, vs, row0=row0)
    for w, part in zip(want, (full[0][0], _bits(full[0][1]), full[1][0], _bits(full[1][1]))):
        for b, r in enumerate(row0.tolist()):
            for s in range(S):
                if 0 <= r + s < cap:
                    w[b, :, r + s] = part[b, :, s]
    assert all(torch.equal(a, b) for a, b in zip(want, (k4, _bits(ks), v4, _bits(vs))))
    # rows that start on odd elements, and outputs of any strides
    odd = torch.zeros(B, H, S, d + 3, dtype=torch.bfloat16, device=dev)[..., 1:d + 1]
    odd.copy_(k)
    k4b, ksb = _cache(dev, B, H, S, d)
    apex.append4(odd, v, k4b, ksb, *full[1])
    assert torch.equal(k4b, full[0][0]) and torch.equal(_bits(ksb), _bits(full[0][1]))
    ko, vo = apex.unpack4(k4, ks, v4, vs, row0=row0, n_rows=S)
    out = torch.full((B, S, H, d + 3), 7.0, dtype=torch.bfloat16, device=dev)
    into = out[..., 1:d + 1].transpose(1, 2)
    apex.unpack4(k4, ks, v4, vs, row0=row0, n_rows=S, k_out=into)
    assert torch.equal(into, ko) and (out[..., 0] == 7).all() and (out[..., d + 1:] == 7).all()
    for b, r in enumerate(row0.tolist()):
        for s in range(S):
            inside = 0 <= r + s < cap
            assert inside or (ko[b, :, s] == 0).all() and (vo[b, :, s] == 0).all()


# ------------------------------------------------------------------------------------------------- attention
def _attn_ref(q, k, v, lens, window=0, n_sink=0, scale=None):
    """(out, tolerance) in 64 bits of q [B,Hq,T,d] over the values k, v [B,Hkv,cap,d]."""
    q = q.double().cpu()
    B, Hq, T, d = q.shape
    Hkv, cap, dv = v.shape[1:]
    G = Hq // Hkv
    scale = 1 / math.sqrt(d) if not scale else scale
    out, tol = torch.zeros(B, Hq, T, dv, dtype=torch.float64), torch.zeros(B, Hq, T, dv, dtype=torch.float64)
    j = torch.arange(cap)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        for t in range(T):
            m = n + t
            seen = j <= m
            if window > 0:
                seen &= (m - j < window) | (j < n_sink)
            idx = seen.nonzero().flatten()
            if not len(idx):
                continue
            for h in range(Hkv):
                kk, vv, x = k[b, h, idx], v[b, h, idx], q[b, h * G:(h + 1) * G, t]
                s = x @ kk.T * scale
                p = torch.softmax(s, -1)
                o, A = p @ vv, p @ vv.abs()
                e = scale * (d * 2.0 ** -24 * (x.abs() @ kk.abs().T)
                             + 2.0 ** -29 * x.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)) + 2.0 ** -23 * s.abs()
                e = e.amax(-1, keepdim=True)
                out[b, h * G:(h + 1) * G, t] = o
                tol[b, h * G:(h + 1) * G, t] = U * o.abs() + A * (2.0 ** -11 + 2 * e + 2.0 ** -13) \
                    + len(idx) * 2.0 ** -36 * vv.abs().max()
    return out, tol


def _close(got, ref, tol):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(err).all()
    assert (err <= tol).all(), float((err - tol).max())


def _attn_inputs(dev, seed, Hq, Hkv, T, dk, dv, cap, lens, factors=False, q_scale=1.5):
    g = _gen(dev, seed)
    B = len(lens)
    q = _normal(g, dev, B, Hq, T, dk, scale=q_scale)
    fk = 2.0 ** -(2 + torch.arange(Hkv, device=dev, dtype=torch.float32) % 3) if factors else None
    fv = 0.3 * torch.rand(Hkv, generator=g, device=dev) + 0.1 if factors else None
    cache = _cache(dev, B, Hkv, cap, dk) + _cache(dev, B, Hkv, cap, dv)
    apex.append4(_normal(g, dev, B, Hkv, cap, dk), _normal(g, dev, B, Hkv, cap, dv), *cache, k_factor=fk, v_factor=fv)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    vals = _values(cache[0], cache[1], fk), _values(cache[2], cache[3], fv)
    return q, cache, ln, dict(k_factor=fk, v_factor=fv), vals


ATTN = [  # Hq, Hkv, T, dk, dv, cap, lens, window, sinks
    (4, 2, 1, 64, 64, 1, [0], 0, 0),
    (4, 2, 1, 64, 64, 130, [0, 1, 129, 64], 0, 0),
    (8, 8, 1, 128, 128, 300, [299, 17], 0, 0),
    (32, 8, 1, 128, 128, 2100, [2099, 5, 1000], 0, 0),
    (16, 1, 1, 128, 128, 777, [700, 776], 100, 4),
    (32, 8, 1, 128, 128, 1500, [1499, 130, 3, 700], 128, 4),
    (32, 8, 4, 128, 128, 1500, [1400, 130, 3], 1, 1),
    (32, 8, 2, 128, 128, 1501, [1400, 130, 3], 200, 130),
    (8, 2, 3, 192, 128, 403, [400, 255, 0], 0, 0),
    (16, 1, 1, 192, 128, 3000, [2999], 1000, 300),
    (8, 2, 5, 64, 64, 500, [495, 100], 64, 7),
    (16, 1, 3, 64, 64, 260, [257, 30], 0, 0),     # 48 rows: three groups
    (8, 1, 64, 128, 128, 400, [336, 0], 50, 2),   # 512 rows
    (4, 4, 16, 128, 128, 2000, [1900, 1984], 0, 0),
    (4, 2, 1, 128, 128, 40000, [39999], 0, 0),
    (16, 1, 2, 192, 128, 900, [898, 5], 200, 140),   # 32 rows: the kernel for many
    (32, 2, 6, 192, 128, 1300, [1294, 600, 0], 0, 0),
    (16, 1, 16, 64, 64, 1000, [984, 130], 100, 4),   # 256 rows: two groups
    (8, 1, 9, 128, 128, 3000, [2991, 2000, 64], 0, 0),
    (16, 2, 40, 128, 128, 700, [660, 1], 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("factors", [False, True])
@pytest.mark.parametrize("Hq,Hkv,T,dk,dv,cap,lens,window,sinks", ATTN)
def test_decode4_matches_the_formula(Hq, Hkv, T, dk, dv, cap, lens, window, sinks, factors):
    dev = _gpu()
    q, cache, ln, f, vals = _attn_inputs(dev, cap + T, Hq, Hkv, T, dk, dv, cap, lens, factors)
    got = apex.decode4(q, *cache, ln, window=window, n_sink=sinks, **f)
    _close(got, *_attn_ref(q, *vals, lens, window, sinks))
    assert torch.equal(got, apex.decode4(q, *cache, ln, window=window, n_sink=sinks, **f))


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 3), (200, 100)])
def test_rows_that_nobody_sees_may_hold_anything(window, sinks):
    dev = _gpu()
    lens, T, cap = [500, 0, 130, 1000], 2, 1003
    q, cache, ln, f, vals = _attn_inputs(dev, 7, 16, 2, T, 128, 128, cap, lens)
    want = apex.decode4(q, *cache, ln, window=window, n_sink=sinks)
    _close(want, *_attn_ref(q, *vals, lens, window, sinks))
    j = torch.arange(cap, device=dev)
    for b, n in enumerate(lens):
        hidden = j >= n + T
        if window:
            hidden |= (j < n - window + 1) & (j >= sinks)
        for i in (0, 2):
            cache[i][b, :, hidden] = 0xFF
            _bits(cache[i + 1])[b, :, hidden] = 0x7F  # NaN
    assert torch.equal(apex.decode4(q, *cache, ln, window=window, n_sink=sinks), want)


@pytest.mark.gpu
def test_lengths_out_of_range_and_past_the_capacity():
    dev = _gpu()
    lens = [-5, 200, 10 ** 9, 197]
    q, cache, ln, f, vals = _attn_inputs(dev, 8, 8, 2, 6, 64, 64, 200, lens)
    _close(apex.decode4(q, *cache, ln), *_attn_ref(q, *vals, lens))
    # a window past which the cache has no row: nothing is seen
    got = apex.decode4(q, *cache, ln, window=2)
    ref, tol = _attn_ref(q, *vals, lens, 2)
    _close(got, ref, tol)
    assert (got[1, :, 2:] == 0).all() and (got[2, :, 2:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 20])
def test_rising_and_peaked_scores(T):
    """Every slice outgrows the ones before it; one key takes nearly all; scales of the scores."""
    dev = _gpu()
    g = _gen(dev, 9)
    cap, d = 1200, 128
    q = torch.ones(1, 4, T, d, dtype=torch.bfloat16, device=dev)
    up = torch.linspace(0, 40, cap, device=dev)[None, None, :, None].expand(1, 2, cap, d)
    k = (up + 0.1 * torch.randn(1, 2, cap, d, generator=g, device=dev)).to(torch.bfloat16)
    v = _normal(g, dev, 1, 2, cap, d)
    cache = _cache(dev, 1, 2, cap, d) + _cache(dev, 1, 2, cap, d)
    ln = torch.tensor([cap - T], dtype=torch.int32, device=dev)
    for kk in (k, k.flip(2)):
        apex.append4(kk, v, *cache)
        vals = _values(cache[0], cache[1], None), _values(cache[2], cache[3], None)
        for scale in (None, 0.001, 1.0):
            got = apex.decode4(q, *cache, ln, scale=scale)
            _close(got, *_attn_ref(q, *vals, [cap - T], scale=scale))


@pytest.mark.gpu
@pytest.mark.parametrize("s", [2.0 ** -100, 2.0 ** -20, 2.0 ** 60])
def test_queries_of_any_size(s):
    dev = _gpu()
    q, cache, ln, f, vals = _attn_inputs(dev, 10, 8, 2, 2, 128, 128, 300, [290])
    big = (q.double() * s).to(torch.bfloat16)
    _close(apex.decode4(big, *cache, ln, scale=0.1 / s), *_attn_ref(big, *vals, [290], scale=0.1 / s))
    small = q.clone()
    small[:, :, :, 5:] *= 2.0 ** -16  # entries far below the row's largest
    _close(apex.decode4(small, *cache, ln), *_attn_ref(small, *vals, [290]))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [None, 1e-30])
def test_queries_of_zeros(scale):
    """Scores of 0: the mean of the values that are seen, with masked keys beside them."""
    dev = _gpu()
    lens = [200, 3, 0]
    q, cache, ln, f, vals = _attn_inputs(dev, 19, 8, 2, 3, 128, 128, 300, lens)
    q[:, 1:5] = 0
    q[:, 5] *= 2.0 ** -120
    got = apex.decode4(q, *cache, ln, window=50, n_sink=2, scale=scale)
    _close(got, *_attn_ref(q, *vals, lens, 50, 2, scale=scale))


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_alone():
    dev = _gpu()
    q, cache, ln, f, vals = _attn_inputs(dev, 11, 8, 2, 3, 128, 128, 300, [290, 100])
    want = apex.decode4(q, *cache, ln)
    bad = q.clone()
    bad[0, 1, 1, 7] = float("nan")
    got = apex.decode4(bad, *cache, ln)
    assert torch.isnan(got[0, 1, 1]).all()
    got[0, 1, 1] = want[0, 1, 1]
    assert torch.equal(got, want)
    _bits(cache[1])[1, 0, 50, 0] = 0x7F  # a key of NaN: every row of its head
    got = apex.decode4(q, *cache, ln)
    assert torch.isnan(got[1, :4]).all() and torch.equal(got[0], want[0]) and torch.equal(got[1, 4:], want[1, 4:])


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,T,d,cap", [(33, 4, 2, 3, 64, 300), (70, 8, 2, 1, 128, 700), (300, 4, 1, 1, 64, 140),
                                              (5, 32, 8, 1, 128, 3000)])
def test_many_sequences(B, Hq, Hkv, T, d, cap):
    dev = _gpu()
    lens = torch.randint(0, cap - T + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    q, cache, ln, f, vals = _attn_inputs(dev, B, Hq, Hkv, T, d, d, cap, lens)
    for window, sinks in ((0, 0), (90, 5)):
        _close(apex.decode4(q, *cache, ln, window=window, n_sink=sinks), *_attn_ref(q, *vals, lens, window, sinks))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(25))
def test_random_configurations(seed):
    dev = _gpu()
    r = torch.Generator().manual_seed(1000 + seed)
    pick = lambda xs: xs[int(torch.randint(0, len(xs), (1,), generator=r))]  # noqa: E731
    Hq, Hkv = pick([(4, 2), (8, 8), (16, 1), (32, 8), (2, 1)])
    dk, dv = pick([(64, 64), (128, 128), (192, 128)])
    T, cap, B = pick([1, 1, 2, 5, 9]), pick([20, 127, 128, 257, 900]), pick([1, 2, 5])
    lens = [int(torch.randint(0, cap + 1, (1,), generator=r)) for _ in range(B)]
    window, sinks = pick([0, 1, 17, 128, 300]), pick([0, 1, 16, 129])
    q, cache, ln, f, vals = _attn_inputs(dev, seed, Hq, Hkv, T, dk, dv, cap, lens, pick([False, True]))
    _close(apex.decode4(q, *cache, ln, window=window, n_sink=sinks, **f), *_attn_ref(q, *vals, lens, window, sinks))


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    dev = _gpu()
    g = _gen(dev, 12)
    H, d, cap = 2, 128, 1 << 24  # 2 GB of codes a head: the second head's rows start there
    B = 3
    try:
        cache = _cache(dev, B, H, cap, d) + _cache(dev, B, H, cap, d)
    except torch.OutOfMemoryError:
        pytest.skip("needs 14 GB")
    n = 300
    k, v = _normal(g, dev, B, H, n, d), _normal(g, dev, B, H, n, d)
    row0 = torch.full((B,), cap - n, dtype=torch.int32, device=dev)
    apex.append4(k, v, *cache, row0=row0)
    ko, vo = apex.unpack4(*cache, row0=row0, n_rows=n)
    assert torch.equal(ko.double().cpu(), _pack_ref(k, None)[2]) and torch.equal(vo.double().cpu(), _pack_ref(v, None)[2])
    q = _normal(g, dev, B, 8, 1, d)
    ln = torch.full((B,), cap - 1, dtype=torch.int32, device=dev)
    got = apex.decode4(q, *cache, ln, window=n)
    small = _cache(dev, B, H, n, d) + _cache(dev, B, H, n, d)
    apex.append4(k, v, *small)
    vals = _values(small[0], small[1], None), _values(small[2], small[3], None)
    _close(got, *_attn_ref(q, *vals, [n - 1] * B))


# ------------------------------------------------------------------------------------------------- in use
@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv,layout", [(64, 64, "half"), (128, 128, "interleaved"), (192, 128, "half")])
def test_a_cache_served(dk, dv, layout):
    """A prompt and then tokens: heads normed and turned, packed, attended to under a window with sinks;
    the prompt's rows read back."""
    dev = _gpu()
    g = _gen(dev, 13)
    B, Hq, Hkv, cap, window, sinks = 2, 8, 2, 160, 48, 4
    qw, kw = 1 + 0.1 * torch.randn(dk, generator=g, device=dev), 1 + 0.1 * torch.randn(dk, generator=g, device=dev)
    fk, fv = torch.full((Hkv,), 2.0 ** -7, device=dev), torch.full((Hkv,), 2.0 ** -8, device=dev)
    f = dict(k_factor=fk, v_factor=fv)
    cache = _cache(dev, B, Hkv, cap, dk) + _cache(dev, B, Hkv, cap, dv)
    lens = torch.tensor([90, 7], dtype=torch.int32, device=dev)
    pos = torch.arange(90, dtype=torch.int32, device=dev)
    k, v = _normal(g, dev, B, Hkv, 90, dk), _normal(g, dev, B, Hkv, 90, dv)
    _, kr = apex.norm_rope(_normal(g, dev, B, Hq, 90, dk), k, positions=pos, q_weight=qw, k_weight=kw, layout=layout)
    apex.append4(kr, v, *cache, **f)
    back = apex.unpack4(*cache, n_rows=90, **f)
    assert ((back[0].float() - kr.float()).abs().amax() / kr.float().abs().amax()) < 0.2  # one step of e2m1
    for step in range(12):
        T = 1 + step % 3
        q, k, v = _normal(g, dev, B, Hq, T, dk), _normal(g, dev, B, Hkv, T, dk), _normal(g, dev, B, Hkv, T, dv)
        at = lens[:, None] + torch.arange(T, dtype=torch.int32, device=dev)
        qr, kr = apex.norm_rope(q, k, positions=at, q_weight=qw, k_weight=kw, layout=layout)
        apex.append4(kr, v, *cache, row0=lens, **f)
        out = apex.decode4(qr, *cache, lens, window=window, n_sink=sinks, **f)
        vals = _values(cache[0], cache[1], fk), _values(cache[2], cache[3], fv)
        _close(out, *_attn_ref(qr, *vals, lens.tolist(), window, sinks))
        lens += T


@pytest.mark.gpu
def test_captured_and_replayed_with_new_lengths():
    dev = _gpu()
    B, Hq, Hkv, T, d, cap = 2, 32, 8, 2, 128, 2000
    q, cache, lens, f, _ = _attn_inputs(dev, 14, Hq, Hkv, T, d, d, cap, [1500, 10], True)
    g = _gen(dev, 15)
    k, v = _normal(g, dev, B, Hkv, T, d), _normal(g, dev, B, Hkv, T, d)
    ws = torch.empty(apex.decode4_workspace_bytes(B, Hq, Hkv, T, cap, d), dtype=torch.uint8, device=dev)

    def calls():
        apex.append4(k, v, *cache, row0=lens, **f)
        out = [apex.decode4(q, *cache, lens, window=w, n_sink=4, workspace=ws, **f) for w in (0, 300)]
        return out + list(apex.unpack4(*cache, row0=lens, n_rows=T, **f))

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for a, b in ((1998, 401), (0, 1), (777, 1300)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        for x in (q, k, v):
            x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        assert all(torch.equal(x, y) for x, y in zip(got, calls()))


@pytest.mark.gpu
def test_two_streams_with_their_own_workspaces():
    dev = _gpu()
    q, cache, ln, f, _ = _attn_inputs(dev, 16, 32, 8, 1, 128, 128, 3000, [2990, 1000, 5])
    want = apex.decode4(q, *cache, ln), *apex.unpack4(*cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = [(apex.decode4(q, *cache, ln, stream=s), *apex.unpack4(*cache, stream=s)) for s in streams * 3]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x in got for a, b in zip(x, want))


@pytest.mark.gpu
def test_outputs_and_workspaces_stay_within_their_bounds():
    dev = _gpu()
    pad = 4096
    for Hq, Hkv, T, dk, dv, cap, lens, window, sinks in ATTN:
        q, cache, ln, f, _ = _attn_inputs(dev, 17, Hq, Hkv, T, dk, dv, cap, lens)
        B = len(lens)
        bufs = []
        for n in (B * Hq * T * dv * 2, apex.decode4_workspace_bytes(B, Hq, Hkv, T, cap, dk, dv)):
            bufs.append((torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device=dev), n))
        o, w = (b[pad:pad + n] for b, n in bufs)
        apex.decode4(q, *cache, ln, window=window, n_sink=sinks, out=o.view(torch.bfloat16).view(B, Hq, T, dv), workspace=w)
        for b, n in bufs:
            assert (b[:pad] == 0xA5).all() and (b[pad + n:] == 0xA5).all()


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
    f = dict(rows=P, bytes=2 * P, scales=3 * P, factor=None, b=512, h=128, s=512, d=128)
    f.update(o)
    return apex.Bits4Tensor(*[f[n] for n, _ in apex.Bits4Tensor._fields_])


MOVE = [
    (dict(rows=None), {}, BAD), (dict(bytes=None), {}, BAD), (dict(scales=None), {}, BAD), (dict(rows=P + 1), {}, BAD),
    (dict(bytes=2 * P + 8), {}, BAD), (dict(scales=3 * P + 4), {}, BAD), (dict(factor=P + 2), {}, BAD),
    (dict(d=0), {}, BAD), (dict(d=72), {}, UNSUPPORTED), (dict(d=528), {}, UNSUPPORTED), ({}, dict(B=0), BAD),
    ({}, dict(H=-1), BAD), ({}, dict(S=0), BAD), ({}, dict(cap=0), BAD), ({}, dict(row0=P + 1), BAD),
    ({}, dict(cap=(1 << 24) + 1), UNSUPPORTED), ({}, dict(B=1 << 16, S=1 << 14), UNSUPPORTED),
    (dict(rows=2 * P + 64), {}, BAD), (dict(rows=3 * P), {}, BAD),  # rows on the packed tensors
]


@pytest.mark.parametrize("tensor,args,code", MOVE)
def test_append4_and_unpack4_refuse(lib, tensor, args, code):
    a = dict(B=1, H=2, S=1, cap=16, row0=None)
    a.update(args)
    other = _tensor(rows=8 * P, bytes=9 * P, scales=10 * P)
    for f in (apex.apex_attn_append4, apex.apex_attn_unpack4):
        for pair in ((_tensor(**tensor), other), (other, _tensor(**tensor))):
            assert f(*pair, a["B"], a["H"], a["S"], a["cap"], a["row0"], None) == code
        assert f(None, other, 1, 2, 1, 16, None, None) == BAD and f(other, None, 1, 2, 1, 16, None, None) == BAD


def test_append4_and_unpack4_refuse_outputs_on_one_another(lib):
    a, b = _tensor(), _tensor(rows=8 * P, bytes=2 * P + 1024, scales=10 * P)  # 2 heads x 16 rows x 64 bytes at 2 P
    assert apex.apex_attn_append4(a, b, 1, 2, 1, 16, None, None) == BAD
    b = _tensor(rows=P + 128, bytes=9 * P, scales=10 * P)
    assert apex.apex_attn_unpack4(a, b, 1, 2, 1, 16, None, None) == BAD
    assert apex.apex_attn_unpack4(_tensor(h=64), _tensor(rows=8 * P, bytes=9 * P, scales=10 * P), 1, 2, 1, 16, None, None) == BAD


ATTN_ARGS = dict(q=P, k=P, ks=P, v=P, vs=P, out=8 * P, B=1, H_q=8, H_kv=2, T=4, S_cap=64, d_qk=128, d_v=128, lens=P,
                 window=0, n_sink=0, fk=None, fv=None, scale=0.0, ws=P, n=1 << 40)


@pytest.mark.parametrize("o,code", [(dict([(x, None)]), BAD) for x in ("q", "k", "ks", "v", "vs", "out", "lens", "ws")] + [
    (dict(q=P + 2), BAD), (dict(k=P + 8), BAD), (dict(ks=P + 8), BAD), (dict(v=P + 4), BAD), (dict(vs=P + 1), BAD),
    (dict(out=P + 8), BAD), (dict(ws=P + 8), BAD), (dict(lens=P + 1), BAD), (dict(fk=P + 2), BAD), (dict(fv=P + 1), BAD),
    (dict(n_sink=-1), BAD), (dict(B=0), BAD), (dict(H_q=0), BAD), (dict(H_kv=3), BAD), (dict(T=0), BAD),
    (dict(S_cap=0), BAD), (dict(d_qk=0), BAD), (dict(T=65), UNSUPPORTED), (dict(S_cap=(1 << 24) + 1), UNSUPPORTED),
    (dict(B=65537), UNSUPPORTED), (dict(d_qk=64), UNSUPPORTED), (dict(d_qk=192, d_v=192), UNSUPPORTED),
    (dict(H_q=6), UNSUPPORTED), (dict(H_q=64), UNSUPPORTED), (dict(scale=float("inf")), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=-0.3), BAD), (dict(n=15), BAD),
    # the output (8192 bytes) on the queries, the keys (8192 bytes), their scales (1024), the values, the lengths
    (dict(q=8 * P + 8176), BAD), (dict(k=8 * P - 8176), BAD), (dict(ks=8 * P - 1008), BAD), (dict(v=8 * P), BAD),
    (dict(vs=8 * P + 16), BAD), (dict(lens=8 * P + 4), BAD), (dict(fk=8 * P), BAD), (dict(fv=8 * P), BAD),
])
def test_decode4_refuses(lib, o, code):
    a = dict(ATTN_ARGS)
    a.update(o)
    assert apex.apex_attn_decode4(a["q"], a["k"], a["ks"], a["v"], a["vs"], a["out"], a["B"], a["H_q"], a["H_kv"],
                                  a["T"], a["S_cap"], a["d_qk"], a["d_v"], a["lens"], a["window"], a["n_sink"], a["fk"],
                                  a["fv"], a["scale"], a["ws"], a["n"], None) == code
    names = ("B", "H_q", "H_kv", "T", "S_cap", "d_qk", "d_v")
    assert (apex.decode4_workspace_bytes(*[a[n] for n in names]) == 0) == any(n in o for n in names)


def test_conveniences_refuse_cpu_tensors(lib):
    x, x4 = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 3, 32, dtype=torch.uint8)
    s = torch.zeros(1, 2, 3, 4).to(torch.float8_e4m3fn)
    with pytest.raises(TypeError):
        apex.append4(x, x, x4, s, x4, s)
    with pytest.raises(TypeError):
        apex.unpack4(x4, s, x4, s)
    with pytest.raises(TypeError):
        apex.decode4(x, x4, s, x4, s, torch.zeros(1, dtype=torch.int32))


@pytest.mark.gpu
def test_conveniences_refuse_what_does_not_fit():
    dev = _gpu()
    q, c, ln, f, _ = _attn_inputs(dev, 18, 8, 2, 2, 128, 128, 64, [32, 40])
    k = torch.zeros(2, 2, 3, 128, dtype=torch.bfloat16, device=dev)
    for bad in (lambda: apex.decode4(q, *c, ln.long()), lambda: apex.decode4(q.float(), *c, ln),
                lambda: apex.decode4(q, c[0], _bits(c[1]), c[2], c[3], ln), lambda: apex.decode4(q, c[0].char(), *c[1:], ln),
                lambda: apex.append4(k.float(), k, *c), lambda: apex.append4(k, k, *c, row0=ln.long())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: apex.decode4(q, *c, ln[:1]), lambda: apex.decode4(q[:1], *c, ln),
                lambda: apex.decode4(q[..., :64].contiguous(), *c, ln), lambda: apex.decode4(q, *c, ln, n_sink=-1),
                lambda: apex.decode4(q, c[0], c[1][:, :1], c[2], c[3], ln),
                lambda: apex.decode4(q, *c, ln, k_factor=torch.ones(8, device=dev)),
                lambda: apex.append4(k[..., :64].contiguous(), k, *c), lambda: apex.append4(k, k[:, :, :2], *c),
                lambda: apex.append4(k, k, c[0], c[1], c[2][:1], c[3]), lambda: apex.unpack4(*c, n_rows=0),
                lambda: apex.unpack4(*c, n_rows=3, k_out=q)):
        with pytest.raises(ValueError):
            bad()
    ws = torch.empty(16, dtype=torch.uint8, device=dev)
    with pytest.raises(apex.ApexError):
        apex.decode4(q, *c, ln, workspace=ws)


# Sizes past 2 GiB of codes: B x 8 heads x cap rows of 128 entries (64 bytes of codes, 8 of scales).
@pytest.mark.parametrize("B,cap", [(32, 65536), (80, 65536), (96, 65536), (160, 65536), (7, 1000003), (1, 3)])
def test_packed_tensors_end_where_they_end(lib, B, cap):
    """Tensors right behind one another share nothing; one that starts a byte sooner does."""
    if torch.cuda.is_available():
        pytest.skip("calls that pass the checks would run on addresses that hold nothing")
    codes, scales = B * 8 * cap * 64, B * 8 * cap * 8
    rows = B * 8 * 2 * 256  # two tokens of each sequence

    def call(f, **moved):
        at, end = {}, 1 << 32
        for name, size in (("k4", codes), ("ks", scales), ("v4", codes), ("vs", scales), ("k", rows), ("v", rows)):
            at[name] = end
            end += size
        at.update((n, at[n] - by) for n, by in moved.items())
        t = [_tensor(rows=at[n], bytes=at[n + "4"], scales=at[n + "s"], b=2048, h=256, s=128) for n in ("k", "v")]
        return f(*t, B, 8, 2, cap, None, None)
    for f in (apex.apex_attn_append4, apex.apex_attn_unpack4):
        assert call(f) not in (BAD, UNSUPPORTED)
        assert call(f, k=2) == BAD  # the first rows on the last scale
    # one packed tensor on the end of another: refused where they are written
    for n in ("ks", "v4", "vs"):
        assert call(apex.apex_attn_append4, **{n: 16}) == BAD


@pytest.mark.gpu
def test_packed_tensors_right_behind_one_another():
    """2.5 GiB of codes with what is next in memory: the calls run and keep to their rows."""
    dev = _gpu()
    B, H, d, cap, n = 80, 8, 128, 65536, 3
    codes, scales, rows = B * H * cap * d // 2, B * H * cap * d // 16, B * H * n * d * 2
    sizes = [codes, scales, codes, scales, rows, rows]
    try:
        buf = torch.zeros(sum(sizes), dtype=torch.uint8, device=dev)
    except torch.OutOfMemoryError:
        pytest.skip("needs 6 GB")
    k4, ks, v4, vs, k, v = torch.split(buf, sizes)
    f8 = torch.float8_e4m3fn
    cache = (k4.view(B, H, cap, d // 2), ks.view(f8).view(B, H, cap, d // 16), v4.view(B, H, cap, d // 2),
             vs.view(f8).view(B, H, cap, d // 16))
    k, v = (x.view(torch.bfloat16).view(B, H, n, d) for x in (k, v))
    g = _gen(dev, 31)
    k.copy_(_normal(g, dev, B, H, n, d))
    v.copy_(_normal(g, dev, B, H, n, d))
    row0 = torch.full((B,), cap - n, dtype=torch.int32, device=dev)
    apex.append4(k, v, *cache, row0=row0)
    for x, (x4, s) in ((k, cache[:2]), (v, cache[2:])):
        code, sb, _ = _pack_ref(x, None)
        assert torch.equal(_codes(x4[:, :, -n:]), code) and torch.equal(_bits(s)[:, :, -n:].cpu(), sb)
        assert int(x4[:, :, -n - 1].count_nonzero()) == 0 and int(_bits(s)[:, :, -n - 1].count_nonzero()) == 0
    want = [_pack_ref(x, None)[2] for x in (k, v)]
    apex.unpack4(*cache, row0=row0, n_rows=n, k_out=k, v_out=v)
    assert torch.equal(k.double().cpu(), want[0]) and torch.equal(v.double().cpu(), want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 16])  # 4, 16 and 64 query rows of a KV head
@pytest.mark.parametrize("power", [-90, 90])
def test_factors_at_both_ends_of_their_range(T, power):
    dev = _gpu()
    f = torch.full((1,), 2.0 ** power, device=dev)
    # equal scores, all values the largest there are: sums over a long cut cache are 2^17 of them
    cap, d = 130000, 128
    k4, ks = _cache(dev, 1, 1, cap, d)
    v4, vs = _cache(dev, 1, 1, cap, d, fill=0x77)
    _bits(vs).fill_(0x7E)
    ln = torch.tensor([cap - T], dtype=torch.int32, device=dev)
    q = torch.ones(1, 4, T, d, dtype=torch.bfloat16, device=dev)
    got = apex.decode4(q, k4, ks, v4, vs, ln, k_factor=f, v_factor=f)
    # weights are powers of two here, sums of them whole numbers times one: exact but for the division
    assert (got.double() / (6 * 448 * 2.0 ** power) - 1).abs().max() <= U
    # other values, whole and cut; queries that bring the scores back
    for cap in (200, 3000):
        lens = [cap - T, 77]
        _, cache, ln, _, vals = _attn_inputs(dev, cap, 4, 1, T, d, d, cap, lens)
        q = _normal(_gen(dev, cap), dev, 2, 4, T, d)
        out = apex.decode4((q.double() * 2.0 ** -power).to(torch.bfloat16), *cache, ln, k_factor=f, v_factor=f)
        ref, tol = _attn_ref(q, *vals, lens)
        _close(out.double() * 2.0 ** -power, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 16])
@pytest.mark.parametrize("power", [12, 18, 24, 70])
def test_scores_of_any_size(T, power):
    """Scores of which one key's is the largest by far, or two keys' are, of either sign: that key's value, or
    the mean of the two."""
    dev = _gpu()
    cap, d = 3000, 128
    g = _gen(dev, power + T)
    q, cache, ln, _, vals = _attn_inputs(dev, power, 4, 1, T, d, d, cap, [cap - T])
    q = q[:, :, :1].expand(1, 4, T, d).contiguous()  # the tokens of a head alike
    f = torch.full((1,), 2.0 ** power, device=dev)
    vv = vals[1][0, 0]
    twin = torch.randperm(cap - T, generator=torch.Generator().manual_seed(T))
    for sign in (1, -1):
        x = sign * q.abs()
        s = (x[0, :, 0].double().cpu() @ vals[0][0, 0].T) / math.sqrt(d) * 2.0 ** power
        s = s[:, :cap - T]  # a prompt's keys: all tokens see them
        best = s.argmax(-1)
        c = [y.clone() for y in cache]
        for i in (0, 1):  # tokens' own keys score nothing like the best: the first key's negative codes
            c[i].view(torch.uint8)[:, :, cap - T:] = c[i].view(torch.uint8)[:, :, best[0]:best[0] + 1]
        c[0][:, :, cap - T:] ^= 0x88
        other = int(twin[0]) if int(twin[0]) not in best.tolist() else int(twin[1])
        for y in c:  # a twin of head 0's best key and of its value
            z = y.view(torch.uint8)
            z[:, :, other] = z[:, :, best[0]]
        got = apex.decode4(x, *c, ln, k_factor=f).double().cpu()
        assert torch.isfinite(got).all()
        s[:, other] = s[:, best[0]]
        for h in range(4):
            # the next one is far below, by more than 2^-20 of the scores' size: scores of fp32 tell them apart
            order = s[h].sort(descending=True)
            low = 2 if int(order.indices[0]) in (int(best[0]), other) else 1
            gap = (order.values[0] - order.values[low]) - 2.0 ** -20 * s[h].abs().max()
            if gap < 40:
                continue
            want = vv[best[h]] if int(best[h]) != other else vv[best[0]]
            rest = cap * math.exp(-40) * vv.abs().max()  # the formula's weights of all other keys
            assert ((got[0, h] - want).abs() <= (U + 2.0 ** -11) * want.abs() + rest).all()
