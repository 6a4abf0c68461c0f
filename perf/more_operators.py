"""Cases of a second set of operators: norms of query and key heads with the rotary positions in the same pass,
and their gradient; rows of a cache held in 4 bits, written, read back and attended to; attention with a sliding
window whose first tokens stay visible (sinks), for prompts and for single tokens.

``run`` computes a case either in plain torch operations (``own`` false) or through the package's entry points
(``own`` true), on the inputs that ``prepare`` makes.  Tensors follow the package's conventions: bf16 [B, H, S, d]
rows, caches [B, H_kv, S_cap, d], int32 lengths and positions.  A 4-bit cache holds e2m1 values, two to a byte (the
even entry in the low half), with one e4m3 scale for 16 entries and an fp32 factor for each KV head.
"""
import math
import random

import torch

own = False

NEG = float("-inf")
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the newest token of one sequence: heads normed and turned, its key and value appended (latency)
        {"name": "norm_token", "op": "norm", "B": 1, "S": 1, "Hq": 32, "Hkv": 8, "d": 128, "d_rot": 128,
         "rot_start": 0, "half": True, "append": True, "S_cap": 4096, "far": 3000, "yarn": 1.0, "weights": "bf16",
         "per_head": False},
        # a long prompt's queries and keys, odd length
        {"name": "norm_prompt", "op": "norm", "B": 1, "S": 8191, "Hq": 128, "Hkv": 8, "d": 128, "d_rot": 128,
         "rot_start": 0, "half": True, "append": False, "S_cap": 0, "far": 0, "yarn": 1.0, "weights": "bf16",
         "per_head": False},
        # a short training step, weights for each head, part of the row turned
        {"name": "grad_short", "op": "grad", "B": 2, "S": 513, "Hq": 32, "Hkv": 8, "d": 128, "d_rot": 64,
         "rot_start": 64, "half": False, "far": 0, "yarn": 1.0, "weights": "fp32", "per_head": True},
        # a training step of many tokens
        {"name": "grad_long", "op": "grad", "B": 4, "S": 4096, "Hq": 32, "Hkv": 8, "d": 128, "d_rot": 128,
         "rot_start": 0, "half": True, "far": 0, "yarn": 1.0, "weights": "bf16", "per_head": False},
        # one step of a batch of conversations: each writes its newest row (latency)
        {"name": "pack_token", "op": "pack", "B": 16, "S": 1, "Hkv": 8, "d_k": 128, "d_v": 128, "S_cap": 4096,
         "factors": True},
        # a prompt's keys and values go into 4 bits and come back for the prompt that follows, odd length
        {"name": "pack_prompt", "op": "pack", "B": 1, "S": 32767, "Hkv": 8, "d_k": 128, "d_v": 128, "S_cap": 32768,
         "factors": True},
        # one conversation on a sliding-window layer with four sinks (latency)
        {"name": "bits4_window", "op": "bits4", "B": 1, "Hq": 32, "Hkv": 8, "T": 1, "d_qk": 128, "d_v": 128,
         "S_cap": 8192, "len_lo": 5003, "len_hi": 5003, "window": 1024, "n_sink": 4, "factors": False},
        # four drafted tokens over a ragged batch
        {"name": "bits4_drafts", "op": "bits4", "B": 8, "Hq": 32, "Hkv": 8, "T": 4, "d_qk": 128, "d_v": 128,
         "S_cap": 32784, "len_lo": 9001, "len_hi": 32768, "window": 0, "n_sink": 0, "factors": True},
        # the batch that the cache's 4 bits make room for: bound by the cache's bytes
        {"name": "bits4_batch", "op": "bits4", "B": 64, "Hq": 32, "Hkv": 8, "T": 1, "d_qk": 128, "d_v": 128,
         "S_cap": 32768, "len_lo": 9001, "len_hi": 32767, "window": 0, "n_sink": 0, "factors": True},
        # a batch of prompts on a sliding-window layer with four sinks
        {"name": "sink_prompts", "op": "sink", "B": 4, "Hq": 32, "Hkv": 8, "Sq": 4096, "Sk": 4096, "d": 128, "d_r": 0,
         "window": 1024, "n_sink": 4},
        # a long context: the rule that only the window's tiles and the sinks' are worked on
        {"name": "sink_long", "op": "sink", "B": 1, "Hq": 32, "Hkv": 8, "Sq": 65536, "Sk": 65536, "d": 128, "d_r": 0,
         "window": 4096, "n_sink": 64},
        # one token for each of a batch, bf16 cache of raw keys
        {"name": "sink_token", "op": "sink", "B": 16, "Hq": 32, "Hkv": 8, "Sq": 1, "Sk": 32768, "d": 128, "d_r": 0,
         "window": 4096, "n_sink": 4},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)) - 1e-9)))))


_HEADS = [(4, 2), (8, 8), (16, 1), (32, 8), (64, 8), (128, 8)]
_ROWS = [(64, 64), (128, 128), (192, 128)]


def _draw(rng):
    op = rng.choice(["norm", "grad", "pack", "bits4", "sink"])
    Hq, Hkv = rng.choice(_HEADS)
    dk, dv = rng.choice(_ROWS)
    B = _log(rng, 1, 16)
    if op in ("norm", "grad"):
        d = rng.choice([64, 80, 128, 128, 192, 256])
        d_rot = d if rng.random() < 0.6 else 64 if d == 192 else 16 * rng.randint(1, d // 16)
        c = {"op": op, "B": B, "S": _log(rng, 1, 8192), "Hq": Hq, "Hkv": Hkv, "d": d, "d_rot": d_rot,
             "rot_start": d - d_rot if rng.random() < 0.5 else 0, "half": rng.random() < 0.5,
             "far": _log(rng, 1, 1 << 20), "yarn": rng.choice([1.0, 1.0, 4.0, 32.0]),
             "weights": rng.choice(["bf16", "fp32"]), "per_head": rng.random() < 0.3}
        if op == "norm":
            c["append"] = c["S"] <= 64 and rng.random() < 0.7
            c["S_cap"] = c["S"] + _log(rng, 1, 4096) if c["append"] else 0
        return c
    if op == "pack":
        S = _log(rng, 1, 32768)
        return {"op": op, "B": B, "S": S, "Hkv": Hkv, "d_k": dk, "d_v": dv, "S_cap": S + _log(rng, 1, 4096),
                "factors": rng.random() < 0.5}
    if op == "bits4":
        T = rng.choice([1, 1, 1, 2, 3, 4, 8, 16])
        hi = _log(rng, 1, 32768)
        return {"op": op, "B": _log(rng, 1, 64), "Hq": Hq, "Hkv": Hkv, "T": T, "d_qk": dk, "d_v": dv, "S_cap": hi + T,
                "len_lo": rng.randint(max(1, hi // 4), hi), "len_hi": hi,
                "window": rng.choice([0, 0, _log(rng, 16, 4096)]), "n_sink": rng.choice([0, 1, 4, 64, 200]),
                "factors": rng.random() < 0.5}
    one = rng.random() < 0.4
    Sk = _log(rng, 1, 32768)
    return {"op": op, "B": _log(rng, 1, 16 if one else 4), "Hq": Hq, "Hkv": Hkv,
            "Sq": 1 if one else rng.choice([Sk, rng.randint(1, Sk)]), "Sk": Sk, "d": dv, "d_r": dk - dv,
            "window": _log(rng, 16, 4096), "n_sink": rng.choice([1, 4, 64, 200])}


def draw(rng):
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and _cache_elements(c) <= 5 << 30:
            return c


def _cache_elements(c):
    if c["op"] in ("norm", "pack"):
        return c["B"] * c["S_cap"] * c["Hkv"] * 2 * c.get("d", c.get("d_k"))
    if c["op"] == "bits4":
        return c["B"] * c["Hkv"] * c["S_cap"] * (c["d_qk"] + c["d_v"])
    return 0


def _lens(c, rng=None):
    """Lengths evenly spread from len_lo to len_hi; the seed only shuffles them."""
    B, lo, hi = c["B"], c["len_lo"], c["len_hi"]
    lens = [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]
    if rng is not None:
        rng.shuffle(lens)
    return lens


def _seen(m, window, n_sink):
    """Keys that the token at position m sees, itself among them."""
    if window <= 0:
        return m + 1
    return min(m + 1, window) + min(n_sink, max(0, m + 1 - window))


def work(case):
    c = case
    if c["op"] in ("norm", "grad"):
        rows = c["B"] * c["S"] * (c["Hq"] + c["Hkv"])
        if c["op"] == "grad":
            n = (c["Hq"] + c["Hkv"] if c["per_head"] else 2) * c["d"]
            return {"bytes": rows * c["d"] * 6 + c["B"] * c["S"] * 4 + 8 * n, "flops": rows * (c["d"] * 10 + c["d_rot"] * 3)}
        copied = c["B"] * c["S"] * c["Hkv"] * c["d"] * 4 if c["append"] else 0
        return {"bytes": rows * c["d"] * 4 + copied + c["B"] * c["S"] * 4, "flops": rows * (c["d"] * 4 + c["d_rot"] * 3)}
    if c["op"] == "pack":  # written: bf16 to 4 bits and scales; read back the other way
        n = c["B"] * c["S"] * c["Hkv"] * (c["d_k"] + c["d_v"])
        return {"bytes": 2 * (2 * n + n // 2 + n // 16), "flops": 4 * n}
    if c["op"] == "bits4":
        T, row = c["T"], c["d_qk"] + c["d_v"]
        keys = pairs = 0
        for n in _lens(c):
            pairs += sum(_seen(n + t, c["window"], c["n_sink"]) for t in range(T))
            w = c["window"] + T - 1 if c["window"] else 0  # what any of the T sees
            keys += min(_seen(n + T - 1, w, c["n_sink"]), n + T)
        return {"bytes": keys * c["Hkv"] * (row // 2 + row // 16) + c["B"] * c["Hq"] * T * row * 2,
                "flops": pairs * c["Hq"] * row * 2}
    d_qk, d_v = c["d"] + c["d_r"], c["d"]
    q0 = c["Sk"] - c["Sq"]
    pairs = sum(_seen(m, c["window"], c["n_sink"]) for m in range(q0, c["Sk"]))
    keys = min(c["Sk"], _seen(c["Sk"] - 1, c["window"] + c["Sq"] - 1, c["n_sink"]))
    return {"bytes": 2 * c["B"] * (d_qk + d_v) * (c["Hq"] * c["Sq"] + c["Hkv"] * keys),
            "flops": 2 * c["B"] * c["Hq"] * pairs * (d_qk + d_v)}


# ---------------------------------------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")


def _codes(x):
    """e2m1 codes of fp32 values: nearest, ties to the even code, up to +-6."""
    a = x.abs()
    code = torch.zeros_like(x, dtype=torch.uint8)
    for mid, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= mid) if up else (a > mid)
    return code | (torch.signbit(x).to(torch.uint8) << 3)


def _packed(x, factor):
    """x [..., H, S, d] in 4 bits: (bytes [..., d/2], scales [..., d/16]); factor [H] or None."""
    f = factor[:, None, None] if factor is not None else torch.ones((), device=x.device)
    g = x.float().unflatten(-1, (-1, 16))
    scale = (g.abs().amax(dim=-1) / (6.0 * f)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (scale.float() * f).unsqueeze(-1)
    c = _codes(torch.where(step > 0, g / torch.where(step > 0, step, 1.0), torch.zeros_like(g))).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale


def _values(x4, scale, factor):
    """fp32 values [..., d] that packed rows stand for."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=x4.device)
    c = torch.stack([x4 & 15, x4 >> 4], dim=-1).flatten(-2)
    v = table[c.int()].unflatten(-1, (-1, 16)) * scale.float().unsqueeze(-1)
    v = v.flatten(-2)
    return v if factor is None else v * factor[:, None, None]


def prepare(case, seed):
    c, dev = case, _device()
    rng = random.Random(seed)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16) * scale

    s = {"case": c}
    B = c["B"]
    if c["op"] in ("norm", "grad"):
        # as projections leave them: [B, S, H, d], seen as [B, H, S, d]; some heads louder than others
        loud = torch.exp(torch.randn(c["Hq"] + c["Hkv"], 1, generator=g, device=dev)).to(torch.bfloat16)
        s["q"] = (normal(B, c["S"], c["Hq"], c["d"]) * loud[:c["Hq"]]).transpose(1, 2)
        s["k"] = (normal(B, c["S"], c["Hkv"], c["d"]) * loud[c["Hq"]:]).transpose(1, 2)
        dtype = torch.bfloat16 if c["weights"] == "bf16" else torch.float32
        for n, heads in (("q", c["Hq"]), ("k", c["Hkv"])):
            shape = (heads, c["d"]) if c["per_head"] else (c["d"],)
            s[n + "_weight"] = (1.0 + 0.2 * torch.randn(shape, generator=g, device=dev)).to(dtype)
        far = [rng.randint(c["far"] // 2, max(1, c["far"])) for _ in range(B)]
        start = torch.tensor(far, dtype=torch.int32, device=dev)[:, None]
        s["positions"] = (start + torch.arange(c["S"], dtype=torch.int32, device=dev)[None]).contiguous()
        if c["op"] == "grad":
            s["q_grad"] = normal(B, c["S"], c["Hq"], c["d"]).transpose(1, 2)
            s["k_grad"] = normal(B, c["S"], c["Hkv"], c["d"]).transpose(1, 2)
        elif c["append"]:
            s["v"] = normal(B, c["S"], c["Hkv"], c["d"]).transpose(1, 2)
            s["k_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d"])
            s["v_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d"])
            rows = [rng.randint(0, c["S_cap"] - c["S"]) for _ in range(B)]
            s["row0"] = torch.tensor(rows, dtype=torch.int32, device=dev)
        return s
    if c["op"] == "sink":
        s["q"] = normal(B, c["Hq"], c["Sq"], c["d"] + c["d_r"], scale=1.5)
        s["k"] = normal(B, c["Hkv"], c["Sk"], c["d"] + c["d_r"])
        s["v"] = normal(B, c["Hkv"], c["Sk"], c["d"])
        return s
    # powers of two near what brings a head's largest scales to the middle of e4m3's range
    for n in ("k", "v"):
        exps = [rng.randint(-5, -2) for _ in range(c["Hkv"])]
        s[n + "_factor"] = torch.tensor([2.0 ** e for e in exps], device=dev) if c["factors"] else None
    if c["op"] == "pack":
        s["k"] = normal(B, c["S"], c["Hkv"], c["d_k"]).transpose(1, 2)
        s["v"] = (normal(B, c["S"], c["Hkv"], c["d_v"]) * 0.3).transpose(1, 2)
        rows = [rng.randint(0, c["S_cap"] - c["S"]) for _ in range(B)]
        s["row0"] = torch.tensor(rows, dtype=torch.int32, device=dev)
        for n in ("k", "v"):
            d = c["d_" + n]
            s[n + "4"] = torch.zeros(B, c["Hkv"], c["S_cap"], d // 2, dtype=torch.uint8, device=dev)
            s[n + "_scale"] = torch.zeros(B, c["Hkv"], c["S_cap"], d // 16, dtype=torch.uint8,
                                          device=dev).view(torch.float8_e4m3fn)
        return s
    lens = _lens(c, rng)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["q"] = normal(B, c["Hq"], c["T"], c["d_qk"], scale=1.5)
    for n, d in (("k", c["d_qk"]), ("v", c["d_v"])):
        parts = [_packed(normal(c["Hkv"], c["S_cap"], d), s[n + "_factor"]) for _ in range(B)]
        s[n + "4"] = torch.stack([p[0] for p in parts])
        s[n + "_scale"] = torch.stack([p[1].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _frequencies(c, d_rot, device):
    """theta_i in 64 bits, with YaRN's three regimes (beta_fast 32, beta_slow 1)."""
    i = torch.arange(d_rot // 2, dtype=torch.float64, device=device)
    theta = 10000.0 ** (-2.0 * i / d_rot)
    scale = c.get("yarn", 1.0)
    if scale > 1.0:
        lam = 2 * math.pi / theta
        t = ((lam - 1.0) / (scale - 1.0)).clamp(0, 1)
        mid = theta / (t * scale + 1 - t)
        theta = torch.where(lam < 32.0, theta, torch.where(lam > scale, theta / scale, mid))
    return theta


def _turned(x, cos, sin, start, n, half):
    """Entries [start, start + n) of fp32 rows turned."""
    part = x[..., start:start + n]
    if half:
        u, w = part[..., :n // 2], part[..., n // 2:]
        turned = torch.cat([u * cos - w * sin, u * sin + w * cos], dim=-1)
    else:
        u, w = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([u * cos - w * sin, u * sin + w * cos], dim=-1).flatten(-2)
    return torch.cat([x[..., :start], turned, x[..., start + n:]], dim=-1)


EPS = 1e-6


def _plain_norm(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, :, None] * _frequencies(c, c["d_rot"], s["q"].device)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    outs = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"].float()
        w = w[:, None, :] if c["per_head"] else w
        rs = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
        if c["op"] == "norm":
            outs[n] = _turned(x * rs * w, cos, sin, c["rot_start"], c["d_rot"], c["half"]).to(torch.bfloat16)
            continue
        back = _turned(s[n + "_grad"].float(), cos, -sin, c["rot_start"], c["d_rot"], c["half"])
        xh, gw = x * rs, back * w
        outs[n] = (rs * (gw - xh * (gw * xh).mean(dim=-1, keepdim=True))).to(torch.bfloat16)
        outs[n + "_weight"] = (back * xh).sum(dim=(0, 2) if c["per_head"] else (0, 1, 2), dtype=torch.float64).float()
    if c["op"] == "norm" and c["append"]:
        rows = s["row0"].long()[:, None] + torch.arange(c["S"], device=s["q"].device)
        b = torch.arange(c["B"], device=s["q"].device)[:, None]
        s["k_cache"][b, :, rows] = outs["k"].transpose(1, 2)
        s["v_cache"][b, :, rows] = s["v"].transpose(1, 2)
        return {"q": outs["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return outs


def _plain_pack(s):
    c = s["case"]
    rows = s["row0"].long()[:, None] + torch.arange(c["S"], device=s["k"].device)
    b = torch.arange(c["B"], device=rows.device)[:, None]
    out = {}
    for n in ("k", "v"):
        x4, scale = _packed(s[n], s[n + "_factor"])
        s[n + "4"][b, :, rows] = x4.transpose(1, 2)
        bytes_ = s[n + "_scale"].view(torch.uint8)
        bytes_[b, :, rows] = scale.view(torch.uint8).transpose(1, 2)
        back = s[n + "4"][b, :, rows].transpose(1, 2), bytes_[b, :, rows].transpose(1, 2).contiguous()
        out[n] = _values(back[0], back[1].view(torch.float8_e4m3fn), s[n + "_factor"]).to(torch.bfloat16)
    return out


def _attend(q, k, v, seen, scale):
    """fp32 attention of q [H, G, T, d] over k [H, S, d], v [H, S, d_v] where seen [T, S]."""
    x = torch.matmul(q.flatten(1, 2), k.transpose(-1, -2)).unflatten(1, q.shape[1:3])
    x = torch.where(seen, x * scale, NEG)
    top = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - torch.where(top == NEG, 0.0, top))
    total = e.sum(dim=-1, keepdim=True)
    o = torch.matmul(e.flatten(1, 2), v).unflatten(1, q.shape[1:3])
    return o / torch.where(total == 0, 1.0, total)


def _plain_bits4(s):
    c, q = s["case"], s["q"]
    B, Hq, T, d = q.shape
    out = torch.empty(B, Hq, T, c["d_v"], dtype=torch.bfloat16, device=q.device)
    j = torch.arange(c["S_cap"], device=q.device)
    for b in range(B):
        k = _values(s["k4"][b], s["k_scale"][b], s["k_factor"])
        v = _values(s["v4"][b], s["v_scale"][b], s["v_factor"])
        m = s["lens"][b] + torch.arange(T, device=q.device)
        seen = j <= m[:, None]
        if c["window"] > 0:
            seen = seen & ((m[:, None] - j < c["window"]) | (j < c["n_sink"]))
        x = q[b].float().reshape(c["Hkv"], -1, T, d)
        out[b] = _attend(x, k, v, seen, 1.0 / math.sqrt(d)).reshape(Hq, T, -1).to(torch.bfloat16)
    return out


_BLOCK = 1024  # query rows worked on together


def _plain_sink(s):
    c, q = s["case"], s["q"]
    B, Hq, Sq, d = q.shape
    W, q0, Hkv = c["window"], c["Sk"] - c["Sq"], c["Hkv"]
    n_rot = c["d_r"] or d
    angle = torch.arange(c["Sk"], dtype=torch.float64, device=q.device)[:, None] * _frequencies(c, n_rot, q.device)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = torch.empty(B, Hq, Sq, c["d"], dtype=torch.bfloat16, device=q.device)
    for b in range(B):
        k = _turned(s["k"][b].float(), cos, sin, d - n_rot, n_rot, False)
        x = _turned(q[b].float(), cos[q0:], sin[q0:], d - n_rot, n_rot, False).reshape(Hkv, -1, Sq, d)
        v = s["v"][b].float()
        for r in range(0, Sq, _BLOCK):
            n = min(_BLOCK, Sq - r)
            m = q0 + r + torch.arange(n, device=q.device)[:, None]
            lo, hi = max(0, q0 + r - W + 1), q0 + r + n
            first = min(c["n_sink"], lo)
            at = torch.cat([torch.arange(first, device=q.device), torch.arange(lo, hi, device=q.device)])
            seen = (at <= m) & ((m - at < W) | (at < c["n_sink"]))
            o = _attend(x[:, :, r:r + n], torch.cat([k[:, :first], k[:, lo:hi]], dim=1),
                        torch.cat([v[:, :first], v[:, lo:hi]], dim=1), seen, 1.0 / math.sqrt(d))
            out[b, :, r:r + n] = o.reshape(Hq, n, -1).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------------------------- the package's calls
def _own_run(s):
    import transformer_attention_rope_gb300 as apex
    c = s["case"]
    if c["op"] in ("norm", "grad"):
        how = dict(positions=s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                   layout="half" if c["half"] else "interleaved", d_rot=c["d_rot"], rot_start=c["rot_start"],
                   yarn_scale=c["yarn"])
        if c["op"] == "grad":
            q, k, qw, kw = apex.norm_rope_grad(s["q_grad"], s["q"], s["k_grad"], s["k"], **how)
            return {"q": q, "q_weight": qw, "k": k, "k_weight": kw}
        if c["append"]:
            q, k, v = apex.norm_rope(s["q"], s["k"], s["v"], k_out=s["k_cache"], v_out=s["v_cache"], row0=s["row0"],
                                     **how)
            return {"q": q, "k_cache": k, "v_cache": v}
        q, k = apex.norm_rope(s["q"], s["k"], **how)
        return {"q": q, "k": k}
    if c["op"] == "sink":
        q0 = c["Sk"] - c["Sq"]
        how = dict(window=c["window"], n_sink=c["n_sink"])
        if c["Sq"] == 1:
            if c["d_r"]:
                return apex.mla_decode(s["q"], s["k"], s["v"], q0, c["d_r"], **how)
            return apex.decode(s["q"], s["k"], s["v"], q0, **how)
        if c["d_r"]:
            return apex.mla_fwd(s["q"], s["k"], s["v"], c["d_r"], q_pos0=q0, **how)
        return apex.fwd(s["q"], s["k"], s["v"], q_pos0=q0, **how)
    cache = (s["k4"], s["k_scale"], s["v4"], s["v_scale"])
    factors = dict(k_factor=s["k_factor"], v_factor=s["v_factor"])
    if c["op"] == "pack":
        apex.append4(s["k"], s["v"], *cache, row0=s["row0"], **factors)
        k, v = apex.unpack4(*cache, row0=s["row0"], n_rows=c["S"], **factors)
        return {"k": k, "v": v}
    return apex.decode4(s["q"], *cache, s["lens"], window=c["window"], n_sink=c["n_sink"], **factors)


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return {"norm": _plain_norm, "grad": _plain_norm, "pack": _plain_pack, "bits4": _plain_bits4,
            "sink": _plain_sink}[op](state)


# ---------------------------------------------------------------------------------------------- in 64 bits
def _turns(c, positions, d_rot, device):
    """exp(i m theta) as complex numbers."""
    theta = []
    for i in range(d_rot // 2):
        th = 10000.0 ** (-2.0 * i / d_rot)
        scale = c.get("yarn", 1.0)
        if scale > 1.0:
            lam = 2.0 * math.pi / th
            if lam > scale:
                div = scale
            else:
                t = min(1.0, max(0.0, (lam - 1.0) / (scale - 1.0)))
                div = t * scale + 1.0 - t
            th = th if lam < 32.0 else th / div
        theta.append(th)
    ang = positions.double()[..., None] * torch.tensor(theta, dtype=torch.float64, device=device)
    return torch.polar(torch.ones_like(ang), ang)


def _spin(y, turn, start, d_rot, half):
    """Rows y (64 bits) turned in place."""
    n = d_rot // 2
    at = start + torch.arange(n, device=y.device) * (1 if half else 2)
    to = at + (n if half else 1)
    z = torch.complex(y[..., at], y[..., to]) * turn
    y[..., at], y[..., to] = z.real, z.imag
    return y


def _rows64(x4, scale, factor):
    """Values of one head's packed rows, from the bits: sign, two of exponent, one of mantissa."""
    low, high = (x4 & 15).int(), (x4.int() >> 4)
    bits = torch.stack([low, high], dim=-1).reshape(*x4.shape[:-1], -1)
    e, m = (bits >> 1) & 3, (bits & 1).double()
    mag = torch.where(e == 0, 0.5 * m, torch.ldexp(1.0 + 0.5 * m, (e - 1).double()))
    v = torch.where(bits >= 8, -mag, mag) * scale.double().repeat_interleave(16, dim=-1)
    return v if factor is None else v * float(factor)


def exact(case, seed):
    """The definitions in 64 bits, one head or one sequence at a time."""
    c, s = case, prepare(case, seed)
    dev = s["lens" if c["op"] == "bits4" else "k"].device
    if c["op"] in ("norm", "grad"):
        turn = _turns(c, s["positions"], c["d_rot"], dev)
        res = {}
        for n in ("q", "k"):
            x = s[n]
            H, w = x.shape[1], s[n + "_weight"].double()
            y = torch.empty(x.shape, dtype=torch.float64, device=dev)
            dw = torch.zeros(H, c["d"], dtype=torch.float64, device=dev)
            for h in range(H):
                row = x[:, h].double().contiguous()
                wh = w[h] if c["per_head"] else w
                length = torch.sqrt(row.pow(2).sum(dim=-1, keepdim=True) / c["d"] + EPS)
                if c["op"] == "norm":
                    y[:, h] = _spin(row / length * wh, turn, c["rot_start"], c["d_rot"], c["half"])
                else:
                    back = _spin(s[n + "_grad"][:, h].double().contiguous(), turn.conj(), c["rot_start"], c["d_rot"],
                                 c["half"])
                    unit = row / length
                    y[:, h] = (back * wh - unit * ((back * wh * unit).sum(dim=-1, keepdim=True) / c["d"])) / length
                    dw[h] = (back * unit).sum(dim=(0, 1))
            res[n] = y
            if c["op"] == "grad":
                res[n + "_weight"] = dw if c["per_head"] else dw.sum(dim=0)
        if c["op"] == "norm" and c["append"]:
            kc, vc = s["k_cache"].double(), s["v_cache"].double()
            for b, r in enumerate(s["row0"].tolist()):
                kc[b, :, r:r + c["S"]] = res["k"][b]
                vc[b, :, r:r + c["S"]] = s["v"][b].double()
            return {"q": res["q"], "k_cache": kc, "v_cache": vc}
        return res
    if c["op"] == "pack":
        res = {}
        steps = torch.tensor([v / 2.0 for v in (0, 1, 2, 3, 4, 6, 8, 12)], dtype=torch.float64, device=dev)
        order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=dev)  # even codes first: ties go to them
        for n in ("k", "v"):
            x = s[n]
            y = torch.empty(x.shape, dtype=torch.float64, device=dev)
            for h in range(c["Hkv"]):
                f = 1.0 if s[n + "_factor"] is None else float(s[n + "_factor"][h])
                g = x[:, h].double().reshape(-1, 16)
                top = g.abs().amax(dim=-1, keepdim=True) / (6.0 * f)
                scale = top.clamp(max=448.0).float().to(torch.float8_e4m3fn).double() * f
                best = torch.full_like(g, float("inf"))
                value = torch.zeros_like(g)
                for v in steps[order].tolist():
                    far = (g.abs() - v * scale).abs()
                    value = torch.where(far < best, v * scale.expand_as(g), value)
                    best = torch.minimum(best, far)
                y[:, h] = torch.where(g < 0, -value, value).reshape(x[:, h].shape)
            res[n] = y
        return res
    if c["op"] == "bits4":
        B, Hq, T, d = s["q"].shape
        G = Hq // c["Hkv"]
        out = torch.empty(B, Hq, T, c["d_v"], dtype=torch.float64, device=dev)
        for b, n in enumerate(s["lens"].tolist()):
            m = min(n + T, c["S_cap"])
            seen = torch.zeros(T, m, dtype=torch.bool, device=dev)
            for t in range(T):
                p = n + t
                seen[t, 0 if c["window"] <= 0 else max(0, p - c["window"] + 1):p + 1] = True
                seen[t, :min(c["n_sink"], p + 1)] = True
            for h in range(c["Hkv"]):
                fk, fv = (None if s[x] is None else s[x][h] for x in ("k_factor", "v_factor"))
                k = _rows64(s["k4"][b, h, :m], s["k_scale"][b, h, :m].float(), fk)
                x = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
                p = torch.softmax(x.masked_fill(~seen, NEG), dim=-1)
                out[b, h * G:(h + 1) * G] = p @ _rows64(s["v4"][b, h, :m], s["v_scale"][b, h, :m].float(), fv)
        return out
    B, Hq, Sq, d = s["q"].shape
    G, q0, n_rot = Hq // c["Hkv"], c["Sk"] - c["Sq"], c["d_r"] or d
    turn = _turns(c, torch.arange(c["Sk"], device=dev), n_rot, dev)
    out = torch.empty(B, Hq, Sq, c["d"], dtype=torch.float64, device=dev)
    step = 2048
    for b in range(B):
        for h in range(c["Hkv"]):
            k = _spin(s["k"][b, h].double(), turn, d - n_rot, n_rot, False)
            v = s["v"][b, h].double()
            q = _spin(s["q"][b, h * G:(h + 1) * G].double(), turn[q0:], d - n_rot, n_rot, False)
            for r in range(0, Sq, step):
                rows = q[:, r:r + step]
                p0 = q0 + r
                end = p0 + rows.shape[1]
                near = max(0, p0 - c["window"] + 1)
                keep = list(range(min(c["n_sink"], near))) + list(range(near, end))
                idx = torch.tensor(keep, device=dev)
                gap = torch.arange(p0, end, device=dev)[:, None] - idx
                hidden = (gap < 0) | ((gap >= c["window"]) & (idx >= c["n_sink"]))
                x = (rows @ k[idx].T / math.sqrt(d)).masked_fill_(hidden, NEG)
                out[b, h * G:(h + 1) * G, r:r + step] = torch.softmax(x, dim=-1) @ v[idx]
    return out
