"""Cases of the cache operators: rotary positions, attention of a drafted tree over a cache, decode that
accumulates attention weights, eviction by those weights.

``run`` computes a case either in plain torch operations (``own`` false) or through the package's entry points
(``own`` true), on the inputs that ``prepare`` makes.  All tensors follow the package's conventions: bf16
[B, H, S, d] rows, caches [B, H_kv, S_cap, d] whose keys are already rotated, int32 lengths and positions.
"""
import math
import random

import torch

own = False

NEG = float("-inf")


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # rotary positions: the newest token of one sequence, its key and value appended to the cache (latency)
        {"name": "rope_token", "op": "rope", "B": 1, "S": 1, "Hq": 32, "Hkv": 8, "d": 128, "d_rot": 128,
         "rot_start": 0, "half": False, "inverse": False, "append": True, "S_cap": 4096, "far": 3000, "yarn": 1.0},
        # the drafted tokens of a batch, half layout, a model stretched to a long context by YaRN
        {"name": "rope_drafts", "op": "rope", "B": 8, "S": 16, "Hq": 32, "Hkv": 8, "d": 128, "d_rot": 128,
         "rot_start": 0, "half": True, "inverse": False, "append": True, "S_cap": 2048, "far": 131072, "yarn": 32.0},
        # gradients of a long prompt's queries and keys, decoupled rows [content 128 | rope part 64], odd length
        {"name": "rope_grad", "op": "rope", "B": 1, "S": 8191, "Hq": 128, "Hkv": 8, "d": 192, "d_rot": 64,
         "rot_start": 128, "half": False, "inverse": True, "append": False, "S_cap": 0, "far": 0, "yarn": 1.0},
        # a small model's tree of five drafts over a short cache (latency)
        {"name": "tree_tiny", "op": "tree", "B": 1, "Hq": 4, "Hkv": 2, "T": 5, "d_qk": 64, "d_v": 64,
         "S_cap": 160, "len_lo": 128, "len_hi": 128, "window": 0},
        # one conversation on a sliding-window layer, sixteen drafts
        {"name": "tree_window", "op": "tree", "B": 1, "Hq": 32, "Hkv": 8, "T": 16, "d_qk": 128, "d_v": 128,
         "S_cap": 4224, "len_lo": 4097, "len_hi": 4097, "window": 1024},
        # a ragged batch of long conversations, eight drafts: bound by the cache's bytes
        {"name": "tree_batch", "op": "tree", "B": 8, "Hq": 32, "Hkv": 8, "T": 8, "d_qk": 128, "d_v": 128,
         "S_cap": 32784, "len_lo": 9001, "len_hi": 32768, "window": 0},
        # wide groups and a full tree of 64: bound by the matrix products
        {"name": "tree_wide", "op": "tree", "B": 4, "Hq": 128, "Hkv": 8, "T": 64, "d_qk": 128, "d_v": 128,
         "S_cap": 8256, "len_lo": 4100, "len_hi": 8192, "window": 0},
        # decode with weights: one conversation
        {"name": "weights_token", "op": "weights", "B": 1, "Hq": 32, "Hkv": 8, "d_qk": 128, "d_v": 128,
         "S_cap": 4096, "len_lo": 1001, "len_hi": 1001},
        # a ragged batch of long caches before its eviction
        {"name": "weights_batch", "op": "weights", "B": 8, "Hq": 32, "Hkv": 8, "d_qk": 128, "d_v": 128,
         "S_cap": 32768, "len_lo": 12345, "len_hi": 32768},
        # decoupled rows and wide groups
        {"name": "weights_decoupled", "op": "weights", "B": 6, "Hq": 128, "Hkv": 8, "d_qk": 192, "d_v": 128,
         "S_cap": 8192, "len_lo": 2000, "len_hi": 8190},
        # the steady state of a bounded cache: a little over its budget after a few steps
        {"name": "evict_step", "op": "evict", "B": 8, "Hkv": 8, "d_k": 128, "d_v": 128, "S_cap": 4224,
         "len_lo": 4100, "len_hi": 4224, "budget": 4096, "n_sink": 4, "n_recent": 1024, "aged": True},
        # a long prompt's cache cut down to its budget
        {"name": "evict_prompt", "op": "evict", "B": 4, "Hkv": 8, "d_k": 128, "d_v": 128, "S_cap": 32768,
         "len_lo": 20001, "len_hi": 32768, "budget": 4096, "n_sink": 4, "n_recent": 512, "aged": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)) - 1e-9)))))


_HEADS = [(4, 2), (8, 8), (16, 1), (32, 8), (64, 8), (128, 8)]
_ROWS = [(64, 64), (128, 128), (192, 128)]


def _draw(rng):
    op = rng.choice(["rope", "tree", "weights", "evict"])
    Hq, Hkv = rng.choice(_HEADS)
    dk, dv = rng.choice(_ROWS)
    B = _log(rng, 1, 16)
    if op == "rope":
        S = _log(rng, 1, 8192)
        append = S <= 64 and rng.random() < 0.7
        whole = dk != 192
        d_rot = dk if whole and rng.random() < 0.6 else 64 if not whole else dk // 2
        return {"op": op, "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "d": dk, "d_rot": d_rot,
                "rot_start": dk - d_rot if rng.random() < 0.5 else 0, "half": rng.random() < 0.5,
                "inverse": not append and rng.random() < 0.5, "append": append,
                "S_cap": S + _log(rng, 1, 4096) if append else 0, "far": _log(rng, 1, 1 << 20),
                "yarn": rng.choice([1.0, 1.0, 4.0, 32.0])}
    if op == "tree":
        T = _log(rng, 1, 64)
        hi = _log(rng, 1, 32768)
        return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d_qk": dk, "d_v": dv, "S_cap": hi + T,
                "len_lo": rng.randint(max(1, hi // 4), hi), "len_hi": hi,
                "window": rng.choice([0, 0, _log(rng, 16, 4096)])}
    if op == "weights":
        hi = _log(rng, 1, 32768)
        return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "d_qk": dk, "d_v": dv, "S_cap": hi + rng.randint(0, 200),
                "len_lo": rng.randint(max(1, hi // 4), hi), "len_hi": hi}
    budget = _log(rng, 32, 8192)
    hi = budget + _log(rng, 1, 24576)
    sink = rng.randint(0, 8)
    return {"op": op, "B": B, "Hkv": Hkv, "d_k": dk, "d_v": dv, "S_cap": hi, "len_lo": rng.randint(budget, hi),
            "len_hi": hi, "budget": budget, "n_sink": sink, "n_recent": rng.randint(0, budget - sink),
            "aged": rng.random() < 0.5}


def draw(rng):
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and _cache_bytes(c) <= 3 << 30:
            return c


def _cache_bytes(c):
    if c["op"] == "rope":
        return 2 * c["B"] * c["S_cap"] * c["Hkv"] * 2 * c["d"]
    dk = c["d_k"] if c["op"] == "evict" else c["d_qk"]
    return c["B"] * c["Hkv"] * c["S_cap"] * (dk + c["d_v"]) * 2


def _lens(c, rng=None):
    """Lengths evenly spread from len_lo to len_hi; the seed only shuffles them."""
    B, lo, hi = c["B"], c["len_lo"], c["len_hi"]
    lens = [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]
    if rng is not None:
        rng.shuffle(lens)
    return lens


def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["B"] * c["S"] * (c["Hq"] + c["Hkv"])
        b = rows * c["d"] * 4 + (c["B"] * c["S"] * c["Hkv"] * c["d"] * 4 if c["append"] else 0) + c["B"] * c["S"] * 4
        return {"bytes": b, "flops": rows * (c["d_rot"] // 2) * 6}
    if c["op"] == "evict":
        total = 0
        for n in _lens(c):
            total += 8 * n + 8 * c["S_cap"]
            if n > c["budget"]:
                must = c["n_sink"] + c["n_recent"]
                free, cand = c["budget"] - must, n - must
                newest = min(c["n_recent"], n - c["budget"])
                moved = newest + free * max(0, n - c["budget"] - newest) / max(1, cand)
                total += moved * (c["d_k"] + c["d_v"]) * 2 * 2
        return {"bytes": int(total * c["Hkv"]), "flops": int(sum(_lens(c)) * c["Hkv"])}
    T = c["T"] if c["op"] == "tree" else 1
    row = c["d_qk"] + c["d_v"]
    keys = pairs = 0
    for n in _lens(c):
        w = c.get("window", 0)
        seen = min(n, w) if w else n
        keys += seen + (T if c["op"] == "tree" else 0)
        pairs += (seen + 1) * T
    by = keys * c["Hkv"] * row * 2 + c["B"] * c["Hq"] * T * row * 2
    if c["op"] == "weights":
        by += keys * c["Hkv"] * 8
    return {"bytes": int(by), "flops": int(pairs * c["Hq"] * row * 2)}


# ---------------------------------------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")


def prepare(case, seed):
    c, dev = case, _device()
    rng = random.Random(seed)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16) * scale

    s = {"case": c}
    B = c["B"]
    if c["op"] == "rope":
        # as projections leave them: [B, S, H, d], seen as [B, H, S, d]
        s["q"] = normal(B, c["S"], c["Hq"], c["d"]).transpose(1, 2)
        s["k"] = normal(B, c["S"], c["Hkv"], c["d"]).transpose(1, 2)
        far = [rng.randint(c["far"] // 2, max(1, c["far"])) for _ in range(B)]
        start = torch.tensor(far, dtype=torch.int32, device=dev)[:, None]
        step = torch.arange(c["S"], dtype=torch.int32, device=dev)[None]
        if c["append"]:  # drafted tokens: several share a depth
            step = torch.div(step, 2, rounding_mode="floor")
            s["v"] = normal(B, c["S"], c["Hkv"], c["d"]).transpose(1, 2)
            s["k_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d"])
            s["v_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d"])
            rows = [rng.randint(0, c["S_cap"] - c["S"]) for _ in range(B)]
            s["row0"] = torch.tensor(rows, dtype=torch.int32, device=dev)
        s["positions"] = (start + step).to(torch.int32).contiguous()
        return s
    lens = _lens(c, rng)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if c["op"] == "evict":
        s["k_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d_k"])
        s["v_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d_v"])
        # weights gathered so far: a few rows hold most of them
        s["acc"] = torch.exp(1.5 * torch.randn(B, c["Hkv"], c["S_cap"], generator=g, device=dev))
        if c["aged"]:
            # a cache that was cut before: older rows in any order with gaps, the newest ones behind them
            old = torch.rand(B, c["Hkv"], c["budget"], generator=g, device=dev).argsort(dim=-1) * 3
            new = 3 * c["budget"] + torch.arange(c["S_cap"] - c["budget"], device=dev).expand(B, c["Hkv"], -1)
            s["positions"] = torch.cat([old, new], dim=-1).to(torch.int32).contiguous()
            s["next_pos"] = s["lens"] - c["budget"] + 3 * c["budget"]
        else:
            s["positions"] = s["next_pos"] = None
        return s
    T = c["T"] if c["op"] == "tree" else 1
    s["q"] = normal(B, c["Hq"], T, c["d_qk"], scale=1.5)
    s["k_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d_qk"])
    s["v_cache"] = normal(B, c["Hkv"], c["S_cap"], c["d_v"])
    if c["op"] == "weights":
        s["acc"] = torch.rand(B, c["Hkv"], c["S_cap"], generator=g, device=dev)
        return s
    words, places = [], []
    for b in range(B):
        mask, depth = [], []
        for t in range(T):
            p = rng.randint(max(-1, t - 6), t - 1)  # parent; -1: the cache's last token
            mask.append((1 << t) | (mask[p] if p >= 0 else 0))
            depth.append(depth[p] + 1 if p >= 0 else 0)
        words.append([m - (1 << 64) if m >> 63 else m for m in mask])
        places.append([lens[b] + d for d in depth])
    s["tree_mask"] = torch.tensor(words, dtype=torch.int64, device=dev)
    s["positions"] = torch.tensor(places, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _frequencies(c, device):
    """theta_i in 64 bits, with YaRN's three regimes (beta_fast 32, beta_slow 1)."""
    i = torch.arange(c["d_rot"] // 2, dtype=torch.float64, device=device)
    theta = 10000.0 ** (-2.0 * i / c["d_rot"])
    if c["yarn"] > 1.0:
        lam = 2 * math.pi / theta
        t = ((lam - 1.0) / (c["yarn"] - 1.0)).clamp(0, 1)
        mid = theta / (t * c["yarn"] + 1 - t)
        theta = torch.where(lam < 32.0, theta, torch.where(lam > c["yarn"], theta / c["yarn"], mid))
    return theta


def _rotated(x, cos, sin, c):
    a, n = c["rot_start"], c["d_rot"]
    x = x.float()
    part = x[..., a:a + n]
    if c["half"]:
        u, w = part[..., :n // 2], part[..., n // 2:]
        turned = torch.cat([u * cos - w * sin, u * sin + w * cos], dim=-1)
    else:
        u, w = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([u * cos - w * sin, u * sin + w * cos], dim=-1).flatten(-2)
    return torch.cat([x[..., :a], turned, x[..., a + n:]], dim=-1).to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, :, None] * _frequencies(c, s["q"].device)
    if c["inverse"]:
        angle = -angle
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q, k = _rotated(s["q"], cos, sin, c), _rotated(s["k"], cos, sin, c)
    if not c["append"]:
        return {"q": q, "k": k}
    rows = s["row0"].long()[:, None] + torch.arange(c["S"], device=q.device)
    b = torch.arange(c["B"], device=q.device)[:, None]
    s["k_cache"][b, :, rows] = k.transpose(1, 2)
    s["v_cache"][b, :, rows] = s["v"].transpose(1, 2)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _tree_visible(s):
    """[B, T, S_cap]: which cache rows each drafted token sees."""
    c, lens, pos = s["case"], s["lens"].long(), s["positions"].long()
    j = torch.arange(c["S_cap"], device=lens.device)
    u = j[None, :] - lens[:, None]  # draft number of each row
    old = (u < 0)[:, None, :].expand(-1, c["T"], -1)
    draft = (u >= 0) & (u < c["T"])
    uc = u.clamp(0, c["T"] - 1)
    bit = (s["tree_mask"][:, :, None] >> uc[:, None, :]) & 1
    seen = old | (draft[:, None, :] & (bit == 1))
    if c["window"] > 0:
        at = torch.where(draft, torch.gather(pos, 1, uc), j[None, :])
        seen = seen & (pos[:, :, None] - at[:, None, :] < c["window"])
    return seen


def _softmax_rows(q, k, seen, Hkv, scale):
    """Weights [B, Hkv, G, T, S] of q [B, Hq, T, d] over k [B, Hkv, S, d]."""
    B, Hq, T, d = q.shape
    x = torch.matmul(q.float().reshape(B, Hkv, -1, d), k.float().transpose(-1, -2)).reshape(B, Hkv, Hq // Hkv, T, -1)
    x = torch.where(seen[:, None, None], x * scale, NEG)
    top = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - torch.where(top == NEG, 0.0, top))
    total = e.sum(dim=-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def _plain_attention(s):
    c = s["case"]
    q = s["q"]
    B, Hq, T, d = q.shape
    if c["op"] == "tree":
        seen = _tree_visible(s)
    else:
        seen = (torch.arange(c["S_cap"], device=q.device)[None] < s["lens"][:, None])[:, None]
    p = _softmax_rows(q, s["k_cache"], seen, c["Hkv"], 1.0 / math.sqrt(d))
    out = torch.matmul(p.reshape(B, c["Hkv"], -1, c["S_cap"]), s["v_cache"].float())
    out = out.reshape(B, Hq, T, c["d_v"]).to(torch.bfloat16)
    if c["op"] == "tree":
        return out
    s["acc"] += p.sum(dim=(2, 3))
    return {"out": out, "acc": s["acc"]}


def _plain_evict(s):
    c, acc, lens = s["case"], s["acc"], s["lens"].long()
    n, budget = c["S_cap"], c["budget"]
    j = torch.arange(n, device=acc.device)
    pos = s["positions"].long() if s["positions"] is not None else j.expand_as(acc)
    nxt = (s["next_pos"].long() if s["next_pos"] is not None else lens)[:, None, None]
    there = (j < lens[:, None, None]).expand_as(acc)
    must = (pos < c["n_sink"]) | (pos >= nxt - c["n_recent"])
    key = torch.where(must, float("inf"), acc)
    key = torch.where(there, key, NEG)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices  # ties: the lowest row first
    kept = torch.zeros_like(there).scatter_(-1, order[..., :budget], True) & there
    low = (j < budget)
    hb, hh, hole = (there & ~kept & low).nonzero(as_tuple=True)
    sb, sh, src = (kept & ~low).nonzero(as_tuple=True)
    s["k_cache"][hb, hh, hole] = s["k_cache"][sb, sh, src]
    s["v_cache"][hb, hh, hole] = s["v_cache"][sb, sh, src]
    acc_out, pos_out = acc.clone(), pos.to(torch.int32).clone()
    acc_out[hb, hh, hole] = acc[sb, sh, src]
    pos_out[hb, hh, hole] = pos[sb, sh, src].to(torch.int32)
    lens_out = lens.clamp(max=budget)
    behind = j >= lens_out[:, None, None]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "acc": acc_out.masked_fill_(behind, 0.0),
            "positions": pos_out.masked_fill_(behind, -1), "lens": lens_out.to(torch.int32)}


# ---------------------------------------------------------------------------------------------- the package's calls
def _own_run(s):
    import transformer_attention_rope_gb300 as apex
    c = s["case"]
    if c["op"] == "rope":
        how = dict(positions=s["positions"], layout="half" if c["half"] else "interleaved", d_rot=c["d_rot"],
                   rot_start=c["rot_start"], inverse=c["inverse"], yarn_scale=c["yarn"])
        if c["append"]:
            q, k, v = apex.rope(s["q"], s["k"], s["v"], k_out=s["k_cache"], v_out=s["v_cache"], row0=s["row0"], **how)
            return {"q": q, "k_cache": k, "v_cache": v}
        q, k = apex.rope(s["q"], s["k"], **how)
        return {"q": q, "k": k}
    if c["op"] == "tree":
        return apex.tree_decode(s["q"], s["k_cache"], s["v_cache"], s["lens"], tree_mask=s["tree_mask"],
                                positions=s["positions"], window=c["window"])
    if c["op"] == "weights":
        out = apex.decode_weights(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["acc"])
        return {"out": out, "acc": s["acc"]}
    acc, pos, lens = apex.evict(s["k_cache"], s["v_cache"], s["acc"], s["lens"], c["budget"], n_sink=c["n_sink"],
                                n_recent=c["n_recent"], positions=s["positions"], next_pos=s["next_pos"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "acc": acc, "positions": pos, "lens": lens}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return _plain_rope(state) if op == "rope" else _plain_evict(state) if op == "evict" else _plain_attention(state)


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time."""
    c, s = case, prepare(case, seed)
    dev = s["k_cache" if "k_cache" in s else "q"].device
    if c["op"] == "rope":
        pairs = c["d_rot"] // 2
        theta = []
        for i in range(pairs):
            th = 10000.0 ** (-2.0 * i / c["d_rot"])
            if c["yarn"] > 1.0:
                lam = 2.0 * math.pi / th
                if lam > c["yarn"]:
                    div = c["yarn"]
                else:
                    t = min(1.0, max(0.0, (lam - 1.0) / (c["yarn"] - 1.0)))
                    div = t * c["yarn"] + 1.0 - t
                th = th if lam < 32.0 else th / div
            theta.append(th)
        ang = s["positions"].double()[:, None, :, None] * torch.tensor(theta, dtype=torch.float64, device=dev)
        turn = torch.polar(torch.ones_like(ang), -ang if c["inverse"] else ang)
        at = c["rot_start"] + torch.arange(pairs, device=dev) * (1 if c["half"] else 2)
        to = at + (pairs if c["half"] else 1)

        def rotate(x):
            y = x.double().contiguous()
            z = torch.complex(y[..., at], y[..., to]) * turn
            y[..., at], y[..., to] = z.real, z.imag
            return y

        q, k = rotate(s["q"]), rotate(s["k"])
        if not c["append"]:
            return {"q": q, "k": k}
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, r in enumerate(s["row0"].tolist()):
            kc[b, :, r:r + c["S"]] = k[b]
            vc[b, :, r:r + c["S"]] = s["v"][b].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    lens = s["lens"].tolist()
    if c["op"] == "evict":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        acc_out = torch.zeros_like(s["acc"], dtype=torch.float64)
        for b, n in enumerate(lens):
            nxt = int(s["next_pos"][b]) if s["next_pos"] is not None else n
            for h in range(c["Hkv"]):
                acc = s["acc"][b, h, :n].double()
                pos = s["positions"][b, h, :n].long() if s["positions"] is not None else torch.arange(n, device=dev)
                rank = torch.where((pos < c["n_sink"]) | (pos >= nxt - c["n_recent"]), float("inf"), acc)
                keep = torch.argsort(-rank, stable=True)[:c["budget"]].sort().values
                stay, come = keep[keep < c["budget"]], keep[keep >= c["budget"]]
                free = torch.ones(min(n, c["budget"]), dtype=torch.bool, device=dev)
                free[stay] = False
                free = free.nonzero().flatten()
                kc[b, h, free], vc[b, h, free] = kc[b, h, come], vc[b, h, come]
                acc_out[b, h, stay], acc_out[b, h, free] = acc[stay], acc[come]
        return {"k_cache": kc, "v_cache": vc, "acc": acc_out, "positions": None, "lens": None}
    B, Hq, T, d = s["q"].shape
    G = Hq // c["Hkv"]
    out = torch.empty(B, Hq, T, c["d_v"], dtype=torch.float64, device=dev)
    acc = s["acc"].double() if c["op"] == "weights" else None
    for b, n in enumerate(lens):
        m = n + (T if c["op"] == "tree" else 0)
        if c["op"] == "tree":
            seen = torch.ones(T, m, dtype=torch.bool, device=dev)
            word = s["tree_mask"][b].tolist()
            seen[:, n:] = torch.tensor([[bool((w >> u) & 1) for u in range(T)] for w in word], device=dev)
            if c["window"] > 0:
                here = s["positions"][b].long()
                seen &= here[:, None] - torch.cat([torch.arange(n, device=dev), here])[None] < c["window"]
        else:
            seen = torch.ones(1, m, dtype=torch.bool, device=dev)
        for h in range(c["Hkv"]):
            x = s["q"][b, h * G:(h + 1) * G].double() @ s["k_cache"][b, h, :m].double().T / math.sqrt(d)
            p = torch.softmax(x.masked_fill(~seen, NEG), dim=-1)
            out[b, h * G:(h + 1) * G] = p @ s["v_cache"][b, h, :m].double()
            if acc is not None:
                acc[b, h, :m] += p.sum(dim=(0, 1))
    return out if acc is None else {"out": out, "acc": acc}
