"""Edges of the operators over caches of rotated keys: windows that begin past the cached keys' end, outputs
on inputs, sizes that do not fit, lengths and positions that a cut left behind.  Plain forms and tolerances are
those of test_cache_operators.py."""
import pytest
import torch

import transformer_attention_rope_gb300 as apex
from test_cache_operators import _attn_inputs, _attn_ref, _close, _gpu, _tree


# ------------------------------------------------------------------------------------------------- windows
def _seen_by_some(T, n, cap, mask, pos, window):
    """[m]: rows of one sequence that some draft sees; mask [T] words, pos [T] positions, n cached keys."""
    m = min(n + T, cap)
    seen = torch.zeros(m, dtype=torch.bool)
    for t in range(T):
        at = max(int(pos[t]), n)
        seen[max(0, min(n, at - window + 1)):n] = True
        for u in range(m - n):
            if (int(mask[t]) >> u) & 1 and at - max(int(pos[u]), n) < window:
                seen[n + u] = True
    return seen


WINDOWS = [  # Hq, Hkv, T, d_qk, d_v, S_cap, lens, window
    (8, 2, 1, 128, 128, 300, [100, 290], 4),
    (8, 2, 2, 128, 128, 300, [100, 298], 4),
    (8, 2, 6, 128, 128, 2000, [1500, 1994, 3], 100),
    (8, 2, 20, 64, 64, 1100, [1080, 4], 3),
    (4, 4, 4, 128, 128, 5000, [4996, 2500], 1024),
    (16, 1, 40, 192, 128, 600, [128, 560], 130),
    (16, 1, 12, 64, 64, 900, [880, 128], 300),     # two M tiles on one CTA
    (16, 1, 12, 128, 128, 900, [880, 256], 300),   # pairs, one M tile
    (16, 1, 33, 128, 128, 900, [860, 640], 300),   # pairs, two M tiles
    (8, 2, 3, 192, 128, 800, [797, 513], 257),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 3, 150, 2000])
@pytest.mark.parametrize("Hq,Hkv,T,dk,dv,cap,lens,window", WINDOWS)
def test_tree_decode_rows_before_every_window_may_hold_anything(Hq, Hkv, T, dk, dv, cap, lens, window, shift):
    """Drafts whose positions begin `shift` past the cached keys: the windows' far edge is theirs, not len's.
    A shift of 150 leaves whole tiles of keys to nobody, 2000 every cached key."""
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, cap + shift, Hq, Hkv, T, dk, dv, cap, lens)
    mask, pos = _tree(T, len(lens), T, lens)
    pos = pos + shift
    for b, n in enumerate(lens):
        seen = torch.zeros(cap, dtype=torch.bool)
        some = _seen_by_some(T, n, cap, mask[b], pos[b], window)
        seen[:len(some)] = some
        seen = seen.to(dev)
        k[b, :, ~seen], v[b, :, ~seen] = float("inf"), float("nan")
    got = apex.tree_decode(q, k, v, ln, tree_mask=mask.to(dev), positions=pos.to(dev), window=window)
    ref, tol, _, _ = _attn_ref(q, k, v, lens, True, mask, pos, window)
    _close(got, ref, tol)
    assert apex.apex_attn_device_status() == 0


# ------------------------------------------------------------------------------------------------- rope: outputs on inputs
@pytest.fixture(scope="module")
def lib():
    try:
        return apex.load_library()
    except RuntimeError:
        pytest.skip("library not built")


P = 1 << 20  # an aligned address that a refused call never touches
BAD = 1


def _rows(at, out, heads, d, strides, out_strides=None):
    return apex.RopeTensor(at, out, heads, d, *strides, *(out_strides or strides))


def _rope_status(q, k=None, v=None, B=2, S=4, row0=None, out_rows=0):
    return apex.apex_attn_rope(q, k, v, B, S, P, S, row0, out_rows, apex.RopeOptions(), None)


DENSE = (2 * 4 * 64, 4 * 64, 64)       # [2, 2, 4, 64]
CACHE = (2 * 32 * 64, 32 * 64, 64)     # rows of [2, 2, 32, 64]


@pytest.mark.parametrize("what", ["shifted by a row", "shifted by an entry", "transposed", "q on k", "k on v's input",
                                  "one output for both", "in place with row0", "rows of the cache itself",
                                  "v on the queries", "an output over itself", "one head's rows again"])
def test_rope_refuses_outputs_that_other_threads_still_read(lib, what):
    """One thread would write a row that another has not read, or has written."""
    q = _rows(P, 2 * P, 2, 64, DENSE)
    k = _rows(4 * P, 8 * P, 2, 64, DENSE, CACHE)
    v = _rows(5 * P, 16 * P, 2, 64, DENSE, CACHE)
    more = dict(row0=P, out_rows=32)
    if what == "shifted by a row":
        q, k, v, more = _rows(P, P + 2 * 64, 2, 64, DENSE), None, None, {}
    elif what == "shifted by an entry":
        q, k, v, more = _rows(P, P + 2, 2, 64, DENSE), None, None, {}
    elif what == "transposed":
        q, k, v, more = _rows(P, P, 2, 64, DENSE, (2 * 4 * 64, 64, 2 * 64)), None, None, {}
    elif what == "q on k":
        q.out = 4 * P + 2 * 1023  # the last entry of k
    elif what == "k on v's input":
        k.out = 5 * P
    elif what == "one output for both":
        v.out = 8 * P + 2 * 32 * 64
    elif what == "in place with row0":
        k = _rows(4 * P, 4 * P, 2, 64, DENSE)
        more = dict(row0=P, out_rows=4)
    elif what == "rows of the cache itself":
        k = _rows(8 * P + 2 * 10 * 64, 8 * P, 2, 64, CACHE)
    elif what == "v on the queries":
        v.out = P
    elif what == "an output over itself":
        q, k, v, more = _rows(P, 2 * P, 2, 64, DENSE, (2 * 4 * 64, 32, 64)), None, None, {}
    else:
        q, k, v, more = _rows(P, 2 * P, 2, 64, DENSE, (2 * 4 * 64, 0, 64)), None, None, {}
    assert _rope_status(q, k, v, **more) == BAD


def test_rope_refuses_exactly_the_outputs_that_share_elements(lib):
    """Random small layouts against their elements, listed one by one."""
    if torch.cuda.is_available():
        pytest.skip("calls that pass the checks would run on addresses that hold nothing")
    import itertools
    import random
    r = random.Random(5)

    def elements(at, heads, d, strides, S):
        return [at // 2 + b * strides[0] + h * strides[1] + s * strides[2] + e
                for b, h, s, e in itertools.product(range(2), range(heads), range(S), range(d))]

    def layout(heads, d, S):
        sizes, step, strides = [(0, 2), (1, heads), (2, S)], d, [0, 0, 0]
        r.shuffle(sizes)
        for i, n in sizes:
            step += r.choice([0, 0, 0, d, 2 * d, 1, -1])
            strides[i] = step * r.choice([1, 1, 1, 1, -1])
            step *= n
        return tuple(strides)

    counts = [0, 0]
    for trial in range(3000):
        S, row0 = r.randint(1, 4), r.random() < 0.4
        rows = S + r.randint(0, 3) if row0 else S
        tensors = []
        for i in range(3):
            heads, d = r.randint(1, 3), r.choice([2, 4])
            a = layout(heads, d, S)
            o = a if r.random() < 0.5 else layout(heads, d, rows)
            at = P + 2 * r.randint(0, 300)
            tensors.append((at, at if r.random() < 0.3 else P + 2 * r.randint(0, 300), heads, d, a, o))
        tensors = [t if r.random() < 0.7 else None for t in tensors]
        if tensors[0] and tensors[1] and tensors[0][3] != tensors[1][3] or not any(tensors):
            continue
        ins = [t and elements(t[0], t[2], t[3], t[4], S) for t in tensors]
        outs = [t and elements(t[1], t[2], t[3], t[5], rows if row0 and i else S) for i, t in enumerate(tensors)]
        bad = False
        for i, t in enumerate(tensors):
            if not t:
                continue
            bad |= len(set(outs[i])) < len(outs[i])
            bad |= any(set(outs[i]) & set(outs[k]) for k in range(i) if tensors[k])
            for k in range(3):
                if tensors[k] and not (k == i and outs[i] == ins[i] and not (row0 and i)):
                    bad |= bool(set(outs[i]) & set(ins[k]))
        args = [t and _rows(t[0], t[1], t[2], t[3], t[4], t[5]) for t in tensors]
        status = _rope_status(*args, S=S, row0=P if row0 else None, out_rows=rows)
        assert (status == BAD) == bad, (trial, tensors, S, row0, rows)
        counts[bad] += 1
    assert min(counts) > 200, counts


@pytest.mark.gpu
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_rope_turns_the_parts_of_one_projection_in_place(half, pad):
    """q and k interleaved in one buffer with v, both in place: their spans overlap, their elements do not."""
    from test_cache_operators import _gen, _normal, _rope_close, _rope_ref
    dev = _gpu()
    g = _gen(dev, 90 + pad)
    B, S, Hq, Hkv, d = 2, 9, 6, 2, 64
    fused = _normal(g, dev, B, S, (Hq + 2 * Hkv) * d + pad)
    before = fused.clone()
    part = lambda x, a, n: x[..., a * d:(a + n) * d].view(B, S, n, d).transpose(1, 2)
    q, k, v = part(fused, 0, Hq), part(fused, Hq, Hkv), part(fused, Hq + Hkv, Hkv)
    pos = torch.randint(0, 999, (B, S), generator=g, device=dev, dtype=torch.int32)
    how = dict(positions=pos, layout="half" if half else "interleaved")
    q2, k2, v2 = apex.rope(q, k, v, q_out=q, k_out=k, **how)
    assert q2 is q and k2 is k and torch.equal(v2, part(before, Hq + Hkv, Hkv))
    for x, a, n in ((q, 0, Hq), (k, Hq, Hkv)):
        _rope_close(x, *_rope_ref(part(before, a, n), pos, half=half))
    assert torch.equal(fused[..., (Hq + Hkv) * d:], before[..., (Hq + Hkv) * d:])
    with pytest.raises(apex.ApexError):
        apex.rope(q, k, positions=pos, q_out=q, k_out=q[:, :Hkv])


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["b s kv h", "b h s kv", "s b kv h", "kv b h s"])
def test_rope_appends_to_caches_that_share_a_buffer(order):
    """Keys and values side by side in one buffer, in any order of dimensions."""
    from test_cache_operators import _gen, _normal, _rope_close, _rope_ref
    dev = _gpu()
    g = _gen(dev, 95)
    size = dict(b=2, h=3, s=40, kv=2)
    names = order.split()
    buf = _normal(g, dev, *[size[n] for n in names], 64)
    view = buf.permute(*[names.index(n) for n in ("kv", "b", "h", "s")], 4)
    kc, vc = view[0], view[1]
    before = kc.clone(), vc.clone()
    S, row0 = 5, [0, 37]  # the second loses its last two rows
    q, k, v = (_normal(g, dev, 2, h, S, 64) for h in (6, 3, 3))
    pos = torch.randint(0, 999, (2, S), generator=g, device=dev, dtype=torch.int32)
    apex.rope(q, k, v, positions=pos, k_out=kc, v_out=vc, row0=torch.tensor(row0, dtype=torch.int32, device=dev))
    want, slack = _rope_ref(k, pos)
    for b, r in enumerate(row0):
        n = min(S, 40 - r)
        _rope_close(kc[b, :, r:r + n], want[b, :, :n], slack[b, :, :n])
        assert torch.equal(vc[b, :, r:r + n], v[b, :, :n])
        for c, old in zip((kc, vc), before):
            c[b, :, r:r + n] = old[b, :, r:r + n]
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


# ------------------------------------------------------------------------------------------------- rope: which kernel runs
def _launched(call):
    """(name, grid) of the kernels that `call` launches."""
    import json
    import os
    import tempfile
    from torch.profiler import ProfilerActivity, profile
    call()
    torch.cuda.synchronize()
    found = []
    for _ in range(3):  # a process's first records may be lost
        with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
        with tempfile.TemporaryDirectory() as d:
            at = os.path.join(d, "trace.json")
            p.export_chrome_trace(at)
            with open(at) as f:
                events = json.load(f)["traceEvents"]
        found = found or [(e["name"], e["args"]["grid"]) for e in events if e.get("cat") == "kernel"]
    if not found:
        pytest.skip("no kernel records from the profiler")
    return found


@pytest.mark.gpu
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("d,wide", [(128, True), (72, True), (66, False)])
def test_rope_of_values_alone(d, wide, half):
    """Values appended without queries and keys: rows of 16 bytes go 16 bytes at a time."""
    from test_cache_operators import _gen, _normal
    dev = _gpu()
    g = _gen(dev, 97)
    B, H, S, cap = 2, 3, 5, 20
    v, vc = _normal(g, dev, B, H, S, d), _normal(g, dev, B, H, cap, d)
    want = vc.clone()
    want[0, :, 7:12], want[1, :, 17:20] = v[0], v[1, :, :3]
    row0 = torch.tensor([7, 17], dtype=torch.int32, device=dev)
    pos = torch.zeros(S, dtype=torch.int32, device=dev)
    t = apex.RopeTensor(v.data_ptr(), vc.data_ptr(), H, d, *v.stride()[:3], *vc.stride()[:3])
    opt = apex.RopeOptions(layout=half)

    def call():
        assert apex.apex_attn_rope(None, None, t, B, S, pos.data_ptr(), 0, row0.data_ptr(), cap, opt,
                                   torch.cuda.current_stream(dev).cuda_stream) == 0

    call()
    assert torch.equal(vc, want)
    names = [n for n, _ in _launched(call) if "rope" in n]
    assert len(names) == 1 and ("rope_rows" in names[0]) == wide, names


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,groups", [(32, 8, 48), (33, 8, 25), (24, 12, 48), (46, 1, 48), (48, 48, 48), (1, 1, 3)])
def test_rope_of_one_token_spreads_its_heads(Hq, Hkv, groups):
    """Few tokens: a head of q, k or v to a group as far as groups go, then two, and so on."""
    from test_cache_operators import _gen, _normal, _rope_close, _rope_ref
    dev = _gpu()
    g = _gen(dev, Hq)
    q, k, v = (_normal(g, dev, 1, h, 1, 128) for h in (Hq, Hkv, Hkv))
    pos = torch.tensor([4321], dtype=torch.int32, device=dev)
    got = apex.rope(q, k, v, positions=pos)
    for x, y in zip((q, k), got):
        _rope_close(y, *_rope_ref(x, pos[None]))
    assert torch.equal(got[2], v)
    grids = [at for n, at in _launched(lambda: apex.rope(q, k, v, positions=pos)) if "rope_rows" in n]
    assert len(grids) == 1 and grids[0][1] == groups, grids


# ------------------------------------------------------------------------------------------------- evict
@pytest.mark.gpu
@pytest.mark.parametrize("cap,lens,budget,sink,recent", [
    (300, [300, 250, 0], 200, 4, 20), (300, [300, 290], 64, 0, 0), (5000, [5000, 4300], 600, 4, 64),
    (40000, [40000], 3000, 7, 100)])
def test_evict_finds_the_newest_position_of_a_cache_that_was_cut_before(cap, lens, budget, sink, recent):
    """Without next_pos the newest rows are those behind the largest position, not behind the length:
    positions far past the lengths would all count as new, and the lowest rows stay whatever their weights."""
    from test_cache_operators import _evict_check, _evict_ref, _gen, _normal
    dev = _gpu()
    g = _gen(dev, cap + budget)
    B, H = len(lens), 2
    k, v = _normal(g, dev, B, H, cap, 8), _normal(g, dev, B, H, cap, 8)
    acc = torch.exp(torch.randn(B, H, cap, generator=g, device=dev))
    pos = (torch.rand(B, H, cap, generator=g, device=dev).argsort(-1) * 3 + cap).to(torch.int32).contiguous()
    for head in range(H):  # the heads' newest rows differ
        pos[:, head, ::7] += 5 * head
    wants = []
    for head in range(H):
        own = [int(pos[b, head, :n].max()) + 1 if n else 0 for b, n in enumerate(lens)]
        one = slice(head, head + 1)
        wants.append(_evict_ref(k[:, one], v[:, one], acc[:, one], lens, budget, sink, recent, pos[:, one], own))
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    a, p, n = apex.evict(k, v, acc, ln, budget, n_sink=sink, n_recent=recent, positions=pos)
    for head in range(H):
        want = wants[head]
        assert torch.equal(p[:, head].cpu(), want[3][:, 0]) and n.tolist() == want[4]
        assert torch.equal(a[:, head].double().cpu(), want[2][:, 0])
        assert torch.equal(k[:, head].cpu(), want[0][:, 0]) and torch.equal(v[:, head].cpu(), want[1][:, 0])
    # rows in order, none cut before: the length, as without positions
    k, v = _normal(g, dev, B, H, cap, 8), _normal(g, dev, B, H, cap, 8)
    rows = torch.arange(cap, dtype=torch.int32, device=dev).expand(B, H, cap).contiguous()
    k2, v2 = k.clone(), v.clone()
    got = apex.evict(k, v, acc, ln, budget, n_sink=sink, n_recent=recent, positions=rows)
    want = apex.evict(k2, v2, acc, ln, budget, n_sink=sink, n_recent=recent)
    assert all(torch.equal(x, y) for x, y in zip((*got, k, v), (*want, k2, v2)))


@pytest.mark.gpu
def test_evict_newest_position_at_the_ends_of_the_range():
    """Positions up to the largest integer, and negative ones alone."""
    from test_cache_operators import _evict_check, _gen, _normal
    dev = _gpu()
    g = _gen(dev, 7)
    for top in (2 ** 31 - 1, 40, -3):
        k, v = _normal(g, dev, 1, 1, 60, 8), _normal(g, dev, 1, 1, 60, 8)
        acc = torch.rand(1, 1, 60, generator=g, device=dev)
        pos = (top - torch.randperm(60, generator=g, device=dev)).to(torch.int32).view(1, 1, 60)
        nxt = max(60, top + 1)
        if nxt < 2 ** 31:
            _evict_check(dev, k.clone(), v.clone(), acc, [60], 20, 0, 9, pos, [nxt])
            b = apex.evict(k.clone(), v.clone(), acc, torch.tensor([60], dtype=torch.int32, device=dev), 20,
                           n_recent=9, positions=pos, next_pos=torch.tensor([nxt], dtype=torch.int32, device=dev))
        else:  # the same with positions moved down
            b = apex.evict(k.clone(), v.clone(), acc, torch.tensor([60], dtype=torch.int32, device=dev), 20,
                           n_recent=9, positions=pos - 1000, next_pos=torch.tensor([nxt - 1000], dtype=torch.int32,
                                                                                   device=dev))
            b = (b[0], torch.where(b[1] >= 0, b[1] + 1000, b[1]), b[2])
        a = apex.evict(k, v, acc, torch.tensor([60], dtype=torch.int32, device=dev), 20, n_recent=9, positions=pos)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------------------------------------- sizes that do not fit
@pytest.mark.parametrize("o", [dict(budget=2 ** 32 + 2), dict(budget=2 ** 31), dict(budget=-2 ** 32 + 2),
                               dict(budget=2, n_sink=2 ** 32), dict(budget=2, n_recent=2 ** 32 + 1)])
def test_evict_refuses_sizes_that_do_not_fit_an_int(lib, o):
    """Cut to 32 bits, a budget of 2^32 + 2 would leave two rows of each cache."""
    x = torch.zeros(1, 2, 3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        apex.evict(x, x, torch.zeros(1, 2, 3), torch.zeros(1, dtype=torch.int32), **o)


@pytest.mark.gpu
def test_sizes_that_do_not_fit_an_int():
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 3, 8, 2, 4, 128, 128, 304, [300, 290])
    whole = apex.tree_decode(q, k, v, ln)
    for window in (-5, -2 ** 32 + 7, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 7, 2 ** 63):
        assert torch.equal(apex.tree_decode(q, k, v, ln, window=window), whole)
    assert not torch.equal(apex.tree_decode(q, k, v, ln, window=7), whole)
    acc, kept = torch.rand(2, 2, 304, device=dev), k.clone()
    with pytest.raises(ValueError):
        apex.evict(k, v, acc, ln, 2 ** 32 + 4)
    assert torch.equal(k, kept)
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    for o in (dict(d_rot=2 ** 32 + 64), dict(rot_start=2 ** 32), dict(rot_start=0.5)):
        with pytest.raises(ValueError):
            apex.rope(q, positions=pos, **o)
    with pytest.raises(apex.ApexError):  # an infinity in 32 bits
        apex.rope(q, positions=pos, rope_base=1e39)


@pytest.mark.gpu
def test_rope_refuses_outputs_of_other_shapes():
    dev = _gpu()
    q, k, v, ln = _attn_inputs(dev, 4, 8, 2, 4, 128, 128, 4, [0, 0])
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    for o in (dict(k_out=k[0, 0]), dict(k_out=k[0, 0], row0=ln), dict(k_out=k[0], row0=ln),
              dict(v=v, k_out=torch.empty_like(k), v_out=v[0, 0], row0=ln),
              dict(v=v, k_out=torch.empty_like(k), v_out=torch.empty_like(v)[:, :, :3], row0=ln)):
        with pytest.raises(ValueError):
            apex.rope(q, k, positions=pos, **o)


@pytest.mark.gpu
@pytest.mark.parametrize("off,S,per", [(0, 64, None), (1, 1, 1), (1, 64, None), (1, 512, 8)])
def test_rope_of_some_tokens_spreads_its_heads(off, S, per):
    """One block an SM where rows go 16 bytes at a time, four where they go 2 bytes at a time, heads in fours or
    up to eight."""
    from test_cache_operators import _gen, _normal, _rope_close, _rope_ref
    dev = _gpu()
    g = _gen(dev, 70 + S)
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    q, k, v = (_normal(g, dev, 1, S, h * 128 + off)[..., off:].view(1, S, h, 128).transpose(1, 2) for h in (32, 8, 8))
    pos = torch.arange(S, dtype=torch.int32, device=dev)
    got = apex.rope(q, k, v, positions=pos)
    for x, y in zip((q, k), got):
        _rope_close(y, *_rope_ref(x, pos[None]))
    assert torch.equal(got[2], v)
    blocks, room = (S * 128 // 256, 4 * sms) if off else (S * 16 // 256, sms)
    share = max(1, -(-blocks * 48 // room))
    want = min(share, 8) if off or share >= 8 else min(share, 4)
    assert per is None or want == per
    grids = [at for n, at in _launched(lambda: apex.rope(q, k, v, positions=pos)) if "rope_" in n]
    assert len(grids) == 1 and grids[0][1] == sum(-(-h // want) for h in (32, 8, 8)), grids
