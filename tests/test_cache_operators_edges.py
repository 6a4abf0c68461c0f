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
