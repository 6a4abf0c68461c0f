"""The operators of a layer with normed heads, a window with sinks and a cache in 4 bits, together as a
program has them: a prompt, then its tokens, over a bf16 cache and over a packed one; then a step of
training on the heads.  References and tolerances are those of each operator's own tests, on what the
operator before it gave."""
import pytest
import torch

import test_bits4
import test_norm_rope
import test_sinks
import transformer_attention_rope_gb300 as apex


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,Hkv,window,sinks", [(64, 4, 2, 40, 4), (128, 8, 2, 128, 1), (128, 32, 2, 100, 130)])
def test_prompt_tokens_and_gradients(d, Hq, Hkv, window, sinks):
    dev = test_sinks._gpu()
    g = torch.Generator(device=dev)
    g.manual_seed(d + Hq)
    B, S, cap = 2, 301, 330
    normal = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    weight = lambda: 1 + 0.1 * torch.randn(d, generator=g, device=dev)  # noqa: E731
    wq, wk = weight(), weight()
    pos = torch.arange(S, dtype=torch.int32, device=dev)
    # projections leave a token's heads side by side
    q, k, v = (normal(B, S, H, d).transpose(1, 2) for H in (Hq, Hkv, Hkv))
    qn = apex.norm_rope(q, positions=torch.zeros_like(pos), q_weight=wq)
    kn = apex.norm_rope(k, positions=pos, q_weight=wk)
    v = v.contiguous()
    out = apex.fwd(qn, kn, v, window=window, n_sink=sinks, keys_prerotated=True)
    ref, tol = test_sinks._ref(qn, kn, v, 0, window, sinks, turned=True)
    test_sinks._close(out, ref, tol)

    # both caches hold the prompt
    k_cache, v_cache = (torch.full((B, Hkv, cap, d), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    k_cache[:, :, :S], v_cache[:, :, :S] = kn, v
    packed = test_bits4._cache(dev, B, Hkv, cap, d) + test_bits4._cache(dev, B, Hkv, cap, d)
    how = dict(k_factor=torch.full((Hkv,), 2.0 ** -7, device=dev), v_factor=torch.full((Hkv,), 2.0 ** -8, device=dev))
    apex.append4(kn, v, *packed, **how)
    lens = torch.full((B,), S, dtype=torch.int32, device=dev)
    for T in (1, 4, 1, 9):
        q1, k1, v1 = normal(B, Hq, T, d), normal(B, Hkv, T, d), normal(B, Hkv, T, d)
        at = lens[:, None] + torch.arange(T, dtype=torch.int32, device=dev)
        qr, _, _ = apex.norm_rope(q1, k1, v1, positions=at, q_weight=wq, k_weight=wk, k_out=k_cache, v_out=v_cache,
                                  row0=lens)
        n = int(lens[0])
        apex.append4(k_cache[:, :, n:n + T], v1, *packed, row0=lens, **how)
        values = (test_bits4._values(packed[0], packed[1], how["k_factor"]),
                  test_bits4._values(packed[2], packed[3], how["v_factor"]))
        exact, tol = test_bits4._attn_ref(qr, *values, lens.tolist(), window, sinks)
        test_bits4._close(apex.decode4(qr, *packed, lens, window=window, n_sink=sinks, **how), exact, tol)
        # the same queries over the packed rows as bf16 and as 4 bits: weights in bf16 here, in fp16 there
        kb, vb = apex.unpack4(*packed, n_rows=n + T, **how)
        rows = apex.tree_decode(qr, kb, vb, lens, window=window, n_sink=sinks)
        # two roundings to bf16 of what is at most the largest value, and fp32 sums
        assert (rows.double().cpu() - exact).abs().max() <= (2.0 ** -7 + 2.0 ** -12) * vb.abs().max().item()
        drafts = apex.tree_decode(qr, k_cache, v_cache, lens, window=window, n_sink=sinks)
        assert torch.isfinite(drafts).all()
        lens += T

    # a step of training on the heads: the formula's gradients
    dq = normal(B, S, Hq, d).transpose(1, 2)
    dk = normal(B, S, Hkv, d).transpose(1, 2)
    gq, gk, gwq, gwk = apex.norm_rope_grad(dq, q, dk, k, positions=pos, q_weight=wq, k_weight=wk)
    for x, w, dy, dx, dw in ((q, wq, dq, gq, gwq), (k, wk, dk, gk, gwk)):
        rx, slack, rw, ew, terms, n = test_norm_rope._grad_ref(dy, x, w, pos[None], 1e-6, {})
        test_norm_rope._close(dx, rx, test_norm_rope.U * rx.abs() + slack)
        test_norm_rope._close(dw, rw.sum(0), ew.sum(0) + terms.sum(0) * (n * x.shape[1] / 8 + 32) * 2.0 ** -24)
