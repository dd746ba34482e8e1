"""The decode step of examples/decode_step.py against plain fp32 operations, several steps from an empty
cache: the operators run together as a decoder uses them.  The expert layer's output is taken from the step
itself, and its input compared (its own tests compare it with the oracle; run here on an input that is a
rounding off, it would quantise some activations to the next E4M3 value, which the bound below does not
count).

Tolerance: a layer rounds to bf16 about eight times on its path (norms, projections, cache, attention,
residual), each by at most 2^-8 of the value, to be taken as independent: sqrt(8) 2^-8 = 1.1e-2 of a branch
a layer at most in the L2 norm, and the branches are a part of the residual.  Held to 2e-2 for two layers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_decode_steps(cache, monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as moe
    from examples import decode_step as ex
    dtype = moe.binding.MOE_E4M3 if cache == "e4m3" else moe.binding.MOE_BF16
    batch, heads, hk, dim = 3, 8, 2, 64
    dec = ex.build(2, batch, 64, heads=heads, kv_heads=hk, dim=dim, d=512, ffn=128, experts=16, page=16, cache_dtype=dtype)
    dec.blocks[0].window = 4  # shorter than the steps, so that the window moves
    keys = [[[] for _ in dec.blocks], [[] for _ in dec.blocks]]

    def norm(t, w):
        return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w

    def stored(t):  # what a cache row holds
        if cache == "bf16":
            return t.bfloat16().float()
        m, e = torch.frexp(t.abs().amax(-1, keepdim=True))
        unit = torch.exp2((e - 9 + (m > 0.875)).float())
        return (t / unit).to(torch.float8_e4m3fn).float() * unit

    seen = []
    forward = moe.forward

    def recorded(x, *args, **kw):
        out = forward(x, *args, **kw)
        seen.append((x.float(), out[0].clone()))
        return out

    monkeypatch.setattr(ex.moe, "forward", recorded)
    g = torch.Generator(device="cuda").manual_seed(9)
    for step in range(7):
        embed = torch.randn(batch, 512, generator=g, device="cuda").bfloat16()
        dec.residual.copy_(embed)
        seen.clear()
        got = dec.step().float()
        r = embed.float()
        for i, b in enumerate(dec.blocks):
            x = norm(r, b.attn_norm)
            qkv = (x @ b.w_qkv.float()).view(batch, heads + 2 * hk, dim)
            for kind, rows in ((0, qkv[:, heads:heads + hk]), (1, qkv[:, heads + hk:])):
                keys[kind][i].append(stored(rows))
            k, v = (torch.stack(keys[kind][i][-(b.window or 99):], 1) for kind in (0, 1))  # [batch, n, hk, dim]
            q = qkv[:, :heads].view(batch, hk, heads // hk, dim)
            p = torch.softmax(torch.einsum("bkgd,bnkd->bkgn", q, k) * dim ** -0.5, -1)
            a = torch.einsum("bkgn,bnkd->bkgd", p, v).reshape(batch, heads * dim)
            r = r + a @ b.w_out.float()
            x = norm(r, b.moe_norm)
            x_seen, y = seen[i]
            rel = float((x_seen - x).norm() / x.norm())
            assert rel < 2e-2, f"step {step}, layer {i}: the expert layer's input, relative L2 {rel:.3e}"
            r = r + dec.alpha * norm(y, b.moe_post_norm)
        rel = float((got - r).norm() / r.norm())
        assert rel < 2e-2, f"step {step}: relative L2 {rel:.3e}"
    assert moe.get_status(dec.attn_ws) == 0 and moe.get_status(dec.moe_ws) == 0
    assert dec.lens.tolist() == [8] * batch
