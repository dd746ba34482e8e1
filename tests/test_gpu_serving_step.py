"""The serving step of examples/decode_step.py against plain fp32 operations: prompts admitted, several steps with pages
from a shared pool, sequences that end and begin again, eager and as a replayed graph.

What the plain form attends to is the cache as it is read back (tests/test_gpu_feed.py holds what is written to the
formulas): keys and values in 4 bits fall to the next code where the step's own roundings, which the plain form does not
have, take them over a border.  The expert layer's output is taken from the step itself, as in the decode step's test.

Tolerance: as there, about eight roundings to bf16 a layer, each by at most 2^-8 of the value and taken as independent:
sqrt(8) 2^-8 = 1.1e-2 of a branch a layer at most in the L2 norm, the branches being a part of the residual.  The turned
queries are one more rounding: sqrt(9) 2^-8.  Held to 2e-2 for two layers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(cache, graph, monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as moe
    from examples import decode_step as ex
    from tests import feed_oracle as fo
    dtype = {"bf16": 1, "e4m3": 2, "int4": 4}[cache]
    batch, heads, hk, dim, d = 3, 8, 2, 64, 512
    srv = ex.build(2, batch, 64, heads=heads, kv_heads=hk, dim=dim, d=d, ffn=128, experts=16, page=16, cache_dtype=dtype,
                   serve=True)
    srv.blocks[0].window, srv.blocks[1].window = 20, 0
    assert isinstance(srv, ex.Server)
    freq, _ = fo.frequencies(dim)
    g = torch.Generator(device="cuda").manual_seed(11)
    seen = []
    forward = moe.forward

    def recorded(x, *args, **kw):
        out = forward(x, *args, **kw)
        seen.append((x, out[0].clone()))  # in a graph: buffers that each replay fills
        return out

    monkeypatch.setattr(ex.moe, "forward", recorded)

    def norm(t, w):
        return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w

    def turned(t, pos):
        a = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
        c, s, x, y = a.cos().float(), a.sin().float(), t[..., : dim // 2], t[..., dim // 2:]
        return torch.cat([x * c - y * s, y * c + x * s], -1)

    def prompts(new):
        plan = srv.admit(torch.tensor(new, dtype=torch.int32, device="cuda"), sum(new))
        for b in srv.blocks:
            x = torch.randn(sum(new), heads + 2 * hk, dim, generator=g, device="cuda").bfloat16()
            q, k, v = x[:, :heads], x[:, heads:heads + hk], x[:, heads + hk:]
            if b.window:
                moe.rope_kv_write(q, k, v, b.cache, srv.rope, plan.pos, plan.slot, srv.attn_ws)
            else:
                moe.kv_write(k, v, b.cache, plan.pos, srv.page_table, srv.attn_ws, seq=plan.seq)

    prompts([17, 0, 30])
    captured = None
    if graph:
        state = [t.clone() for t in (srv.lens, srv.n_free, srv.page_table)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            srv.step()
        torch.cuda.synchronize()
        seen.clear()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured, stream=side):
            srv.step()
        for t, s in zip((srv.lens, srv.n_free, srv.page_table), state):
            t.copy_(s)
        buffers = list(seen)
    for step in range(20):
        if step == 9:  # one leaves, and another takes its place
            srv.release(torch.tensor([False, False, True], device="cuda"))
            prompts([0, 0, 5])
        before = srv.lens.clone()
        embed = torch.randn(batch, d, generator=g, device="cuda").bfloat16()
        srv.residual.copy_(embed)
        seen.clear()
        if graph:
            captured.replay()
        else:
            srv.step()
        got, ys = srv.residual.float(), [y for _, y in (buffers if graph else seen)]
        assert torch.equal(srv.lens, before + 1) and torch.equal(srv.pos, before)
        r = embed.float()
        for i, b in enumerate(srv.blocks):
            qkv = (norm(r, b.attn_norm) @ b.w_qkv.float()).view(batch, heads + 2 * hk, dim)
            q = turned(qkv[:, :heads], before) if b.window else qkv[:, :heads]
            out = []
            for s in range(batch):
                n = int(srv.lens[s])
                first = max(0, n - b.window) if b.window else 0
                pos = torch.arange(first, n, dtype=torch.int32, device="cuda")
                k, v = moe.kv_read(b.cache, pos, srv.page_table, srv.attn_ws, seq=torch.full_like(pos, s), dtype=torch.float32)
                p = torch.softmax(torch.einsum("kgd,nkd->kgn", q[s].view(hk, heads // hk, dim), k) * dim ** -0.5, -1)
                out.append(torch.einsum("kgn,nkd->kgd", p, v).reshape(heads * dim))
            r = r + torch.stack(out) @ b.w_out.float()
            r = r + srv.alpha * norm(ys[i], b.moe_post_norm)
        rel = float((got - r).norm() / r.norm())
        assert rel < 2e-2, f"step {step}: relative L2 {rel:.3e}"
    for ws in (srv.attn_ws, srv.moe_ws, srv.plan_ws):
        assert moe.get_status(ws) == 0
    held = [srv.page_table[b, : -(-n // 16)].tolist() for b, n in enumerate(srv.lens.tolist())]
    assert sorted(sum(held, []) + srv.free[: int(srv.n_free)].tolist()) == list(range(srv.n_pages))


def test_the_example_serves(capsys, monkeypatch):
    import sys
    import __graft_entry__
    __graft_entry__.build()
    from examples import decode_step as ex
    monkeypatch.setattr(sys, "argv", ["decode_step.py", "--batch", "4", "--context", "64", "--layers", "2", "--steps", "5",
                                      "--cache", "int4", "--serve"])
    ex.main()
    assert "serving" in capsys.readouterr().out
