"""Rows of examples/decode_step.py's server whose sequence has ended and that no other has taken: they hold no pages, decode
nothing and leave the others' places as they are, eager and in a replayed graph."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("window", [0, 20])  # of the last block: places by position, and by slot
def test_ended_rows_stay_empty(graph, window):
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as moe
    from examples import decode_step as ex
    batch, heads, hk, dim, d, page = 5, 8, 2, 64, 512, 16
    srv = ex.build(2, batch, 64, heads=heads, kv_heads=hk, dim=dim, d=d, ffn=128, experts=16, page=page, cache_dtype=1,
                   serve=True)
    srv.blocks[0].window, srv.blocks[1].window = 20, window
    g = torch.Generator(device="cuda").manual_seed(3)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def ended(*rows):
        return torch.tensor([b in rows for b in range(batch)], device="cuda")

    def prompts(new):
        plan = srv.admit(ints(new), sum(new))
        for b in srv.blocks:
            x = torch.randn(sum(new), heads + 2 * hk, dim, generator=g, device="cuda").bfloat16()
            moe.rope_kv_write(x[:, :heads], x[:, heads:heads + hk], x[:, heads + hk:], b.cache, srv.rope, plan.pos, plan.slot,
                              srv.attn_ws)

    prompts([17, 3, 30, 5, 16])
    step = srv.step
    if graph:
        state = [t.clone() for t in (srv.lens, srv.n_free, srv.page_table)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            srv.step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured, stream=side):
            srv.step()
        for t, s in zip((srv.lens, srv.n_free, srv.page_table), state):
            t.copy_(s)
        step = captured.replay
    lens, idle = [17, 3, 30, 5, 16], set()
    for i in range(24):
        if i == 2:
            srv.release(ended(0, 3))
            lens[0] = lens[3] = 0
            idle = {0, 3}
        if i == 9:  # another takes the place of one
            prompts([0, 0, 0, 9, 0])
            lens[3] = 9
            idle = {0}
        if i == 15:  # (a row twice)
            srv.release(ended(0, 4))
            lens[4] = 0
            idle = {0, 4}
        srv.residual.copy_(torch.randn(batch, d, generator=g, device="cuda").bfloat16())
        step()
        now = srv.residual.float()
        assert torch.isfinite(now).all()
        pos = [-1 if b in idle else n for b, n in enumerate(lens)]
        lens = [n if b in idle else n + 1 for b, n in enumerate(lens)]
        assert srv.lens.tolist() == lens and srv.pos.tolist() == pos
        table = srv.page_table.tolist()
        assert srv.slot.tolist() == [-1 if p < 0 else table[b][p // page] * page + p % page for b, p in enumerate(pos)]
        held = [table[b][: -(-n // page)] for b, n in enumerate(lens)]
        assert sorted(sum(held, []) + srv.free[: int(srv.n_free)].tolist()) == list(range(srv.n_pages))
        # the last block's values: each row's own, at its place
        rows = [b for b in range(batch) if b not in idle]
        _, v = moe.kv_read(srv.blocks[1].cache, ints([pos[b] for b in rows]), srv.page_table, srv.attn_ws, seq=ints(rows))
        assert torch.equal(v, srv.qkv.view(batch, heads + 2 * hk, dim)[rows, heads + hk:])
    for ws in (srv.attn_ws, srv.moe_ws, srv.plan_ws):
        assert moe.get_status(ws) == 0


def test_a_prompt_that_found_no_pages_leaves_its_row_empty():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as moe
    from examples import decode_step as ex
    srv = ex.build(1, 2, 64, heads=2, kv_heads=1, dim=64, d=512, ffn=128, experts=16, page=16, cache_dtype=1, serve=True)
    srv.release(torch.ones(2, dtype=torch.bool, device="cuda"))
    srv.n_free.fill_(2)
    srv.admit(torch.tensor([40, 20], dtype=torch.int32, device="cuda"), 60)
    assert moe.get_status(srv.plan_ws) == -9 and srv.lens.tolist() == [0, 0]
    srv.admit(torch.tensor([0, 20], dtype=torch.int32, device="cuda"), 60)
    srv.step()
    assert moe.get_status(srv.plan_ws) == 0 and srv.lens.tolist() == [0, 21] and srv.pos.tolist() == [-1, 20]
