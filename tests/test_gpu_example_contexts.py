"""examples/decode_step.py with more tokens in its contexts than one call of the library takes (2^20): in several sequences
together, and in one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,context", [(2, 600_000), (1, 1_100_000)])
@pytest.mark.parametrize("serve", [False, True])
def test_long_contexts(serve, batch, context):
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as moe
    from examples import decode_step as ex
    dec = ex.build(1, batch, context, heads=1, kv_heads=1, dim=32, d=512, ffn=128, experts=16, page=64, cache_dtype=1,
                   serve=serve)
    cache, start = dec.blocks[0].cache, context - 58
    for t in (cache.k, cache.v):
        t.fill_(float("nan"))
    ex.fill(dec, context, start)
    if serve:
        assert dec.lens.tolist() == [start] * batch
    n = start if serve else context
    for b in range(batch):
        for first in range(0, n, 1 << 19):  # every position has a number of its own
            pos = torch.arange(first, min(n, first + (1 << 19)), dtype=torch.int32, device="cuda")
            k, v = moe.kv_read(cache, pos, dec.page_table, dec.attn_ws, seq=torch.full_like(pos, b))
            assert torch.isfinite(k).all() and torch.isfinite(v).all()
            assert (v[1:] != v[:-1]).flatten(1).any(1).all()
    if not serve:
        dec.pos.fill_(start), dec.lens.fill_(start + 1)
    dec.residual.copy_(torch.randn_like(dec.residual))
    dec.step()
    assert torch.isfinite(dec.residual.float()).all()
    for ws in (dec.attn_ws, dec.moe_ws) + ((dec.plan_ws,) if serve else ()):
        assert moe.get_status(ws) == 0
