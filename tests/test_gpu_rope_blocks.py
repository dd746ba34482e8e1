"""rope_kv_write with so many tokens that a block takes several heads: blocks that go from keys to values, that have values
alone, and a last one with fewer heads.  The cache bit for bit as rope in fp32 and kv_write fill it, and, like the queries,
a sample of it against the formula in 64 bits."""
import pytest
import torch

from tests import feed_oracle as fo
from tests.decoder_oracle import power
from tests.test_gpu_feed import close, gen, ints

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


def pools(cache):
    return [t for t in (cache.k, cache.v, cache.k_exp, cache.v_exp, cache.k_scale, cache.v_scale) if t is not None]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("src", [BF, F32])
@pytest.mark.parametrize("each", [2, 3, 4])
@pytest.mark.parametrize("hk,dim,rot,interleaved", [(1, 256, 64, True), (3, 128, 128, False), (5, 64, 24, False)])
def test_several_heads_a_block(moe, kind, src, each, hk, dim, rot, interleaved):
    # tokens that make up `each` heads' rows (a row is dim / 8 lanes) for every 1024 lanes of each multiprocessor
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = -(-each * sms * 1024 * 8 // (dim * 2 * hk)) + 5
    g, heads, page = gen(T + dim), 5, 64
    n_pages = T // page + 2
    table, (freq, m) = moe.Rope(rot, interleaved=interleaved), fo.frequencies(rot)
    dtype = {"bf16": 1, "e4m3": 2, "int4": 4}[kind]
    cache, other = (moe.KVCache.empty(n_pages, hk, page, dim, dtype) for _ in range(2))
    for t in pools(cache) + pools(other):
        t.fill_(3)
    ws = moe.attn_workspace(cache, hk, 1)
    x = torch.randn(T, heads + 2 * hk, dim, generator=g).to(src)
    pos = torch.randint(0, 100000, (T,), generator=g).int()
    slot = torch.randperm(n_pages * page, generator=g)[:T].int()
    slot[::7] = -1
    dev = x.cuda()
    q, k, v = dev[:, :heads], dev[:, heads:heads + hk], dev[:, heads + hk:]
    got = moe.rope_kv_write(q, k, v, cache, table, pos.cuda(), slot.cuda(), ws)
    assert moe.get_status(ws) == 0 and torch.equal(dev.cpu(), x)
    turned = moe.rope(k.float(), table, pos.cuda())
    moe.kv_write(turned, v.float().contiguous(), other, slot.cuda(), ints([list(range(n_pages))]), ws, seq=ints([0] * T))
    assert moe.get_status(ws) == 0
    for a, b in zip(pools(cache), pools(other)):
        assert torch.equal(a, b)
    some = torch.cat([torch.arange(0, T, 41), torch.arange(T - 9, T)])
    want, tol = fo.turned(x[some, :heads], pos[some], freq, m, interleaved, out=BF)
    close(got.cpu()[some], want, tol, "queries")
    want, tol = fo.turned(x[some, heads:heads + hk], pos[some], freq, m, interleaved)
    close(turned.cpu()[some], want, tol, "keys in fp32")
    there = some[slot[some] >= 0]
    at, rows = slot[there].long(), [t.cpu() for t in pools(cache)]
    rows = [t[at // page, :, at % page] for t in rows]
    if kind == "bf16":
        want, tol = fo.turned(x[there, heads:heads + hk], pos[there], freq, m, interleaved, out=BF)
        close(rows[0], want, tol, "keys")
        assert torch.equal(rows[1], x[there, heads + hk:].to(BF))
    if kind == "int4":  # off by half a step of the scale at most, and by the turned key's own error
        for n, (raw, exps, scales) in enumerate((rows[::2], rows[1::2])):
            want, tol = fo.turned(x[there, heads:heads + hk], pos[there], freq, m, interleaved)
            if n:
                want, tol = x[there, heads + hk:].double(), torch.zeros_like(want)
            got = fo.values4(fo.unpack4(raw), scales, exps)
            step = fo.SCALES[scales[..., :dim // 16].long()] * power(exps.long() - 127)[..., None]
            assert ((got - want).abs() <= step.repeat_interleave(16, -1) / 2 + tol).all()
