"""The operators that make and feed the paged cache at the edges of what they take: query heads of many blocks, 65536
sequences, pages planned and released by a replayed graph and on two streams at once, rows of one token."""
import random

import pytest
import torch

from tests import feed_oracle as fo
from tests.test_gpu_feed import attend, close, gen, ints, pool

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


@pytest.mark.parametrize("H,hk,dim", [(17, 1, 128), (40, 1, 64), (66, 2, 256), (1024, 1, 128), (1024, 2, 32)])
@pytest.mark.parametrize("width", [None, 65])
def test_attention_of_many_heads_a_key(moe, H, hk, dim, width):
    assert attend(moe, gen(H + dim), [3, 0, 300], H, hk, dim, 16 if width is None else 32, width=width) == 0


@pytest.mark.parametrize("width", [1, 65])
def test_attention_of_65536_sequences(moe, width):
    """None or one token each: the result is that token's value, exactly."""
    B, dim, page, g = 65536, 32, 16, gen(3)
    cache = moe.KVCache.empty(B, 1, page, dim, moe.binding.MOE_INT4)
    x = torch.randn(B, 2, dim, generator=g).to(BF).cuda()
    table = torch.zeros(B, width, dtype=torch.int32)
    table[:, 0] = torch.randperm(B, generator=g).int()
    ws = moe.attn_workspace(cache, 2, B)
    zero, seq = torch.zeros(B, dtype=torch.int32).cuda(), torch.arange(B, dtype=torch.int32).cuda()
    moe.kv_write(x[:, :1], x[:, 1:], cache, zero, table.cuda(), ws, seq=seq)
    v = fo.values4(*fo.quantise4(x[:, 1].cpu()))
    lens = torch.randint(0, 2, (B,), generator=g).int()
    q = torch.randn(B, 2, dim, generator=g).to(BF).cuda()
    out = moe.attn_decode(q, cache, lens.cuda(), table.cuda(), ws)
    assert moe.get_status(ws) == 0
    want = torch.where((lens > 0)[:, None, None], v[:, None].expand(B, 2, dim), torch.zeros((), dtype=torch.float64))
    assert torch.equal(out.double().cpu(), want)


def sequences(moe, seed, B, width, page, spare):
    rng = random.Random(seed)
    lens = [rng.randint(0, 60) for _ in range(B)]
    table, free = pool(rng, lens, page, width, spare)
    host = dict(lens=lens, table=table, free=free, n_free=spare)
    dev = dict(lens=ints(lens), table=ints(table), free=ints(free), n_free=ints([spare]), new=ints([0] * B),
               ended=torch.zeros(B, dtype=torch.bool).cuda(), ws=moe.pages_workspace(B), out={
                   "starts": ints([0] * (B + 1)), **{n: ints([0] * MOST) for n in ("seq", "pos", "slot")}})
    return rng, host, dev


MOST = 400


def step(moe, dev, page):
    n = len(dev["free"])
    moe.page_release(dev["lens"], dev["ended"], dev["table"], dev["free"], dev["n_free"], page, dev["ws"])
    moe.page_plan(dev["lens"], dev["new"], dev["table"], dev["free"], dev["n_free"], page, n, MOST, dev["ws"], **dev["out"])


def choose(rng, host, dev):
    B = len(host["lens"])
    ended, new = [rng.random() < 0.2 for _ in range(B)], [rng.choice([0, 1, rng.randint(0, 70)]) for _ in range(B)]
    dev["ended"].copy_(torch.tensor(ended)), dev["new"].copy_(torch.tensor(new, dtype=torch.int32))
    return ended, new


def expect(host, dev, ended, new, page):
    host["lens"], host["n_free"], host["free"] = fo.release(host["lens"], ended, host["table"], host["free"], host["n_free"], page)
    seq, pos, slot, starts, host["lens"], host["n_free"], host["table"], refused = fo.plan(
        host["lens"], new, host["table"], host["free"], host["n_free"], page, MOST)
    for name, want in (("seq", seq), ("pos", pos), ("slot", slot), ("starts", starts)):
        assert dev["out"][name].tolist() == want
    assert dev["lens"].tolist() == host["lens"] and dev["n_free"].tolist() == [host["n_free"]]
    assert dev["table"].tolist() == host["table"] and dev["free"].tolist() == host["free"]
    return refused


@pytest.mark.parametrize("width", [10, 700])  # a release of one launch and of two
def test_pages_in_a_replayed_graph(moe, width):
    page, B = 16, 11
    rng, host, dev = sequences(moe, width, B, width, page, 30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(moe, dev, page)  # nobody ended, no new tokens: nothing changes
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(moe, dev, page)
    refusals = 0
    for _ in range(25):
        ended, new = choose(rng, host, dev)
        graph.replay()
        refused = expect(host, dev, ended, new, page)
        assert moe.get_status(dev["ws"]) == (-9 if refused else 0)
        refusals += refused
    assert 0 < refusals < 25


def test_two_pools_on_two_streams(moe):
    page, streams = 16, [torch.cuda.Stream() for _ in range(2)]
    sets = [sequences(moe, 5 + i, 9 + i, 12, page, 40) for i in range(2)]
    for _ in range(15):
        picks = [choose(rng, host, dev) for rng, host, dev in sets]
        torch.cuda.synchronize()
        for (_, _, dev), s in zip(sets, streams):
            with torch.cuda.stream(s):
                step(moe, dev, page)
        torch.cuda.synchronize()
        for (_, host, dev), (ended, new) in zip(sets, picks):
            expect(host, dev, ended, new, page)


@pytest.mark.parametrize("kind", [BF, F32])
def test_one_row_among_others(moe, kind):
    """A step of one token whose rows are slices of wider ones, turned in place and apart."""
    table, (freq, m), pos = moe.Rope(64), fo.frequencies(64), ints([777])
    x = torch.randn(1, 12, 64, generator=gen(2)).to(kind)
    dev = x.cuda()
    want, tol = fo.turned(x[:, 2:6], pos.cpu(), freq, m, False, out=kind)
    wide = torch.full((1, 9, 64), 5.0, dtype=kind).cuda()
    moe.rope(dev[:, 2:6], table, pos, out=wide[:, 3:7])
    close(wide[:, 3:7], want, tol, "apart")
    assert (wide[:, :3] == 5).all() and (wide[:, 7:] == 5).all()
    moe.rope(dev[:, 2:6], table, pos, out=dev[:, 2:6])
    assert torch.equal(dev[:, 2:6], wide[:, 3:7])
    assert torch.equal(dev[:, :2].cpu(), x[:, :2]) and torch.equal(dev[:, 6:].cpu(), x[:, 6:])
