"""The operators that make and feed the paged cache, on the GPU, against plain 64-bit implementations
(tests/feed_oracle.py, tests/decoder_oracle.py): whole numbers, codes, scales and exponents bit for bit, floating
results within bounds that count their roundings."""
import math
import random

import pytest
import torch

from tests import decoder_oracle as o
from tests import feed_oracle as fo
from tests.test_feed_abi import calls

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def close(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    assert not torch.isnan(err).any(), f"{what}: NaN"
    over = err > tol
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} over the bound, worst {float((err / tol)[over].max()):.3g} x"


# -------------------------------------------------------------------------------- rows ------

def rows(g, T, heads, dim):
    """Rows of many sizes, some at the borders of what 4 bits tell apart."""
    x = torch.randn(T, heads, dim, generator=g) * torch.exp(2 * torch.randn(T, heads, 1, generator=g))
    x *= torch.exp(1.5 * torch.randn(T, heads, dim // 16, generator=g)).repeat_interleave(16, -1)
    edge = [lambda r: r * 0, lambda r: r * 2.0 ** -110, lambda r: r * 2.0 ** 118, lambda r: r.sign() * 3.0e38]
    for t in range(min(T, 4)):
        x[t] = edge[t](x[t].clamp(-64, 64))
    if T > 7:
        x[4, :, 0], x[4, :, 1:] = 105.0, 7.5       # at the exponent's border; codes half way between two
        x[5, :, 0], x[5, :, 1:] = 105.0078125, -2.5
        x[6, :, ::16], x[6, :, 1::16] = 7.0, 3.5
        x[7, :, ::16] = 7.03125                    # past a scale's border
    return x


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 48)])
@pytest.mark.parametrize("src", [BF, F32])
def test_4_bit_rows_written_then_read(moe, dim, heads, page, src):
    g = gen(dim + heads)
    n_seqs, width, T = 3, 3, 41
    cache = moe.KVCache.empty(n_seqs * width + 1, heads, page, dim, moe.binding.MOE_INT4)
    for t in (cache.k, cache.v, cache.k_exp, cache.v_exp, cache.k_scale, cache.v_scale):
        t.fill_(0xA5)
    table = torch.randperm(cache.n_pages, generator=g)[: n_seqs * width].view(n_seqs, width).int()
    spots = torch.randperm(n_seqs * width * page, generator=g)[:T]
    seq, pos = (spots // (width * page)).int(), (spots % (width * page)).int()
    x = torch.cat([rows(g, T, heads, dim), rows(g, T, heads, dim), torch.randn(T, 1, dim, generator=g)], 1).to(src)
    dev = x.cuda()
    ws = moe.attn_workspace(cache, heads, n_seqs)
    args = (pos.cuda(), table.cuda(), ws)
    moe.kv_write(dev[:, :heads], dev[:, heads:2 * heads], cache, *args, seq=seq.cuda())
    out = [moe.kv_read(cache, *args, seq=seq.cuda(), dtype=t) for t in (BF, F32)]
    assert moe.get_status(ws) == 0
    touched = torch.zeros(cache.n_pages, page, dtype=torch.bool)
    for i, (pool, exps, scales) in enumerate(((cache.k, cache.k_exp, cache.k_scale), (cache.v, cache.v_exp, cache.v_scale))):
        part = x[:, i * heads:(i + 1) * heads]
        n, b, e = fo.quantise4(part)
        want = fo.values4(n, b, e)
        for t in range(T):
            p, r = o.place(page, table, int(seq[t]), int(pos[t]))
            touched[p, r] = True
            assert torch.equal(pool[p, :, r].cpu(), fo.pack4(n[t]))
            assert torch.equal(scales[p, :, r].cpu(), fo.padded(b[t], dim))
            assert torch.equal(exps[p, :, r].cpu(), e[t])
        assert torch.equal(out[0][i].double().cpu(), want) and torch.equal(out[1][i].double().cpu(), want)
        # a value is off by half its group's scale at most, where the row's size is in range
        unit = (fo.SCALES[b.long()] * o.power(e.long() - 127)[..., None]).repeat_interleave(16, -1)
        inside = part.double().abs() <= 105 * 2.0 ** 119
        assert ((want - part.double()).abs() <= unit / 2)[inside].all()
        rest = ~touched
        for t in (pool, exps, scales):  # every other row as it was
            assert (t.cpu().transpose(1, 2)[rest] == 0xA5).all()


def test_a_row_with_no_number_reads_as_nan(moe):
    cache = moe.KVCache.empty(2, 2, 16, 64, moe.binding.MOE_INT4)
    ws, table = moe.attn_workspace(cache, 2, 1), ints([[1, 0]])
    x = torch.randn(4, 2, 64, generator=gen(1))
    x[0, 0, 3], x[1, 1, 63], x[2, 0, 0] = math.nan, math.inf, -math.inf
    args = (ints([0, 5, 17, 31]), table, ws)
    moe.kv_write(x.cuda(), x.cuda(), cache, *args, seq=ints([0] * 4))
    k, v = moe.kv_read(cache, *args, seq=ints([0] * 4), dtype=F32)
    lost = torch.zeros(4, 2, dtype=torch.bool)
    lost[0, 0] = lost[1, 1] = lost[2, 0] = True
    for t in (k, v):
        assert torch.equal(torch.isnan(t).all(-1).cpu(), lost) and torch.equal(torch.isnan(t).any(-1).cpu(), lost)
    q = torch.randn(1, 2, 64, generator=gen(2)).to(BF).cuda()
    out = moe.attn_decode(q, cache, ints([32]), table, ws, window=14)      # position 31 alone and unwritten rows
    assert moe.get_status(ws) == 0 and out.shape == (1, 2, 64)
    out = moe.attn_decode(q, cache, ints([1]), table, ws)
    assert torch.isnan(out[0, 0]).all() and torch.isfinite(out[0, 1]).all()


def test_skipped_and_refused_places_in_4_bits(moe):
    cache = moe.KVCache.empty(3, 1, 16, 32, moe.binding.MOE_INT4)
    pools = (cache.k, cache.v, cache.k_exp, cache.v_exp, cache.k_scale, cache.v_scale)
    for t in pools:
        t.fill_(7)
    ws, table = moe.attn_workspace(cache, 1, 2), ints([[0, 9], [2, 1]])
    x = torch.randn(1, 1, 32).cuda()
    for pos, seq, status in ((-1, 0, 0), (16, 0, -8), (32, 1, -8), (0, 2, -8)):
        moe.kv_write(x, x, cache, ints([pos]), table, ws, seq=ints([seq]))
        k, v = moe.kv_read(cache, ints([pos]), table, ws, seq=ints([seq]))
        assert moe.get_status(ws) == status and not k.any() and not v.any()
        assert all((t == 7).all() for t in pools)


# ------------------------------------------------------------------------- attention --------

def host_cache(g, n_pages, heads, page, dim, spread=1.0):
    """A 4-bit cache of normal rows whose sizes vary: (the pools, their values in bf16, which holds them exactly)."""
    shape = (n_pages, heads, page)
    pools, values = [], []
    for _ in range(2):
        x = torch.randn(*shape, dim, generator=g) * torch.exp(spread * torch.randn(shape, generator=g))[..., None]
        x *= torch.exp(0.5 * torch.randn(heads, 1, dim, generator=g))
        n, b, e = fo.quantise4(x)
        pools.append((fo.pack4(n), e, fo.padded(b, dim)))
        values.append(fo.values4(n, b, e).to(BF))
    (k, ke, ks), (v, ve, vs) = pools
    return [k, v, ke, ve, ks, vs], values


def below_fp32(lens, v):
    """What the shared bound leaves out.  Weights are fp32 numbers relative to the largest, 1: one below 2^-126 is 0 (exp2
    flushes it), so that each token may be missing with 2^-126 of its value, n max|v| 2^-126 in all before the division by
    a sum of 1 or more; and bf16's steps below 2^-126 are 2^-133, half of which a rounding takes."""
    return max(lens) * float(v.double().abs().max()) * 2.0 ** -126 + 2.0 ** -134


def attend(moe, g, lens, H, hk, dim, page, window=0, scale=None, n_more=2, mutate=None, spread=1.0, width=None):
    B = len(lens)
    width = width or max(1, max(-(-max(n, 1) // page) for n in lens))
    n_pages = B * width + n_more
    pools, (k, v) = host_cache(g, n_pages, hk, page, dim, spread)
    table = torch.randperm(n_pages, generator=g)[: B * width].view(B, width).int()
    lens_t = torch.tensor(lens, dtype=torch.int32)
    rows = torch.randn(B, H + 3, dim, generator=g).to(BF)
    q = rows[:, 1:1 + H]
    if mutate:
        mutate(pools, table, lens_t)
    cache = moe.KVCache(*[t.cuda() for t in pools])
    ws = moe.attn_workspace(cache, H, B)
    lse = torch.full((B, H), 7.0).cuda()
    scale = dim ** -0.5 if scale is None else scale
    args = (rows.cuda()[:, 1:1 + H], cache, lens_t.cuda(), table.cuda(), ws)
    out = moe.attn_decode(*args, scale=scale, window=window, lse=lse)
    again = moe.attn_decode(*args, scale=scale, window=window)
    status = moe.get_status(ws)
    want, want_lse, tol, tol_lse = o.attention(q, k, v, None, None, lens_t, table, scale, window)
    close(out, want, tol + below_fp32(lens, v), "out")
    close(lse, want_lse, tol_lse, "lse")
    assert torch.equal(out, again)  # nothing depends on the order in which CTAs finish
    return status


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("H,hk", [(1, 1), (8, 1), (6, 2), (12, 1), (32, 2), (9, 3)])
def test_attention_shapes(moe, dim, H, hk):
    assert attend(moe, gen(dim * 100 + H), [1, 0, 130, 33, 257], H, hk, dim, 16) == 0


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 240, 256])
@pytest.mark.parametrize("dim", [64, 128, 192])
@pytest.mark.parametrize("window", [0, 1, 31, 200])
def test_attention_pages_and_windows(moe, page, dim, window):
    assert attend(moe, gen(page + window), [1, 300, 16, 129, 0, 128, 517], 4, 2, dim, page, window) == 0


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 5003])
def test_attention_lengths(moe, n):
    assert attend(moe, gen(n), [n], 7, 1, 128, 64) == 0
    assert attend(moe, gen(n), [n], 2, 2, 96, 16, window=n - 1) == 0


# A page table wide enough for segments of more than 1024 tokens takes the kernels with larger tiles.
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192])
@pytest.mark.parametrize("H,hk", [(1, 1), (8, 1), (6, 2), (12, 1), (32, 2)])
def test_attention_shapes_with_large_tiles(moe, dim, H, hk):
    assert attend(moe, gen(dim * 10 + H), [1, 0, 130, 33, 257, 300], H, hk, dim, 64, width=17) == 0


@pytest.mark.parametrize("page", [16, 48, 64, 240, 256])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 1025])
def test_attention_pages_and_windows_with_large_tiles(moe, page, dim, window):
    assert attend(moe, gen(page + dim), [1, 300, 1100, 255, 0, 256, 1300], 10, 1, dim, page, window,
                  width=-(-1301 // page)) == 0


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 255, 256, 257, 511, 512, 513])
def test_attention_lengths_with_large_tiles(moe, n):
    assert attend(moe, gen(n), [n, 7], 7, 1, 128, 64, width=17) == 0
    assert attend(moe, gen(n), [n, 7], 2, 2, 64, 16, width=65) == 0


def test_attention_of_many_short_sequences_with_large_tiles(moe):
    rng = random.Random(14)
    assert attend(moe, gen(15), [rng.randint(0, 90) for _ in range(150)], 8, 2, 64, 256, width=5) == 0


def test_attention_of_many_sequences(moe):
    rng = random.Random(4)
    assert attend(moe, gen(11), [rng.randint(0, 90) for _ in range(331)], 8, 2, 64, 16) == 0
    assert attend(moe, gen(12), [0] * 40 + [1] * 200, 2, 1, 32, 32) == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_ignores_what_it_does_not_see(moe, dim):
    """Bytes of any kind in rows outside the window and behind the last token, exponents and scales that no row has."""
    lens, page, window = [5, 70, 33, 128, 200], 16, 40

    def rubbish(pools, table, lens_t):
        seen = torch.zeros(pools[0].shape[0], page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(max(0, n - window), n):
                seen[int(table[b, j // page]), j % page] = True
        g = gen(99)
        for i, t in enumerate(pools):
            dirt = torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8)
            dirt[::2] = 255
            keep = seen[:, None, :] if t.dim() == 3 else seen[:, None, :, None]
            t.copy_(torch.where(keep, t, dirt))

    assert attend(moe, gen(dim), lens, 4, 2, dim, page, window, mutate=rubbish) == 0
    window = 1030  # with large tiles: everything but what lies behind the last token is seen
    assert attend(moe, gen(dim), lens, 4, 2, dim, page, window, mutate=rubbish, width=65) == 0


@pytest.mark.parametrize("dim,page,hk", [(128, 4096, 1), (64, 1024, 3), (128, 16, 70), (256, 4096, 2)])
def test_attention_of_large_pages_and_many_heads(moe, dim, page, hk):
    assert attend(moe, gen(dim + page), [300, 1, 77], 2 * hk, hk, dim, page, width=1 if page > 300 else None) == 0


def test_two_streams_with_a_workspace_each(moe):
    """Calls on two streams at once, over one cache."""
    g = gen(55)
    pools, (k, v) = host_cache(g, 64, 2, 64, 128)
    cache = moe.KVCache(*[t.cuda() for t in pools])
    table = torch.randperm(64, generator=g).view(2, 32).int()
    lens = [ints([2000, 1500]), ints([700, 2048])]
    q = torch.randn(2, 2, 16, 128, generator=g).to(BF)
    dev, t = q.cuda(), table.cuda()
    ws = [moe.attn_workspace(cache, 16, 2) for _ in range(2)]
    alone = [moe.attn_decode(dev[i], cache, lens[i], t, ws[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(moe.attn_decode(dev[i], cache, lens[i], t, ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert moe.get_status(ws[i]) == 0 and all(torch.equal(o_, alone[i]) for o_ in outs[i])


def test_attention_with_bad_pages(moe):
    def bad(pools, table, lens_t):
        table[0, 1], table[1, 0], table[1, 2] = -1, 1 << 20, 9999
        table[2] = -7

    assert attend(moe, gen(3), [60, 60, 40], 4, 2, 128, 16, mutate=bad) == -8
    assert attend(moe, gen(3), [60, 60, 40], 4, 2, 128, 16, mutate=bad, width=65) == -8

    def long(pools, table, lens_t):
        lens_t[0] = 1000

    assert attend(moe, gen(4), [60, 1, 40], 4, 2, 128, 16, mutate=long) == -8


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_attention_scales_and_sizes(moe, scale):
    assert attend(moe, gen(8), [300, 77], 4, 1, 128, 16, scale=scale, spread=3.0) == 0


def test_attention_gives_each_size_of_weight_its_precision(moe):
    """A token that outweighs the others by e^60 with values of 0, and others far apart, with values of their own:
    elements that only small weights reach."""
    dim, n, page = 64, 100, 16
    k = torch.zeros(n, 1, dim)
    k[:, :, 0] = -2.0 * torch.arange(n)[:, None]
    v = torch.zeros(n, 1, dim)
    for d in range(dim):
        v[d, 0, d] = 1.0
    v[0] = 0.0
    cache = moe.KVCache.empty(7, 1, page, dim, moe.binding.MOE_INT4)
    ws, table = moe.attn_workspace(cache, 1, 1), torch.arange(7, dtype=torch.int32).view(1, 7)
    pos, seq = torch.arange(n, dtype=torch.int32).cuda(), ints([0] * n)
    moe.kv_write(k.cuda(), v.cuda(), cache, pos, table.cuda(), ws, seq=seq)
    values = [t.cpu() for t in moe.kv_read(cache, pos, table.cuda(), ws, seq=seq)]
    q = torch.zeros(1, 1, dim, dtype=BF)
    q[..., 0] = 1.0
    out = moe.attn_decode(q.cuda(), cache, ints([n]), table.cuda(), ws, scale=0.5)
    host = [torch.zeros(7, 1, page, dim, dtype=BF) for _ in range(2)]
    for h, x in zip(host, values):
        h.view(7 * page, dim)[:n] = x[:, 0]
    want, _, tol, _ = o.attention(q, *host, None, None, [n], table, 0.5, 0)
    close(out, want, tol, "out")
    assert (want[0, 0, 1:60] > 0).all()


def test_attention_over_4_bits_is_that_over_the_same_values_in_bf16(moe):
    """The two differ by the order of the products' sums, which the shared bound counts twice."""
    g = gen(21)
    pools, (k, v) = host_cache(g, 40, 2, 64, 128)
    table = torch.randperm(40, generator=g).view(2, 20).int()
    lens = ints([1200, 900])
    q = torch.randn(2, 8, 128, generator=g).to(BF).cuda()
    outs = []
    for cache in (moe.KVCache(*[t.cuda() for t in pools]), moe.KVCache(k.cuda(), v.cuda())):
        ws = moe.attn_workspace(cache, 8, 2)
        outs.append(moe.attn_decode(q, cache, lens, table.cuda(), ws))
    _, _, tol, _ = o.attention(q.cpu(), k, v, None, None, lens.cpu(), table, 128 ** -0.5, 0)
    close(outs[0], outs[1].double().cpu(), 2 * tol, "out")


def test_a_long_cache_in_4_bits(moe):
    """Rows and scales past 2^31 bytes of a pool."""
    dim, heads, page = 256, 8, 256
    n_pages = (1 << 31) // (heads * page * dim // 2) + 40
    cache = moe.KVCache.empty(n_pages, heads, page, dim, moe.binding.MOE_INT4)
    g = gen(5)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 20]], dtype=torch.int32)
    ws = moe.attn_workspace(cache, heads, 1)
    n = 600
    x = torch.randn(n, 2 * heads, dim, generator=g).to(BF).cuda()
    pos, seq = torch.arange(n, dtype=torch.int32).cuda(), ints([0] * n)
    moe.kv_write(x[:, :heads], x[:, heads:], cache, pos, table.cuda(), ws, seq=seq)
    k, v = moe.kv_read(cache, pos, table.cuda(), ws, seq=seq)
    for got, part in ((k, x[:, :heads]), (v, x[:, heads:])):
        assert torch.equal(got.double().cpu(), fo.values4(*fo.quantise4(part.cpu())))
    q = torch.randn(1, heads, dim, generator=g).to(BF)
    out = moe.attn_decode(q.cuda(), cache, ints([n]), table.cuda(), ws)
    assert moe.get_status(ws) == 0
    host = []
    for t in (k, v):
        flat = torch.zeros(3 * page, heads, dim, dtype=BF)
        flat[:n] = t.cpu()
        host.append(flat.view(3, page, heads, dim).transpose(1, 2).contiguous())
    want, _, tol, _ = o.attention(q, *host, None, None, [n], torch.tensor([[0, 1, 2]]), dim ** -0.5, 0)
    close(out, want, tol, "out")


# --------------------------------------------------------------------------------- pages ----

def planned(moe, lens, new, table, free, n_free, page, max_tokens, in_place=False):
    B, n_pages = len(lens), len(free)
    t, f = ints(table).view(B, -1), ints(free)
    ln, nf, ws = ints(lens), ints([n_free]), moe.pages_workspace(B)
    out = {} if in_place else dict(lens_out=torch.empty_like(ln), n_free_out=torch.empty_like(nf))
    got = moe.page_plan(ln, None if new is None else ints(new), t, f, nf, page, n_pages, max_tokens, ws, **out)
    status = moe.get_status(ws)
    if not in_place:
        assert ln.tolist() == list(lens) and nf.tolist() == [n_free]
    assert f.tolist() == list(free)
    seq, pos, slot, starts, after, left, want_table, refused = fo.plan(lens, [1] * B if new is None else new, table, free,
                                                                       n_free, page, max_tokens)
    assert got.starts.tolist() == starts
    assert got.lens.tolist() == after and got.n_free.tolist() == [left]
    assert got.seq.tolist() == seq and got.pos.tolist() == pos and got.slot.tolist() == slot
    assert t.tolist() == want_table
    assert status == (-9 if refused else 0)


def pool(rng, lens, page, width, spare):
    held = [-(-max(n, 0) // page) for n in lens]
    order = list(range(sum(held) + spare))
    rng.shuffle(order)
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-1] * (width - h))
        at += h
    return table, order[at:] + [0] * sum(held)


@pytest.mark.parametrize("B,page,top,more", [(1, 16, 100, 1), (1, 1, 5, 40), (7, 48, 500, 300), (64, 64, 4096, 1),
                                             (200, 16, 900, 700), (1025, 32, 60, 3), (3000, 16, 90, 40), (2, 4096, 9000, 9000)])
@pytest.mark.parametrize("spare", ["enough", "few"])
def test_plan(moe, B, page, top, more, spare):
    rng = random.Random(B + page)
    lens = [rng.choice([0, page, rng.randint(0, top)]) for _ in range(B)]
    new = [rng.choice([0, 1, rng.randint(0, more)]) for _ in range(B)]
    width = -(-(top + more) // page) + 2
    need = sum(-(-(a + b) // page) + (-a // page) for a, b in zip(lens, new))
    table, free = pool(rng, lens, page, width, max(1, need if spare == "enough" else need // 2))
    n_free = max(1, need if spare == "enough" else need // 2)
    for max_tokens in (sum(new), sum(new) + 13):
        planned(moe, lens, new, table, free, n_free, page, max_tokens, in_place=max_tokens == sum(new))
    planned(moe, lens, new, table, free, n_free, page, sum(new) // 2)  # a list without room for all


def test_plan_and_release_of_very_many(moe):
    """65536 sequences and a list of 2^20 places, against the formulas in whole tensors (the oracle goes one by one)."""
    B, page, most = 65536, 16, 1 << 20
    g = gen(77)
    lens, new = torch.randint(0, 200, (B,), generator=g), torch.randint(0, 33, (B,), generator=g)
    held, wanted = (lens + page - 1) // page, (lens + new + page - 1) // page
    ends = new.cumsum(0)
    fits = ends <= most
    got = torch.where(fits, wanted - held, torch.zeros_like(held))
    n_pages = int(held.sum() + got.sum())
    order = torch.randperm(n_pages, generator=g)
    width = int(wanted.max())
    table, first = torch.full((B, width), -1), held.cumsum(0) - held
    column = torch.arange(width)
    table = torch.where(column < held[:, None], order[(first[:, None] + column).clamp(max=n_pages - 1)], table)
    free = torch.zeros(n_pages, dtype=torch.int64)
    n_free = int(got.sum())
    free[:n_free] = order[int(held.sum()):]
    dev = [t.int().cuda() for t in (lens, new, table, free)]
    nf, ws = ints([n_free]), moe.pages_workspace(B)
    plan = moe.page_plan(*dev, nf, page, n_pages, most, ws)
    assert moe.get_status(ws) == (0 if fits.all() else -9)
    take = got.cumsum(0) - got
    nth = column - held[:, None]
    mine = (nth >= 0) & (nth < got[:, None])
    table[mine] = free[(n_free - 1 - take[:, None] - nth)[mine]]
    assert torch.equal(dev[2].cpu(), table.int()) and int(plan.n_free) == 0
    after = lens + torch.where(fits, new, torch.zeros_like(new))
    assert torch.equal(plan.lens.cpu(), after.int())
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).clamp(max=most)
    assert torch.equal(plan.starts.cpu(), starts.int())
    seq = torch.repeat_interleave(torch.arange(B), new)[:most]
    pos = lens[seq] + torch.arange(len(seq)) - (ends - new)[seq]
    ok = fits[seq]
    slot = table[seq, (pos // page).clamp(max=width - 1)] * page + pos % page
    pad = most - len(seq)
    for mine, want in ((plan.seq, seq), (plan.pos, torch.where(ok, pos, -1)), (plan.slot, torch.where(ok, slot, -1))):
        assert torch.equal(mine.cpu(), torch.cat([want, torch.full((pad,), -1)]).int())
    ended = torch.randint(0, 2, (B,), generator=g).bool()
    moe.page_release(dev[0], ended.cuda(), dev[2], dev[3], nf, page, ws)
    assert moe.get_status(ws) == 0
    back = torch.where(ended, (after + page - 1) // page, torch.zeros_like(after))
    assert torch.equal(dev[0].cpu(), torch.where(ended, torch.zeros_like(after), after).int())
    assert nf.tolist() == [int(back.sum())]
    assert torch.equal(dev[3].cpu()[: int(back.sum())], table[column < back[:, None]].int())


def test_plan_edges(moe):
    planned(moe, [0], [0], [[-1]], [3, 1, 0, 2], 4, 16, 5)
    planned(moe, [16, 0, 5], None, [[0, -1], [-1, -1], [1, -1]], [2, 3, 0, 0], 2, 16, 8)
    planned(moe, [16, 0, 5], None, [[0, -1], [-1, -1], [1, -1]], [2, 3, 0, 0], 1, 16, 3)     # one page for two
    planned(moe, [16, 15, 3], [1, 1, 1], [[0], [1], [2]], [3, 4, 0, 0, 0], 2, 16, 3)          # a row without room
    planned(moe, [-4, 2], [-7, 3], [[-1], [0]], [1, 0], 1, 16, 4)                            # negative: none
    planned(moe, [16, 16], [1, 2 ** 31 - 1], [[0, -1], [1, -1]], [2, 3, 0, 0], 2, 16, 6)      # more than can be
    planned(moe, [3], [0], [[0]], [0], 0, 16, 0)
    planned(moe, [3], [2], [[0]], [0], 0, 16, 0)


def test_plan_of_nobody(moe):
    ws = moe.pages_workspace(0)
    got = moe.page_plan(ints([]), None, torch.zeros(0, 4, dtype=torch.int32).cuda(), ints([1, 0]), ints([2]), 16, 2, 3, ws)
    assert got.starts.tolist() == [0] and got.slot.tolist() == [-1] * 3 and got.n_free.tolist() == [2]


def test_plan_with_bad_pages(moe):
    """A page outside the pool in the table, or on the stack, gives no place; a count of free pages outside the stack is
    taken for the nearest."""
    ws = moe.pages_workspace(2)
    got = moe.page_plan(ints([3, 16]), ints([1, 1]), ints([[9, 0], [1, 0]]), ints([0, 7]), ints([2]), 16, 2, 2, ws)
    assert moe.get_status(ws) == -8 and got.slot.tolist() == [-1, -1] and got.pos.tolist() == [3, 16]
    for n, left, status in ((5, 1, -8), (-3, 0, -8)):
        got = moe.page_plan(ints([16, 1]), ints([1, 0]), ints([[0, 0], [1, 0]]), ints([0, 1]), ints([n]), 16, 2, 2, ws)
        assert moe.get_status(ws) == status and got.n_free.tolist() == [left]


@pytest.mark.parametrize("B,page,top", [(1, 16, 40), (9, 48, 500), (300, 16, 5000), (1500, 64, 300)])
@pytest.mark.parametrize("flags", [torch.bool, torch.uint8])
def test_release(moe, B, page, top, flags):
    rng = random.Random(B)
    lens = [rng.choice([0, -3, page, rng.randint(0, top)]) for _ in range(B)]
    table, free = pool(rng, lens, page, -(-top // page) + 1, 5)
    ended = [rng.random() < 0.4 for _ in range(B)]
    ended[0] = True
    t, ws = ints(table), moe.pages_workspace(B)
    for in_place in (False, True):
        f, ln, nf = ints(free), ints(lens), ints([5])
        out = {} if in_place else dict(lens_out=torch.empty_like(ln), n_free_out=torch.empty_like(nf))
        after, left = moe.page_release(ln, torch.tensor(ended).to(flags).cuda(), t, f, nf, page, ws, **out)
        assert moe.get_status(ws) == 0
        want_lens, want_left, want_free = fo.release(lens, ended, table, free, 5, page)
        assert after.tolist() == want_lens and left.tolist() == [want_left] and f.tolist() == want_free
        assert t.tolist() == table


def test_release_past_the_stack_and_the_table(moe):
    ws = moe.pages_workspace(2)
    table, ended = ints([[0, 1], [2, 3]]), torch.ones(2, dtype=torch.bool).cuda()
    free = ints([9, 9, 9])
    after, left = moe.page_release(ints([32, 32]), ended, table, free, ints([1]), 16, ws)
    assert moe.get_status(ws) == -8 and left.tolist() == [3] and free.tolist() == [9, 0, 1] and after.tolist() == [0, 0]
    free = ints([9, 9, 9])
    _, left = moe.page_release(ints([1000, 0]), ended, table, free, ints([0]), 16, ws)
    assert moe.get_status(ws) == -8 and left.tolist() == [2] and free.tolist() == [0, 1, 9]


def test_pages_go_round(moe):
    """A pool shared by sequences that grow, end and begin again: at each step every page has one owner or is free."""
    rng, page, n_pages, B = random.Random(6), 16, 61, 9
    lens, n_free, free = ints([0] * B), ints([n_pages]), ints(list(range(n_pages)))
    table, ws = torch.full((B, 12), -1, dtype=torch.int32).cuda(), moe.pages_workspace(B)
    refused = 0
    for _ in range(60):
        ended = torch.tensor([rng.random() < 0.1 for _ in range(B)]).cuda()
        moe.page_release(lens, ended, table, free, n_free, page, ws)
        new = ints([rng.choice([0, 1, rng.randint(1, 60)]) for _ in range(B)])
        moe.page_plan(lens, new, table, free, n_free, page, n_pages, 300, ws)
        refused += moe.get_status(ws) == -9
        held = [table[b, : -(-n // page)].tolist() for b, n in enumerate(lens.tolist())]
        assert sorted(sum(held, []) + free[: int(n_free)].tolist()) == list(range(n_pages))
    assert refused > 0


# -------------------------------------------------------------------------------- rotary ----

@pytest.mark.parametrize("dim,rot", [(8, 8), (64, 64), (72, 24), (80, 40), (96, 96), (128, 128), (128, 32), (136, 136),
                                     (192, 64), (248, 200), (256, 256), (256, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", [BF, F32])
def test_rope(moe, dim, rot, interleaved, kind):
    g = gen(dim + rot)
    T, heads = 37, 3
    freq, magnitude = fo.frequencies(rot, "by_index")
    table = moe.Rope(rot, interleaved=interleaved, scaling="by_index", factor=8.0)
    x = torch.randn(T, heads + 2, dim, generator=g).to(kind)
    x[:, :, rot:] *= 100.0
    pos = torch.randint(0, 1 << 20, (T,), generator=g).int()
    pos[:6] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 12345])
    dev = x.cuda()
    part = dev[:, 1:1 + heads]
    got = moe.rope(part, table, pos.cuda())
    want, tol = fo.turned(x[:, 1:1 + heads], pos, freq, magnitude, interleaved, out=kind)
    close(got, want, tol, "turned")
    assert torch.equal(got[..., rot:], part[..., rot:])
    wide = torch.full((T, heads + 1, dim), 7.0, dtype=kind).cuda()
    moe.rope(part, table, pos.cuda(), out=wide[:, :heads])  # rows that lie further apart
    assert torch.equal(wide[:, :heads], got) and (wide[:, heads] == 7).all()
    back = moe.rope(part, table, pos.cuda(), inverse=True)
    want, tol = fo.turned(x[:, 1:1 + heads], pos, freq, magnitude, interleaved, inverse=True, out=kind)
    close(back, want, tol, "turned back")
    assert moe.rope(part, table, pos.cuda(), out=part) is part  # in place, of a slice
    assert torch.equal(part, got)
    assert torch.equal(dev[:, 0].cpu(), x[:, 0]) and torch.equal(dev[:, -1].cpu(), x[:, -1])


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "by_index", "by_turns"])
@pytest.mark.parametrize("T,heads", [(1, 1), (1, 128), (700, 40), (5000, 12)])
def test_rope_scalings_and_sizes(moe, scaling, T, heads):
    g = gen(T + heads)
    freq, magnitude = fo.frequencies(64, scaling, 500000.0, 4.0, 8192.0, 1.0, 4.0)
    table = moe.Rope(64, base=500000.0, scaling=scaling, factor=4.0, original=8192.0, low=1.0, high=4.0)
    x, pos = torch.randn(T, heads, 64, generator=g), torch.randint(0, 40000, (T,), generator=g).int()
    want, tol = fo.turned(x, pos, freq, magnitude, False)
    close(moe.rope(x.cuda(), table, pos.cuda()), want, tol, "turned")


@pytest.mark.parametrize("kind", [BF, F32])
def test_rope_of_very_many_heads_and_tokens(moe, kind):
    table = moe.Rope(8)
    freq, m = fo.frequencies(8)
    for T, heads in ((3, 1024), (70001, 1)):
        g = gen(T)
        x, pos = torch.randn(T, heads, 16, generator=g).to(kind), torch.randint(0, 9000, (T,), generator=g).int()
        want, tol = fo.turned(x, pos, freq, m, False, out=kind)
        close(moe.rope(x.cuda(), table, pos.cuda()), want, tol, "turned")


def test_rope_of_given_frequencies_and_no_tokens(moe):
    freq = [1.0, 0.25, -0.5, 3.0]
    table = moe.Rope(8, frequencies=freq, magnitude=0.5, interleaved=True)
    x, pos = torch.randn(9, 1, 8, generator=gen(1)), torch.arange(9, dtype=torch.int32) * 100003
    want, tol = fo.turned(x, pos, freq, 0.5, True)
    close(moe.rope(x.cuda(), table, pos.cuda()), want, tol, "turned")
    assert moe.rope(x[:0].cuda(), table, pos[:0].cuda()).shape == (0, 1, 8)


def test_rope_keeps_no_numbers_in_their_pair(moe):
    """What is not turned, and other pairs, know nothing of an infinity or a NaN."""
    for interleaved in (False, True):
        table = moe.Rope(16, interleaved=interleaved)
        x = torch.ones(1, 1, 32)
        x[..., 3], x[..., 20] = math.nan, math.inf
        y = moe.rope(x.cuda(), table, ints([5])).cpu()[0, 0]
        pair = [2, 3] if interleaved else [3, 11]
        assert torch.isnan(y[pair]).all() and math.isinf(y[20])
        rest = [i for i in range(32) if i not in pair + [20]]
        assert torch.isfinite(y[rest]).all() and (y[[i for i in rest if i >= 16]] == 1).all()


def test_rope_is_its_own_gradient_turned_back(moe):
    """The gradient of sum(w * rope(x)) with respect to x is w turned back: against differences."""
    table = moe.Rope(32, scaling="by_index", factor=4.0)
    g = gen(9)
    x, w, pos = torch.randn(3, 2, 40, generator=g), torch.randn(3, 2, 40, generator=g), ints([3, 77, 4000])
    grad = moe.rope(w.cuda(), table, pos, inverse=True).cpu()
    base = (moe.rope(x.cuda(), table, pos).cpu().double() * w).sum(-1)
    for d in (0, 9, 16, 31, 35):
        y = x.clone()
        y[..., d] += 0.5
        moved = (moe.rope(y.cuda(), table, pos).cpu().double() * w).sum(-1)
        # linear: the difference is the gradient but for some fp32 roundings of elements of size 4
        assert ((moved - base) / 0.5 - grad[..., d]).abs().max() < 40 * 8 * 2.0 ** -23


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("src", [BF, F32])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (96, 24, False), (128, 128, False), (160, 80, True), (256, 256, True)])
@pytest.mark.parametrize("T,heads,hk", [(1, 4, 2), (45, 6, 3)])
def test_rope_kv_write(moe, kind, src, dim, rot, interleaved, T, heads, hk):
    g = gen(dim + T)
    page = 32
    table = moe.Rope(rot, interleaved=interleaved)
    freq, m = fo.frequencies(rot)
    cache = moe.KVCache.empty(4, hk, page, dim, {"bf16": 1, "e4m3": 2, "int4": 4}[kind])
    pools = [t for t in (cache.k, cache.v, cache.k_exp, cache.v_exp, cache.k_scale, cache.v_scale) if t is not None]
    for t in pools:
        t.fill_(3)
    ws = moe.attn_workspace(cache, heads, 1)
    x = torch.randn(T, heads + 2 * hk, dim, generator=g).to(src)
    pos = torch.randint(0, 100000, (T,), generator=g).int()
    slot = torch.randperm(4 * page, generator=g)[:T].int()
    skipped = T // 3 if T > 1 else -1
    if T > 1:
        slot[skipped] = -1
    dev = x.cuda()
    q, k, v = dev[:, :heads], dev[:, heads:heads + hk], dev[:, heads + hk:]
    got = moe.rope_kv_write(q, k, v, cache, table, pos.cuda(), slot.cuda(), ws)
    assert moe.get_status(ws) == 0 and torch.equal(dev.cpu(), x)
    want, tol = fo.turned(x[:, :heads], pos, freq, m, interleaved, out=BF)
    close(got, want, tol, "queries")
    # the keys as rope gives them in fp32 and kv_write stores them, bit for bit: the values are the same
    turned = moe.rope(k.float(), table, pos.cuda())
    other = moe.KVCache.empty(4, hk, page, dim, cache.dtype)
    for t in (other.k, other.v, other.k_exp, other.v_exp, other.k_scale, other.v_scale):
        if t is not None:
            t.fill_(3)
    where = torch.where(slot < 0, torch.full_like(slot, -1), slot)
    moe.kv_write(turned, v.float().contiguous(), other, where.cuda(), ints([[0, 1, 2, 3]]), ws, seq=ints([0] * T))
    for a, b in zip(pools, [t for t in (other.k, other.v, other.k_exp, other.v_exp, other.k_scale, other.v_scale) if t is not None]):
        assert torch.equal(a, b)
    apart = torch.full((T, heads + 1, dim), 7.0, dtype=BF).cuda()
    moe.rope_kv_write(q, k, v, cache, table, pos.cuda(), slot.cuda(), ws, q_out=apart[:, 1:])
    assert torch.equal(apart[:, 1:], got) and (apart[:, 0] == 7).all()
    if src is BF:  # queries in place
        assert moe.rope_kv_write(q, k, v, cache, table, pos.cuda(), slot.cuda(), ws, q_out=q) is q
        assert torch.equal(q, got)


def test_rope_kv_write_refuses_places_past_the_cache(moe):
    cache, table = moe.KVCache.empty(2, 1, 16, 64), moe.Rope(64)
    cache.k.zero_(), cache.v.zero_()
    ws = moe.attn_workspace(cache, 1, 1)
    x = torch.ones(3, 1, 64, dtype=BF).cuda()
    for slots, status in (([32, -1, 2 ** 31 - 1], -8), ([-5, -1, -2 ** 31], 0)):
        moe.rope_kv_write(x, x, x, cache, table, ints([0, 1, 2]), ints(slots), ws)
        assert moe.get_status(ws) == status and not cache.k.any() and not cache.v.any()


# ------------------------------------------------------------------------------ together ----

@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("graph", [False, True])
def test_plan_place_and_attend(moe, kind, graph):
    """Prompts of mixed lengths, then single tokens, as a server runs them: pages planned, keys turned into the cache,
    attention over it; captured once and replayed.  Against each sequence's own history in 64 bits, the bound being that of
    attention plus the stored keys' possible difference: a key near the border of two codes may fall either way, so that
    the cache's own contents are read back for the comparison, and compared themselves where they are bf16."""
    g = gen(33)
    B, heads, hk, dim, page, n_pages, width = 5, 4, 2, 64, 16, 64, 12
    cache = moe.KVCache.empty(n_pages, hk, page, dim, {"bf16": 1, "int4": 4}[kind])
    table = moe.Rope(32, interleaved=True, base=500.0)
    freq, m = fo.frequencies(32, base=500.0)
    lens, n_free, free = ints([0] * B), ints([n_pages]), ints(torch.randperm(n_pages, generator=g).tolist())
    pages = torch.full((B, width), -1, dtype=torch.int32).cuda()
    ws, pws = moe.attn_workspace(cache, heads, B), moe.pages_workspace(B)
    prompt = [40, 1, 0, 17, 33]
    T = sum(prompt) + 3
    x = torch.randn(T, heads + 2 * hk, dim, generator=g).to(BF).cuda()
    plan = moe.page_plan(lens, ints(prompt), pages, free, n_free, page, n_pages, T, pws)
    moe.rope_kv_write(x[:, :heads], x[:, heads:heads + hk], x[:, heads + hk:], cache, table, plan.pos, plan.slot, ws)
    history = [[x[sum(prompt[:b]) + i].cpu() for i in range(n)] for b, n in enumerate(prompt)]

    step_x = torch.zeros(B, heads + 2 * hk, dim, dtype=BF).cuda()
    q_out, out = torch.empty(B, heads, dim, dtype=BF).cuda(), torch.empty(B, heads, dim, dtype=BF).cuda()
    outs = {n: torch.empty(k, dtype=torch.int32).cuda() for n, k in (("starts", B + 1), ("seq", B), ("pos", B), ("slot", B))}

    def step():
        p = moe.page_plan(lens, None, pages, free, n_free, page, n_pages, B, pws, **outs)
        moe.rope_kv_write(step_x[:, :heads], step_x[:, heads:heads + hk], step_x[:, heads + hk:], cache, table, p.pos, p.slot,
                          ws, q_out=q_out)
        moe.attn_decode(q_out, cache, lens, pages, ws, out=out)

    if graph:
        state = [t.clone() for t in (lens, n_free, pages)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured, stream=side):
            step()
        for t, s in zip((lens, n_free, pages), state):
            t.copy_(s)
    for n in range(20):
        new = torch.randn(B, heads + 2 * hk, dim, generator=g).to(BF)
        step_x.copy_(new)
        captured.replay() if graph else step()
        for b in range(B):
            history[b].append(new[b])
        assert lens.tolist() == [len(h) for h in history]
        want_q, tol_q = fo.turned(new[:, :heads], lens.cpu() - 1, freq, m, True, out=BF)
        close(q_out, want_q, tol_q, "queries")
        if n % 6 != 1:
            continue
        for b in range(B):
            L = len(history[b])
            pos, seq = torch.arange(L, dtype=torch.int32).cuda(), ints([b] * L)
            k, v = (t.cpu() for t in moe.kv_read(cache, pos, pages, ws, seq=seq))
            rows = torch.stack(history[b])
            turned, tol = fo.turned(rows[:, heads:heads + hk], pos.cpu(), freq, m, True, out=BF)
            if kind == "bf16":
                close(k, turned, tol, "keys")
                assert torch.equal(v, rows[:, heads + hk:])
            else:  # off by half a step of the group, and by the turned key's own error
                nn, bb, ee = fo.quantise4(turned)
                unit = (fo.SCALES[bb.long()] * o.power(ee.long() - 127)[..., None]).repeat_interleave(16, -1)
                assert ((k.double() - turned).abs() <= 0.57 * unit).all()   # the scale may be the next: 1 + 1/8 times it
                assert torch.equal(v.double(), fo.values4(*fo.quantise4(rows[:, heads + hk:])))
            flat = [torch.zeros(-(-L // page) * page, hk, dim, dtype=BF) for _ in range(2)]
            flat[0][:L], flat[1][:L] = k, v
            host = [f.view(-1, page, hk, dim).transpose(1, 2).contiguous() for f in flat]
            want, _, tol, _ = o.attention(q_out[b:b + 1].cpu(), *host, None, None, [L],
                                          torch.arange(len(host[0])).view(1, -1), dim ** -0.5, 0)
            close(out[b:b + 1], want, tol, "out")
    assert moe.get_status(ws) == 0 and moe.get_status(pws) == 0
    held = [pages[b, : -(-n // page)].tolist() for b, n in enumerate(lens.tolist())]
    assert sorted(sum(held, []) + free[: int(n_free)].tolist()) == list(range(n_pages))


def test_tensors_of_another_device_are_refused(moe, monkeypatch):
    from routed_expert_layer_fp32_gb300 import decoder
    todo = calls(moe, moe.KVCache.empty(1, 1, 16, 64, moe.binding.MOE_INT4), "cuda")
    for call in todo:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(decoder, "_devices", 2)
    monkeypatch.setattr(decoder, "_current_device", lambda: 1)  # as if the program had gone on to another
    for call in todo:
        with pytest.raises(ValueError, match="GPU 0"):
            call()
