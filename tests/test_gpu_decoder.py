"""The decode-step operators on the GPU against plain 64-bit implementations (tests/decoder_oracle.py):
codes and exponents bit for bit, floating results within bounds that count their roundings."""
import math

import pytest
import torch

from tests import decoder_oracle as o

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


def host_cache(g, n_pages, heads, page, dim, e4m3, spread=1.0):
    """Host pools with normal rows whose sizes vary; E4M3: their codes and exponents."""
    shape = (n_pages, heads, page, dim)
    x = [torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[:3], generator=g))[..., None]
         for _ in range(2)]
    if not e4m3:
        return [t.to(BF) for t in x] + [None, None]
    q = [o.quantise(t.to(BF)) for t in x]
    codes = [c.float().to(torch.float8_e4m3fn).view(torch.uint8) for c, _ in q]
    return codes + [e for _, e in q]


def to_device(moe, pools):
    return moe.KVCache(*[None if t is None else t.cuda() for t in pools])


def tables(g, n_seqs, width, n_pages):
    assert n_seqs * width <= n_pages
    return torch.randperm(n_pages, generator=g)[: n_seqs * width].view(n_seqs, width).int()


def close(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape
    same = got == want  # infinities among them
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    assert not torch.isnan(err).any(), f"{what}: NaN"
    over = err > tol
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} over the bound, worst {float((err / tol)[over].max()):.3g} x"


# ------------------------------------------------------------------------------ cache -------

@pytest.mark.parametrize("dim", [16, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 48), (8, 64)])
@pytest.mark.parametrize("src", [BF, F32])
@pytest.mark.parametrize("e4m3", [False, True])
def test_write_then_read(moe, dim, heads, page, src, e4m3):
    g = gen(dim * heads + page)
    n_seqs, width, T = 3, 4, 37
    pools = host_cache(g, n_seqs * width + 2, heads, page, dim, e4m3)
    cache = to_device(moe, pools)
    table = tables(g, n_seqs, width, cache.n_pages)
    spots = torch.randperm(n_seqs * width * page, generator=g)[:T]
    seq, pos = (spots // (width * page)).int(), (spots % (width * page)).int()
    wide = torch.randn(T, 2 * heads + 1, dim, generator=g) * torch.exp(2 * torch.randn(T, 2 * heads + 1, 1, generator=g))
    wide[0] = 0.0                                                  # a row of zeros
    wide[1, :, 0], wide[2, :, 0] = 448.0, 449.0                     # at the exponent's border and past it
    wide[1, :, 1:], wide[2, :, 1:] = 1.0625, -1.1875               # codes half way between two
    wide[3] *= 2.0 ** -126                                          # around the smallest exponent
    wide = wide.to(src)
    dev = wide.cuda()
    k, v = dev[:, :heads], dev[:, heads:2 * heads]                  # slices of a projection's rows
    ws = moe.attn_workspace(cache, heads, n_seqs)
    moe.kv_write(k, v, cache, pos.cuda(), table.cuda(), ws, seq=seq.cuda())
    kr, vr = moe.kv_read(cache, pos.cuda(), table.cuda(), ws, seq=seq.cuda())
    kf, vf = moe.kv_read(cache, pos.cuda(), table.cuda(), ws, seq=seq.cuda(), dtype=F32)
    assert moe.get_status(ws) == 0
    want = [None if t is None else t.clone() for t in pools]
    for t in range(T):
        p, r = o.place(page, table, int(seq[t]), int(pos[t]))
        for i, x in enumerate((wide[t, :heads], wide[t, heads:2 * heads])):
            if e4m3:
                c, e = o.quantise(x)
                want[i][p, :, r], want[2 + i][p, :, r] = c.float().to(torch.float8_e4m3fn).view(torch.uint8), e
            else:
                want[i][p, :, r] = x.to(BF)
    for got, w in zip((cache.k, cache.v, cache.k_exp, cache.v_exp), want):
        if w is not None:  # every written row, and every other one as it was
            bits = torch.uint8 if e4m3 else torch.int16
            # +0 and -0 are one value
            eq = got.cpu().view(bits) == w.view(bits)
            zero = (w.view(torch.float8_e4m3fn).float() == 0) if e4m3 and w.dim() == 4 else torch.zeros_like(eq)
            both0 = zero & ((got.cpu().view(torch.float8_e4m3fn).float() == 0) if e4m3 and w.dim() == 4 else zero)
            assert (eq | both0).all()
    for t in range(T):
        p, r = o.place(page, table, int(seq[t]), int(pos[t]))
        for i, (b, f) in enumerate(((kr, kf), (vr, vf))):
            vals = torch.stack([o.cached(want[i], want[2 + i], p, h, r) for h in range(heads)])
            assert torch.equal(f[t].cpu(), vals.float())
            assert torch.equal(b[t].cpu(), vals.to(BF))  # exact but for values below bf16's range


def test_write_and_read_edges(moe):
    """Skipped positions, sequences by number, one token, none; refused places leave the cache alone."""
    g = gen(5)
    heads, page, dim = 2, 16, 64
    pools = host_cache(g, 9, heads, page, dim, True)
    cache = to_device(moe, pools)
    table = tables(g, 4, 2, 8)
    table[3, 1] = 9          # not a page
    table[2, 1] = -5
    ws = moe.attn_workspace(cache, heads, 4)
    k = torch.randn(4, heads, dim, generator=g).to(BF).cuda()

    def run(pos, seq=None, n=4):
        pos = torch.tensor(pos, dtype=torch.int32).cuda()
        seq = None if seq is None else torch.tensor(seq, dtype=torch.int32).cuda()
        before = [t.clone() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
        moe.kv_write(k[:n], k[:n], cache, pos, table.cuda(), ws, seq=seq)
        kr, vr = moe.kv_read(cache, pos, table.cuda(), ws, seq=seq)
        same = [torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_exp, cache.v_exp))]
        return kr, vr, moe.get_status(ws), all(same)

    kr, vr, st, same = run([-1, -7, -1, -1])
    assert st == 0 and same and not kr.any() and not vr.any()
    kr, _, st, same = run([31, 16], [0, 1], 2)
    assert st == 0 and not same
    c, e = o.quantise(k[:2].cpu())
    assert torch.equal(kr.double().cpu(), c * o.power(e.long() - 127)[..., None])
    for pos, seq in (([32], [0]), ([2 ** 31 - 1], [1]), ([0], [4]), ([0], [-1]), ([16], [3]), ([31], [2])):
        kr, vr, st, same = run(pos, seq, 1)
        assert st == -8 and same and not kr.any() and not vr.any()
    kr, _, st, _ = run([3, 5, -1, 0])      # token t of sequence t
    assert st == 0 and kr[:2].any() and not kr[2].any() and kr[3].any()
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    moe.kv_write(k[:0], k[:0], cache, empty, table.cuda(), ws)
    assert moe.kv_read(cache, empty, table.cuda(), ws)[0].shape == (0, heads, dim)


def test_infinities_and_nan_are_kept(moe):
    cache = moe.KVCache.empty(1, 1, 16, 32, moe.binding.MOE_E4M3)
    cache.k.zero_(), cache.v.zero_(), cache.k_exp.zero_(), cache.v_exp.zero_()
    x = torch.ones(2, 1, 32)
    x[0, 0, 3], x[1, 0, 5] = math.inf, math.nan
    ws = moe.attn_workspace(cache, 1, 1)
    at = torch.tensor([0, 1], dtype=torch.int32).cuda()
    seq, table = torch.zeros(2, dtype=torch.int32).cuda(), torch.zeros(1, 1, dtype=torch.int32).cuda()
    moe.kv_write(x.cuda(), x.cuda(), cache, at, table, ws, seq=seq)
    k, _ = moe.kv_read(cache, at, table, ws, seq=seq)
    assert torch.isinf(k[0, 0, 3]) and torch.isfinite(k[0, 0, :3]).all() and torch.isfinite(k[0, 0, 4:]).all()
    assert torch.isnan(k[1, 0, 5]) and (k[1, 0, :5] == 1).all() and (k[1, 0, 6:] == 1).all()


# -------------------------------------------------------------------------- attention -------

def check_attention(moe, seed, lens, heads, kv_heads, dim, page, e4m3, window=0, width=None, scale=None, spread=0.5,
                    poison=True, q_size=1.0):
    g = gen(seed)
    B = len(lens)
    need = max(1, max(-(-n // page) for n in lens))
    width = width or need
    n_pages = B * width + 2
    pools = host_cache(g, n_pages, kv_heads, page, dim, e4m3, spread)
    table = tables(g, B, width, n_pages)
    scale = dim ** -0.5 if scale is None else scale
    q = (q_size * torch.randn(B, heads + 2 * kv_heads, dim, generator=g)).to(BF)[:, :heads]
    lens_t = torch.tensor(lens, dtype=torch.int32)
    want, lse, tol, tol_lse = o.attention(q, *pools, lens_t, table, scale, window)
    if poison:  # what no sequence sees may hold anything
        used = torch.zeros(n_pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            n = min(n, width * page)
            for j in range(max(0, n - window) if window else 0, max(n, 0)):
                p, r = o.place(page, table, b, j)
                if 0 <= p < n_pages:
                    used[p, r] = True
        mask = ~used[:, None, :].expand(n_pages, kv_heads, page)
        for i in range(2):
            if e4m3:
                pools[i][mask], pools[2 + i][mask] = 0x7F, 255
            else:
                pools[i][mask] = math.nan if i else math.inf
    cache = to_device(moe, pools)
    ws = moe.attn_workspace(cache, heads, B)
    got_lse = torch.full((B, heads), 7.0, device="cuda")
    qd = q.cuda() if seed % 2 else torch.cat([q, q], 1).cuda()[:, :heads]     # rows of a wider tensor too
    out = moe.attn_decode(qd, cache, lens_t.cuda(), table.cuda(), ws, scale=scale, window=window, lse=got_lse)
    assert moe.get_status(ws) == 0
    what = f"lens {lens} heads {heads}/{kv_heads} dim {dim} page {page} e4m3 {e4m3} window {window}"
    close(out, want, tol, what)
    close(got_lse, lse, tol_lse, what + " lse")
    again = moe.attn_decode(qd, cache, lens_t.cuda(), table.cuda(), ws, scale=scale, window=window)
    assert torch.equal(out, again), what + ": not repeatable"
    return out


LENS = [[1], [2, 0, 15, 16, 17], [63, 64, 65, 127, 128, 129], [0], [0, 0, 0], [257, 1, 0, 400], [1000]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_lengths(moe, lens, e4m3):
    check_attention(moe, len(lens), lens, 8, 2, 128, 16, e4m3)


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_widths(moe, dim, e4m3):
    check_attention(moe, dim, [97, 1, 200, 64], 6, 2, dim, 32, e4m3)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (2, 1), (7, 1), (8, 1), (9, 1), (15, 3), (16, 1), (17, 1),
                                            (24, 1), (32, 2), (33, 1), (64, 1), (40, 40)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_head_layouts(moe, heads, kv_heads, e4m3):
    check_attention(moe, heads, [70, 0, 131], heads, kv_heads, 64, 16, e4m3)
    if heads <= 17:
        check_attention(moe, heads, [70, 33], heads, kv_heads, 256, 16, e4m3)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 96, 128, 256, 1008])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_pages(moe, page, e4m3):
    check_attention(moe, page, [page, page + 1, 2 * page - 1, 150, 5], 4, 2, 128, page, e4m3)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 128, 200, 513, 5000])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_windows(moe, window, e4m3):
    check_attention(moe, window, [700, 1, 0, 64, 65, 513, 514], 4, 1, 128, 48, e4m3, window=window, width=16)


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_split_long_rows(moe, e4m3):
    """One long row among short ones, so that many CTAs share it and a few take several rows."""
    check_attention(moe, 3, [9001, 5, 0, 130, 64, 1], 4, 2, 64, 64, e4m3)
    check_attention(moe, 4, [40 + 7 * i for i in range(70)], 4, 2, 64, 32, e4m3)


def check_dense(moe, dim, heads, kv_heads, e4m3, lens):
    """Long sequences against a 64-bit form gathered on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(dim + heads)
    page, B = 64, len(lens)
    width = max(lens) // page + 1
    lens = torch.tensor(lens, dtype=torch.int32)
    n_pages = B * width
    shape = (n_pages, kv_heads, page, dim)
    pools = [torch.randn(shape, generator=g, device="cuda").to(BF) for _ in range(2)]
    exps = [None, None]
    if e4m3:
        pools = [(32 * x.float()).to(torch.float8_e4m3fn).view(torch.uint8) for x in pools]
        exps = [torch.randint(120, 125, shape[:3], generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    cache = moe.KVCache(*pools, *exps)
    table = torch.randperm(n_pages, generator=g, device="cuda").view(B, width).int()
    q = torch.randn(B, heads, dim, generator=g, device="cuda").to(BF)
    ws = moe.attn_workspace(cache, heads, B)
    lse = torch.empty(B, heads, device="cuda")
    outs = [moe.attn_decode(q, cache, lens.cuda(), table, ws, lse=lse) for _ in range(5)]
    assert moe.get_status(ws) == 0
    for out in outs[1:]:
        assert torch.equal(out, outs[0])
    scale = dim ** -0.5
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            assert not outs[0][b].any() and (lse[b] == -math.inf).all()
            continue
        at = torch.arange(n, device="cuda")
        pg, row = table[b].long()[at // page], at % page
        k, v = (x.permute(0, 2, 1, 3)[pg, row] for x in pools)
        if e4m3:
            k, v = (x.view(torch.float8_e4m3fn).double() * torch.exp2(e.permute(0, 2, 1)[pg, row].double() - 127)[..., None]
                    for x, e in zip((k, v), exps))
        else:
            k, v = k.double(), v.double()
        qh = q[b].double().view(kv_heads, heads // kv_heads, dim)
        s = torch.einsum("kgd,nkd->kgn", qh, k) * scale
        p = torch.softmax(s, -1)
        want = torch.einsum("kgn,nkd->kgd", p, v)
        size = (torch.einsum("kgd,nkd->kgn", qh.abs(), k.abs()).amax(-1) * scale)[..., None]
        eps = (2 * dim + 6) * o.U32 * size + 4 * o.U32 * (2 + n / 16)
        tol = o.UBF * want.abs() + (1 + o.UBF) * (o.UBF + 2 * eps + 2 * o.U32 * (n + 8)) * torch.einsum("kgn,nkd->kgd", p, v.abs())
        close(outs[0][b].view_as(want), want.cpu(), tol.cpu(), f"sequence {b}")
        want_lse = torch.logsumexp(s, -1)
        close(lse[b].view_as(want_lse), want_lse.cpu(), (eps[..., 0] + 2 * o.U32 * n + 4 * o.U32 * want_lse.abs()).cpu(), f"lse {b}")


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 8, 8), (128, 16, 8), (128, 80, 8), (256, 8, 4)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_many_tiles_a_cta(moe, dim, heads, kv_heads, e4m3):
    """Tens of tiles and several segments for every CTA: the ring goes round many times, and the page
    table is read far past its first entries."""
    check_dense(moe, dim, heads, kv_heads, e4m3, [9000, 12000, 8123, 1, 0, 11111, 6400])


@pytest.mark.parametrize("dim,heads", [(64, 16), (128, 16), (128, 8), (256, 8), (256, 3)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_one_row_over_all_ctas(moe, dim, heads, e4m3):
    """One sequence and kv head cut between all CTAs: more partial results than the last of them has room
    to hold at once."""
    check_dense(moe, dim, heads, 1, e4m3, [40000])


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_many_short_sequences(moe, e4m3):
    """More sequences than threads that count them, most of them short, many empty."""
    g = gen(77)
    lens = torch.randint(0, 40, (1500,), generator=g)
    lens[torch.randperm(1500, generator=g)[:500]] = 0
    lens[700], lens[1499] = 300, 171
    check_attention(moe, 78, lens.tolist(), 2, 1, 64, 16, e4m3, poison=False)


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 12, 4), (128, 16, 4), (128, 32, 2), (192, 24, 4), (256, 20, 4)])
@pytest.mark.parametrize("window", [0, 45])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_short_sequences_side_by_side(moe, dim, heads, kv_heads, window, e4m3):
    """Several segments of one or a few tiles a CTA, a different number of tiles each, some cut between
    two CTAs, and rows in every tile that are not seen and hold no numbers."""
    g = gen(dim + heads + window)
    lens = torch.randint(1, 150, (180,), generator=g)
    lens[::17] = 0
    lens[5], lens[60], lens[179] = 700, 1, 333
    check_attention(moe, 90 + dim, lens.tolist(), heads, kv_heads, dim, 48, e4m3, window=window)


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_nan_stays_in_its_head(moe, e4m3):
    """A query with a NaN or an infinity, and a key row with a NaN, spoil their heads and no other."""
    g = gen(81)
    pools = host_cache(g, 12, 2, 16, 64, e4m3)
    table = tables(g, 2, 6, 12)
    lens = torch.tensor([90, 33], dtype=torch.int32)
    q = torch.randn(2, 8, 64, generator=g).to(BF)
    want, _, tol, _ = o.attention(q, *pools, lens, table, 0.125, 0)
    q[0, 1, 5], q[1, 6, 0] = math.nan, math.inf
    p, r = o.place(16, table, 0, 37)
    if e4m3:
        pools[0][p, 1, r, 3] = 0x7F
    else:
        pools[0][p, 1, r, 3] = math.nan
    cache = to_device(moe, pools)
    ws = moe.attn_workspace(cache, 8, 2)
    out = moe.attn_decode(q.cuda(), cache, lens.cuda(), table.cuda(), ws, scale=0.125)
    spoilt = torch.zeros(2, 8, dtype=torch.bool)
    spoilt[0, 1] = spoilt[1, 6] = True
    spoilt[0, 4:] = True            # kv head 1 of sequence 0
    assert torch.isnan(out.cpu()[spoilt]).all()
    close(out.cpu()[~spoilt], want[~spoilt], tol[~spoilt], "the other heads")
    assert moe.get_status(ws) == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_sharp_and_scaled_rows(moe, e4m3):
    """Scores far apart (single tokens take all), a negative scale, a zero scale, row sizes over many
    powers of two, tiny and huge queries."""
    check_attention(moe, 11, [300, 64], 8, 2, 128, 16, e4m3, q_size=40.0)
    check_attention(moe, 12, [300, 64], 8, 2, 128, 16, e4m3, scale=-0.3)
    check_attention(moe, 13, [300, 64], 8, 2, 128, 16, e4m3, scale=0.0)
    check_attention(moe, 14, [300, 64], 8, 2, 128, 16, e4m3, spread=3.0, scale=1e-3)
    check_attention(moe, 15, [300, 64], 8, 2, 128, 16, e4m3, q_size=1e-30)
    check_attention(moe, 16, [300, 64], 8, 2, 128, 16, e4m3, q_size=1e15, scale=1e-15)


@pytest.mark.parametrize("dim,heads", [(64, 5), (128, 4), (128, 8), (256, 3)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_small_weights_alone_in_their_elements(moe, dim, heads, e4m3):
    """Weights of six sizes down to e^-48, side by side in every tile, each with elements in which no
    other token has a value: every size keeps its own precision."""
    g = gen(5)
    n, page = 200, 16
    level = torch.arange(n) % 6
    k = torch.tensor([0.0, -11.0, -20.0, -30.0, -40.0, -48.0])[level][:, None].expand(n, dim)
    v = torch.randn(n, dim, generator=g) * (torch.arange(dim) % 6 == level[:, None])
    n_pages = -(-n // page)
    pools = [torch.cat([x, torch.zeros(n_pages * page - n, dim)]).view(n_pages, 1, page, dim).to(BF) for x in (k, v)]
    exps = [None, None]
    if e4m3:
        codes, exps = zip(*[o.quantise(x) for x in pools])
        pools = [c.float().to(torch.float8_e4m3fn).view(torch.uint8) for c in codes]
    pools = [*pools, *exps]
    q = torch.ones(1, heads, dim).to(BF)
    table = torch.randperm(n_pages, generator=g)
    pools = [t if t is None else t[torch.argsort(table)] for t in pools]
    table, lens = table.int().view(1, -1), torch.tensor([n], dtype=torch.int32)
    want, lse, tol, tol_lse = o.attention(q, *pools, lens, table, 1 / dim, 0)
    cache = to_device(moe, pools)
    ws = moe.attn_workspace(cache, heads, 1)
    got_lse = torch.empty(1, heads, device="cuda")
    out = moe.attn_decode(q.cuda(), cache, lens.cuda(), table.cuda(), ws, scale=1 / dim, lse=got_lse)
    close(out, want, tol, "out")
    close(got_lse, lse, tol_lse, "lse")


def test_attention_scores_of_minus_infinity_and_rows_of_zeros(moe):
    """Keys that give -infinity are masked tokens; with nothing else the row is empty.  E4M3 rows of zeros
    (the smallest exponent) beside others, and nothing but them."""
    page, dim = 16, 64
    g = gen(8)
    pools = host_cache(g, 4, 1, page, dim, False)
    pools[0][0, 0, 3:9, 0] = -math.inf
    pools[0][1, 0, :, 0] = -math.inf
    q = torch.ones(2, 2, dim).to(BF)
    cache = to_device(moe, pools)
    ws = moe.attn_workspace(cache, 2, 2)
    table = torch.tensor([[0], [1]], dtype=torch.int32)
    lens = torch.tensor([16, 16], dtype=torch.int32)
    lse = torch.empty(2, 2, device="cuda")
    out = moe.attn_decode(q.cuda(), cache, lens.cuda(), table.cuda(), ws, lse=lse)
    keep = [j for j in range(16) if not 3 <= j < 9]
    s = pools[0][0, 0, keep].double().sum(-1) * dim ** -0.5
    p = torch.softmax(s, 0)
    v = pools[1][0, 0, keep].double()
    close(out[0, 0], p @ v, o.UBF * (p @ v).abs() + (o.UBF + 1e-4) * (p @ v.abs()), "masked by -infinity")
    assert not out[1].any() and (lse[1] == -math.inf).all()
    pools = host_cache(g, 2, 1, page, dim, True)
    pools[1][0, 0, ::2], pools[3][0, 0, ::2] = 0, 0
    pools[1][1], pools[3][1] = 0, 0
    want, lse_w, tol, tol_lse = o.attention(q, *pools, lens, table, 0.125, 0)
    cache = to_device(moe, pools)
    out = moe.attn_decode(q.cuda(), cache, lens.cuda(), table.cuda(), ws, scale=0.125, lse=lse)
    close(out, want, tol, "rows of zeros")
    close(lse, lse_w, tol_lse, "rows of zeros, lse")
    assert not out[1].any()


def test_attention_bad_pages_and_lengths(moe):
    """Pages outside the pool count as masked, lengths past the table are cut, negative ones empty."""
    g = gen(21)
    for e4m3 in (False, True):
        pools = host_cache(g, 20, 2, 16, 64, e4m3)
        cache = to_device(moe, pools)
        table = tables(g, 4, 5, 20)
        table[0, 1], table[0, 4], table[1, :] = 20, -1, 99
        lens = torch.tensor([80, 33, 1000, -4], dtype=torch.int32)
        q = torch.randn(4, 4, 64, generator=g).to(BF)
        want, lse, tol, tol_lse = o.attention(q, *pools, lens, table, 0.125, 0)
        ws = moe.attn_workspace(cache, 4, 4)
        got_lse = torch.empty(4, 4, device="cuda")
        out = moe.attn_decode(q.cuda(), cache, lens.cuda(), table.cuda(), ws, lse=got_lse)
        assert moe.get_status(ws) == -8
        assert moe.get_status(ws) == 0
        close(out, want, tol, "bad pages")
        close(got_lse, lse, tol_lse, "bad pages lse")
        good = tables(g, 4, 5, 20)
        lens = torch.tensor([80, 33, 0, 1], dtype=torch.int32)  # the workspace serves the next call
        want, _, tol, _ = o.attention(q, *pools, lens, good, 0.125, 0)
        close(moe.attn_decode(q.cuda(), cache, lens.cuda(), good.cuda(), ws), want, tol, "after bad pages")
        assert moe.get_status(ws) == 0


def test_attention_workspace_serves_smaller_calls(moe):
    """One workspace, calls of other sizes in a row: nothing of one call is left for the next."""
    g = gen(31)
    pools = host_cache(g, 200, 2, 16, 64, False)
    cache = to_device(moe, pools)
    ws = moe.attn_workspace(cache, 16, 8)
    for n, (B, heads) in enumerate([(8, 16), (1, 2), (3, 16), (8, 4), (1, 16)]):
        width = 200 // B
        table = tables(g, B, width, 200)
        lens = torch.randint(0, min(width * 16, 900) + 1, (B,), generator=g).int()
        q = torch.randn(B, heads, 64, generator=g).to(BF)
        want, _, tol, _ = o.attention(q, *pools, lens, table, 0.125, 0)
        close(moe.attn_decode(q.cuda(), cache, lens.cuda(), table.cuda(), ws), want, tol, f"call {n}")


def test_attention_joins_by_lse(moe):
    """Two halves of a context joined by their log-sum-exps give the whole."""
    g = gen(41)
    pools = host_cache(g, 8, 1, 16, 128, False)
    cache = to_device(moe, pools)
    table = tables(g, 1, 8, 8)
    q = torch.randn(1, 4, 128, generator=g).to(BF).cuda()
    ws = moe.attn_workspace(cache, 4, 1)
    parts = []
    for t, n in ((table, 128), (table[:, :4].contiguous(), 64), (table[:, 4:].contiguous(), 64)):
        lse = torch.empty(1, 4, device="cuda")
        out = moe.attn_decode(q, cache, torch.tensor([n], dtype=torch.int32).cuda(), t.cuda(), ws, lse=lse)
        parts.append((out.double(), lse.double()))
    (whole, lse), (a, la), (b, lb) = parts
    assert torch.allclose(torch.logaddexp(la, lb), lse, atol=1e-5)
    joined = a * torch.exp(la - lse)[..., None] + b * torch.exp(lb - lse)[..., None]
    assert (joined - whole).abs().max() <= 4 * o.UBF * max(a.abs().max(), b.abs().max())


def test_far_pages_of_a_large_pool(moe):
    """Rows beyond 2^31 elements and 2^32 bytes from the pool's start: written, read and attended to."""
    heads, page, dim = 8, 64, 128
    n_pages = (5 << 30) // (heads * page * dim * 2) + 1
    cache = moe.KVCache.empty(n_pages, heads, page, dim)
    g = gen(51)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32).cuda()
    T = 150
    k, v = (torch.randn(T, heads, dim, generator=g).to(BF) for _ in range(2))
    pos, seq = torch.arange(T, dtype=torch.int32).cuda(), torch.zeros(T, dtype=torch.int32).cuda()
    ws = moe.attn_workspace(cache, heads, 1)
    moe.kv_write(k.cuda(), v.cuda(), cache, pos, table, ws, seq=seq)
    kr, vr = moe.kv_read(cache, pos, table, ws, seq=seq)
    assert torch.equal(kr.cpu(), k) and torch.equal(vr.cpu(), v)
    q = torch.randn(1, heads, dim, generator=g).to(BF)
    out = moe.attn_decode(q.cuda(), cache, torch.tensor([T], dtype=torch.int32).cuda(), table, ws, scale=0.1)
    pools = [torch.zeros(3, heads, page, dim, dtype=BF) for _ in range(2)]
    for t in range(T):
        pools[0][t // page, :, t % page], pools[1][t // page, :, t % page] = k[t], v[t]
    want, _, tol, _ = o.attention(q, *pools, None, None, torch.tensor([T]), torch.tensor([[0, 1, 2]]), 0.1, 0)
    close(out, want, tol, "far pages")
    assert moe.get_status(ws) == 0


def test_other_streams_and_graphs(moe):
    """On a side stream, and captured as a graph whose lengths and inputs change between replays."""
    g = gen(61)
    heads, kv, page, dim, B = 8, 2, 16, 64, 3
    pools = host_cache(g, 30, kv, page, dim, True)
    cache = to_device(moe, pools)
    table = tables(g, B, 10, 30)
    td, ws = table.cuda(), moe.attn_workspace(cache, heads, B)
    qkv = torch.zeros(B, heads + 2 * kv, dim, dtype=BF, device="cuda")
    lens, pos = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty(B, heads, dim, dtype=BF, device="cuda")

    def step():
        moe.kv_write(qkv[:, heads:heads + kv], qkv[:, heads + kv:], cache, pos, td, ws)
        moe.attn_decode(qkv[:, :heads], cache, lens, td, ws, out=out, scale=0.125)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in ([1, 2, 3], [160, 17, 90], [64, 159, 1]):
        x = torch.randn(B, heads + 2 * kv, dim, generator=g).to(BF)
        qkv.copy_(x)
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        pos.copy_(torch.tensor(n, dtype=torch.int32) - 1)
        for b in range(B):
            p, r = o.place(page, table, b, n[b] - 1)
            for i, lo in enumerate((heads, heads + kv)):
                c, e = o.quantise(x[b, lo:lo + kv])
                pools[i][p, :, r] = c.float().to(torch.float8_e4m3fn).view(torch.uint8)
                pools[2 + i][p, :, r] = e
        # position 0 took the zeros of the warm-up calls until its first real token
        host = [t.cpu() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i in range(4):
            for b in range(B):
                p, r = o.place(page, table, b, n[b] - 1)
                host[i][p, :, r] = pools[i][p, :, r]
        want, _, tol, _ = o.attention(x[:, :heads], *host, torch.tensor(n), table, 0.125, 0)
        close(out, want, tol, f"replay at {n}")
    assert moe.get_status(ws) == 0


# ------------------------------------------------------------------------- block norm -------

@pytest.mark.parametrize("d", [8, 16, 128, 264, 1000, 2048, 4096, 4104, 7168, 16384])
@pytest.mark.parametrize("T", [1, 3, 37])
def test_block_norm(moe, d, T):
    g = gen(d + T)
    kinds = [(a, b, c) for a in (BF, F32) for b in (BF, F32) for c in (BF, F32)]
    for n, (ty, tr, tx) in enumerate(kinds):
        for post in (False, True):
            for gate in (None, "channel", "token"):
                y = (2 * torch.randn(T, d, generator=g)).to(ty)
                r = (3 * torch.randn(T, d, generator=g)).to(tr)
                w_pre, w_post = 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
                gt = None
                if gate == "channel":
                    gt = torch.randn(d, generator=g).to(ty)
                elif gate == "token":
                    gt = torch.randn(T, 2 * d, generator=g).to(tx)[:, d:]
                want_r, want_x, tol_r, tol_x = o.block_norm(y, w_post if post else None, gt, 0.6, r, w_pre, 1e-5, tr, tx)
                r_dev = r.cuda()
                if n % 2:
                    r_out, x = moe.block_norm(r_dev, w_pre.cuda(), y=y.cuda(), w_post=w_post.cuda() if post else None,
                                              gate=None if gt is None else gt.cuda(), alpha=0.6, eps=1e-5, x_dtype=tx)
                    assert r_out is r_dev
                else:
                    wide = None
                    if gt is not None and gate == "token":
                        wide = torch.zeros(T, 2 * d, dtype=gt.dtype, device="cuda")
                        wide[:, d:] = gt.cuda()
                    r_out, x = moe.block_norm(r_dev, w_pre.cuda(), y=y.cuda(), w_post=w_post.cuda() if post else None,
                                              gate=wide[:, d:] if wide is not None else None if gt is None else gt.cuda(),
                                              alpha=0.6, eps=1e-5, x_dtype=tx, residual_out=torch.empty_like(r_dev))
                    assert torch.equal(r_dev.cpu(), r)
                what = f"T {T} d {d} {ty} {tr} {tx} post {post} gate {gate}"
                close(r_out, want_r, tol_r, what + " residual")
                close(x, want_x, tol_x, what + " x")


def test_block_norm_parts(moe):
    """The first block's norm alone, the last block's sum alone, a zero row, many rows."""
    g = gen(71)
    r = torch.randn(5, 2048, generator=g).to(BF)
    w = 1 + 0.1 * torch.randn(2048, generator=g)
    rd = r.cuda()
    r_out, x = moe.block_norm(rd, w.cuda())
    want_r, want_x, _, tol = o.block_norm(None, None, None, 1.0, r, w, 1e-6, BF, BF)
    assert r_out is rd and torch.equal(rd.cpu(), r)
    close(x, want_x, tol, "norm alone")
    copy, x2 = moe.block_norm(rd, w.cuda(), residual_out=torch.zeros_like(rd))
    assert torch.equal(copy, rd) and torch.equal(x, x2)
    y = torch.randn(5, 2048, generator=g)
    r_out, none = moe.block_norm(rd, None, y=y.cuda(), alpha=-2.0)
    want_r, _, tol_r, _ = o.block_norm(y, None, None, -2.0, r, None, 1e-6, BF, BF)
    assert none is None
    close(r_out, want_r, tol_r, "sum alone")
    zero = torch.zeros(2, 64, device="cuda")
    _, x = moe.block_norm(zero, torch.ones(64, device="cuda"), y=torch.zeros(2, 64, device="cuda"),
                          w_post=torch.ones(64, device="cuda"), x_dtype=F32)
    assert not x.any()
    T, d = 70000, 64
    r, y = torch.randn(T, d, generator=g).to(BF), torch.randn(T, d, generator=g).to(BF)
    want_r, want_x, tol_r, tol_x = o.block_norm(y, w[:d], None, 1.0, r, w[:d], 1e-6, BF, BF)
    r_out, x = moe.block_norm(r.cuda(), w[:d].cuda(), y=y.cuda(), w_post=w[:d].cuda())
    close(r_out, want_r, tol_r, "many rows")
    close(x, want_x, tol_x, "many rows x")
    assert moe.block_norm(rd[:0], w.cuda(), y=rd[:0])[1].shape == (0, 2048)


@pytest.mark.parametrize("d", [264, 4104, 6200, 8192, 10000, 16384])
@pytest.mark.parametrize("ty,tr", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_block_norm_rows_in_turn(moe, d, ty, tr):
    """More rows than run at once, in place: a row is read ahead of its turn and written in it."""
    g = gen(d)
    T = 5000 if d == 264 else 331
    y, r = (2 * torch.randn(T, d, generator=g)).to(ty), (3 * torch.randn(T, d, generator=g)).to(tr)
    w_pre, w_post = 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
    want_r, want_x, tol_r, tol_x = o.block_norm(y, w_post, None, 0.6, r, w_pre, 1e-5, tr, BF)
    r_dev = r.cuda()
    r_out, x = moe.block_norm(r_dev, w_pre.cuda(), y=y.cuda(), w_post=w_post.cuda(), alpha=0.6, eps=1e-5, x_dtype=BF)
    assert r_out is r_dev
    close(r_out, want_r, tol_r, f"d {d} residual")
    close(x, want_x, tol_x, f"d {d} x")


def test_binding_refuses_tensors_that_do_not_fit(moe):
    cache = moe.KVCache.empty(4, 2, 16, 64)
    ws = moe.attn_workspace(cache, 4, 2)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.zeros(2, 2, **i32), torch.ones(2, **i32)
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=BF, device="cuda")
    bad_attn = [dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.transpose(1, 2)), dict(q=q.cpu()), dict(lens=lens.long()),
                dict(lens=lens[:1]), dict(page_table=table[:1]), dict(page_table=table.t()), dict(out=q.float()),
                dict(out=q[:1]), dict(lse=torch.zeros(2, 3, device="cuda")), dict(lse=torch.zeros(2, 4, dtype=BF, device="cuda"))]
    for change in bad_attn:
        args = dict(q=q, cache=cache, lens=lens, page_table=table, ws=ws)
        args.update(change)
        with pytest.raises(ValueError):
            moe.attn_decode(**args)
    for change in (dict(k=k.half()), dict(v=k.float()), dict(v=k[:1]), dict(k=k[:, :1]), dict(pos=lens.long()),
                   dict(pos=lens[:1]), dict(seq=lens[:1]), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        args = dict(k=k, v=k, cache=cache, pos=lens, page_table=table, ws=ws)
        args.update(change)
        with pytest.raises(ValueError):
            moe.kv_write(**args)
    with pytest.raises(moe.MoeError):
        moe.attn_decode(q, cache, lens, table, ws[:512])
    with pytest.raises(moe.MoeError):
        moe.attn_workspace(cache, 5, 2)
    with pytest.raises(moe.MoeError):  # rows that start off a 16-byte boundary
        odd = torch.as_strided(torch.zeros(400, dtype=BF, device="cuda"), (2, 2, 64), (130, 64, 1))
        moe.kv_write(odd, odd, cache, lens, table, ws)
    r = torch.zeros(2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for change in (dict(y=r[:1]), dict(w_pre=w.double()), dict(w_post=w[:32]), dict(y=r, gate=w[:32]), dict(out=r[:1]),
                   dict(residual=r.half()), dict(residual_out=r.to(BF)), dict(w_pre=None, y=r, out=r.clone())):
        args = dict(residual=r, w_pre=w)
        args.update(change)
        with pytest.raises(ValueError):
            moe.block_norm(**args)
