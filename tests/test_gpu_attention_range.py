"""Attention over E4M3 caches whose values are far from 1: rows of every exponent that kv_write gives, and
rows of zeros (whose exponent is the smallest) beside large ones.  Tolerances are those of
tests/decoder_oracle.py."""
import math

import pytest
import torch

from tests import decoder_oracle as o
from tests.test_gpu_decoder import BF, close, gen, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


def check(moe, v, dim, heads, page=16, lift=None, seed=0):
    """v [n, dim]: the values of one sequence of one kv head; lift [n] is added to the tokens' scores."""
    g = gen(seed)
    n = v.shape[0]
    n_pages = -(-n // page)
    k = torch.randn(n, dim, generator=g)
    q = torch.randn(1, heads, dim, generator=g)
    if lift is not None:
        q[..., 0], k[:, 0] = 16.0, lift / (16.0 * dim ** -0.5)
    pools, exps = [], []
    for x in (k, v):
        x = torch.cat([x.to(BF), torch.zeros(n_pages * page - n, dim, dtype=BF)]).view(n_pages, 1, page, dim)
        c, e = o.quantise(x)
        pools.append(c.float().to(torch.float8_e4m3fn).view(torch.uint8))
        exps.append(e)
    pools += exps
    table, lens = torch.arange(n_pages).int().view(1, -1), torch.tensor([n], dtype=torch.int32)
    q = q.to(BF)
    want, lse, tol, tol_lse = o.attention(q, *pools, lens, table, dim ** -0.5, 0)
    cache = to_device(moe, pools)
    ws = moe.attn_workspace(cache, heads, 1)
    got_lse = torch.empty(1, heads, device="cuda")
    out = moe.attn_decode(q.cuda(), cache, lens.cuda(), table.cuda(), ws, lse=got_lse)
    # what may be rounded to 2^128 (3.3e38 is stored as that) is an infinity in bf16
    beyond = (want.abs() + tol >= (2 - 2 ** -8) * 2.0 ** 127) & (out.double().cpu() == torch.sign(want) * math.inf)
    close(torch.where(beyond, want, out.double().cpu()), want, tol, "out")
    close(got_lse, lse, tol_lse, "lse")


@pytest.mark.parametrize("dim,heads", [(64, 4), (128, 8), (256, 3)])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_values_near_the_largest_number(moe, dim, heads, n):
    v = (torch.rand(n, dim, generator=gen(n)) * 2 - 1) * 3.3e38
    v[:, 1] = 3.3e38
    check(moe, v, dim, heads)
    v[::2] *= 1e-38       # beside rows of ordinary size
    check(moe, v, dim, heads)
    v[::3] = 0.0
    check(moe, v, dim, heads)


@pytest.mark.parametrize("dim,heads", [(64, 4), (128, 8), (256, 3)])
@pytest.mark.parametrize("size", [-110, -90, -60, -30, 0, 10, 24, 32, 48, 60, 80, 110, 124])
def test_rows_of_zeros_take_their_share_beside_rows_of_any_size(moe, dim, heads, size):
    """Tokens without values, in tiles of their own and with the larger weights, count in the sum."""
    n = 700
    v = torch.randn(n, dim, generator=gen(size + 200)) * 2.0 ** size
    lift = torch.zeros(n)
    v[:500], lift[:500] = 0.0, 3.0
    check(moe, v, dim, heads, lift=lift)
    v[::2], lift[::2] = 0.0, 3.0     # and in every tile
    check(moe, v, dim, heads, lift=lift)


@pytest.mark.parametrize("dim,heads", [(64, 4), (128, 8), (256, 3)])
def test_tiles_of_every_size_side_by_side(moe, dim, heads):
    """Stretches of 128 tokens whose values differ by factors up to 2^240 count alike in the sum."""
    sizes = torch.tensor([120.0, -120.0, 0.0, 60.0, -60.0, 100.0, -20.0, 20.0])
    v = torch.randn(1024, dim, generator=gen(9)) * torch.exp2(sizes).repeat_interleave(128)[:, None]
    lift = torch.linspace(2.0, -2.0, 1024)
    check(moe, v, dim, heads, lift=lift)
    check(moe, v.flip(0), dim, heads, lift=lift)
    check(moe, v.flip(0), dim, heads, lift=lift.flip(0))
