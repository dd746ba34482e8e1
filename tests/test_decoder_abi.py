"""Refusals of the decode-step operators without a GPU: the C entry points reject bad arguments before
any launch, and the binding rejects tensors that do not fit."""
import ctypes
import math

import pytest
import torch

P, WS, BIG = 1 << 20, 1 << 21, 1 << 40  # fake 16-byte aligned addresses: never dereferenced


@pytest.fixture(scope="module")
def moe():
    from routed_expert_layer_fp32_gb300 import _build
    _build.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


def desc(moe, **kw):
    f = dict(n_pages=64, page_size=16, n_kv_heads=4, head_dim=128, dtype=moe.binding.MOE_E4M3, k=P, v=P, k_exp=P, v_exp=P)
    f.update(kw)
    return ctypes.byref(moe.decoder.MoeKvCacheC(*f.values()))


BAD_CACHES = [(dict(n_pages=0), -1), (dict(page_size=0), -1), (dict(page_size=24), -2), (dict(page_size=8192), -2),
              (dict(head_dim=0), -1), (dict(head_dim=72), -2), (dict(head_dim=272), -2), (dict(n_kv_heads=0), -1),
              (dict(dtype=0), -1), (dict(dtype=3), -1), (dict(k=0), -1), (dict(v=P + 8), -1), (dict(k_exp=0), -1),
              (dict(v_exp=P + 4), -1), (dict(n_pages=1 << 25), -2), (dict(n_kv_heads=1025), -2)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(moe, bad, status):
    lib, c = moe.binding.lib(), desc(moe, **bad)
    assert lib.moe_kv_write(c, P, P, 1, 512, 512, 4, None, P, P, 4, 8, WS, BIG, None) == status
    assert lib.moe_kv_read(c, 4, None, P, P, 4, 8, P, P, 1, WS, BIG, None) == status
    assert lib.moe_attn_decode(c, P, 2048, 16, 4, P, P, 8, 0.1, 0, P, None, WS, BIG, None) == status
    assert lib.moe_attn_workspace_bytes(c, 16, 4) == 0


def test_no_cache(moe):
    lib = moe.binding.lib()
    assert lib.moe_kv_write(None, P, P, 1, 512, 512, 4, None, P, P, 4, 8, WS, BIG, None) == -1
    assert lib.moe_attn_workspace_bytes(None, 16, 4) == 0


@pytest.mark.parametrize("at,value,status", [
    (1, None, -1), (2, None, -1), (1, P + 8, -1), (3, 2, -1), (4, 511, -1), (4, 516, -1), (5, 256, -1), (6, -1, -1),
    (6, (1 << 20) + 1, -1), (6, 5, -1), (8, None, -1), (8, P + 2, -1), (9, None, -1), (10, 0, -1), (11, 0, -1),
    (12, None, -1), (12, WS + 4, -1), (13, 64, -3)])
def test_kv_write_refusals(moe, at, value, status):
    args = [desc(moe), P, P, 1, 512, 512, 4, None, P, P, 4, 8, WS, BIG, None]
    args[at] = value
    assert moe.binding.lib().moe_kv_write(*args) == status


@pytest.mark.parametrize("at,value,status", [
    (1, -1, -1), (1, 5, -1), (3, None, -1), (4, None, -1), (5, 0, -1), (6, -3, -1), (7, None, -1), (8, P + 4, -1),
    (9, 2, -1), (10, None, -1), (11, 700, -3)])
def test_kv_read_refusals(moe, at, value, status):
    args = [desc(moe), 4, None, P, P, 4, 8, P, P, 1, WS, BIG, None]
    args[at] = value
    assert moe.binding.lib().moe_kv_read(*args) == status


@pytest.mark.parametrize("at,value,status", [
    (1, None, -1), (1, P + 4, -1), (2, 2047, -1), (2, 2052, -1), (3, 18, -1), (3, 0, -1), (3, 2048, -2), (4, -1, -1),
    (4, 70000, -2), (5, None, -1), (5, P + 1, -1), (6, None, -1), (7, 0, -1), (7, 1 << 27, -2), (7, (1 << 24) + 1, -2), (8, math.nan, -1),
    (8, math.inf, -1), (9, -1, -1), (10, None, -1), (10, P + 2, -1), (11, P + 1, -1), (12, None, -1), (13, 4096, -3)])
def test_attn_decode_refusals(moe, at, value, status):
    args = [desc(moe), P, 2048, 16, 4, P, P, 8, 0.1, 0, P, None, WS, BIG, None]
    args[at] = value
    assert moe.binding.lib().moe_attn_decode(*args) == status


def test_attn_workspace(moe):
    lib = moe.binding.lib()
    need = lib.moe_attn_workspace_bytes(desc(moe), 16, 4)
    assert need > 0
    assert lib.moe_attn_workspace_bytes(desc(moe), 18, 4) == 0
    assert lib.moe_attn_workspace_bytes(desc(moe), 16, -1) == 0
    # as large as the calls it serves need: any larger batch or shape may need more, never less
    assert lib.moe_attn_workspace_bytes(desc(moe), 16, 400) >= need
    assert lib.moe_attn_workspace_init(None, BIG, None) == -1
    assert lib.moe_attn_workspace_init(WS + 8, BIG, None) == -1
    assert lib.moe_attn_workspace_init(WS, 1024, None) == -3


NORM = [P, 1, P, P, 1, 0, 1.0, P, P, 1, P, P, 1, 4, 2048, 1e-6, None]


@pytest.mark.parametrize("change,status", [
    ({13: -1}, -1), ({14: 0}, -1), ({14: 2044}, -2), ({14: 16392}, -2), ({1: 2}, -1), ({4: 3}, -1), ({9: 2}, -1),
    ({12: 7}, -1), ({6: math.nan}, -1), ({6: math.inf}, -1), ({15: -1e-6}, -1), ({15: math.nan}, -1), ({7: None}, -1),
    ({8: None}, -1), ({10: None}, -1), ({0: None}, -1), ({0: None, 2: None, 3: None, 11: None}, -1), ({0: P + 8}, -1),
    ({2: P + 4}, -1), ({3: P + 2}, -1), ({7: P + 8}, -1), ({8: P + 8}, -1), ({10: P + 4}, -1), ({11: P + 8}, -1),
    ({5: 2047}, -1), ({5: 1024}, -1), ({5: 2052}, -1)])
def test_block_norm_refusals(moe, change, status):
    args = list(NORM)
    for i, v in change.items():
        args[i] = v
    assert moe.binding.lib().moe_block_norm(*args) == status


def test_nothing_to_do_is_no_error(moe):
    lib, c = moe.binding.lib(), desc(moe)
    assert lib.moe_kv_write(c, None, None, 1, 0, 0, 0, None, None, None, 0, 0, None, 0, None) == 0
    assert lib.moe_kv_read(c, 0, None, None, None, 0, 0, None, None, 1, None, 0, None) == 0
    assert lib.moe_attn_decode(c, None, 0, 16, 0, None, None, 0, 0.1, 0, None, None, None, 0, None) == 0
    assert lib.moe_block_norm(*[0 if i == 13 else a for i, a in enumerate(NORM)]) == 0


def test_bad_page_has_a_name(moe):
    assert "page" in moe.binding.status_string(-8)
    assert moe.binding.STATUS[-8] == "MOE_ERR_BAD_PAGE"


def test_cache_tensors_are_checked(moe):
    bf = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    codes, exps = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 16, dtype=torch.uint8)
    for bad in ((bf.float(), bf.float()), (bf, bf[:1]), (bf, codes), (bf[0], bf[0]), (codes, codes),
                (codes, codes, exps, exps[:1]), (codes, codes, exps, exps.int()), (bf, bf, exps, exps)):
        with pytest.raises(ValueError):
            moe.KVCache(*bad)
    with pytest.raises(ValueError, match="CUDA"):
        moe.KVCache(bf, bf)
