"""Refusals of the operators that make and feed the paged cache, without a GPU: the C entry points reject bad
arguments before any launch, the binding tensors that do not fit, and tensors of a device that is not the current one."""
import ctypes
import math

import pytest
import torch

from tests import feed_oracle as fo

P, WS, BIG = 1 << 20, 1 << 21, 1 << 40  # fake 16-byte aligned addresses: never dereferenced


@pytest.fixture(scope="module")
def moe():
    from routed_expert_layer_fp32_gb300 import _build
    _build.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


def cache(moe, **kw):
    f = dict(n_pages=64, page_size=16, n_kv_heads=4, head_dim=128, dtype=moe.binding.MOE_INT4, k=P, v=P, k_exp=P, v_exp=P,
             k_scale=P, v_scale=P)
    f.update(kw)
    return ctypes.byref(moe.decoder.MoeKvCacheC(*f.values()))


def table(moe, **kw):
    f = dict(dim=128, interleaved=0, magnitude=1.0, turns=P)
    f.update(kw)
    return ctypes.byref(moe.decoder.MoeRopeC(*f.values()))


@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=144), -2), (dict(head_dim=80), -2), (dict(head_dim=288), -2), (dict(k_scale=0), -1), (dict(v_scale=0), -1),
    (dict(k_scale=P + 8), -1), (dict(v_scale=P + 4), -1), (dict(k_exp=0), -1), (dict(v_exp=0), -1), (dict(k=0), -1),
    (dict(page_size=24), -2), (dict(dtype=5), -1), (dict(dtype=3), -1)])
def test_every_call_refuses_a_bad_4_bit_cache(moe, bad, status):
    lib, c = moe.binding.lib(), cache(moe, **bad)
    assert lib.moe_kv_write(c, P, P, 1, 512, 512, 4, None, P, P, 4, 8, WS, BIG, None) == status
    assert lib.moe_kv_read(c, 4, None, P, P, 4, 8, P, P, 1, WS, BIG, None) == status
    assert lib.moe_attn_decode(c, P, 2048, 16, 4, P, P, 8, 0.1, 0, P, None, WS, BIG, None) == status
    assert lib.moe_attn_workspace_bytes(c, 16, 4) == 0
    assert lib.moe_rope_kv_write(table(moe, dim=64), c, P, 2048, 16, P, 2048, P, P, 1, 512, 512, 4, P, P, WS, BIG,
                                 None) == status


def test_a_good_4_bit_cache_has_a_workspace(moe):
    lib = moe.binding.lib()
    for dim in range(32, 257, 32):
        assert lib.moe_attn_workspace_bytes(cache(moe, head_dim=dim), 16, 4) > 0


PLAN = [P, P, 4, P, 8, P, P, 64, 16, 32, P, P, P, P, P, P, WS, BIG, None]


@pytest.mark.parametrize("at,value,status", [
    (0, None, -1), (0, P + 2, -1), (1, P + 1, -1), (2, -1, -1), (2, 65537, -2), (3, None, -1), (4, 0, -1), (4, 1 << 25, -2),
    (5, None, -1), (6, None, -1), (7, 0, -1), (7, 1 << 28, -2), (8, 0, -1), (8, 4097, -2), (9, -1, -1), (9, (1 << 20) + 1, -1),
    (10, None, -1), (11, None, -1), (12, None, -1), (13, None, -1), (14, None, -1), (15, None, -1), (13, P + 4, -1),
    (14, P + 8, -1), (15, P + 4, -1), (16, None, -1), (16, WS + 8, -1), (17, 64, -3), (17, 768, -3)])
def test_page_plan_refusals(moe, at, value, status):
    args = list(PLAN)
    args[at] = value
    assert moe.binding.lib().moe_page_plan(*args) == status


RELEASE = [P, P, 4, P, 8, P, P, 64, 16, P, P, WS, BIG, None]


@pytest.mark.parametrize("at,value,status", [
    (0, None, -1), (1, None, -1), (2, -1, -1), (2, 65537, -2), (3, None, -1), (4, 0, -1), (5, None, -1), (6, None, -1),
    (7, 0, -1), (8, 0, -1), (8, 5000, -2), (9, None, -1), (10, None, -1), (10, P + 2, -1), (11, None, -1), (12, 700, -3)])
def test_page_release_refusals(moe, at, value, status):
    args = list(RELEASE)
    args[at] = value
    assert moe.binding.lib().moe_page_release(*args) == status


def test_pages_workspace(moe):
    lib = moe.binding.lib()
    assert lib.moe_pages_workspace_bytes(-1) == 0 and lib.moe_pages_workspace_bytes(65537) == 0
    assert 768 <= lib.moe_pages_workspace_bytes(0) <= lib.moe_pages_workspace_bytes(65536)


@pytest.mark.parametrize("bad,status", [(dict(dim=0), -1), (dict(dim=136), -1), (dict(dim=12), -2), (dict(turns=0), -1),
                                        (dict(turns=P + 4), -1), (dict(magnitude=math.nan), -1),
                                        (dict(magnitude=math.inf), -1)])
def test_a_bad_table_is_refused(moe, bad, status):
    lib, t = moe.binding.lib(), table(moe, **bad)
    assert lib.moe_rope_apply(t, P, 2048, P, 2048, 1, 4, 16, 128, P, 0, None) == status
    assert lib.moe_rope_kv_write(t, cache(moe), P, 2048, 16, P, 2048, P, P, 1, 512, 512, 4, P, P, WS, BIG, None) == status


@pytest.mark.parametrize("change,status", [
    ({0: None}, -1), ({1: None}, -1), ({1: P + 8}, -1), ({2: 2047}, -1), ({2: 2052}, -1), ({2: 1024}, -1), ({3: None}, -1),
    ({3: P + 4}, -1), ({4: 2040}, -1), ({5: 2}, -1), ({6: -1}, -1), ({6: (1 << 20) + 1}, -1), ({7: 0}, -1), ({7: 1025}, -2),
    ({8: 124}, -1), ({8: 132}, -2), ({8: 264}, -2), ({9: None}, -1), ({9: P + 2}, -1), ({1: P, 3: P, 4: 4096}, -1)])
def test_rope_refusals(moe, change, status):
    args = [table(moe), P, 2048, 2 * P, 2048, 1, 4, 16, 128, P, 0, None]
    for at, value in change.items():
        args[at] = value
    assert moe.binding.lib().moe_rope_apply(*args) == status


@pytest.mark.parametrize("change,status", [
    ({1: None}, -1), ({2: None}, -1), ({2: P + 8}, -1), ({3: 1000}, -1), ({3: 2052}, -1), ({4: 0}, -1), ({4: 1025}, -2),
    ({5: None}, -1), ({5: P + 2}, -1), ({6: 2047}, -1), ({7: None}, -1), ({8: P + 8}, -1), ({9: 4}, -1), ({10: 511}, -1),
    ({11: 256}, -1), ({12: -1}, -1), ({12: (1 << 20) + 1}, -1), ({13: None}, -1), ({14: None}, -1), ({14: P + 2}, -1),
    ({15: None}, -1), ({15: WS + 4}, -1), ({16: 100}, -3), ({9: 0, 5: P}, -1), ({5: P, 6: 4096}, -1)])
def test_rope_kv_write_refusals(moe, change, status):
    args = [table(moe), cache(moe), P, 2048, 16, 2 * P, 2048, P, P, 1, 512, 512, 4, P, P, WS, BIG, None]
    for at, value in change.items():
        args[at] = value
    assert moe.binding.lib().moe_rope_kv_write(*args) == status


def test_nothing_to_do_is_no_error(moe):
    lib = moe.binding.lib()
    assert lib.moe_rope_apply(table(moe), None, 0, None, 0, 1, 0, 16, 128, None, 0, None) == 0
    assert lib.moe_rope_kv_write(table(moe), cache(moe), None, 0, 16, None, 0, None, None, 1, 0, 0, 0, None, None, None, 0,
                                 None) == 0


def test_the_new_status_has_a_name(moe):
    assert "page" in moe.binding.status_string(-9)
    assert moe.binding.STATUS[-9] == "MOE_ERR_NO_PAGES"


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1, 1, 1, 2), (7, 1e4, 0, 1, 1, 1, 2), (258, 1e4, 0, 1, 1, 1, 2), (64, 1.0, 0, 1, 1, 1, 2),
    (64, math.nan, 0, 1, 1, 1, 2), (64, math.inf, 0, 1, 1, 1, 2), (64, 1e4, 5, 1, 1, 1, 2), (64, 1e4, -1, 1, 1, 1, 2),
    (64, 1e4, 1, 0.5, 1, 1, 2), (64, 1e4, 1, math.nan, 1, 1, 2), (64, 1e4, 3, 2, 0, 1, 2), (64, 1e4, 3, 2, 1, 0, 2),
    (64, 1e4, 4, 2, 4096, 2, 2), (64, 1e4, 4, 2, 4096, 2, math.inf), (2, 1e4, 2, 2, 1, 1, 2), (4, 1e300, 2, 1e300, 1, 1, 2)])
def test_frequency_refusals(moe, args):
    turns, m = (ctypes.c_uint64 * 256)(), ctypes.c_float()
    assert moe.binding.lib().moe_rope_frequencies(*args, turns, ctypes.byref(m)) == -1
    assert moe.binding.lib().moe_rope_frequencies(64, 1e4, 0, 1, 1, 1, 2, None, ctypes.byref(m)) == -1


def test_turns_refuse_what_is_no_frequency(moe):
    out = (ctypes.c_uint64 * 1)()
    for f in (math.nan, math.inf, -math.inf, 2.0 ** 31):
        assert moe.binding.lib().moe_rope_turns((ctypes.c_double * 1)(f), 1, out) == -1
    assert moe.binding.lib().moe_rope_turns(None, 1, out) == -1
    assert moe.binding.lib().moe_rope_turns(None, 0, None) == 0


@pytest.mark.parametrize("f", [0.0, 1.0, 1e-4, 0.1, -0.3, 6.283185307179586, 12345.678, -1e-19, 2.0 ** 30 + 0.25])
def test_turns_are_the_fraction_of_a_turn(moe, f):
    """Against 1 / (2 pi) to 60 digits.  A double's own product error aside the table is a whole number: off by 2 units
    for frequencies up to 1, and by 2^-64 of the frequency in turns for larger ones."""
    from fractions import Fraction
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    out = (ctypes.c_uint64 * 1)()
    assert moe.binding.lib().moe_rope_turns((ctypes.c_double * 1)(f), 1, out) == 0
    turns = Fraction(f) / two_pi
    want = (turns - math.floor(turns)) * 2 ** 64
    err = abs(out[0] - want)
    err = min(err, 2 ** 64 - err)
    assert err <= 2 + abs(turns) * 2


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "by_index", "by_turns"])
@pytest.mark.parametrize("rot", [8, 64, 72, 128, 256])
def test_frequencies_are_the_formulas(moe, scaling, rot):
    """exp and log in 64 bits: some 2^-50 of the frequency."""
    turns, m = (ctypes.c_uint64 * (rot // 2))(), ctypes.c_float()
    assert moe.binding.lib().moe_rope_frequencies(rot, 500000.0, moe.Rope.SCALINGS.index(scaling), 16.0, 8192.0, 1.0, 4.0,
                                                  turns, ctypes.byref(m)) == 0
    want, magnitude = fo.frequencies(rot, scaling, 500000.0, 16.0, 8192.0, 1.0, 4.0)
    assert abs(m.value - magnitude) <= 2 ** -23
    for t, f in zip(turns, want):
        assert abs(t * 2.0 ** -64 * 2 * math.pi - f) <= 2.0 ** -48 * f + 2.0 ** -60


def test_tensors_are_checked(moe):
    rows, codes, scales = torch.zeros(2, 1, 16), torch.zeros(2, 1, 16, 48), torch.zeros(2, 1, 16, 8)
    e, c, s = rows.to(torch.uint8), codes.to(torch.uint8), scales.to(torch.uint8)
    for bad in ((c, c, e, e, s, None), (c, c, e, e, s[..., :6], s), (c, c, None, e, s, s), (c, c, e, e, s, s.int()),
                (codes.bfloat16(), codes.bfloat16(), e, e, s, s), (c[:1], c, e, e, s, s)):
        with pytest.raises(ValueError):
            moe.KVCache(*bad)
    with pytest.raises(ValueError, match="CUDA"):
        moe.KVCache(c, c, e, e, s, s)
    with pytest.raises(ValueError, match="32"):
        moe.KVCache.empty(1, 1, 16, 80, moe.binding.MOE_INT4, device="cpu")
    for bad in (dict(dim=12), dict(dim=264), dict(dim=64, scaling="other"), dict(dim=64, frequencies=[1.0]),
                dict(dim=8, frequencies=[1.0] * 4, scaling="linear")):
        with pytest.raises(ValueError):
            moe.Rope(device="cpu", **bad)


def calls(moe, four, dev):
    """One good call of each operator: they run on a GPU, and fail where the tensors are on another than the current one."""
    def ints(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device=dev)

    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=dev)
    ws, table = torch.zeros(1 << 22, dtype=torch.uint8, device=dev), moe.Rope(64, device=dev)
    return [lambda: moe.page_plan(ints(1), None, ints(1, 2), ints(4), ints(1), 16, 4, 8, ws),
            lambda: moe.page_release(ints(1), torch.ones(1, dtype=torch.bool, device=dev), ints(1, 2), ints(4), ints(1), 16, ws),
            lambda: moe.rope(x, table, ints(1)), lambda: moe.rope_kv_write(x, x, x, four, table, ints(1), ints(1), ws),
            lambda: moe.kv_write(x, x, four, ints(1), ints(1, 1), ws), lambda: moe.kv_read(four, ints(1), ints(1, 1), ws),
            lambda: moe.attn_decode(x, four, ints(1), ints(1, 1), ws)]


def test_tensors_of_another_device_are_refused_without_a_gpu(moe, monkeypatch):
    from routed_expert_layer_fp32_gb300 import decoder
    monkeypatch.setattr(moe.binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(decoder, "_devices", 2)
    monkeypatch.setattr(decoder, "_current_device", lambda: 0)
    monkeypatch.setattr(decoder, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)  # host tensors that say they lie on GPU 1
    four = moe.KVCache.empty(1, 1, 16, 64, moe.binding.MOE_INT4, device="cpu")
    todo = calls(moe, four, "cpu")

    def launched(*args):
        raise AssertionError("the library was called")

    class NoLibrary:
        def __getattr__(self, name):
            return launched

    monkeypatch.setattr(moe.binding, "lib", NoLibrary)
    for call in todo:
        with pytest.raises(ValueError, match="GPU 1"):
            call()
