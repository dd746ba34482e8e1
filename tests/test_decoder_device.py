"""The decode-step calls refuse tensors of a device that is not the current one, before any launch."""
import pytest
import torch


def calls(moe, cache, residual):
    i32 = dict(dtype=torch.int32, device=residual.device)
    bf = dict(dtype=torch.bfloat16, device=residual.device)
    at, table = torch.zeros(1, **i32), torch.zeros(1, 1, **i32)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=residual.device)
    kv, w = torch.zeros(1, 1, 64, **bf), torch.ones(64, device=residual.device)
    return [lambda: moe.kv_write(kv, kv, cache, at, table, ws), lambda: moe.kv_read(cache, at, table, ws),
            lambda: moe.attn_decode(kv, cache, at, table, ws), lambda: moe.attn_workspace(cache, 1, 1),
            lambda: moe.block_norm(residual, w)]


def test_tensors_of_another_device_are_refused_without_a_gpu(monkeypatch):
    from routed_expert_layer_fp32_gb300 import _build
    _build.build()
    import routed_expert_layer_fp32_gb300 as moe
    from routed_expert_layer_fp32_gb300 import decoder

    def launched(*args):
        raise AssertionError("the library was called")

    class NoLibrary:
        def __getattr__(self, name):
            return launched

    monkeypatch.setattr(moe.binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(moe.binding, "lib", NoLibrary)
    monkeypatch.setattr(decoder, "_devices", 2)
    monkeypatch.setattr(decoder, "_current_device", lambda: 0)
    monkeypatch.setattr(decoder, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)  # host tensors that say they lie on GPU 1
    pool = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    for call in calls(moe, moe.KVCache(pool, pool), torch.zeros(1, 64)):
        with pytest.raises(ValueError, match="GPU 1"):
            call()


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as moe
    from routed_expert_layer_fp32_gb300 import decoder
    todo = calls(moe, moe.KVCache.empty(1, 1, 16, 64), torch.zeros(1, 64, device="cuda"))
    for call in todo:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(decoder, "_devices", 2)
    monkeypatch.setattr(decoder, "_current_device", lambda: 1)  # as if the program had gone on to another
    for call in todo:
        with pytest.raises(ValueError, match="GPU 0"):
            call()
