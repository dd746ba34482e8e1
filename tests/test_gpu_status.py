"""Which of several recorded errors moe_get_status reports, and that it clears them all.  The flags are
written from the host."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FORCED, TIMEOUT, INDEX, PAGE = 1, 2, 4, 8


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_layer_fp32_gb300 as m
    return m


@pytest.mark.parametrize("flags,status", [(0, 0), (FORCED, -4), (TIMEOUT, -5), (INDEX, -7), (PAGE, -8),
                                          (PAGE | TIMEOUT, -5), (FORCED | TIMEOUT, -5), (FORCED | PAGE, -4),
                                          (FORCED | PAGE | TIMEOUT, -5), (INDEX | TIMEOUT | PAGE, -7)])
def test_the_worst_error_is_reported(moe, flags, status):
    ws = moe.attn_workspace(moe.KVCache.empty(1, 1, 16, 64), 1, 1)
    ws.view(torch.int32)[0] = flags
    assert moe.get_status(ws) == status
    assert moe.get_status(ws) == 0
