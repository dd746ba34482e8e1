"""The page calls' workspace: the status record of 768 bytes, a word a sequence and one more, in whole 256 bytes."""
import pytest


@pytest.mark.parametrize("B", [0, 1, 62, 63, 64, 127, 1000, 65536])
def test_no_word_more_than_is_used(B):
    from routed_expert_layer_fp32_gb300 import _build
    _build.build()
    import routed_expert_layer_fp32_gb300 as moe
    want = -(-(768 + 4 * (B + 1)) // 256) * 256
    lib = moe.binding.lib()
    assert lib.moe_pages_workspace_bytes(B) == want
    P, WS = 1 << 20, 1 << 21  # fake addresses: refused before a launch
    assert lib.moe_page_plan(P, P, B, P, 8, P, P, 64, 16, 32, P, P, P, P, P, P, WS, want - 1, None) == -3
    assert lib.moe_page_release(P, P, B, P, 8, P, P, 64, 16, P, P, WS, want - 1, None) == -3
