"""A cache descriptor of a program built before MOE_INT4 ends with v_exp: calls on bf16 and E4M3 caches read nothing behind
it.  In a process of its own, with the descriptor at the end of a page of memory and a page that cannot be read behind it."""
import subprocess
import sys

import pytest

CHILD = """
import ctypes, mmap
import routed_expert_layer_fp32_gb300 as moe
from routed_expert_layer_fp32_gb300.decoder import MoeKvCacheC
lib, libc, size = moe.binding.lib(), ctypes.CDLL(None, use_errno=True), mmap.PAGESIZE
libc.mmap.restype = ctypes.c_void_p
libc.mmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long]
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
at = libc.mmap(None, 2 * size, mmap.PROT_READ | mmap.PROT_WRITE, mmap.MAP_PRIVATE | mmap.MAP_ANONYMOUS, -1, 0)
assert libc.mprotect(at + size, size, 0) == 0
P, WS = 1 << 20, 1 << 21  # fake addresses: no call below comes to a launch
exps = P if DTYPE == 2 else None
full = MoeKvCacheC(64, 16, 4, 128, DTYPE, P, P, exps, exps, None, None)
old = MoeKvCacheC.k_scale.offset
desc = at + size - old
ctypes.memmove(desc, ctypes.byref(full), old)
n = lib.moe_attn_workspace_bytes(desc, 16, 4)
assert n == lib.moe_attn_workspace_bytes(ctypes.byref(full), 16, 4) > 0
assert lib.moe_attn_decode(desc, P, 2048, 16, 4, P, P, 8, 0.1, 0, P, None, WS, n - 256, None) == -3
assert lib.moe_kv_write(desc, P, P, 1, 512, 512, 0, None, P, P, 4, 8, WS, n, None) == 0
assert lib.moe_kv_read(desc, 0, None, P, P, 4, 8, P, P, 1, WS, n, None) == 0
"""


@pytest.mark.parametrize("dtype", [1, 2])
def test_nothing_behind_an_earlier_descriptor_is_read(dtype):
    from routed_expert_layer_fp32_gb300 import _build
    _build.build()
    run = subprocess.run([sys.executable, "-c", CHILD.replace("DTYPE", str(dtype))], capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr[-500:]
