"""GB300-native routed mixture-of-experts expert layer (libmoe) and the decode-step operators around
it: CUDA kernels behind a C ABI, with a thin ctypes binding (`binding`, `decoder`)."""
from . import binding  # noqa: F401
from .binding import (GraphedForward, GraphedStack, Layer, MoeError, dispatch, e4m3_encode, forward,  # noqa: F401
                      forward_stack, get_status, route, workspace, workspace_bytes)
from .decoder import (KVCache, PagePlan, Rope, attn_decode, attn_workspace, block_norm, kv_read, kv_write,  # noqa: F401
                      page_plan, page_release, pages_workspace, rope, rope_kv_write)
