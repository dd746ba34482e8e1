"""The decode-step operators around the expert layer: a paged key-value cache (written as it is or
quantised, and read back), the attention of one new token over it, and the norms, gate and residual
between two blocks.  Argument marshalling only; include/libmoe.h states the operators.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as _b
from .binding import MOE_BF16, MOE_E4M3, MOE_F32

# A decode step calls these operators a few times a layer with microseconds of GPU work each, so what
# the host spends on a call counts: each tensor is looked at once, and only with the cheap accessors.
_CODES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
# the current stream's handle alone: 0.1 us, a torch.cuda.Stream 3 us (absent from builds without CUDA)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_devices = 0  # of the process; 0: not counted yet


class MoeKvCacheC(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p)]


class KVCache:
    """A paged cache's pools as device tensors, plus the C descriptor that borrows them.

    k, v [n_pages, n_kv_heads, page_size, head_dim]: bf16, or E4M3 codes (uint8 or
    torch.float8_e4m3fn) with their rows' exponents k_exp, v_exp [n_pages, n_kv_heads, page_size]
    uint8.  Pages are handed out by the caller: position p of sequence s is in row p % page_size of
    page page_table[s, p // page_size]."""

    def __init__(self, k, v, k_exp=None, v_exp=None):
        e4m3 = k.dtype in (torch.uint8, torch.float8_e4m3fn)
        if not e4m3 and k.dtype != torch.bfloat16:
            raise ValueError(f"a cache holds bf16 values or E4M3 codes, not {k.dtype}")
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v are [n_pages, n_kv_heads, page_size, head_dim] of one type")
        if e4m3:
            for t in (k_exp, v_exp):
                if t is None or t.dtype != torch.uint8 or t.shape != k.shape[:3]:
                    raise ValueError("an E4M3 cache needs k_exp and v_exp, uint8 [n_pages, n_kv_heads, page_size]")
        elif k_exp is not None or v_exp is not None:
            raise ValueError("a bf16 cache has no exponents")
        if any(t is not None and t.device != k.device for t in (v, k_exp, v_exp)):
            raise ValueError("a cache's pools lie on one device")
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.dtype = MOE_E4M3 if e4m3 else MOE_BF16
        self.c = MoeKvCacheC(self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, self.dtype, _b._ptr(k),
                             _b._ptr(v), _b._ptr(k_exp), _b._ptr(v_exp))
        self.ref = ctypes.byref(self.c)
        self.device = k.get_device()

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, dtype: int = MOE_BF16,
              device="cuda") -> "KVCache":
        """Pools for n_pages pages, their contents undefined (no call reads a row that was not written)."""
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        if dtype == MOE_BF16:
            k, v = (torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2))
            return cls(k, v)
        if dtype != MOE_E4M3:
            raise ValueError("a cache is MOE_BF16 or MOE_E4M3")
        k, v = (torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)))


def _misfit(name: str, t: torch.Tensor, what: str):
    return ValueError(f"{name} must be {what}, on the same GPU as the others; got {t.dtype} {list(t.shape)} with strides "
                      f"{list(t.stride())} on {t.device}")


def _check_device(dev: int):
    """The library launches on the current device, and handle 0, the default stream, is that device's own:
    a call on another device's tensors would run here with that one's addresses.  (Asking for the current
    device takes 0.4 us, so calls ask only where there are several.)"""
    global _devices
    if _devices == 0:
        _devices = torch.cuda.device_count()
    if _devices != 1 and dev != _current_device():
        raise ValueError(f"the tensors are on GPU {dev}, not on the current one: call under torch.cuda.device({dev})")


def attn_workspace(cache: KVCache, n_heads: int, B: int) -> torch.Tensor:
    """Workspace of attn_decode for up to B sequences (kept by the caller, one call at a time)."""
    _check_device(cache.device)
    n = int(_b.lib().moe_attn_workspace_bytes(cache.ref, n_heads, B))
    if n == 0:
        raise _b.MoeError(-2, "moe_attn_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.k.device)
    _b._check(_b.lib().moe_attn_workspace_init(ws.data_ptr(), n, _raw_stream(cache.device)), "moe_attn_workspace_init")
    return ws


def _row_stride(t: torch.Tensor, name: str, heads: int, dim: int) -> int:
    """Elements from one row [heads, dim] of t [T, heads, dim] to the next; the rows are contiguous in themselves."""
    s0, s1, s2 = t.stride()
    if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
        raise _misfit(name, t, f"rows of [{heads}, {dim}] that are contiguous in themselves")
    return s0 if t.shape[0] > 1 else heads * dim


def _tokens(pos, seq, page_table, ws, T: int, dev: int):
    """Addresses of pos and seq (or None), and the page table's and the workspace's address and size."""
    if pos.dtype is not torch.int32 or pos.shape != (T,) or pos.get_device() != dev or not pos.is_contiguous():
        raise _misfit("pos", pos, f"int32 [{T}], contiguous")
    sp = None
    if seq is not None:
        if seq.dtype is not torch.int32 or seq.shape != (T,) or seq.get_device() != dev or not seq.is_contiguous():
            raise _misfit("seq", seq, f"int32 [{T}], contiguous")
        sp = seq.data_ptr()
    return (pos.data_ptr(), sp, *_table(page_table, ws, dev))


def _table(page_table, ws, dev: int):
    if (page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.get_device() != dev
            or not page_table.is_contiguous()):
        raise _misfit("page_table", page_table, "int32 [sequences, pages], contiguous")
    if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise _misfit("ws", ws, "uint8, contiguous")
    n_seqs, width = page_table.shape
    return page_table.data_ptr(), n_seqs, width, ws.data_ptr(), ws.numel()


def kv_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, pos: torch.Tensor, page_table: torch.Tensor,
             ws: torch.Tensor, seq: Optional[torch.Tensor] = None) -> None:
    """Writes tokens' keys and values, k and v [T, n_kv_heads, head_dim] bf16 or fp32 (rows may be
    slices of a fused projection's output), at position pos[t] of sequence seq[t] (None: t)."""
    T, dev, heads, dim = k.shape[0], cache.device, cache.n_kv_heads, cache.head_dim
    if _devices != 1:
        _check_device(dev)
    code, shape = _CODES.get(k.dtype), (T, heads, dim)
    if code is None or k.shape != shape or k.get_device() != dev:
        raise _misfit("k", k, f"bf16 or fp32 {list(shape)}")
    if v.dtype is not k.dtype or v.shape != shape or v.get_device() != dev:
        raise _misfit("v", v, f"{k.dtype} {list(shape)}, as k")
    pp, sp, table, n_seqs, width, wp, wn = _tokens(pos, seq, page_table, ws, T, dev)
    rc = _b.lib().moe_kv_write(cache.ref, k.data_ptr(), v.data_ptr(), code, _row_stride(k, "k", heads, dim),
                               _row_stride(v, "v", heads, dim), T, sp, pp, table, n_seqs, width, wp, wn, _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_kv_write")


def kv_read(cache: KVCache, pos: torch.Tensor, page_table: torch.Tensor, ws: torch.Tensor,
            seq: Optional[torch.Tensor] = None, dtype=torch.bfloat16, k: Optional[torch.Tensor] = None,
            v: Optional[torch.Tensor] = None):
    """The keys and values at position pos[t] of sequence seq[t] (None: t): (k, v), each
    [T, n_kv_heads, head_dim] of `dtype`, or of the given output tensors."""
    T, dev = pos.shape[0], cache.device
    if _devices != 1:
        _check_device(dev)
    shape = (T, cache.n_kv_heads, cache.head_dim)
    if k is None:
        k = torch.empty(shape, dtype=dtype if v is None else v.dtype, device=cache.k.device)
    if v is None:
        v = torch.empty(shape, dtype=k.dtype, device=cache.k.device)
    code = _CODES.get(k.dtype)
    if code is None or k.shape != shape or k.get_device() != dev or not k.is_contiguous():
        raise _misfit("k", k, f"bf16 or fp32 {list(shape)}, contiguous")
    if v.dtype is not k.dtype or v.shape != shape or v.get_device() != dev or not v.is_contiguous():
        raise _misfit("v", v, f"{k.dtype} {list(shape)}, contiguous")
    pp, sp, table, n_seqs, width, wp, wn = _tokens(pos, seq, page_table, ws, T, dev)
    rc = _b.lib().moe_kv_read(cache.ref, T, sp, pp, table, n_seqs, width, k.data_ptr(), v.data_ptr(), code, wp, wn,
                              _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_kv_read")
    return k, v


def attn_decode(q: torch.Tensor, cache: KVCache, lens: torch.Tensor, page_table: torch.Tensor, ws: torch.Tensor,
                scale: Optional[float] = None, window: int = 0, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token a sequence: q [B, n_heads, head_dim] bf16 (rows may be slices of a
    fused projection's output) over the last `window` (0: all) of lens[b] cached tokens.  scale
    defaults to head_dim ** -0.5.  Returns out [B, n_heads, head_dim] bf16; lse [B, n_heads] fp32,
    where given, receives the log-sum-exp of the scores."""
    dev, dim, shape = cache.device, cache.head_dim, q.shape
    if _devices != 1:
        _check_device(dev)
    if q.dtype is not torch.bfloat16 or len(shape) != 3 or shape[2] != dim or q.get_device() != dev:
        raise _misfit("q", q, f"bf16 [sequences, n_heads, {dim}]")
    B, H, _ = shape
    if lens.dtype is not torch.int32 or lens.shape != (B,) or lens.get_device() != dev or not lens.is_contiguous():
        raise _misfit("lens", lens, f"int32 [{B}], contiguous")
    table, n_seqs, width, wp, wn = _table(page_table, ws, dev)
    if n_seqs != B:
        raise _misfit("page_table", page_table, f"int32 [{B}, pages], a row a sequence")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    elif out.dtype is not torch.bfloat16 or out.shape != shape or out.get_device() != dev or not out.is_contiguous():
        raise _misfit("out", out, f"bf16 {list(shape)}, contiguous")
    lp = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (B, H) or lse.get_device() != dev or not lse.is_contiguous():
            raise _misfit("lse", lse, f"fp32 [{B}, {H}], contiguous")
        lp = lse.data_ptr()
    rc = _b.lib().moe_attn_decode(cache.ref, q.data_ptr(), _row_stride(q, "q", H, dim), H, B, lens.data_ptr(), table, width,
                                  dim ** -0.5 if scale is None else scale, window, out.data_ptr(), lp, wp, wn,
                                  _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_attn_decode")
    return out


def block_norm(residual: torch.Tensor, w_pre: Optional[torch.Tensor], y: Optional[torch.Tensor] = None,
               w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
               eps: float = 1e-6, x_dtype=torch.bfloat16, residual_out: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None):
    """residual [T, d] plus alpha * gate * norm(y) * w_post, and the next block's input norm(.) * w_pre.
    y None: the norm of the residual alone; w_post or gate None: without them; gate [d] (for all
    tokens) or [T, d]; w_pre None: the residual sum alone.  Returns (residual_out, x): residual_out
    defaults to `residual`, updated in place."""
    shape, dev, code = residual.shape, residual.get_device(), _CODES.get(residual.dtype)
    if dev < 0 or code is None or len(shape) != 2 or not residual.is_contiguous():
        raise _misfit("residual", residual, "bf16 or fp32 [tokens, d], contiguous and on a GPU")
    if _devices != 1:
        _check_device(dev)
    T, d = shape
    rp = residual.data_ptr()
    yp, y_code, post, pre, gp, gs, g_code, xp, x_code = None, 0, None, None, None, 0, 0, None, 0
    if y is not None:
        y_code = _CODES.get(y.dtype)
        if y_code is None or y.shape != shape or y.get_device() != dev or not y.is_contiguous():
            raise _misfit("y", y, f"bf16 or fp32 {list(shape)}, contiguous")
        yp = y.data_ptr()
    if w_post is not None:
        if (w_post.dtype is not torch.float32 or w_post.shape != (d,) or w_post.get_device() != dev
                or not w_post.is_contiguous()):
            raise _misfit("w_post", w_post, f"fp32 [{d}], contiguous")
        post = w_post.data_ptr()
    if gate is not None:
        g_code, per_token = _CODES.get(gate.dtype), gate.dim() == 2
        if (g_code is None or gate.shape != (shape if per_token else (d,)) or gate.get_device() != dev
                or (gate.stride(-1) != 1 and d > 1)):
            raise _misfit("gate", gate, f"bf16 or fp32 [{d}] or {list(shape)} with contiguous rows")
        gp = gate.data_ptr()
        gs = gate.stride(0) if per_token and T > 1 else 0
    if residual_out is None:
        residual_out = residual
        op = None if y is None else rp  # without y the residual stays as it is
    else:
        if (residual_out.dtype is not residual.dtype or residual_out.shape != shape or residual_out.get_device() != dev
                or not residual_out.is_contiguous()):
            raise _misfit("residual_out", residual_out, f"{residual.dtype} {list(shape)}, contiguous, as the residual")
        op = residual_out.data_ptr()
    if w_pre is not None:
        if w_pre.dtype is not torch.float32 or w_pre.shape != (d,) or w_pre.get_device() != dev or not w_pre.is_contiguous():
            raise _misfit("w_pre", w_pre, f"fp32 [{d}], contiguous")
        pre = w_pre.data_ptr()
        if out is None:
            out = torch.empty(shape, dtype=x_dtype, device=residual.device)
        x_code = _CODES.get(out.dtype)
        if x_code is None or out.shape != shape or out.get_device() != dev or not out.is_contiguous():
            raise _misfit("out", out, f"bf16 or fp32 {list(shape)}, contiguous")
        xp = out.data_ptr()
    elif out is not None:
        raise ValueError("an output norm needs w_pre")
    rc = _b.lib().moe_block_norm(yp, y_code, post, gp, g_code, gs, alpha, rp, op, code, pre, xp, x_code, T, d, eps,
                                 _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_block_norm")
    return residual_out, out
