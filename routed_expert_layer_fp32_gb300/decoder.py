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
_raw_stream = torch._C._cuda_getCurrentRawStream  # the handle alone: 0.1 us, a torch.cuda.Stream 3 us


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
    return ValueError(f"{name} is {what}, contiguous and on the cache's GPU; got {t.dtype} {list(t.shape)} on {t.device}")


def _int32(t: torch.Tensor, name: str, shape, dev: int) -> int:
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise _misfit(name, t, f"int32 {list(shape)}")
    return t.data_ptr()


def _table(t: torch.Tensor, dev: int):
    if t.dtype is not torch.int32 or t.dim() != 2 or t.get_device() != dev or not t.is_contiguous():
        raise _misfit("page_table", t, "int32 [sequences, pages]")
    n, width = t.shape
    return t.data_ptr(), n, width


def _workspace(ws: torch.Tensor, dev: int):
    if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise _misfit("ws", ws, "uint8")
    return ws.data_ptr(), ws.numel()


def _rows(t: torch.Tensor, name: str, T: int, heads: int, dim: int, dev: int):
    """(address, row stride) of [T, heads, dim] rows that are contiguous in themselves."""
    if t.shape != (T, heads, dim) or t.get_device() != dev:
        raise ValueError(f"{name} is [{T}, {heads}, {dim}] on the cache's GPU; got {list(t.shape)} on {t.device}")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
        raise ValueError(f"{name}'s rows of [{heads}, {dim}] must be contiguous")
    return t.data_ptr(), (s0 if T > 1 else heads * dim)


def _full(t: torch.Tensor, name: str, shape, dev: int) -> int:
    if t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} is {list(shape)}, contiguous and on the same GPU; got {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _code(t: torch.Tensor, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} is bf16 or fp32, not {t.dtype}")
    return code


def attn_workspace(cache: KVCache, n_heads: int, B: int) -> torch.Tensor:
    """Workspace of attn_decode for up to B sequences (kept by the caller, one call at a time)."""
    n = int(_b.lib().moe_attn_workspace_bytes(cache.ref, n_heads, B))
    if n == 0:
        raise _b.MoeError(-2, "moe_attn_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.k.device)
    _b._check(_b.lib().moe_attn_workspace_init(ws.data_ptr(), n, _raw_stream(cache.device)), "moe_attn_workspace_init")
    return ws


def kv_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, pos: torch.Tensor, page_table: torch.Tensor,
             ws: torch.Tensor, seq: Optional[torch.Tensor] = None) -> None:
    """Writes tokens' keys and values, k and v [T, n_kv_heads, head_dim] bf16 or fp32 (rows may be
    slices of a fused projection's output), at position pos[t] of sequence seq[t] (None: t)."""
    T, dev = k.shape[0], cache.device
    code = _code(k, "k")
    if v.dtype is not k.dtype:
        raise ValueError("k and v have one type")
    kp, ks = _rows(k, "k", T, cache.n_kv_heads, cache.head_dim, dev)
    vp, vs = _rows(v, "v", T, cache.n_kv_heads, cache.head_dim, dev)
    table, n_seqs, width = _table(page_table, dev)
    wp, wn = _workspace(ws, dev)
    rc = _b.lib().moe_kv_write(cache.ref, kp, vp, code, ks, vs, T, None if seq is None else _int32(seq, "seq", (T,), dev),
                               _int32(pos, "pos", (T,), dev), table, n_seqs, width, wp, wn, _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_kv_write")


def kv_read(cache: KVCache, pos: torch.Tensor, page_table: torch.Tensor, ws: torch.Tensor,
            seq: Optional[torch.Tensor] = None, dtype=torch.bfloat16, k: Optional[torch.Tensor] = None,
            v: Optional[torch.Tensor] = None):
    """The keys and values at position pos[t] of sequence seq[t] (None: t): (k, v), each
    [T, n_kv_heads, head_dim] of `dtype`, or of the given output tensors."""
    T, dev = pos.shape[0], cache.device
    shape = (T, cache.n_kv_heads, cache.head_dim)
    k = k if k is not None else torch.empty(shape, dtype=dtype, device=cache.k.device)
    v = v if v is not None else torch.empty(shape, dtype=k.dtype, device=cache.k.device)
    code = _code(k, "k")
    if v.dtype is not k.dtype:
        raise ValueError("k and v have one type")
    table, n_seqs, width = _table(page_table, dev)
    wp, wn = _workspace(ws, dev)
    rc = _b.lib().moe_kv_read(cache.ref, T, None if seq is None else _int32(seq, "seq", (T,), dev),
                              _int32(pos, "pos", (T,), dev), table, n_seqs, width, _full(k, "k", shape, dev),
                              _full(v, "v", shape, dev), code, wp, wn, _raw_stream(dev))
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
    if q.dim() != 3 or q.dtype is not torch.bfloat16:
        raise ValueError("q is [sequences, n_heads, head_dim] bf16")
    dev, dim = cache.device, cache.head_dim
    B, H, _ = shape = q.shape
    qp, qs = _rows(q, "q", B, H, dim, dev)
    lp = _int32(lens, "lens", (B,), dev)
    table, n_seqs, width = _table(page_table, dev)
    if n_seqs != B:
        raise ValueError("page_table holds one row a sequence")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    elif out.dtype is not torch.bfloat16:
        raise ValueError("out is bf16")
    if lse is not None and lse.dtype is not torch.float32:
        raise ValueError("lse is fp32")
    wp, wn = _workspace(ws, dev)
    rc = _b.lib().moe_attn_decode(cache.ref, qp, qs, H, B, lp, table, width, dim ** -0.5 if scale is None else scale,
                                  window, _full(out, "out", shape, dev),
                                  None if lse is None else _full(lse, "lse", (B, H), dev), wp, wn, _raw_stream(dev))
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
    if residual.dim() != 2:
        raise ValueError("residual is [tokens, d]")
    T, d = shape = residual.shape
    dev = residual.get_device()
    if dev < 0:
        raise ValueError("libmoe takes CUDA tensors")
    code = _code(residual, "residual")
    rp = _full(residual, "residual", shape, dev)
    yp, y_code, post, pre, gp, gs, g_code, xp, x_code = None, 0, None, None, None, 0, 0, None, 0
    if y is not None:
        yp, y_code = _full(y, "y", shape, dev), _code(y, "y")
    if w_post is not None:
        post = _full(w_post, "w_post", (d,), dev)
        if w_post.dtype is not torch.float32:
            raise ValueError("w_post is fp32")
    if gate is not None:
        per_token = gate.dim() == 2
        if gate.shape != (shape if per_token else (d,)) or gate.get_device() != dev or (gate.stride(-1) != 1 and d > 1):
            raise ValueError("gate is [d] or [tokens, d], its rows contiguous and on the same GPU")
        gp, g_code = gate.data_ptr(), _code(gate, "gate")
        gs = gate.stride(0) if per_token and T > 1 else 0
    if residual_out is None:
        residual_out = residual
        op = None if y is None else rp  # without y the residual stays as it is
    else:
        op = _full(residual_out, "residual_out", shape, dev)
        if residual_out.dtype is not residual.dtype:
            raise ValueError("residual_out has the residual's type")
    if w_pre is not None:
        pre = _full(w_pre, "w_pre", (d,), dev)
        if w_pre.dtype is not torch.float32:
            raise ValueError("w_pre is fp32")
        if out is None:
            out = torch.empty(shape, dtype=x_dtype, device=residual.device)
        xp, x_code = _full(out, "out", shape, dev), _code(out, "out")
    elif out is not None:
        raise ValueError("an output norm needs w_pre")
    rc = _b.lib().moe_block_norm(yp, y_code, post, gp, g_code, gs, alpha, rp, op, code, pre, xp, x_code, T, d, eps,
                                 _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_block_norm")
    return residual_out, out
