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


def _check_int32(t: torch.Tensor, name: str, dims: int):
    if t.dtype != torch.int32 or t.dim() != dims:
        raise ValueError(f"{name} is an int32 tensor of {dims} dimension{'s' if dims > 1 else ''}")


def _rows(t: torch.Tensor, name: str, heads: int, dim: int):
    """(address, row stride) of [T, heads, dim] rows that are contiguous in themselves."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} is [tokens, {heads}, {dim}]")
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
        raise ValueError(f"{name}'s rows of [{heads}, {dim}] must be contiguous")
    return t.data_ptr(), (s0 if t.shape[0] > 1 else heads * dim)


def _on_one_device(t: torch.Tensor, others):
    for o in others:
        if o is not None and o.device != t.device:
            raise ValueError("libmoe takes tensors of one device")


def attn_workspace(cache: KVCache, n_heads: int, B: int) -> torch.Tensor:
    """Workspace of attn_decode for up to B sequences (kept by the caller, one call at a time)."""
    n = int(_b.lib().moe_attn_workspace_bytes(cache.ref, n_heads, B))
    if n == 0:
        raise _b.MoeError(-2, "moe_attn_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.k.device)
    _b._check(_b.lib().moe_attn_workspace_init(_b._ptr(ws), n, _b._stream()), "moe_attn_workspace_init")
    return ws


def kv_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, pos: torch.Tensor, page_table: torch.Tensor,
             ws: torch.Tensor, seq: Optional[torch.Tensor] = None) -> None:
    """Writes tokens' keys and values, k and v [T, n_kv_heads, head_dim] bf16 or fp32 (rows may be
    slices of a fused projection's output), at position pos[t] of sequence seq[t] (None: t)."""
    T = k.shape[0]
    if v.shape[0] != T or v.dtype != k.dtype:
        raise ValueError("k and v have one length and type")
    _check_tokens(T, pos, seq, page_table)
    _on_one_device(cache.k, (k, v, pos, seq, page_table, ws))
    kp, ks = _rows(k, "k", cache.n_kv_heads, cache.head_dim)
    vp, vs = _rows(v, "v", cache.n_kv_heads, cache.head_dim)
    _b._check(_b.lib().moe_kv_write(cache.ref, kp, vp, _b._dtype_code(k), ks, vs, T, _b._ptr(seq), _b._ptr(pos),
                                    _b._ptr(page_table), page_table.shape[0], page_table.shape[1], _b._ptr(ws),
                                    ws.numel(), _b._stream()), "moe_kv_write")


def kv_read(cache: KVCache, pos: torch.Tensor, page_table: torch.Tensor, ws: torch.Tensor,
            seq: Optional[torch.Tensor] = None, dtype=torch.bfloat16, k: Optional[torch.Tensor] = None,
            v: Optional[torch.Tensor] = None):
    """The keys and values at position pos[t] of sequence seq[t] (None: t): (k, v), each
    [T, n_kv_heads, head_dim] of `dtype`, or of the given output tensors."""
    T = pos.shape[0]
    shape = (T, cache.n_kv_heads, cache.head_dim)
    k = k if k is not None else torch.empty(shape, dtype=dtype, device=cache.k.device)
    v = v if v is not None else torch.empty(shape, dtype=k.dtype, device=cache.k.device)
    if k.shape != shape or v.shape != shape or k.dtype != v.dtype:
        raise ValueError(f"k and v are {list(shape)} of one type")
    _check_tokens(T, pos, seq, page_table)
    _on_one_device(cache.k, (k, v, pos, seq, page_table, ws))
    _b._check(_b.lib().moe_kv_read(cache.ref, T, _b._ptr(seq), _b._ptr(pos), _b._ptr(page_table), page_table.shape[0],
                                   page_table.shape[1], _b._ptr(k), _b._ptr(v), _b._dtype_code(k), _b._ptr(ws),
                                   ws.numel(), _b._stream()), "moe_kv_read")
    return k, v


def _check_tokens(T: int, pos, seq, page_table):
    _check_int32(pos, "pos", 1)
    _check_int32(page_table, "page_table", 2)
    if seq is not None:
        _check_int32(seq, "seq", 1)
    if pos.shape[0] != T or (seq is not None and seq.shape[0] != T):
        raise ValueError("pos and seq hold one entry a token")


def attn_decode(q: torch.Tensor, cache: KVCache, lens: torch.Tensor, page_table: torch.Tensor, ws: torch.Tensor,
                scale: Optional[float] = None, window: int = 0, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token a sequence: q [B, n_heads, head_dim] bf16 (rows may be slices of a
    fused projection's output) over the last `window` (0: all) of lens[b] cached tokens.  scale
    defaults to head_dim ** -0.5.  Returns out [B, n_heads, head_dim] bf16; lse [B, n_heads] fp32,
    where given, receives the log-sum-exp of the scores."""
    if q.dim() != 3 or q.dtype != torch.bfloat16:
        raise ValueError("q is [sequences, n_heads, head_dim] bf16")
    B, H = q.shape[0], q.shape[1]
    qp, qs = _rows(q, "q", H, cache.head_dim)
    _check_int32(lens, "lens", 1)
    _check_int32(page_table, "page_table", 2)
    if lens.shape[0] != B or page_table.shape[0] != B:
        raise ValueError("lens and page_table hold one row a sequence")
    out = out if out is not None else torch.empty((B, H, cache.head_dim), dtype=torch.bfloat16, device=q.device)
    if out.shape != q.shape or out.dtype != torch.bfloat16:
        raise ValueError("out is [sequences, n_heads, head_dim] bf16")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (B, H)):
        raise ValueError("lse is [sequences, n_heads] fp32")
    _on_one_device(cache.k, (q, lens, page_table, ws, out, lse))
    _b._check(_b.lib().moe_attn_decode(cache.ref, qp, qs, H, B, _b._ptr(lens), _b._ptr(page_table),
                                       page_table.shape[1], cache.head_dim ** -0.5 if scale is None else scale, window,
                                       _b._ptr(out), _b._ptr(lse), _b._ptr(ws), ws.numel(), _b._stream()),
              "moe_attn_decode")
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
    T, d = residual.shape
    if y is not None and y.shape != residual.shape:
        raise ValueError("y has the residual's shape")
    for w, name in ((w_pre, "w_pre"), (w_post, "w_post")):
        if w is not None and (w.dtype != torch.float32 or w.shape != (d,)):
            raise ValueError(f"{name} is [d] fp32")
    gp, gs = None, 0
    if gate is not None:
        if gate.shape != (d,) and gate.shape != (T, d):
            raise ValueError("gate is [d] or [tokens, d]")
        if not gate.is_cuda or (gate.stride(-1) != 1 and d > 1):
            raise ValueError("gate's rows are contiguous on the GPU")
        gp, gs = gate.data_ptr(), (gate.stride(0) if gate.dim() == 2 and T > 1 else 0)
    r_out = residual_out if residual_out is not None else residual
    if r_out.shape != residual.shape or r_out.dtype != residual.dtype:
        raise ValueError("residual_out has the residual's shape and type")
    if w_pre is None:
        if out is not None:
            raise ValueError("an output norm needs w_pre")
    elif out is None:
        out = torch.empty((T, d), dtype=x_dtype, device=residual.device)
    elif out.shape != residual.shape:
        raise ValueError("out has the residual's shape")
    _on_one_device(residual, (w_pre, y, w_post, gate, r_out, out))
    code = _b._dtype_code
    if y is None and r_out is residual:
        r_ptr = None  # the residual stays as it is
    else:
        r_ptr = _b._ptr(r_out)
    _b._check(_b.lib().moe_block_norm(_b._ptr(y), MOE_F32 if y is None else code(y), _b._ptr(w_post), gp,
                                      MOE_F32 if gate is None else code(gate), gs, alpha, _b._ptr(residual), r_ptr,
                                      code(residual), _b._ptr(w_pre), _b._ptr(out), MOE_F32 if out is None else code(out),
                                      T, d, eps, _b._stream()), "moe_block_norm")
    return r_out, out
