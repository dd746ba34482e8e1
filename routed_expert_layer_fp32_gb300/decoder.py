"""The decode-step operators around the expert layer: a paged key-value cache (written as it is or
quantised, and read back) with its pages planned on the GPU, rotary positions on the way into it, the attention of
one new token over it, and the norms, gate and residual between two blocks.  Argument marshalling only;
include/libmoe.h states the operators.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

import torch

from . import binding as _b
from .binding import MOE_BF16, MOE_E4M3, MOE_F32, MOE_INT4

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
                ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class KVCache:
    """A paged cache's pools as device tensors, plus the C descriptor that borrows them.

    k, v [n_pages, n_kv_heads, page_size, head_dim]: bf16, or E4M3 codes (uint8 or
    torch.float8_e4m3fn) with their rows' exponents k_exp, v_exp [n_pages, n_kv_heads, page_size]
    uint8, or 4-bit codes (uint8, [.., head_dim / 2]) with exponents and the scales of 16 elements each, k_scale,
    v_scale [n_pages, n_kv_heads, page_size, 4 ceil(head_dim / 64)] uint8.  Pages are handed out by the caller (or by
    page_plan): position p of sequence s is in row p % page_size of page page_table[s, p // page_size]."""

    def __init__(self, k, v, k_exp=None, v_exp=None, k_scale=None, v_scale=None):
        int4 = k_scale is not None or v_scale is not None
        e4m3 = not int4 and k.dtype in (torch.uint8, torch.float8_e4m3fn)
        if not e4m3 and k.dtype != (torch.uint8 if int4 else torch.bfloat16):
            raise ValueError(f"a cache holds bf16 values, E4M3 codes or (with scales) 4-bit codes, not {k.dtype}")
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v are [n_pages, n_kv_heads, page_size, head_dim] of one type")
        if e4m3 or int4:
            for t in (k_exp, v_exp):
                if t is None or t.dtype != torch.uint8 or t.shape != k.shape[:3]:
                    raise ValueError("an E4M3 or 4-bit cache needs k_exp and v_exp, uint8 [n_pages, n_kv_heads, page_size]")
        elif k_exp is not None or v_exp is not None:
            raise ValueError("a bf16 cache has no exponents")
        if int4:
            scales = (*k.shape[:3], _scale_pitch(2 * k.shape[3]))
            for t in (k_scale, v_scale):
                if t is None or t.dtype != torch.uint8 or t.shape != scales:
                    raise ValueError(f"a 4-bit cache needs k_scale and v_scale, uint8 {list(scales)}")
        if any(t is not None and t.device != k.device for t in (v, k_exp, v_exp, k_scale, v_scale)):
            raise ValueError("a cache's pools lie on one device")
        self.k, self.v, self.k_exp, self.v_exp, self.k_scale, self.v_scale = k, v, k_exp, v_exp, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        if int4:
            self.head_dim *= 2
        self.dtype = MOE_INT4 if int4 else MOE_E4M3 if e4m3 else MOE_BF16
        self.c = MoeKvCacheC(self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, self.dtype, _b._ptr(k),
                             _b._ptr(v), _b._ptr(k_exp), _b._ptr(v_exp), _b._ptr(k_scale), _b._ptr(v_scale))
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
        if dtype not in (MOE_E4M3, MOE_INT4):
            raise ValueError("a cache is MOE_BF16, MOE_E4M3 or MOE_INT4")
        rows = shape[:3]

        def pair(*last):
            return [torch.empty((*rows, *last), dtype=torch.uint8, device=device) for _ in range(2)]

        if dtype == MOE_E4M3:
            return cls(*pair(head_dim), *pair())
        if head_dim % 32 != 0:
            raise ValueError("a 4-bit cache's head_dim is a multiple of 32")
        return cls(*pair(head_dim // 2), *pair(), *pair(_scale_pitch(head_dim)))


def _scale_pitch(head_dim: int) -> int:
    return -(-head_dim // 64) * 4


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


class PagePlan(NamedTuple):
    """What page_plan returns: of each new token its sequence, position and slot (page * page_size + row), -1 behind the
    last; where each sequence's tokens begin; the lengths and the count of free pages afterwards."""
    seq: torch.Tensor
    pos: torch.Tensor
    slot: torch.Tensor
    starts: torch.Tensor
    lens: torch.Tensor
    n_free: torch.Tensor


def pages_workspace(B: int, device="cuda") -> torch.Tensor:
    """Workspace of page_plan and page_release for up to B sequences (one call at a time)."""
    n = int(_b.lib().moe_pages_workspace_bytes(B))
    if n == 0:
        raise _b.MoeError(-2, "moe_pages_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _ints(name: str, t: torch.Tensor, n: int, dev: int) -> int:
    # (numel and dim are a third of what the shape costs)
    if t.dtype is not torch.int32 or t.numel() != n or t.dim() != 1 or t.get_device() != dev or not t.is_contiguous():
        raise _misfit(name, t, f"int32 [{n}], contiguous")
    return t.data_ptr()


def _pool(lens, page_table, free_pages, n_free, ws, lens_out, n_free_out):
    """What page_plan and page_release share: sizes, addresses, and the outputs (in place where none are given)."""
    dev = page_table.get_device()
    if dev < 0:
        raise _misfit("page_table", page_table, "int32 [sequences, pages], contiguous and on a GPU")
    if _devices != 1:
        _check_device(dev)
    table, B, width, wp, wn = _table(page_table, ws, dev)
    if free_pages.dim() != 1:
        raise _misfit("free_pages", free_pages, "int32 [pages]")
    n = free_pages.shape[0]
    lens_out = lens if lens_out is None else lens_out
    n_free_out = n_free if n_free_out is None else n_free_out
    return (dev, B, width, table, _ints("lens", lens, B, dev), _ints("free_pages", free_pages, n, dev), n,
            _ints("n_free", n_free, 1, dev), lens_out, _ints("lens_out", lens_out, B, dev), n_free_out,
            _ints("n_free_out", n_free_out, 1, dev), wp, wn)


def page_plan(lens: torch.Tensor, new_tokens: Optional[torch.Tensor], page_table: torch.Tensor, free_pages: torch.Tensor,
              n_free: torch.Tensor, page_size: int, n_pages: int, max_tokens: int, ws: torch.Tensor,
              lens_out: Optional[torch.Tensor] = None, n_free_out: Optional[torch.Tensor] = None,
              starts: Optional[torch.Tensor] = None, seq: Optional[torch.Tensor] = None,
              pos: Optional[torch.Tensor] = None, slot: Optional[torch.Tensor] = None) -> PagePlan:
    """Room for new_tokens[b] (None: one) more tokens of each sequence, which has lens[b] in the cache: pages from the
    stack free_pages [n_pages], whose first n_free[0] entries are free, into page_table [B, max_pages], and the list of
    all new tokens' sequences, positions and slots, padded to max_tokens (seq, pos and slot, where they are given, begin at
    a multiple of 16 bytes).  lens and n_free are updated in place unless lens_out and n_free_out are given."""
    (dev, B, width, table, lp, fp, n, np_, lens_out, lop, n_free_out, nop, wp, wn) = _pool(
        lens, page_table, free_pages, n_free, ws, lens_out, n_free_out)
    if n != n_pages:
        raise _misfit("free_pages", free_pages, f"int32 [{n_pages}], contiguous")
    new = None if new_tokens is None else _ints("new_tokens", new_tokens, B, dev)
    if max_tokens < 0:
        raise ValueError("max_tokens is 0 or more")

    def out(name, t, count):
        if t is None:
            t = torch.empty(count, dtype=torch.int32, device=page_table.device)
        return t, _ints(name, t, count, dev)

    starts, sp = out("starts", starts, B + 1)
    seq, qp = out("seq", seq, max_tokens)
    pos, pp = out("pos", pos, max_tokens)
    slot, tp = out("slot", slot, max_tokens)
    rc = _b.lib().moe_page_plan(lp, new, B, table, width, fp, np_, n, page_size, max_tokens, lop, nop, sp, qp, pp, tp, wp,
                                wn, _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_page_plan")
    return PagePlan(seq, pos, slot, starts, lens_out, n_free_out)


def page_release(lens: torch.Tensor, ended: torch.Tensor, page_table: torch.Tensor, free_pages: torch.Tensor,
                 n_free: torch.Tensor, page_size: int, ws: torch.Tensor, lens_out: Optional[torch.Tensor] = None,
                 n_free_out: Optional[torch.Tensor] = None):
    """The pages of sequences with ended[b] (bool or uint8) back on the stack free_pages, their lengths 0.  Returns
    (lens, n_free): updated in place unless lens_out and n_free_out are given."""
    (dev, B, width, table, lp, fp, n, np_, lens_out, lop, n_free_out, nop, wp, wn) = _pool(
        lens, page_table, free_pages, n_free, ws, lens_out, n_free_out)
    if (ended.dtype not in (torch.bool, torch.uint8) or ended.shape != (B,) or ended.get_device() != dev
            or not ended.is_contiguous()):
        raise _misfit("ended", ended, f"bool or uint8 [{B}], contiguous")
    rc = _b.lib().moe_page_release(lp, ended.data_ptr(), B, table, width, fp, np_, n, page_size, lop, nop, wp, wn,
                                   _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_page_release")
    return lens_out, n_free_out


class MoeRopeC(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("turns", ctypes.c_void_p)]


class Rope:
    """Rotary positions' frequencies on the device.  dim: the elements of each head that are turned (a multiple of 8);
    interleaved: pairs are elements 2i and 2i + 1, else i and i + dim / 2.  scaling: "none", or how frequencies trained
    for a context of `original` positions are changed for one `factor` times as long: "linear", "base", "by_index" (pairs
    with more than `high` turns in the original context stay, those below `low` are slowed, between by their index; with
    a magnitude) or "by_turns" (between by their turns).  frequencies: radians a position of each pair, in place
    of all of that, with `magnitude` on cosine and sine."""
    SCALINGS = ("none", "linear", "base", "by_index", "by_turns")

    def __init__(self, dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original: float = 4096.0, low: float = 1.0, high: float = 32.0,
                 frequencies: Optional[Sequence[float]] = None, magnitude: Optional[float] = None, device="cuda"):
        if dim <= 0 or dim % 8 != 0 or dim > 256:
            raise ValueError("dim is a multiple of 8, from 8 to 256")
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling is one of {', '.join(self.SCALINGS)}")
        turns, own = (ctypes.c_uint64 * (dim // 2))(), ctypes.c_float(1.0)
        if frequencies is None:
            rc = _b.lib().moe_rope_frequencies(dim, base, self.SCALINGS.index(scaling), factor, original, low, high, turns,
                                               ctypes.byref(own))
        else:
            if scaling != "none":
                raise ValueError("frequencies are given, or made by a scaling")
            given = [float(f) for f in frequencies]
            if len(given) != dim // 2:
                raise ValueError(f"a frequency for each of {dim // 2} pairs")
            rc = _b.lib().moe_rope_turns((ctypes.c_double * len(given))(*given), len(given), turns)
        if rc:
            raise _b.MoeError(rc, "moe_rope_frequencies" if frequencies is None else "moe_rope_turns")
        self.dim, self.interleaved = dim, bool(interleaved)
        self.magnitude = own.value if magnitude is None else float(magnitude)
        # torch has no arithmetic for uint64 everywhere: the same bits
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.device = self.turns.get_device()
        self.c = MoeRopeC(dim, int(self.interleaved), self.magnitude, _b._ptr(self.turns))
        self.ref = ctypes.byref(self.c)


def _heads(name: str, t: torch.Tensor, dev: int, code_of=_CODES):
    """Type code, shape and row stride of t [tokens, heads, dim]."""
    code = code_of.get(t.dtype)
    if code is None or t.dim() != 3 or t.get_device() != dev:
        raise _misfit(name, t, "bf16 or fp32 [tokens, heads, head_dim]")
    T, heads, dim = t.shape
    return code, T, heads, dim, _row_stride(t, name, heads, dim)


def rope(x: torch.Tensor, table: Rope, pos: torch.Tensor, out: Optional[torch.Tensor] = None,
         inverse: bool = False) -> torch.Tensor:
    """x [tokens, heads, head_dim] bf16 or fp32 (rows may be slices of a fused projection's output) with the first
    table.dim elements of each head turned by its token's position pos[t]; inverse: turned back.  out may be x."""
    dev = table.device
    if _devices != 1:
        _check_device(dev)
    code, T, heads, dim, stride = _heads("x", x, dev)
    pp = _ints("pos", pos, T, dev)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if out.dtype is not x.dtype or out.shape != x.shape:
        raise _misfit("out", out, f"{x.dtype} {list(x.shape)}, as x")
    out_stride = _heads("out", out, dev)[4]
    rc = _b.lib().moe_rope_apply(table.ref, x.data_ptr(), stride, out.data_ptr(), out_stride, code, T, heads, dim, pp,
                                 int(inverse), _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_rope_apply")
    return out


def rope_kv_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: KVCache, table: Rope, pos: torch.Tensor,
                  slot: torch.Tensor, ws: torch.Tensor, q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """q [T, n_heads, head_dim] and k [T, n_kv_heads, head_dim] turned by their tokens' positions pos[t]; the keys and v
    into the cache at slot[t] (page * page_size + row, as page_plan gives them; negative: not written).  q, k and v bf16
    or fp32, slices of a fused projection's output as it lies.  Returns q_out, bf16, which may be q."""
    dev, dim = cache.device, cache.head_dim
    if _devices != 1:
        _check_device(dev)
    code, T, heads, q_dim, q_stride = _heads("q", q, dev)
    if q_dim != dim or table.device != dev:
        raise _misfit("q", q, f"bf16 or fp32 [tokens, heads, {dim}]")
    shape = (T, cache.n_kv_heads, dim)
    if k.dtype is not q.dtype or k.shape != shape or k.get_device() != dev:
        raise _misfit("k", k, f"{q.dtype} {list(shape)}")
    if v.dtype is not q.dtype or v.shape != shape or v.get_device() != dev:
        raise _misfit("v", v, f"{q.dtype} {list(shape)}")
    pp, sp = _ints("pos", pos, T, dev), _ints("slot", slot, T, dev)
    if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise _misfit("ws", ws, "uint8, contiguous")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    elif q_out.dtype is not torch.bfloat16 or q_out.shape != q.shape or q_out.get_device() != dev:
        raise _misfit("q_out", q_out, f"bf16 {list(q.shape)}")
    rc = _b.lib().moe_rope_kv_write(table.ref, cache.ref, q.data_ptr(), q_stride, heads, q_out.data_ptr(),
                                    _row_stride(q_out, "q_out", heads, dim), k.data_ptr(), v.data_ptr(), code,
                                    _row_stride(k, "k", shape[1], dim), _row_stride(v, "v", shape[1], dim), T, pp, sp,
                                    ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if rc:
        raise _b.MoeError(rc, "moe_rope_kv_write")
    return q_out


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
