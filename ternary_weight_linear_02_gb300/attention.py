"""Rotary positions, the quantised paged cache and attention over it: binding.

What a decode step needs between its fused QKV call and its o call.  Like the
rest of the package this only marshals tensors into the C ABI
(``include/ternary_linear.h``); the work runs on the current stream of the
tensors' device, and errors found on the host raise before anything is enqueued.
Indices that live on the device (positions, slots, page tables, lengths) are
checked there: one out of range skips its work and is reported by
``device_status`` (TL_ERR_VALUE).

    qkv = linear(x, w_qkv, s_qkv).unflatten(-1, (q_heads + 2 * kv_heads, 128))
    q = kv_append(cache, qkv[:, q_heads:-kv_heads], qkv[:, -kv_heads:], slots,
                  q=qkv[:, :q_heads], positions=positions, table=table)
    o = tree_attention(q.unflatten(0, (batch, draft)), cache, page_table, context_len, tree)
    x = linear(o.flatten(-2).flatten(0, 1), w_o, s_o)
"""
from __future__ import annotations

import ctypes

import torch

from . import TL_BF16, TL_F16, TL_F32, _check, load

__all__ = ["KVCache", "KV_FORMATS", "rope_table", "rope", "kv_append", "kv_read", "tree_attention"]

KV_FORMATS = {"int8": 0, "fp8": 1, "int4": 2}
_CODES = {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}
_DT = {torch.float16: TL_F16, torch.bfloat16: TL_BF16, torch.float32: TL_F32}
_INTERLEAVED, _INVERSE = 1, 2

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _stream(dev: torch.device) -> int:
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _cuda(t: torch.Tensor, what: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device (no CPU path)")
    return t


def _index(t: torch.Tensor, what: str, dtype: torch.dtype, n: int) -> torch.Tensor:
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{what} must be a 1-D {dtype} tensor of {n} elements")
    _cuda(t, what)
    return t if t.is_contiguous() else t.contiguous()


def _rows(t: torch.Tensor, what: str, dims: int) -> torch.Tensor:
    if t.dim() != dims:
        raise ValueError(f"{what} must have {dims} dimensions")
    _cuda(t, what)
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _table(table: torch.Tensor) -> torch.Tensor:
    if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous fp32 tensor [positions, rotary_dim] (rope_table)")
    return _cuda(table, "table")


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("format", ctypes.c_int32)]


class KVCache:
    """A paged cache of keys and values in 8 or 4 bits: a handle on four tensors.

    Codes [pages, kv_heads, page_size, head_dim] -- "int8": int8, "fp8":
    float8_e4m3fn, "int4": uint8 with head_dim / 2 bytes per row (two fields of value +
    8, the even element in the low bits) -- and fp32 scales [pages, kv_heads,
    page_size], for keys and for values; value = code * scale.  Slot s is place
    s % page_size of page s // page_size.  head_dim is 64 or 128, page_size a
    multiple of 16.  The tensors stay the caller's: entries may be copied, moved or
    shared between sequences with ordinary indexing.
    """

    __slots__ = ("format", "k_codes", "v_codes", "k_scale", "v_scale", "pages", "kv_heads", "page_size",
                 "head_dim", "_c", "_ref")

    def __init__(self, format: str, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        if format not in KV_FORMATS:
            raise ValueError(f"format must be one of {sorted(KV_FORMATS)}")
        for t in (k_codes, v_codes):
            if t.dtype != _CODES[format] or t.dim() != 4 or not t.is_contiguous():
                raise ValueError(f"codes must be contiguous {_CODES[format]} [pages, kv_heads, page_size, row]")
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or not t.is_contiguous() or t.shape != k_codes.shape[:3]:
                raise ValueError("scales must be contiguous fp32 [pages, kv_heads, page_size]")
        if v_codes.shape != k_codes.shape:
            raise ValueError("key and value codes must have one shape")
        for t in (k_codes, v_codes, k_scale, v_scale):
            if _cuda(t, "the cache").device != k_codes.device:
                raise ValueError("the cache's tensors must be on one device")
        self.format = format
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.pages, self.kv_heads, self.page_size, row = k_codes.shape
        self.head_dim = 2 * row if format == "int4" else row
        if self.head_dim not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        if self.page_size < 16 or self.page_size % 16:
            raise ValueError("page_size must be a multiple of 16")
        self._c = _Cache(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                         self.pages, self.page_size, self.kv_heads, self.head_dim, KV_FORMATS[format])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, format: str, pages: int, page_size: int, kv_heads: int, head_dim: int,
              device="cuda") -> "KVCache":
        """An unwritten cache (its contents are undefined; no call reads a key beyond a
        sequence's length)."""
        if format not in KV_FORMATS:
            raise ValueError(f"format must be one of {sorted(KV_FORMATS)}")
        row = head_dim // 2 if format == "int4" else head_dim
        shape = (pages, kv_heads, page_size)
        codes = [torch.empty((*shape, row), dtype=torch.uint8, device=device).view(_CODES[format]) for _ in "kv"]
        scales = [torch.empty(shape, dtype=torch.float32, device=device) for _ in "kv"]
        return cls(format, *codes, *scales)


def _declare(lib):
    i32, i64, u32, p, f64 = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_double)
    pc = ctypes.POINTER(_Cache)
    lib.ternary_rope_table.argtypes = [p, i64, i32, f64, f64, f64, f64, f64, f64, p]
    lib.ternary_rope.argtypes = [p, i64, i64, p, i64, i64, i32, i64, i32, i32, p, p, i64, i32, u32, p]
    lib.ternary_kv_append.argtypes = [pc, p, i64, i64, p, i64, i64, i32, i64, p, p, i64, i64, p, i64, i64,
                                      i32, p, p, i64, i32, u32, p]
    lib.ternary_kv_read.argtypes = [pc, p, i64, p, p, i32, p]
    lib.ternary_tree_attention_workspace.argtypes = [i64, i64, i32, i32, i32]
    lib.ternary_tree_attention.argtypes = [p, i64, i64, i64, i32, i64, i64, i32, pc, p, i64, i64, p, p, i64,
                                           i64, ctypes.c_float, p, p, p, i64, p]
    for f in (lib.ternary_rope_table, lib.ternary_rope, lib.ternary_kv_append, lib.ternary_kv_read,
              lib.ternary_tree_attention):
        f.restype = ctypes.c_int
    lib.ternary_tree_attention_workspace.restype = i64
    return lib


_ready = None


def _lib():
    global _ready
    if _ready is None:
        _ready = _declare(load())
    return _ready


def rope_table(positions: int, rotary_dim: int, *, base: float = 10000.0, factor: float = 1.0,
               original_len: float = 0.0, ramp: tuple[float, float] = (1.0, 32.0), magnitude: float = 1.0,
               device="cuda") -> torch.Tensor:
    """Cosines and sines of positions 0 .. positions - 1: fp32 [positions, rotary_dim]
    (cosines, then sines), made once per model, angles in fp64.

    factor > 1 stretches the context: frequencies of fewer than ramp[0] full turns
    within original_len positions are divided by factor, those of more than ramp[1]
    stay, those between move over linearly; original_len = 0 divides all of them.
    magnitude multiplies every entry (the attention's temperature at long contexts)."""
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("device must be a CUDA device (no CPU path)")
    if positions < 0 or rotary_dim < 0:
        raise ValueError("positions and rotary_dim must not be negative")
    out = torch.empty((int(positions), int(rotary_dim)), dtype=torch.float32, device=dev)
    _check(_lib().ternary_rope_table(out.data_ptr(), int(positions), int(rotary_dim), float(base),
                                     float(factor), float(original_len), float(ramp[0]), float(ramp[1]),
                                     float(magnitude), _stream(out.device)), "ternary_rope_table")
    return out


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, *, interleaved: bool = False,
         inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """x [tokens, heads, head_dim] (fp16, bf16 or fp32; any token and head stride) with
    the first table.shape[1] elements of each head rotated by its token's position
    (int64 [tokens]): pairs (x[i], x[i + R/2]), or (x[2i], x[2i+1]) interleaved.
    inverse: the negative angle, which takes the output's gradient to the input's.
    out: where to write; x itself rotates in place."""
    if x.dtype not in _DT:
        raise ValueError("x must be fp16, bf16 or fp32")
    x = _rows(x, "x", 3)
    n, heads, dim = x.shape
    positions = _index(positions, "positions", torch.int64, n)
    table = _table(table)
    if out is None:
        out = torch.empty((n, heads, dim), dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != x.device or out.stride(-1) != 1:
        raise ValueError("out must have x's shape, dtype and device, its last axis dense")
    rc = _lib().ternary_rope(x.data_ptr(), x.stride(0), x.stride(1), out.data_ptr(), out.stride(0),
                             out.stride(1), _DT[x.dtype], n, heads, dim, positions.data_ptr(),
                             table.data_ptr(), table.shape[0], table.shape[1],
                             (_INTERLEAVED if interleaved else 0) | (_INVERSE if inverse else 0),
                             _stream(x.device))
    if rc:
        _check(rc, "ternary_rope")
    return out


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *,
              q: torch.Tensor | None = None, positions: torch.Tensor | None = None,
              table: torch.Tensor | None = None, interleaved: bool = False,
              q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Write k, v [tokens, kv_heads, head_dim] (fp16 or bf16, strided views welcome) into
    the cache at slots (int64 [tokens]; negative: padding, not stored).  With a table
    (rope_table, rotary_dim a multiple of 16) k, and q [tokens, q_heads, head_dim] where
    given, are rotated by positions (int64 [tokens]) in the same pass; the rotated q is
    returned (written to q_out; q itself rotates in place).  k is not rounded
    between its rotation and its quantisation."""
    if k.dtype not in (torch.float16, torch.bfloat16) or v.dtype != k.dtype:
        raise ValueError("k and v must be fp16 or bf16, both the same")
    k, v = _rows(k, "k", 3), _rows(v, "v", 3)
    n = k.shape[0]
    want = (n, cache.kv_heads, cache.head_dim)
    if k.shape != want or v.shape != want:
        raise ValueError(f"k and v must be {want}: got {tuple(k.shape)} and {tuple(v.shape)}")
    slots = _index(slots, "slots", torch.int64, n)
    if table is not None:
        table = _table(table)
        if positions is None:
            raise ValueError("a table needs positions")
        positions = _index(positions, "positions", torch.int64, n)
        tp, pp, t_rows, rot = table.data_ptr(), positions.data_ptr(), table.shape[0], table.shape[1]
    else:
        if q is not None or interleaved:
            raise ValueError("q and interleaved need a table")
        tp = pp = None
        t_rows = rot = 0
    if q is not None:
        q = _rows(q, "q", 3)
        if q.dtype != k.dtype or q.shape[0] != n or q.shape[2] != cache.head_dim:
            raise ValueError("q must be [tokens, q_heads, head_dim] in k's dtype")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.device != q.device or q_out.stride(-1) != 1:
            raise ValueError("q_out must have q's shape, dtype and device, its last axis dense")
        qa = (q.data_ptr(), q.stride(0), q.stride(1), q_out.data_ptr(), q_out.stride(0), q_out.stride(1),
              q.shape[1])
    else:
        if q_out is not None:
            raise ValueError("q_out needs q")
        qa = (None, 0, 0, None, 0, 0, 0)
    rc = _lib().ternary_kv_append(cache._ref, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                                  v.stride(0), v.stride(1), _DT[k.dtype], n, slots.data_ptr(), *qa, pp, tp,
                                  t_rows, rot, _INTERLEAVED if interleaved else 0, _stream(k.device))
    if rc:
        _check(rc, "ternary_kv_append")
    return q_out


def kv_read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16
            ) -> tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [tokens, kv_heads, head_dim] in dtype (fp16, bf16 or fp32): the values at
    slots (int64 [tokens]); zeros where a slot is negative."""
    if dtype not in _DT:
        raise ValueError("dtype must be fp16, bf16 or fp32")
    n = slots.shape[0] if slots.dim() == 1 else -1
    slots = _index(slots, "slots", torch.int64, n)
    shape = (n, cache.kv_heads, cache.head_dim)
    k = torch.empty(shape, dtype=dtype, device=slots.device)
    v = torch.empty(shape, dtype=dtype, device=slots.device)
    rc = _lib().ternary_kv_read(cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), _DT[dtype],
                                _stream(slots.device))
    if rc:
        _check(rc, "ternary_kv_read")
    return k, v


_ws_bytes: dict = {}


def tree_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, context_len: torch.Tensor,
                   tree: torch.Tensor | None = None, *, scale: float | None = None,
                   out: torch.Tensor | None = None, return_lse: bool = False):
    """Attention of each sequence's new tokens q [batch, draft, q_heads, head_dim] (fp16 or
    bf16) over its cached keys: the context_len[b] committed ones, and of the new
    tokens' own (at places context_len[b] .. + draft - 1, written by kv_append before)
    those that tree names -- bool or uint8 [draft, draft] or [batch, draft, draft],
    row t listing what token t sees; None: a chain, token t sees tokens 0 .. t.

    page_table int32 [batch, max_pages], context_len int32 [batch].  scale defaults to
    head_dim ** -0.5.  Returns [batch, draft, q_heads, head_dim] in q's dtype (zeros for a
    token that sees nothing) and, with return_lse, ln of the sum of exp of its scores,
    fp32 [batch, draft, q_heads]."""
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("q must be fp16 or bf16")
    q = _rows(q, "q", 4)
    b, t, heads, dim = q.shape
    if dim != cache.head_dim or heads % cache.kv_heads:
        raise ValueError("q must be [batch, draft, a multiple of kv_heads, head_dim]")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != b:
        raise ValueError("page_table must be int32 [batch, max_pages]")
    if page_table.stride(1) != 1:
        page_table = page_table.contiguous()
    _cuda(page_table, "page_table")
    context_len = _index(context_len, "context_len", torch.int32, b)
    tp, tb, tr = None, 0, 0
    if tree is not None:
        if tree.dtype not in (torch.bool, torch.uint8) or tree.shape[-2:] != (t, t) or tree.dim() not in (2, 3) \
                or (tree.dim() == 3 and tree.shape[0] not in (1, b)):
            raise ValueError("tree must be bool or uint8 [draft, draft] or [batch, draft, draft]")
        _cuda(tree, "tree")
        if tree.stride(-1) != 1:
            tree = tree.contiguous()
        tp, tr = tree.data_ptr(), tree.stride(-2)
        tb = tree.stride(0) if tree.dim() == 3 and tree.shape[0] > 1 else 0
    if out is None:
        out = torch.empty((b, t, heads, dim), dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device or not out.is_contiguous():
        raise ValueError("out must be contiguous with q's shape, dtype and device")
    lse = torch.empty((b, t, heads), dtype=torch.float32, device=q.device) if return_lse else None
    lib = _lib()
    key = (b, t, heads, cache.kv_heads, dim)
    need = _ws_bytes.get(key)
    if need is None:
        need = _ws_bytes[key] = int(lib.ternary_tree_attention_workspace(*key))
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 0 else None
    rc = lib.ternary_tree_attention(q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), _DT[q.dtype], b, t,
                                    heads, cache._ref, page_table.data_ptr(), page_table.stride(0),
                                    page_table.shape[1], context_len.data_ptr(), tp, tb, tr,
                                    dim ** -0.5 if scale is None else float(scale), out.data_ptr(),
                                    None if lse is None else lse.data_ptr(),
                                    None if ws is None else ws.data_ptr(), max(need, 0), _stream(q.device))
    if rc:
        _check(rc, "ternary_tree_attention")
    return (out, lse) if return_lse else out
