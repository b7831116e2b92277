"""Rotary positions, the quantised paged cache and attention over it: binding.

What a decode step needs between its fused QKV call and its o call.  Like the
rest of the package this only marshals tensors into the C ABI
(``include/ternary_linear.h``); the work runs on the current stream of the
tensors' device, and errors found on the host raise before anything is enqueued.
Indices that live on the device (positions, slots, page tables, lengths) are
checked there: one out of range is never followed (a position or slot skips its token, a
page is read as page 0, a length is clamped) and is reported by ``device_status``
(TL_ERR_VALUE).

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


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _launch(dev: torch.device, f, *args) -> int:
    """f(*args, stream) on dev, whichever device is the current one."""
    if dev.index == _current_device():
        return f(*args, _stream(dev))
    with torch.cuda.device(dev):
        return f(*args, _stream(dev))


def _cuda(t: torch.Tensor, what: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device (no CPU path)")
    return t.device


def _same(t: torch.Tensor, what: str, dev: torch.device):
    if t.device != dev:
        _cuda(t, what)
        raise ValueError(f"{what} must be on {dev} like the call's other tensors: it is on {t.device}")


def _index(t: torch.Tensor, what: str, dtype: torch.dtype, n: int, dev: torch.device) -> torch.Tensor:
    if t.dtype is not dtype or t.shape != (n,):
        raise ValueError(f"{what} must be a 1-D {dtype} tensor of {n} elements")
    _same(t, what, dev)
    return t if t.is_contiguous() else t.contiguous()


def _rows(t: torch.Tensor, what: str, dev: torch.device) -> tuple[torch.Tensor, tuple]:
    """The tensor with a dense last axis, and its strides."""
    _same(t, what, dev)
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1:
        t = t.contiguous()
        st = t.stride()
    return t, st


def _out(out: torch.Tensor, like: torch.Tensor, what: str) -> tuple:
    st = out.stride()
    if out.shape != like.shape or out.dtype is not like.dtype or out.device != like.device or st[-1] != 1:
        raise ValueError(f"{what} must have the input's shape, dtype and device, its last axis dense")
    return st


def _table(table: torch.Tensor, dev: torch.device) -> tuple[int, int]:
    if table.dtype is not torch.float32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous fp32 tensor [positions, rotary_dim] (rope_table)")
    _same(table, "table", dev)
    return table.shape


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
                 "head_dim", "device", "_c", "_ref")

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
            if not t.is_cuda:
                raise ValueError("the cache must be on a CUDA device (no CPU path)")
            if t.device != k_codes.device:
                raise ValueError("the cache's tensors must be on one device")
        self.format = format
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.device = k_codes.device
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
    lib.ternary_tree_attention_workspace.argtypes = [i64, i64, i32, i32, i32, i64]
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
    _check(_launch(out.device, _lib().ternary_rope_table, out.data_ptr(), int(positions), int(rotary_dim),
                   float(base), float(factor), float(original_len), float(ramp[0]), float(ramp[1]),
                   float(magnitude)), "ternary_rope_table")
    return out


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, *, interleaved: bool = False,
         inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """x [tokens, heads, head_dim] (fp16, bf16 or fp32; any token and head stride) with
    the first table.shape[1] elements of each head rotated by its token's position
    (int64 [tokens]): pairs (x[i], x[i + R/2]), or (x[2i], x[2i+1]) interleaved.
    inverse: the negative angle, which takes the output's gradient to the input's (the
    calls record nothing for autograd, as the linear layers do not).
    out: where to write; x itself rotates in place."""
    dt = _DT.get(x.dtype)
    if dt is None or x.dim() != 3:
        raise ValueError("x must be [tokens, heads, head_dim] in fp16, bf16 or fp32")
    dev = _cuda(x, "x")
    x, xs = _rows(x, "x", dev)
    shape = x.shape
    n, heads, dim = shape
    positions = _index(positions, "positions", torch.int64, n, dev)
    t_rows, rot = _table(table, dev)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=dev)
        ot, oh = heads * dim, dim
    else:
        ot, oh, _ = _out(out, x, "out")
    rc = _launch(
        dev, (_ready or _lib()).ternary_rope, x.data_ptr(), xs[0], xs[1], out.data_ptr(), ot, oh, dt, n, heads, dim,
        positions.data_ptr(), table.data_ptr(), t_rows, rot,
        (_INTERLEAVED if interleaved else 0) | (_INVERSE if inverse else 0))
    if rc:
        _check(rc, "ternary_rope")
    return out


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *,
              q: torch.Tensor | None = None, positions: torch.Tensor | None = None,
              table: torch.Tensor | None = None, interleaved: bool = False,
              q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Write k, v [tokens, kv_heads, head_dim] (fp16 or bf16, strided views welcome) into
    the cache at slots (int64 [tokens]; negative: padding, not stored; a slot named by two
    tokens of one call is left undefined, a mixture of both).  With a table
    (rope_table, rotary_dim a multiple of 16) k, and q [tokens, q_heads, head_dim] where
    given, are rotated by positions (int64 [tokens]) in the same pass; the rotated q is
    returned (written to q_out; q itself rotates in place).  k is not rounded
    between its rotation and its quantisation."""
    dtype = k.dtype
    dt = _DT.get(dtype)
    if dt is None or dt == TL_F32 or v.dtype is not dtype:
        raise ValueError("k and v must be fp16 or bf16, both the same")
    shape = k.shape
    n = shape[0] if shape else 0
    if shape != (n, cache.kv_heads, cache.head_dim) or v.shape != shape:
        raise ValueError(f"k and v must be [tokens, {cache.kv_heads}, {cache.head_dim}]: "
                         f"got {tuple(shape)} and {tuple(v.shape)}")
    dev = cache.device
    k, ks = _rows(k, "k", dev)
    v, vs = _rows(v, "v", dev)
    slots = _index(slots, "slots", torch.int64, n, dev)
    if table is not None:
        t_rows, rot = _table(table, dev)
        if positions is None:
            raise ValueError("a table needs positions")
        positions = _index(positions, "positions", torch.int64, n, dev)  # (a copy lives until the call)
        tp, pp = table.data_ptr(), positions.data_ptr()
    else:
        if q is not None or interleaved:
            raise ValueError("q and interleaved need a table")
        tp = pp = None
        t_rows = rot = 0
    if q is not None:
        qshape = q.shape
        if q.dtype is not dtype or len(qshape) != 3 or qshape[0] != n or qshape[2] != cache.head_dim:
            raise ValueError("q must be [tokens, q_heads, head_dim] in k's dtype")
        q, qs = _rows(q, "q", dev)
        if q_out is None:
            q_out = torch.empty(qshape, dtype=dtype, device=dev)
            ot, oh = qshape[1] * qshape[2], qshape[2]
        else:
            ot, oh, _ = _out(q_out, q, "q_out")
        rc = _launch(
            dev, (_ready or _lib()).ternary_kv_append, cache._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0],
            vs[1], dt, n, slots.data_ptr(), q.data_ptr(), qs[0], qs[1], q_out.data_ptr(), ot, oh, qshape[1], pp, tp,
            t_rows, rot, _INTERLEAVED if interleaved else 0)
    else:
        if q_out is not None:
            raise ValueError("q_out needs q")
        rc = _launch(
            dev, (_ready or _lib()).ternary_kv_append, cache._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0],
            vs[1], dt, n, slots.data_ptr(), None, 0, 0, None, 0, 0, 0, pp, tp, t_rows, rot,
            _INTERLEAVED if interleaved else 0)
    if rc:
        _check(rc, "ternary_kv_append")
    return q_out


def kv_read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16
            ) -> tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [tokens, kv_heads, head_dim] in dtype (fp16, bf16 or fp32): the values at
    slots (int64 [tokens]); zeros where a slot is negative."""
    dt = _DT.get(dtype)
    if dt is None:
        raise ValueError("dtype must be fp16, bf16 or fp32")
    n = slots.shape[0] if slots.dim() == 1 else -1
    dev = cache.device
    slots = _index(slots, "slots", torch.int64, n, dev)
    shape = (n, cache.kv_heads, cache.head_dim)
    k = torch.empty(shape, dtype=dtype, device=dev)
    v = torch.empty(shape, dtype=dtype, device=dev)
    rc = _launch(dev, (_ready or _lib()).ternary_kv_read, cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), dt)
    if rc:
        _check(rc, "ternary_kv_read")
    return k, v


_ws_bytes: dict = {}   # of the sizes met last: a server's page tables grow all the time
_WS_SIZES = 512


def tree_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, context_len: torch.Tensor,
                   tree: torch.Tensor | None = None, *, scale: float | None = None,
                   out: torch.Tensor | None = None, return_lse: bool = False):
    """Attention of each sequence's new tokens q [batch, draft, q_heads, head_dim] (fp16 or
    bf16) over its cached keys: the context_len[b] committed ones, and of the new
    tokens' own (at places context_len[b] .. + draft - 1, written by kv_append before)
    those that tree names -- bool or uint8 [draft, draft] or [batch, draft, draft],
    row t listing what token t sees; None: a chain, token t sees tokens 0 .. t.

    page_table int32 [batch, max_pages], context_len int32 [batch].  scale defaults to
    head_dim ** -0.5.  Scores and sums are fp32; the weights, with their value scales, enter
    the product with the values in fp16.  Returns [batch, draft, q_heads, head_dim] in q's
    dtype (zeros for a token that sees nothing) and, with return_lse, ln of the sum of exp of its scores,
    fp32 [batch, draft, q_heads]."""
    dtype = q.dtype
    dt = _DT.get(dtype)
    if dt is None or dt == TL_F32 or q.dim() != 4:
        raise ValueError("q must be [batch, draft, q_heads, head_dim] in fp16 or bf16")
    dev = cache.device
    q, qs = _rows(q, "q", dev)
    shape = q.shape
    b, t, heads, dim = shape
    if dim != cache.head_dim or heads % cache.kv_heads:
        raise ValueError("q must be [batch, draft, a multiple of kv_heads, head_dim]")
    pshape = page_table.shape
    if page_table.dtype is not torch.int32 or len(pshape) != 2 or pshape[0] != b:
        raise ValueError("page_table must be int32 [batch, max_pages]")
    _same(page_table, "page_table", dev)
    pstride = page_table.stride()
    if pstride[1] != 1:
        page_table = page_table.contiguous()
        pstride = page_table.stride()
    context_len = _index(context_len, "context_len", torch.int32, b, dev)
    tp, tb, tr = None, 0, 0
    if tree is not None:
        tshape = tree.shape
        if (tree.dtype is not torch.bool and tree.dtype is not torch.uint8) or not (
                tshape == (b, t, t) or tshape == (t, t) or tshape == (1, t, t)):
            raise ValueError("tree must be bool or uint8 [draft, draft] or [batch, draft, draft]")
        _same(tree, "tree", dev)
        if tree.stride(-1) != 1:
            tree = tree.contiguous()
        ts = tree.stride()
        tp, tr = tree.data_ptr(), ts[-2]
        tb = ts[0] if len(tshape) == 3 and tshape[0] > 1 else 0
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    elif out.shape != shape or out.dtype is not dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be contiguous with q's shape, dtype and device")
    lse = torch.empty((b, t, heads), dtype=torch.float32, device=dev) if return_lse else None
    lib = _ready or _lib()
    key = (b, t, heads, cache.kv_heads, dim, pshape[1] * cache.page_size)
    need = _ws_bytes.get(key)
    if need is None:
        if len(_ws_bytes) >= _WS_SIZES:
            _ws_bytes.clear()
        need = _ws_bytes[key] = int(lib.ternary_tree_attention_workspace(*key))
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    rc = _launch(
        dev, lib.ternary_tree_attention, q.data_ptr(), qs[0], qs[1], qs[2], dt, b, t, heads, cache._ref,
        page_table.data_ptr(), pstride[0], pshape[1], context_len.data_ptr(), tp, tb, tr,
        dim ** -0.5 if scale is None else float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(),
        None if ws is None else ws.data_ptr(), max(need, 0))
    if rc:
        _check(rc, "ternary_tree_attention")
    return (out, lse) if return_lse else out
