"""Low-rank adapters of many requests beside a shared ternary layer: binding.

The packed weights serve every request; what a request's own fine-tuning adds is a product of two thin matrices, and
one call adds each token's.  Like the rest of the package this only marshals tensors into the C ABI
(``include/ternary_linear.h``).

    qkv = linear(x, w_qkv, s_qkv)
    lora_add(x, qkv_adapters, which, qkv, out=qkv)         # in place
    ...
    gu = linear(x, w_gate_up, s_gate_up)
    h = lora_silu_mul(x, gate_up_adapters, which, gu)      # silu(gate) * up of the adapted layer
"""
from __future__ import annotations

import ctypes

import torch

from . import TL_F32, _DT, _check, load
from .attention import _cuda, _launch, _same

__all__ = ["Adapters", "lora_add", "lora_silu_mul"]


class _Adapters(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("inputs", ctypes.c_int64),
                ("shard_rows", ctypes.c_int64 * 8), ("shards", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("adapters", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Adapters:
    """The adapters of one layer: a handle on their stacked matrices (fp16 or bf16).

    a [adapters, shards * rank, inputs], b [adapters, outputs, rank], scale fp32 [adapters] (None: 1); shards: the
    output rows of each shard of a fused layer (None: one shard), each with `rank` rows of a of its own.
    Column c of shard s gets scale * b[c] . (a[s * rank : (s + 1) * rank] x).  rank is a multiple of 8, 8..128; adapters
    of smaller rank are padded with zeros."""

    __slots__ = ("a", "b", "scale", "shards", "rank", "count", "inputs", "outputs", "dtype", "device", "_c", "_ref")

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor | None = None, shards=None):
        if a.dtype not in (torch.float16, torch.bfloat16) or b.dtype is not a.dtype:
            raise ValueError("a and b must be fp16 or bf16, both the same")
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or not a.is_contiguous() or not b.is_contiguous():
            raise ValueError("a must be [adapters, shards * rank, inputs] and b [adapters, outputs, rank], contiguous")
        self.count, self.outputs, self.rank = b.shape
        self.inputs = a.shape[2]
        self.shards = (self.outputs,) if shards is None else tuple(int(n) for n in shards)
        if not 1 <= len(self.shards) <= 8 or min(self.shards) < 0 or sum(self.shards) != self.outputs:
            raise ValueError("shards must be 1 to 8 sizes that add up to b's outputs")
        if a.shape[1] != len(self.shards) * self.rank:
            raise ValueError("a must have rank rows for each shard")
        if self.rank % 8 or not 8 <= self.rank <= 128:
            raise ValueError("rank must be a multiple of 8, 8 to 128")
        self.device = _cuda(a, "a")
        _same(b, "b", self.device)
        if scale is not None:
            if scale.dtype is not torch.float32 or scale.shape != (self.count,) or not scale.is_contiguous():
                raise ValueError("scale must be a contiguous fp32 tensor [adapters]")
            _same(scale, "scale", self.device)
        self.a, self.b, self.scale, self.dtype = a, b, scale, a.dtype
        self._c = _Adapters(a.data_ptr(), b.data_ptr(), None if scale is None else scale.data_ptr(), self.inputs,
                            (ctypes.c_int64 * 8)(*self.shards), len(self.shards), self.rank, self.count, _DT[a.dtype])
        self._ref = ctypes.byref(self._c)


_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = load()
        i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        lib.ternary_lora_workspace.argtypes = [i64, i64]
        lib.ternary_lora_workspace.restype = i64
        for f in (lib.ternary_lora_add, lib.ternary_lora_silu_mul):
            f.argtypes = [p, i64, ctypes.POINTER(_Adapters), p, p, i64, p, i64, i32, i64, p, i64, p]
            f.restype = ctypes.c_int
        _ready = lib
    return _ready


def _rows(t: torch.Tensor, what: str, cols: int, dev: torch.device) -> tuple[torch.Tensor, int]:
    """[tokens, cols] with a dense last axis, and its token stride."""
    if t.device != dev:
        _same(t, what, dev)
    st = t.stride()
    if len(st) != 2:
        t = t.reshape(-1, cols)
        st = t.stride()
    if st[1] != 1 and cols > 1:
        t = t.contiguous()
        st = t.stride()
    return t, st[0]


def _call(name: str, x, adapters: Adapters, which, y, out, cols: int):
    dev, k, kind = adapters.device, adapters.inputs, y.dtype
    shape = x.shape
    if x.dtype is not adapters.dtype or len(shape) < 1 or shape[-1] != k:
        raise ValueError(f"x must be [..., {k}] in the adapters' dtype")
    n, lead = adapters.outputs, shape[:-1]
    if y.shape != (*lead, n) or (kind is not torch.float32 and kind is not adapters.dtype):
        raise ValueError(f"y must be [..., {n}] with x's leading dimensions, in the adapters' dtype or fp32")
    x, xs = _rows(x, "x", k, dev)
    m = x.shape[0]
    wshape = which.shape
    if which.dtype is not torch.int32 or not (wshape == lead or wshape == (m,)):
        raise ValueError("which must be int32, one number for each token")
    if which.device != dev:
        _same(which, "which", dev)
    if not which.is_contiguous():
        which = which.contiguous()
    if out is None:
        o = out = torch.empty_like(y, memory_format=torch.contiguous_format) if cols == n else y.new_empty((*lead, cols))
        os = cols
        if len(lead) != 1:
            o = out.view(-1, cols)
    else:
        if out.shape != (*lead, cols) or out.dtype is not kind or out.device != dev or len(lead) != 1 and not out.is_contiguous():
            raise ValueError(f"out must be [..., {cols}] with y's leading dimensions, dtype and device (contiguous unless two-dimensional)")
        o = out if len(lead) == 1 else out.view(-1, cols)
        os, dense = o.stride()
        if dense != 1 and cols > 1:
            raise ValueError("out must be dense in its last axis")
    if out is y:
        y, ys = o, os
    else:
        y, ys = _rows(y, "y", n, dev)
    lib = _ready or _lib()
    ws, need = None, 0
    if m > 1024 or adapters.count > 1024:
        need = int(lib.ternary_lora_workspace(m, adapters.count))
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    rc = _launch(dev, getattr(lib, name), x.data_ptr(), xs, adapters._ref, which.data_ptr(), y.data_ptr(), ys, o.data_ptr(), os, _DT[kind], m,
                 None if ws is None else ws.data_ptr(), need)
    if rc:
        _check(rc, name)
    return out


def lora_add(x: torch.Tensor, adapters: Adapters, which: torch.Tensor, y: torch.Tensor, *, out: torch.Tensor | None = None) -> torch.Tensor:
    """y + each token's adapter product: x [..., inputs] (fp16 or bf16, the adapters' dtype), y [..., outputs] (that dtype or
    fp32) what the shared layer gave for x, which int32 [...]: each token's adapter, negative: none.  Sums are fp32, the
    result is rounded once to y's dtype.  out: where to write; y itself adds in place."""
    return _call("ternary_lora_add", x, adapters, which, y, out, adapters.outputs)


def lora_silu_mul(x: torch.Tensor, adapters: Adapters, which: torch.Tensor, y: torch.Tensor, *, out: torch.Tensor | None = None) -> torch.Tensor:
    """silu(g) * u of a fused gate/up layer with adapters: y [..., 2 N] what the shared layer gave (gate columns, then up
    columns), g and u its halves with each token's adapter product added (two shards of N); returns [..., N].  g and u
    stay fp32, the result is rounded once to y's dtype.  16-bit y has g and u rounded already, which linear_silu_mul never does:
    where that matters, take y from the layer with out_dtype=torch.float32 and round what is returned."""
    if len(adapters.shards) != 2 or adapters.shards[0] != adapters.shards[1]:
        raise ValueError("a gated layer has two shards of one size: gate and up")
    return _call("ternary_lora_silu_mul", x, adapters, which, y, out, adapters.outputs // 2)
