"""Verification of drafted tokens: binding.

The last step of a decode step with a drafter: the target's probabilities of a drafted chain or tree decide
which tokens stand.  Like the rest of the package this only marshals tensors into the C ABI
(``include/ternary_linear.h``).
"""
from __future__ import annotations

import ctypes

import torch

from . import _DT, _check, load
from .attention import _cuda, _launch, _same

__all__ = ["verify_drafts"]

_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = load()
        i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        lib.ternary_verify_drafts.argtypes = [p, i64, i64, p, i64, i64, i32, p, i64, p, i64, p, i64, i64, i64, i64, p, p, p, p]
        lib.ternary_verify_drafts.restype = ctypes.c_int
        _ready = lib
    return _ready


def _dense(t: torch.Tensor, what: str, dev: torch.device) -> tuple[torch.Tensor, tuple]:
    """The tensor with a dense last axis, and its strides."""
    if t.device != dev:
        _same(t, what, dev)
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        t = t.contiguous()
        st = t.stride()
    return t, st


def verify_drafts(target: torch.Tensor, tokens: torch.Tensor, uniform: torch.Tensor, *, draft: torch.Tensor | None = None,
                  parent: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Which drafted tokens stand, and the token after them, from given random numbers: the tokens are distributed
    as if the target had drawn them one by one.

    target [batch, draft + 1, vocab] (fp32, fp16 or bf16): probabilities of the token after node 0, where the
    sequence stands, and after each drafted token (node 1 + i).  tokens int64 [batch, draft].  parent int32
    [draft] or [batch, draft]: the drafted token that each follows (-1: none; always an earlier one); None: a
    chain.  draft [batch, draft (or more), vocab] in target's dtype: the probabilities that the drafter drew each
    node's children from (row n: node n); None: it gave tokens only.  uniform fp32 [batch, draft + 1] in [0, 1):
    one number for each drafted token, the last for the token that is drawn.

    At a node, w is its target row and W = 1; children are looked at in order, x the child's token: accepted if
    u W q(x) < w(x), and otherwise w = max(w - W q, 0), W = sum w (without draft: q(x) = 1, and a rejected token is
    taken out of w, W -= w(x)).  The last token is drawn from w.

    Returns (path int32 [batch, draft], count int32 [batch], tokens int64 [batch, draft + 1]): the indexes of the
    accepted tokens in order, how many, and their tokens followed by the drawn one; -1 behind."""
    kind = target.dtype
    dt, shape = _DT.get(kind), target.shape
    if dt is None or len(shape) != 3 or shape[1] < 1:
        raise ValueError("target must be [batch, draft + 1, vocab] in fp32, fp16 or bf16")
    dev = target.device
    if not target.is_cuda:
        _cuda(target, "target")
    b, n, v = shape
    n -= 1
    if tokens.dtype is not torch.int64 or tokens.shape != (b, n):
        raise ValueError(f"tokens must be int64 [batch, draft] = [{b}, {n}]")
    if uniform.dtype is not torch.float32 or uniform.shape != (b, n + 1):
        raise ValueError(f"uniform must be fp32 [batch, draft + 1] = [{b}, {n + 1}]")
    target, (tb, tn, _) = _dense(target, "target", dev)
    tokens, (xb, _) = _dense(tokens, "tokens", dev)
    uniform, (ub, _) = _dense(uniform, "uniform", dev)
    qp, qb, qn = None, 0, 0
    if draft is not None:
        shape = draft.shape
        if draft.dtype is not kind or len(shape) != 3 or shape[0] != b or shape[1] < n or shape[2] != v:
            raise ValueError("draft must be [batch, draft, vocab] in target's dtype")
        draft, (qb, qn, _) = _dense(draft, "draft", dev)
        qp = draft.data_ptr()
    pp, pb = None, 0
    if parent is not None:
        shape = parent.shape
        if parent.dtype is not torch.int32 or not (shape == (b, n) or shape == (n,)):
            raise ValueError("parent must be int32 [draft] or [batch, draft]")
        parent, st = _dense(parent, "parent", dev)
        pp, pb = parent.data_ptr(), st[0] if len(shape) == 2 else 0
    # (of the inputs' shapes: empty_like takes half of empty's time on the host)
    path = torch.empty_like(tokens, dtype=torch.int32, memory_format=torch.contiguous_format)
    count = tokens.new_empty(b, dtype=torch.int32)
    out = torch.empty_like(uniform, dtype=torch.int64, memory_format=torch.contiguous_format)
    rc = _launch(dev, (_ready or _lib()).ternary_verify_drafts, target.data_ptr(), tb, tn, qp, qb, qn, dt, tokens.data_ptr(), xb, pp,
                 pb, uniform.data_ptr(), ub, b, n, v, path.data_ptr(), count.data_ptr(), out.data_ptr())
    if rc:
        _check(rc, "ternary_verify_drafts")
    return path, count, out
