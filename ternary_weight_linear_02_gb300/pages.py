"""Pages and entries of the cache between steps: binding.

What a server does between two passes of its layers: rows take pages for their next tokens and give them
back, answers continue a common prompt, accepted entries of a drafted tree are closed up.  Every decision is
made on the device from arrays that live there (``KVPages``), so a loop of steps needs no answer on
the host and can be captured.  Like the rest of the package this only marshals tensors into the C ABI
(``include/ternary_linear.h``); an index out of range is never followed and is reported by
``device_status`` (TL_ERR_VALUE).

    slots, ok = pages_reserve(pages, extra, draft + 1)    # room for the row's newest token and the drafted ones
    kv_append(cache, k, v, slots.flatten(), ...)          # in every layer, then tree_attention(..)
    path, count, tokens = verify_drafts(target, drafted, uniform, draft=q, parent=parent)
    count = torch.where(ok, count, 0)                     # a row that found no pages: the step did nothing for it
    kv_compact(layers, pages, pages.lens + 1, path, count)             # behind the newest token, the tree's root
    pages_free(pages, torch.where(ok, pages.lens + 1 + count, -1))     # .. and what was not accepted given back

Where ok is False the row's tokens have no slots, and behind the pages that it holds its table names pages of other rows: nothing
that was computed for the row in this step is of use, and its entries must not be moved.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, load
from .attention import KVCache, _Cache, _cuda, _index, _launch, _same

__all__ = ["KVLayers", "KVPages", "pages_free", "pages_reserve", "pages_fork", "kv_copy", "kv_compact"]


class KVLayers:
    """The caches of a model's layers (KVCache, one or more of one geometry on one device, none
    twice), as the calls take them that work on all layers at once."""

    __slots__ = ("caches", "first", "count", "device", "_array")

    def __init__(self, caches):
        self.caches = tuple(caches)
        if not self.caches or not all(isinstance(c, KVCache) for c in self.caches):
            raise ValueError("layers must be one or more KVCache")
        self.first, self.count = self.caches[0], len(self.caches)
        self.device = self.first.device
        for c in self.caches:
            if (c.format, c.pages, c.page_size, c.kv_heads, c.head_dim) != (
                    self.first.format, self.first.pages, self.first.page_size, self.first.kv_heads, self.first.head_dim):
                raise ValueError("the layers' caches must have one format and shape")
            if c.device != self.device:
                raise ValueError("the layers' caches must be on one device")
        ptrs = [t.data_ptr() for c in self.caches for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
        if len(set(ptrs)) != len(ptrs):
            raise ValueError("a cache is named twice")
        self._array = (_Cache * self.count)(*[c._c for c in self.caches])

    def __len__(self):
        return self.count


def _layers(layers) -> KVLayers:
    if isinstance(layers, KVLayers):
        return layers
    return KVLayers([layers] if isinstance(layers, KVCache) else layers)


class _Pages(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("held", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("rows", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class KVPages:
    """The rows (sequences) of a server and their pages: a handle on four int32 tensors.

    refs [pages]: how many rows hold each page (0: free); table [rows, max_pages]; lens [rows]: tokens of
    each row; held [rows]: pages of each row, table[r, :held[r]] -- at least those of its tokens, maybe more
    ahead of them.  One KVPages serves the caches of all layers.  The tensors stay the caller's; the
    calls change them in place on the current stream."""

    __slots__ = ("page_size", "refs", "table", "lens", "held", "pages", "rows", "max_pages", "device", "_c", "_ref")

    def __init__(self, page_size: int, refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, held: torch.Tensor):
        if not 16 <= page_size <= 1 << 20 or page_size % 16:
            raise ValueError("page_size must be a multiple of 16, up to 2^20")
        for t, n in ((refs, 1), (table, 2), (lens, 1), (held, 1)):
            if t.dtype is not torch.int32 or t.dim() != n or t.stride(-1) != 1 and t.shape[-1] > 1:
                raise ValueError("refs [pages], table [rows, max_pages], lens [rows] and held [rows] must be int32, dense")
            if not t.is_cuda:
                raise ValueError("the pages must be on a CUDA device (no CPU path)")
            if t.device != refs.device:
                raise ValueError("the pages' tensors must be on one device")
        self.rows, self.max_pages = table.shape
        if lens.shape[0] != self.rows or held.shape[0] != self.rows:
            raise ValueError("lens and held must have one element for each row of the table")
        stride = table.stride(0) if self.rows > 1 else max(table.stride(0), self.max_pages)
        if stride < self.max_pages:
            raise ValueError("rows of the table must not overlap")
        self.page_size, self.refs, self.table, self.lens, self.held = int(page_size), refs, table, lens, held
        self.pages, self.device = refs.shape[0], refs.device
        self._c = _Pages(refs.data_ptr(), table.data_ptr(), lens.data_ptr(), held.data_ptr(), stride, self.pages,
                         self.max_pages, self.rows, self.page_size)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, pages: int, rows: int, max_pages: int, page_size: int, device="cuda") -> "KVPages":
        """All pages free, all rows without tokens."""
        dev = torch.device(device)
        return cls(page_size, *(torch.zeros(shape, dtype=torch.int32, device=dev) for shape in
                                ((pages,), (rows, max_pages), (rows,), (rows,))))


def _declare(lib):
    i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    pp = ctypes.POINTER(_Pages)
    lib.ternary_pages_free.argtypes = [pp, p, p]
    lib.ternary_pages_reserve.argtypes = [pp, p, p, i32, p, p]
    lib.ternary_pages_fork_workspace.argtypes = [i64]
    lib.ternary_pages_fork_workspace.restype = i64
    lib.ternary_pages_fork.argtypes = [pp, p, p, i32, p, p, i64, p]
    lib.ternary_kv_copy.argtypes = [p, i32, p, p, p, i64, p]
    lib.ternary_kv_compact.argtypes = [p, i32, p, i64, i64, p, p, i64, p, i64, i64, p]
    lib.ternary_pages_compact.argtypes = [pp, p, i32, p, p, i64, p, i64, p]
    for f in (lib.ternary_pages_free, lib.ternary_pages_reserve, lib.ternary_pages_fork, lib.ternary_kv_copy,
              lib.ternary_kv_compact, lib.ternary_pages_compact):
        f.restype = ctypes.c_int
    return lib


_ready = None


def _lib():
    global _ready
    if _ready is None:
        _ready = _declare(load())
    return _ready


def pages_free(pages: KVPages, keep: torch.Tensor) -> None:
    """Row r holds keep[r] tokens from now on (int32 [rows]): pages.lens[r] becomes keep[r], the pages behind the
    last one are given back.  0 ends a row, a negative value leaves it as it is; keep may also be above
    lens, up to the pages held (tokens accepted into pages reserved before)."""
    keep = _index(keep, "keep", torch.int32, pages.rows, pages.device)
    rc = _launch(pages.device, (_ready or _lib()).ternary_pages_free, pages._ref, keep.data_ptr())
    if rc:
        _check(rc, "ternary_pages_free")


def pages_reserve(pages: KVPages, extra: torch.Tensor, width: int) -> tuple[torch.Tensor, torch.Tensor]:
    """Pages for the next extra[r] tokens of each row (int32 [rows]; negative: leave the row) beyond those that it
    holds: the lowest-numbered free ones, to the rows in order, to each all it needs or none.  Returns (slots
    int64 [rows, width], ok bool [rows]): the slots of the row's next min(extra, width) tokens, as kv_append takes
    them, -1 behind them and where ok is False (no page was left).  lens stays: pages_free moves it on
    when the tokens are there.  Where ok is False the row keeps what it has, and nothing else of the step may be done for it
    (this module's loop shows how)."""
    if not 0 <= width < 1 << 31:
        raise ValueError("width must be 0 or more, in 32 bits")
    dev = pages.device
    extra = _index(extra, "extra", torch.int32, pages.rows, dev)
    slots = extra.new_empty((pages.rows, int(width)), dtype=torch.int64)
    ok = torch.empty_like(extra, dtype=torch.bool)
    rc = _launch(dev, (_ready or _lib()).ternary_pages_reserve, pages._ref, extra.data_ptr(), slots.data_ptr(), int(width),
                 ok.data_ptr())
    if rc:
        _check(rc, "ternary_pages_reserve")
    return slots, ok


def pages_fork(pages: KVPages, parent: torch.Tensor, layers=None) -> torch.Tensor:
    """Row r, which must hold no page, continues row parent[r] (int32 [rows]; negative: leave the row): full pages
    are shared, the entries of the last, partly filled one are copied to a page of its own in every
    layer (KVLayers, or KVCache objects; None: only the tables).  Several rows may continue one, which itself is not
    forked in the same call.  Returns ok bool [rows]: False where no page was left."""
    dev = pages.device
    parent = _index(parent, "parent", torch.int32, pages.rows, dev)
    array, n = None, 0
    if layers is not None:
        layers = _layers(layers)
        if (layers.first.pages, layers.first.page_size) != (pages.pages, pages.page_size):
            raise ValueError("the caches must have the pages' number and size")
        if layers.device != dev:
            raise ValueError(f"layers must be on {dev} like the pages: they are on {layers.device}")
        array, n = layers._array, layers.count
    lib = _ready or _lib()
    need = 16 + 32 * pages.rows   # ternary_pages_fork_workspace
    ok = torch.empty_like(parent, dtype=torch.bool)
    ws = parent.new_empty(need, dtype=torch.uint8)
    rc = _launch(dev, lib.ternary_pages_fork, pages._ref, parent.data_ptr(), array, n, ok.data_ptr(), ws.data_ptr(), need)
    if rc:
        _check(rc, "ternary_pages_fork")
    return ok


def kv_copy(layers, src: torch.Tensor, dst: torch.Tensor, tokens: torch.Tensor | None = None) -> None:
    """The first tokens[i] places (None: all) of page src[i] copied to page dst[i] in every layer (KVLayers, or
    KVCache objects); int32 [n], a negative page: no copy.  A page that is written must not be read or written
    by another copy of the call."""
    layers = _layers(layers)
    dev, n = layers.device, src.shape[0] if src.dim() == 1 else -1
    src = _index(src, "src", torch.int32, n, dev)
    dst = _index(dst, "dst", torch.int32, n, dev)
    if tokens is not None:
        tokens = _index(tokens, "tokens", torch.int32, n, dev)
    rc = _launch(dev, (_ready or _lib()).ternary_kv_copy, layers._array, layers.count, src.data_ptr(), dst.data_ptr(),
                 None if tokens is None else tokens.data_ptr(), n)
    if rc:
        _check(rc, "ternary_kv_copy")


def _dense(t: torch.Tensor, what: str, rows: int, dev: torch.device) -> torch.Tensor:
    if t.dtype is not torch.int32 or t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{what} must be int32 with {rows} rows")
    _same(t, what, dev)
    return t if t.stride(1) == 1 or t.shape[1] <= 1 else t.contiguous()


def kv_compact(layers, page_table, start: torch.Tensor, keep: torch.Tensor, count: torch.Tensor) -> None:
    """Closes up entries in place, in every layer (KVLayers, or KVCache objects): of each sequence, the entry
    at place start[b] + keep[b, i] moves to place start[b] + i, for i < count[b].  page_table int32 [batch,
    max_pages], start and count int32 [batch], keep int32 [batch, n] with 0 <= keep[b, 0] < keep[b, 1] < ..

    page_table may be a KVPages: its rows, whose places end with the pages that they hold (a plain table has no such
    end: what it names behind them would be moved).

    verify_drafts' path and count after a drafted tree; or with start 0 the entries that are left of a
    context.  Sequences must not share the pages that are written."""
    layers = _layers(layers)
    pool = page_table if isinstance(page_table, KVPages) else None
    if pool is not None:
        page_table, dev, b = pool.table, pool.device, pool.rows
        if (layers.first.pages, layers.first.page_size) != (pool.pages, pool.page_size):
            raise ValueError("the caches must have the pages' number and size")
    else:
        dev = _cuda(page_table, "page_table")
        b = page_table.shape[0] if page_table.dim() else 0
        page_table = _dense(page_table, "page_table", b, dev)
    if dev != layers.device:
        raise ValueError(f"page_table must be on {layers.device} like the layers: it is on {dev}")
    keep = _dense(keep, "keep", b, dev)
    start = _index(start, "start", torch.int32, b, dev)
    count = _index(count, "count", torch.int32, b, dev)
    lib = _ready or _lib()
    if pool is not None:
        rc = _launch(dev, lib.ternary_pages_compact, pool._ref, layers._array, layers.count, start.data_ptr(), keep.data_ptr(),
                     keep.stride(0), count.data_ptr(), keep.shape[1])
    else:
        rc = _launch(dev, lib.ternary_kv_compact, layers._array, layers.count, page_table.data_ptr(), page_table.stride(0),
                     page_table.shape[1], start.data_ptr(), keep.data_ptr(), keep.stride(0), count.data_ptr(), b, keep.shape[1])
    if rc:
        _check(rc, "ternary_kv_compact" if pool is None else "ternary_pages_compact")
