"""Host-side refusals of the page and entry calls (no GPU, nothing is launched)."""
import ctypes

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import attention, pages

OK, NULL, SHAPE, DTYPE, ALIGN, VALUE, CUDA = 0, 1, 2, 3, 4, 5, 6
A, B, C, D, E = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    tl.build()
    tl.load()
    return pages._lib()


def pool(refs=A, table=B, lens=C, held=D, stride=4, n=9, wide=4, rows=3, page=16):
    return ctypes.byref(pages._Pages(refs, table, lens, held, stride, n, wide, rows, page))


def cache(i=0, **kw):
    at = 0x100000 * (i + 1)
    d = dict(kc=at, vc=at + 0x1000, ks=at + 0x2000, vs=at + 0x3000, pages=9, page=16, heads=2, dim=64, fmt=0)
    d.update(kw)
    return attention._Cache(d["kc"], d["vc"], d["ks"], d["vs"], d["pages"], d["page"], d["heads"], d["dim"], d["fmt"])


def many(*cs):
    return (attention._Cache * len(cs))(*cs)


BAD_POOLS = [(dict(rows=-1), SHAPE), (dict(rows=8193), SHAPE), (dict(page=8), SHAPE), (dict(page=24), SHAPE), (dict(n=0), SHAPE),
             (dict(n=1 << 30), SHAPE), (dict(wide=-1), SHAPE), (dict(wide=1 << 27, stride=1 << 27), SHAPE), (dict(stride=3), SHAPE),
             (dict(refs=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(held=None), NULL),
             (dict(refs=A + 2), ALIGN), (dict(table=B + 1), ALIGN), (dict(lens=C + 2), ALIGN), (dict(held=D + 2), ALIGN)]


@pytest.mark.parametrize("kw,want", BAD_POOLS)
def test_pools(lib, kw, want):
    assert lib.ternary_pages_free(pool(**kw), E, None) == want
    assert lib.ternary_pages_reserve(pool(**kw), E, None, 0, None, None) == want
    assert lib.ternary_pages_fork(pool(**kw), E, None, 0, None, A, 1 << 20, None) == want


def test_free_and_reserve(lib):
    assert lib.ternary_pages_free(None, E, None) == NULL and lib.ternary_pages_free(pool(), None, None) == NULL
    assert lib.ternary_pages_free(pool(), E + 2, None) == ALIGN and lib.ternary_pages_free(pool(rows=0), None, None) == OK

    def reserve(extra=E, slots=A, width=4, ok=B, p=None):
        return lib.ternary_pages_reserve(p or pool(), extra, slots, width, ok, None)

    assert reserve(extra=None) == NULL and reserve(extra=E + 1) == ALIGN and reserve(slots=A + 4) == ALIGN
    assert reserve(width=-1) == SHAPE and reserve(p=pool(rows=0), extra=None) == OK


def test_fork(lib):
    def fork(p=None, parent=E, caches=None, layers=0, ws=A, size=1 << 20):
        return lib.ternary_pages_fork(p or pool(), parent, caches, layers, None, ws, size, None)

    assert fork(parent=None) == NULL and fork(parent=E + 2) == ALIGN and fork(ws=None) == NULL and fork(ws=A + 8) == ALIGN
    assert lib.ternary_pages_fork_workspace(3) == 16 + 3 * 32 and lib.ternary_pages_fork_workspace(-1) == -1
    assert lib.ternary_pages_fork_workspace(8193) == -1
    assert fork(size=15) == SHAPE and fork(layers=-1) == SHAPE and fork(layers=513, caches=many(cache())) == SHAPE
    assert fork(layers=1) == NULL
    assert fork(layers=1, caches=many(cache(pages=8))) == SHAPE     # not the pool's pages
    assert fork(layers=1, caches=many(cache(page=32))) == SHAPE
    assert fork(layers=2, caches=many(cache(), cache(1, dim=128))) == SHAPE
    assert fork(layers=2, caches=many(cache(), cache())) == VALUE   # a cache twice
    assert fork(layers=2, caches=many(cache(), cache(1, vs=0x103000))) == VALUE
    assert fork(layers=1, caches=many(cache(vc=0x100000))) == VALUE
    assert fork(layers=1, caches=many(cache(fmt=3))) == DTYPE
    assert fork(p=pool(rows=0), parent=None, ws=None) == OK


def test_copy(lib):
    def copy(caches=None, layers=1, src=A, dst=B, tokens=C, n=4):
        return lib.ternary_kv_copy(caches or many(cache()), layers, src, dst, tokens, n, None)

    assert lib.ternary_kv_copy(None, 1, A, B, C, 4, None) == NULL
    assert copy(layers=0) == SHAPE and copy(n=-1) == SHAPE and copy(n=1 << 31) == SHAPE
    assert copy(src=None) == NULL and copy(dst=None) == NULL and copy(src=A + 2) == ALIGN and copy(tokens=C + 1) == ALIGN
    assert copy(n=0, src=None) == OK


def test_compact(lib):
    def compact(caches=None, layers=1, table=A, wide=4, start=B, keep=C, count=D, b=2, n=3, stride=3):
        return lib.ternary_kv_compact(caches or many(cache()), layers, table, 4, wide, start, keep, stride, count, b, n, None)

    assert compact(layers=0) == SHAPE and compact(b=-1) == SHAPE and compact(n=-1) == SHAPE and compact(b=(1 << 16) + 1) == SHAPE
    assert compact(wide=-1) == SHAPE and compact(wide=1 << 27) == SHAPE and compact(stride=1 << 41) == SHAPE
    for name in ("table", "start", "keep", "count"):
        assert compact(**{name: None}) == NULL
    assert compact(keep=C + 2) == ALIGN and compact(start=B + 1) == ALIGN
    assert compact(b=0, start=None) == OK and compact(n=0, keep=None) == OK


def test_injected_launch_failure(lib):
    lib.ternary_test_inject_launch_failures(1)
    try:
        assert lib.ternary_pages_free(pool(), E, None) == CUDA
    finally:
        lib.ternary_test_inject_launch_failures(0)


def test_binding_refuses():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tl.KVPages(16, i, torch.zeros(3, 4, dtype=torch.int32), i, i)
    with pytest.raises(ValueError, match="int32"):
        tl.KVPages(16, i.long(), torch.zeros(3, 4, dtype=torch.int32), i, i)
    with pytest.raises(ValueError, match="KVCache"):
        tl.KVLayers([])
    with pytest.raises(ValueError, match="KVCache"):
        tl.KVLayers([i])


class _FakePages:
    device, rows = torch.device("cpu"), 3


def test_binding_refuses_sizes_beyond_32_bits():
    """Sizes are passed in 32 bits: what does not fit is refused, not cut off."""
    i, table = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    for size in (8, 24, (1 << 20) + 16, (1 << 32) + 16):
        with pytest.raises(ValueError, match="page_size"):
            tl.KVPages(size, i, table, i, i)
    for width in (-1, 1 << 31, (1 << 32) + 1):
        with pytest.raises(ValueError, match="width"):
            tl.pages_reserve(_FakePages(), i, width)
