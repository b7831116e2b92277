"""Host-side refusals of closing up a pool's rows (no GPU, nothing is launched)."""
from test_pages_host import ALIGN, B, C, CUDA, D, NULL, OK, SHAPE, cache, lib, many, pool  # noqa: F401


def test_compact_of_a_pool(lib):  # noqa: F811
    def compact(p=None, caches=None, layers=1, start=B, keep=C, count=D, n=3, stride=3):
        return lib.ternary_pages_compact(p or pool(), caches or many(cache()), layers, start, keep, stride, count, n, None)

    assert lib.ternary_pages_compact(None, many(cache()), 1, B, C, 3, D, 3, None) == NULL
    assert lib.ternary_pages_compact(pool(), None, 1, B, C, 3, D, 3, None) == NULL
    assert compact(layers=0) == SHAPE and compact(n=-1) == SHAPE and compact(stride=1 << 41) == SHAPE
    assert compact(caches=many(cache(pages=8))) == SHAPE and compact(caches=many(cache(page=32))) == SHAPE
    assert compact(p=pool(held=None)) == NULL and compact(p=pool(rows=-1)) == SHAPE and compact(p=pool(table=B + 1)) == ALIGN
    for name in ("start", "keep", "count"):
        assert compact(**{name: None}) == NULL
    assert compact(keep=C + 2) == ALIGN and compact(p=pool(rows=0), start=None) == OK and compact(n=0, keep=None) == OK
    lib.ternary_test_inject_launch_failures(1)
    try:
        assert compact() == CUDA
    finally:
        lib.ternary_test_inject_launch_failures(0)
