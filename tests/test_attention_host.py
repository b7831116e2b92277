"""Host-side refusals of the rotary, cache and attention calls (no GPU, nothing is launched)."""
import ctypes

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import attention

OK, NULL, SHAPE, DTYPE, ALIGN, VALUE, CUDA = 0, 1, 2, 3, 4, 5, 6
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    tl.build()
    tl.load()
    return attention._lib()


def cache(kc=A, vc=B, ks=C, vs=D, pages=4, page=16, heads=2, dim=64, fmt=0):
    return ctypes.byref(attention._Cache(kc, vc, ks, vs, pages, page, heads, dim, fmt))


def test_rope_table_refusals(lib):
    def call(table=A, n=8, r=64, base=1e4, factor=1.0, olen=0.0, lo=1.0, hi=32.0, mag=1.0):
        return lib.ternary_rope_table(table, n, r, base, factor, olen, lo, hi, mag, None)

    assert call(n=-1) == SHAPE and call(n=1 << 31) == SHAPE
    assert call(r=0) == SHAPE and call(r=63) == SHAPE and call(r=1026) == SHAPE
    assert call(base=0.0) == VALUE and call(base=float("nan")) == VALUE
    assert call(factor=0.0) == VALUE and call(factor=float("inf")) == VALUE
    assert call(mag=float("nan")) == VALUE and call(olen=float("inf")) == VALUE
    assert call(table=None) == NULL and call(table=A + 4) == ALIGN
    assert call(n=0, table=None) == OK


def test_rope_refusals(lib):
    def call(x=A, xt=128, xh=64, out=B, ot=128, oh=64, dt=1, n=4, h=2, d=64, pos=C, table=D, rows=9, r=64, flags=0):
        return lib.ternary_rope(x, xt, xh, out, ot, oh, dt, n, h, d, pos, table, rows, r, flags, None)

    assert call(dt=3) == DTYPE and call(dt=-1) == DTYPE and call(flags=4) == DTYPE
    assert call(n=-1) == SHAPE and call(h=-1) == SHAPE and call(d=1) == SHAPE and call(d=1026) == SHAPE
    assert call(r=0) == SHAPE and call(r=3) == SHAPE and call(r=66) == SHAPE and call(rows=-1) == SHAPE
    assert call(xt=1 << 41) == SHAPE and call(oh=-(1 << 41)) == SHAPE
    for name in ("x", "out", "pos", "table"):
        assert call(**{name: None}) == NULL
    assert call(x=A + 1) == ALIGN and call(x=A + 2, dt=2) == ALIGN and call(pos=C + 4) == ALIGN
    assert call(table=D + 4) == ALIGN
    assert call(n=0, x=None) == OK and call(h=0, out=None) == OK


def test_cache_refusals(lib):
    def read(c, slots=A, n=4, k=B, v=C, dt=1):
        return lib.ternary_kv_read(c, slots, n, k, v, dt, None)

    assert read(None) == NULL
    for bad in (dict(fmt=3), dict(fmt=-1)):
        assert read(cache(**bad)) == DTYPE
    for bad in (dict(dim=96), dict(dim=256), dict(page=8), dict(page=24), dict(page=0), dict(heads=0),
                dict(pages=0), dict(pages=1 << 31)):
        assert read(cache(**bad)) == SHAPE
    for bad in ("kc", "vc", "ks", "vs"):
        assert read(cache(**{bad: None})) == NULL
        assert read(cache(**{bad: A + 8})) == ALIGN
    assert read(cache(), dt=3) == DTYPE and read(cache(), n=-1) == SHAPE
    assert read(cache(), slots=None) == NULL and read(cache(), slots=A + 4) == ALIGN
    assert read(cache(), k=B + 8) == ALIGN
    assert read(cache(), n=0, slots=None) == OK and read(cache(), k=None, v=None) == OK


def test_append_refusals(lib):
    def call(c=None, k=A, v=B, dt=1, n=4, slots=C, q=None, qo=None, hq=0, pos=None, table=None, rows=0, r=0, flags=0,
             stride=128):
        return lib.ternary_kv_append(c or cache(), k, stride, 64, v, 128, 64, dt, n, slots, q, 128, 64, qo, 128, 64, hq, pos,
                                     table, rows, r, flags, None)

    assert call(dt=2) == DTYPE and call(flags=2, table=D, pos=C, r=16) == DTYPE
    assert call(flags=1) == DTYPE                     # a layout without a table
    assert call(n=-1) == SHAPE and call(hq=-1) == SHAPE and call(stride=1 << 41) == SHAPE
    assert call(table=D, pos=C, rows=4, r=24) == SHAPE and call(table=D, pos=C, rows=4, r=80) == SHAPE
    assert call(table=D, pos=C, rows=4, r=0) == SHAPE
    assert call(k=None) == NULL and call(v=None) == NULL and call(slots=None) == NULL
    assert call(table=D, r=16) == NULL                # a table without positions
    assert call(q=A, qo=B, hq=2) == NULL              # queries without a table
    assert call(q=A, hq=2, table=D, pos=C, r=16) == NULL
    assert call(k=A + 1) == ALIGN and call(slots=C + 4) == ALIGN
    assert call(table=D + 4, pos=C, r=16) == ALIGN
    assert call(n=0, k=None, v=None, slots=None) == OK


def test_attention_refusals(lib):
    def call(q=A, dt=1, b=2, t=3, hq=4, c=None, pages=B, wide=4, lens=C, tree=None, scale=0.125, out=D, ws=A,
             ws_bytes=1 << 40):
        return lib.ternary_tree_attention(q, 768, 256, 64, dt, b, t, hq, c or cache(), pages, 4, wide, lens, tree, 9, 3,
                                          scale, out, None, ws, ws_bytes, None)

    assert call(dt=2) == DTYPE
    assert call(b=-1) == SHAPE and call(t=-1) == SHAPE and call(hq=3) == SHAPE and call(hq=0) == SHAPE
    assert call(t=1 << 17) == SHAPE and call(wide=-1) == SHAPE and call(wide=1 << 30) == SHAPE
    assert call(t=65) == SHAPE                        # more new tokens than a row of pages holds
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == VALUE
    for name in ("q", "pages", "lens", "out"):
        assert call(**{name: None}) == NULL
    assert call(q=A + 1) == ALIGN and call(out=D + 2) == ALIGN and call(pages=B + 2) == ALIGN
    assert call(ws=A + 8) == ALIGN
    assert call(b=0, q=None, out=None) == OK and call(t=0, q=None, out=None) == OK
    w = lib.ternary_tree_attention_workspace
    assert w(-1, 1, 4, 2, 64, 64) == -1 and w(1, 1, 5, 2, 64, 64) == -1 and w(1, 1, 4, 2, 96, 64) == -1
    assert w(1, 1, 4, 2, 64, -1) == -1 and w(1, 1, 4, 2, 64, 1 << 31) == -1
    assert w(0, 1, 4, 2, 64, 64) == 0
    assert w(2, 3, 4, 2, 64, 64) == 0                 # contexts of a page or two: no workspace
    need = w(2, 3, 4, 2, 64, 1 << 16)
    assert need > 0
    assert call(wide=4096, ws=None) == NULL and call(wide=4096, ws_bytes=need - 1) == SHAPE


def test_injected_launch_failure(lib):
    lib.ternary_test_inject_launch_failures(1)
    try:
        assert lib.ternary_kv_read(cache(), A, 4, B, C, 1, None) == CUDA
    finally:
        lib.ternary_test_inject_launch_failures(0)


def test_binding_refuses():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        tl.rope(x, pos, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="fp16"):
        tl.rope(x.double(), pos, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="format"):
        tl.KVCache.empty("int2", 1, 16, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        tl.KVCache.empty("int8", 1, 16, 1, 64, device="cpu")
    codes, scale = torch.zeros(1, 1, 16, 64, dtype=torch.int8), torch.zeros(1, 1, 16)
    with pytest.raises(ValueError, match="codes"):
        tl.KVCache("fp8", codes, codes, scale, scale)
    with pytest.raises(ValueError, match="scales"):
        tl.KVCache("int8", codes, codes, scale.double(), scale)
    with pytest.raises(ValueError, match="CUDA"):
        tl.rope_table(4, 64, device="cpu")
