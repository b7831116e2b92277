"""Host-side refusals of the low-rank adapters (no GPU, nothing is launched)."""
import ctypes

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import lora

OK, NULL, SHAPE, DTYPE, ALIGN, VALUE, CUDA = 0, 1, 2, 3, 4, 5, 6
A, B, C, D, E, F, G = (0x10000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    tl.build()
    tl.load()
    return lora._lib()


def adapters(a=A, b=B, scale=C, inputs=64, rows=(32, 32), shards=None, rank=16, n=3, dtype=1):
    rows = tuple(rows) + (0,) * (8 - len(rows))
    return lora._Adapters(a, b, scale, inputs, (ctypes.c_int64 * 8)(*rows), 2 if shards is None else shards, rank, n, dtype)


@pytest.mark.parametrize("gate", [False, True])
def test_refusals(lib, gate):
    f = lib.ternary_lora_silu_mul if gate else lib.ternary_lora_add

    def call(ad=None, x=D, xs=64, which=E, y=F, ys=64, out=G, os=64, odt=1, m=5, ws=None, size=0):
        return f(x, xs, ctypes.byref(ad or adapters()), which, y, ys, out, os, odt, m, ws, size, None)

    assert f(D, 64, None, E, F, 64, G, 64, 1, 5, None, 0, None) == NULL
    assert call(ad=adapters(dtype=2)) == DTYPE and call(odt=0) == DTYPE and call(odt=3) == DTYPE
    for bad in (dict(n=0), dict(n=2049), dict(shards=0), dict(shards=9), dict(rank=0), dict(rank=12), dict(rank=136), dict(inputs=0),
                dict(inputs=1 << 25), dict(rows=(-8, 8)), dict(rows=(1 << 25, 1 << 25))):
        assert call(ad=adapters(**bad)) == SHAPE
    assert call(m=-1) == SHAPE and call(m=1 << 30) == SHAPE and call(xs=1 << 41) == SHAPE and call(os=-(1 << 41)) == SHAPE
    for name in ("x", "which", "y", "out"):
        assert call(**{name: None}) == NULL
    assert call(ad=adapters(a=None)) == NULL and call(ad=adapters(b=None)) == NULL
    assert call(ad=adapters(a=A + 8)) == ALIGN and call(ad=adapters(b=B + 2)) == ALIGN and call(ad=adapters(scale=C + 2)) == ALIGN
    assert call(x=D + 1) == ALIGN and call(which=E + 2) == ALIGN and call(y=F + 1) == ALIGN and call(out=G + 2, odt=2) == ALIGN
    assert call(out=F, os=72) == VALUE                       # in place with another stride
    assert call(m=1025) == NULL and call(m=1025, ws=A, size=16) == SHAPE and call(m=1025, ws=A + 8, size=1 << 20) == ALIGN
    assert call(m=0, x=None) == OK and call(ad=adapters(rows=(0, 0)), y=None) == OK
    if gate:
        assert call(ad=adapters(rows=(32, 24))) == SHAPE and call(ad=adapters(rows=(32,), shards=1)) == SHAPE
        assert call(out=F) == VALUE
    lib.ternary_test_inject_launch_failures(2)
    try:
        assert call() == CUDA and call(ad=adapters(scale=None)) == CUDA
    finally:
        lib.ternary_test_inject_launch_failures(0)


def test_workspace(lib):
    w = lib.ternary_lora_workspace
    assert w(-1, 1) == -1 and w(1, 0) == -1 and w(1, 2049) == -1 and w(1 << 30, 1) == -1
    assert w(0, 1) == 0 and w(1024, 1024) == 0 and w(1, 1025) > 0
    # the tokens, and three numbers for each tile that there can be
    assert w(8192, 6) >= 4 * (8192 + 3 * (8192 // 16 + 6))


def test_binding_refuses():
    a, b = torch.zeros(2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 32, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tl.Adapters(a, b)
    with pytest.raises(ValueError, match="fp16"):
        tl.Adapters(a.float(), b.float())
    with pytest.raises(ValueError, match="rank rows"):
        tl.Adapters(a, b, shards=(16, 16))
    with pytest.raises(ValueError, match="add up"):
        tl.Adapters(a, b, shards=(16, 8))
    with pytest.raises(ValueError, match="multiple of 8"):
        tl.Adapters(torch.zeros(2, 12, 64).half(), torch.zeros(2, 32, 12).half())
    with pytest.raises(ValueError, match="contiguous"):
        tl.Adapters(a, b.transpose(1, 2))
