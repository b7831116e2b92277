"""Rotary positions against fp64: the table, the rotation of every layout, dtype, rotated
width and alignment, its inverse as its gradient, and what an index out of range does."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from attn_ref import U, rotate, table64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def check(got, x, rows, interleaved, inverse=False):
    """Three fp32 roundings of terms bounded by |a| + |b|, then one to the output type."""
    want = rotate(x.double().cpu(), rows.double().cpu(), interleaved, inverse)
    r = rows.shape[1]
    mag = rotate(x.double().cpu().abs(), torch.ones(x.shape[0], r, dtype=torch.float64), interleaved)
    m = mag.abs()
    if interleaved:
        m[..., 0:r:2] = m[..., 1:r:2]
    else:
        m[..., :r // 2] = m[..., r // 2:r]
    bound = U[x.dtype] * want.abs() + 2.0 ** -23 * m * rows.double().cpu().abs().max() + 2.0 ** -25
    err = (got.double().cpu() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(factor=4.0),
                                dict(factor=8.0, original_len=4096, ramp=(1.0, 32.0), magnitude=1.2),
                                dict(factor=2.0, original_len=100, ramp=(3.0, 3.0))])
def test_table(kw):
    got = tl.rope_table(70001, 64, **kw).double().cpu()
    want = table64(70001, 64, **kw)
    # an angle of p f radians in fp64 is off by a few 2^-53 of itself; the entry is rounded once
    assert ((got - want).abs() <= 2.0 ** -24 * want.abs() + 70001 * 2.0 ** -48).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,h,d,r", [(1, 32, 128, 128), (5, 3, 128, 64), (1, 1, 64, 16), (37, 7, 96, 96),
                                     (3, 2, 80, 32), (4, 5, 64, 62), (2, 3, 17, 6), (300, 1, 256, 256), (2, 1, 2, 2)])
def test_rotation(dtype, interleaved, n, h, d, r):
    g = torch.Generator(device=DEV).manual_seed(n * 1000 + d)
    x = torch.randn(n, h, d, generator=g, device=DEV).to(dtype)
    table = tl.rope_table(5000, r)
    pos = torch.randint(0, 5000, (n,), generator=g, device=DEV)
    pos[0] = 4999
    for inverse in (False, True):
        check(tl.rope(x, pos, table, interleaved=interleaved, inverse=inverse), x, table[pos], interleaved, inverse)


@pytest.mark.parametrize("shift,pad", [(0, 8), (0, 3), (1, 0), (4, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_offsets_and_in_place(shift, pad, interleaved):
    n, h, d = 9, 5, 64
    row = h * d + pad
    flat = torch.randn(n * row + shift + 8, device=DEV).to(torch.bfloat16)
    x = flat[shift:shift + n * row].view(n, row)[:, :h * d].unflatten(1, (h, d))
    table = tl.rope_table(100, 32)
    pos = torch.arange(n, device=DEV) * 7
    before = flat.clone()
    want = tl.rope(x.contiguous(), pos, table, interleaved=interleaved)
    check(want, x, table[pos], interleaved)
    assert torch.equal(tl.rope(x, pos, table, interleaved=interleaved), want)
    byhead = x.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost
    assert torch.equal(tl.rope(byhead, pos, table, interleaved=interleaved), want)
    assert tl.rope(x, pos, table, interleaved=interleaved, out=x) is x
    assert torch.equal(x, want)
    back = torch.ones_like(flat, dtype=torch.bool)
    back[shift:shift + n * row].view(n, row)[:, :h * d] = False
    assert torch.equal(flat[back], before[back])  # nothing beside the heads was touched


def test_inverse_is_the_gradient():
    n, h, d = 4, 3, 32
    x, w = (torch.randn(n, h, d, device=DEV) for _ in range(2))
    table = tl.rope_table(1000, 16, magnitude=1.3)
    pos = torch.tensor([0, 1, 500, 999], device=DEV)
    for inter in (False, True):
        grad = tl.rope(w, pos, table, interleaved=inter, inverse=True).double()
        # the map is linear: central differences have no truncation error, and with a step of 1
        # only the fp32 rounding of outputs (each below 8) and of the sum
        for e in ((0, 0, 0), (1, 2, 7), (2, 1, 8), (3, 0, 15), (3, 2, 31)):
            step = torch.zeros_like(x)
            step[e] = 1.0
            up, down = (tl.rope(x + s * step, pos, table, interleaved=inter).double() for s in (1, -1))
            diff = float(((up - down) / 2 * w.double()).sum())
            assert abs(diff - float(grad[e])) <= 4 * 8 * 2.0 ** -23 * 2 * float(w.abs().max() + 1)
        y = tl.rope(tl.rope(x, pos, table, interleaved=inter), pos, table, interleaved=inter, inverse=True)
        y[..., :16] /= 1.3 ** 2
        assert (y - x).abs().max() <= 2.0 ** -20 * x.abs().max()


def test_empty_and_out_of_range():
    table = tl.rope_table(10, 64)
    x = torch.randn(3, 2, 64, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    assert tl.rope(x[:0], none, table).shape == (0, 2, 64)
    assert tl.rope(x[:, :0], none.new_zeros(3), table).shape == (3, 0, 64)
    for d in (64, 62):  # the vector and the plain form
        xs = x[..., :d].contiguous()
        tb = tl.rope_table(10, d)
        out = torch.full_like(xs, 5.0)
        tl.rope(xs, torch.tensor([3, 10, -1], device=DEV), tb, out=out)
        torch.cuda.synchronize()
        assert tl.device_status(clear=True) == 5
        assert torch.equal(out[1:], torch.full_like(out[1:], 5.0))
        assert torch.equal(out[0], tl.rope(xs[:1], torch.tensor([3], device=DEV), tb)[0])


def test_other_stream_and_graph():
    x = torch.randn(64, 8, 128, device=DEV, dtype=torch.float16)
    table = tl.rope_table(64, 128)
    pos = torch.arange(64, device=DEV)
    want = tl.rope(x, pos, table)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = tl.rope(x, pos, table)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.rope(x, pos, table, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
