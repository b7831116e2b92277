"""The gated product of adapted layers: gates of any size, infinities and NaN, types and ranks that the other cases leave out.

Bounds of silu(g) u, g and u given.  fp32 outputs: g / (1 + expf(-g)) with expf within 2 ulp, a sum, a quotient and a product within
half an ulp each: 2^-21 of the result (3.5 ulp of 2^-23), and where expf overflows (g below -88.7) 0 for what is less than 2^-121 |u|.
16-bit outputs: 2^-16 of the result and 2^-119 |u| (the kernel's comment), then half a step of the output."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from test_gpu_lora import U, close, exact, gated, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


KINDS = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, torch.float32), (torch.float16, torch.float32)]
SIZES = [(64, 16), (33, 16), (96, 24)]  # columns of a half, rank: whole blocks of columns, cut ones, a rank of the general form


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("half,rank", SIZES)
def test_gates_of_any_size(half, rank, dtype, out_dtype):
    """Adapters of zeros, so that y's halves reach the product as they are: gates from -110 to 110, factors from 2^-20 to 2^100 (f16: 2^9)."""
    tokens, n = 40, 3
    gen = torch.Generator(device=DEV).manual_seed(half)
    g = (torch.rand(tokens, half, generator=gen, device=DEV) * 220 - 110).to(out_dtype)
    g[0, :24] = torch.linspace(-89, -86, 24, device=DEV).to(out_dtype)
    g[1, :8] = torch.tensor([0.0, -0.0, 1e-5, -1e-5, 17.0, -17.0, 88.0, -88.0], device=DEV).to(out_dtype)
    top = 9 if out_dtype is torch.float16 else 100
    u = torch.exp2(torch.rand(tokens, half, generator=gen, device=DEV) * (top + 20) - 20).to(out_dtype)
    u[0] = 2.0 ** top
    a, b = torch.zeros(n, 2 * rank, 64, dtype=dtype, device=DEV), torch.randn(n, 2 * half, rank, generator=gen, device=DEV).to(dtype)
    x = torch.randn(tokens, 64, generator=gen, device=DEV).to(dtype)
    which = (torch.arange(tokens, device=DEV) % (n + 1) - 1).int()
    got = tl.lora_silu_mul(x, tl.Adapters(a, b, shards=(half, half)), which, torch.cat([g, u], 1)).double()
    gd, ud = g.double(), u.double()
    want = gd * torch.sigmoid(gd) * ud
    if out_dtype is torch.float32:
        off = 2.0 ** -21 * want.abs() + torch.where(gd < -88.7, 2.0 ** -121 * ud.abs(), 0.0) + 2.0 ** -149
    else:
        step = U[out_dtype]
        off = (2.0 ** -16 * want.abs() + torch.where(gd < -87, 2.0 ** -119 * ud.abs(), 0.0)) * (1 + step) + step * want.abs()
        off += 2.0 ** -25 if out_dtype is torch.float16 else 2.0 ** -134
    err = (got - want).abs()
    assert torch.isfinite(got).all() and bool((err <= off).all()), float((err / off).max())


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("half,rank", SIZES)
def test_infinities_and_nan_of_y(half, rank, dtype, out_dtype):
    """Each stays in its place, and is what the formula gives."""
    odd = [float("inf"), float("-inf"), float("nan"), 0.0, 2.0, -2.0]
    tokens = len(odd)
    y = torch.full((tokens, 2 * half), 1.0, dtype=out_dtype, device=DEV)
    for i, v in enumerate(odd):
        for j, w in enumerate(odd):
            y[i, j], y[i, half + j] = v, w
    gen = torch.Generator(device=DEV).manual_seed(2)
    a, b = torch.zeros(1, 2 * rank, 64, dtype=dtype, device=DEV), torch.randn(1, 2 * half, rank, generator=gen, device=DEV).to(dtype)
    which = torch.tensor([0, -1, 0, -1, 0, -1], dtype=torch.int32, device=DEV)
    for w in (which, -1 - which):
        got = tl.lora_silu_mul(torch.ones(tokens, 64, dtype=dtype, device=DEV), tl.Adapters(a, b, shards=(half, half)), w, y).double()
        g, u = y[:, :half].double(), y[:, half:].double()
        want = g * torch.sigmoid(g) * u
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        fine = want.isfinite()
        assert torch.equal(got[want.isinf()], want[want.isinf()])
        assert bool(((got - want)[fine].abs() <= 2.0 ** -6 * want[fine].abs()).all())


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("half,rank", SIZES)
def test_values_of_x_that_are_no_numbers_stay_in_their_rows(half, rank, dtype, out_dtype):
    x, y, a, b, s, which = make(50, 128, (half, half), rank, 3, dtype, out_dtype, seed=3)
    ad = tl.Adapters(a, b, s, shards=(half, half))
    want = tl.lora_silu_mul(x, ad, which, y)
    which[7], which[20], which[30] = 0, 1, -1
    want = tl.lora_silu_mul(x, ad, which, y)
    x[7, 3], x[20, 5], x[30, 1] = float("nan"), float("inf"), float("nan")
    got = tl.lora_silu_mul(x, ad, which, y)
    keep = torch.ones(50, dtype=torch.bool, device=DEV)
    keep[7] = keep[20] = False
    assert torch.equal(got[keep], want[keep])               # row 30 has no adapter: its x is not looked at
    assert torch.isnan(got[7]).all() and not torch.isfinite(got[20]).all()


@pytest.mark.parametrize("dtype,out_dtype", KINDS)
@pytest.mark.parametrize("tokens,inputs,half,rank,n", [(40, 256, 64, 16, 4), (33, 200, 48, 24, 3), (60, 136, 72, 40, 2), (20, 264, 64, 64, 2), (50, 512, 96, 128, 3),
                                                       (300, 256, 1000, 128, 2), (1100, 72, 64, 24, 3), (9, 72, 31, 128, 2), (200, 64, 128, 8, 2000)])
def test_types_and_ranks(tokens, inputs, half, rank, n, dtype, out_dtype):
    x, y, a, b, s, which = make(tokens, inputs, (half, half), rank, n, dtype, out_dtype, seed=half + rank)
    got = tl.lora_silu_mul(x, tl.Adapters(a, b, s, shards=(half, half)), which, y)
    z, off = exact(x, y, a, b, s, which, (half, half))
    close(got, *gated(z, off, half, out_dtype))
