"""Low-rank adapters on the GPU against the formula in 64 bits.

Bound of one element before its rounding.  The shrink's sum of K exact products in fp32, added in some order and
scaled: off by at most (K + 2) 2^-24 s sum |a||x|.  Split into 16-bit numbers it keeps 2^-17 of itself (2^-16 in
the bound: the first number's half step, 2^-9 for bf16, times the second's), 2^-22 (2^-21) for f16 and where bf16 feeds
fp32; f16 numbers below 2^-24 of a row's largest (scaled to 2^14 at least) are rounded at 2^-39 of it.  The second
sum of up to 3 R products and y: (3 R + 2) 2^-24 (|y| + sum |b||h|).  Tensor cores may cut off what falls below
the largest term of a step instead of rounding: each 2^-24 above is counted as 2^-23."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

pytestmark = pytest.mark.gpu
DEV = "cuda"
VALUE = 5
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def make(tokens, inputs, shards, rank, n, dtype, out_dtype, seed=0, scale=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    total = sum(shards)
    x = torch.randn(tokens, inputs, generator=gen, device=DEV).to(dtype)
    y = torch.randn(tokens, total, generator=gen, device=DEV).to(out_dtype)
    a = (torch.randn(n, len(shards) * rank, inputs, generator=gen, device=DEV) * inputs ** -0.5).to(dtype)
    b = (torch.randn(n, total, rank, generator=gen, device=DEV) * rank ** -0.5).to(dtype)
    s = 0.25 + torch.rand(n, generator=gen, device=DEV) if scale else None
    which = torch.randint(-1, n, (tokens,), generator=gen, device=DEV).int()
    return x, y, a, b, s, which


def exact(x, y, a, b, s, which, shards):
    """z = y + product, and the bound of z, in 64 bits."""
    z, off = y.double(), torch.zeros_like(y, dtype=torch.float64)
    rank, k = b.shape[2], x.shape[1]
    fine = x.dtype is torch.float16 or y.dtype is torch.float32
    e, u = 2.0 ** -23, 2.0 ** -21 if fine else 2.0 ** -16
    off += e * z.abs() * (3 * rank + 2)
    for i in range(a.shape[0]):
        rows = (which == i).nonzero()[:, 0]
        if not len(rows):
            continue
        xi, w, at = x[rows].double(), float(s[i]) if s is not None else 1.0, 0
        hs = [w * xi @ a[i, j * rank:(j + 1) * rank].double().T for j in range(len(shards))]
        mags = [abs(w) * xi.abs() @ a[i, j * rank:(j + 1) * rank].double().abs().T for j in range(len(shards))]
        top = torch.stack([m.amax(1) for m in mags]).amax(0)[:, None]
        for j, n in enumerate(shards):
            bj = b[i, at:at + n].double()
            z[rows, at:at + n] += hs[j] @ bj.T
            dh = (k + 2) * e * mags[j] + u * (hs[j].abs() + (k + 2) * e * mags[j]) + 2.0 ** -38 * top
            off[rows, at:at + n] += dh @ bj.abs().T + (3 * rank + 2) * e * (hs[j].abs() @ bj.abs().T)
            at += n
    return z, off


def close(got, z, off, what=""):
    u = U[got.dtype]
    bound = off * (1 + u) + u * z.abs() + 2.0 ** -24 * (got.dtype is torch.float16)
    err = (got.double() - z).abs()
    assert torch.isfinite(got).all(), what
    assert (err <= bound).all(), f"{what}: {float((err / bound.clamp(min=1e-300)).max()):.3g} of the bound"


def gated(z, off, half, dtype):
    """silu(g) u and its bound: |silu'| < 1.1; division and products 2^-21, as the exponential for fp32 outputs; for 16-bit
    ones that is off by 2 + 1.173 |g| units of 2^-23, |g| below 88 (beyond, the result is below 2^-119): 2^-16."""
    g, u = z[:, :half], z[:, half:]
    h = g * torch.sigmoid(g)
    dg, du = off[:, :half], off[:, half:]
    return h * u, 1.1 * dg * (u.abs() + du) + h.abs() * du + 2.0 ** (-21 if dtype is torch.float32 else -16) * (h * u).abs()


CASES = [  # tokens, inputs, shards, rank, adapters
    (1, 64, (32,), 8, 1), (1, 3584, (3584, 512, 512), 16, 3), (16, 1024, (1024,), 16, 8), (7, 200, (40, 8, 24), 24, 2),
    (33, 1000, (72, 56), 32, 5), (64, 4096, (256,), 64, 64), (100, 264, (96,), 128, 3), (257, 512, (320,), 16, 2),
    (300, 2048, (128, 64), 64, 4), (1024, 256, (64,), 8, 700), (1025, 256, (64,), 8, 3), (3001, 320, (104,), 16, 40),
    (2000, 96, (32,) * 8, 128, 7), (2048, 9000, (256, 96, 100), 64, 3), (2100, 9000, (3500,), 32, 2),
    (1500, 15000, (64,) * 5, 24, 4), (700, 136, (24, 8) * 4, 24, 5), (500, 4096, (48, 16, 16), 64, 2), (129, 8, (40,), 16, 1), (90, 72, (16,), 8, 2000), (1, 8, (8,), 8, 1)]


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
                                             (torch.float16, torch.float32)])
@pytest.mark.parametrize("tokens,inputs,shards,rank,n", CASES)
def test_add(tokens, inputs, shards, rank, n, dtype, out_dtype):
    x, y, a, b, s, which = make(tokens, inputs, shards, rank, n, dtype, out_dtype, seed=tokens + inputs)
    ad = tl.Adapters(a, b, s, shards=shards)
    got = tl.lora_add(x, ad, which, y)
    z, off = exact(x, y, a, b, s, which, shards)
    close(got, z, off)
    none = which < 0
    assert torch.equal(got[none], y[none])
    again = y.clone()
    assert tl.lora_add(x, ad, which, again, out=again) is again and torch.equal(again, got)


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("tokens,inputs,half,rank,n", [(1, 512, 1024, 16, 1), (16, 3584, 2000, 8, 9), (50, 136, 24, 32, 3), (300, 256, 96, 16, 4),
                                                       (1500, 128, 40, 64, 5), (77, 100, 33, 16, 2), (60, 256, 64, 32, 2)])
def test_silu_mul(tokens, inputs, half, rank, n, dtype, out_dtype):
    x, y, a, b, s, which = make(tokens, inputs, (half, half), rank, n, dtype, out_dtype, seed=half)
    got = tl.lora_silu_mul(x, tl.Adapters(a, b, s, shards=(half, half)), which, y)
    z, off = exact(x, y, a, b, s, which, (half, half))
    close(got, *gated(z, off, half, out_dtype))


@pytest.mark.parametrize("tokens,inputs,shards", [(5, 33, (7,)), (40, 129, (31, 1, 12)), (130, 250, (18,))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_odd_sizes(tokens, inputs, shards, dtype):
    """Rows that start anywhere: sizes that are no multiple of eight."""
    x, y, a, b, s, which = make(tokens, inputs, shards, 16, 2, dtype, dtype, seed=9)
    close(tl.lora_add(x, tl.Adapters(a, b, s, shards=shards), which, y), *exact(x, y, a, b, s, which, shards))


def test_strides():
    """x, y and out as views of wider tensors, at even and odd offsets, and leading dimensions."""
    x, y, a, b, s, which = make(48, 128, (64, 32), 16, 5, torch.bfloat16, torch.bfloat16, seed=2)
    ad = tl.Adapters(a, b, s, shards=(64, 32))
    want = tl.lora_add(x, ad, which, y)
    for shift in (0, 8, 3):
        wx, wy, wo = (torch.zeros(48, 160 + shift, dtype=torch.bfloat16, device=DEV) for _ in range(3))
        wx[:, shift:shift + 128], wy[:, shift:shift + 96] = x, y
        out = wo[:, shift:shift + 96]
        tl.lora_add(wx[:, shift:shift + 128], ad, which, wy[:, shift:shift + 96], out=out)
        assert torch.equal(out, want)
        assert float(wo[:, :shift].float().abs().sum()) == 0 and float(wo[:, shift + 96:].float().abs().sum()) == 0
    three = tl.lora_add(x.view(4, 12, 128), ad, which.view(4, 12), y.view(4, 12, 96))
    assert three.shape == (4, 12, 96) and torch.equal(three.view(48, 96), want)
    assert torch.equal(tl.lora_add(x.t().contiguous().t(), ad, which, y), want)
    assert tl.lora_add(x[:0], ad, which[:0], y[:0]).shape == (0, 96)


@pytest.mark.parametrize("tokens,inputs,n", [(40, 512, 3), (900, 512, 4), (5000, 512, 3), (4100, 14000, 3)])
def test_runs_and_orders(tokens, inputs, n):
    """A token's result does not hang on where it stands or on what else is in the batch with tiles of one size."""
    x, y, a, b, s, _ = make(tokens, inputs, (96,), 16, n, torch.bfloat16, torch.bfloat16, seed=tokens)
    gen = torch.Generator(device=DEV).manual_seed(1)
    cuts = torch.randint(0, tokens, (n,), generator=gen, device=DEV).sort().values
    which = torch.searchsorted(cuts, torch.arange(tokens, device=DEV), right=True).int() - 1
    ad = tl.Adapters(a, b, s)
    got = tl.lora_add(x, ad, which, y)
    close(got, *exact(x, y, a, b, s, which, (96,)))
    order = torch.randperm(tokens, generator=gen, device=DEV)
    mixed = tl.lora_add(x[order], ad, which[order], y[order])
    assert torch.equal(mixed, got[order])
    for _ in range(3):
        assert torch.equal(tl.lora_add(x, ad, which, y), got)


def test_no_scale_and_only_one_adapter_in_use():
    x, y, a, b, _, which = make(200, 256, (128,), 32, 50, torch.float16, torch.float16, seed=6, scale=False)
    which.fill_(37)
    close(tl.lora_add(x, tl.Adapters(a, b), which, y), *exact(x, y, a, b, None, which, (128,)))
    which.fill_(-1)
    assert torch.equal(tl.lora_add(x, tl.Adapters(a, b), which, y), y)


@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** -14])
def test_large_and_small_products_in_f16(size):
    """h far outside f16's range, brought back by b: the split's scale carries it."""
    x, y, a, b, s, which = make(20, 512, (64,), 16, 2, torch.float16, torch.float16, seed=8)
    x = (x * (32.0 if size > 1 else 2.0 ** -9)).half()
    a = (a * (512.0 if size > 1 else 2.0 ** -5)).half()
    b = (b / size).half() if size > 1 else (b * 512).half()
    y = torch.zeros_like(y)
    z, off = exact(x, y, a, b, s, which, (64,))
    assert float(z.abs().max()) < 60000
    close(tl.lora_add(x, tl.Adapters(a, b, s), which, y), z, off)


def test_values_that_are_no_numbers_stay_in_their_rows():
    x, y, a, b, s, which = make(70, 256, (64,), 16, 2, torch.bfloat16, torch.bfloat16, seed=4)
    which = (torch.arange(70, device=DEV) % 2).int()
    ad = tl.Adapters(a, b, s)
    want = tl.lora_add(x, ad, which, y)
    bad = x.clone()
    bad[3, 5], bad[10, 0] = float("nan"), float("inf")
    got = tl.lora_add(bad, ad, which, y)
    keep = torch.ones(70, dtype=torch.bool, device=DEV)
    keep[3] = keep[10] = False
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[10]).any()


@pytest.mark.parametrize("tokens", [30, 2000])
def test_adapters_out_of_range(tokens):
    """A number beyond the adapters is none, and sets the status word."""
    x, y, a, b, s, which = make(tokens, 128, (64,), 16, 3, torch.bfloat16, torch.bfloat16, seed=3)
    which[5], which[tokens - 1], which[9] = 3, 1 << 30, -(1 << 31)
    got = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    assert tl.device_status() == VALUE
    inside = torch.where((which >= 0) & (which < 3), which, -1)
    close(got, *exact(x, y, a, b, s, inside, (64,)))
    assert torch.equal(got[inside < 0], y[inside < 0])


@pytest.mark.parametrize("tokens,inputs", [(16, 256), (1500, 256), (2000, 30000)])
def test_replayed_with_other_adapters(tokens, inputs):
    x, y, a, b, s, which = make(tokens, inputs, (96,), 16, 6, torch.bfloat16, torch.bfloat16, seed=5)
    ad = tl.Adapters(a, b, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tl.lora_add(x, ad, which, y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tl.lora_add(x, ad, which, y)
    gen = torch.Generator(device=DEV).manual_seed(7)
    for i in range(5):
        which.copy_(torch.randint(-1, 6, (tokens,), generator=gen, device=DEV) if i else torch.full((tokens,), 2))
        x.normal_(generator=gen)
        graph.replay()
        close(got, *exact(x, y, a, b, s, which, (96,)))


def test_after_the_shared_layer():
    """The layer and its adapters on one stream, as they are used: equal to the sum of the two."""
    from ternary_weight_linear_02_gb300 import synth
    m, k, shards = 24, 512, (256, 64, 64)
    x, _, a, b, s, which = make(m, k, shards, 16, 4, torch.bfloat16, torch.bfloat16, seed=12)
    w = synth.packed_codes(sum(shards), k, 5, DEV)
    sc = synth.scales(sum(shards), 0, 0.005, 0.05, 6, DEV)
    y = tl.linear(x, w, sc, 0, out_dtype=torch.float32)
    ad = tl.Adapters(a, b, s, shards=shards)
    keep = y.clone()
    tl.lora_add(x, ad, which, y, out=y)
    close(y, *exact(x, keep, a, b, s, which, shards))


MANY = [  # tokens, inputs, shards, rank, adapters: tiles of 128 tokens, from one block a tile to eight, columns cut short
    (2048, 520, (264, 96, 104), 64, 3), (2304, 328, (72,), 40, 4), (2048, 17408, (40, 16), 8, 2), (1300, 6800, (64, 8, 72, 136), 16, 4),
    (2100, 264, (128, 40, 0, 24), 48, 5), (5000, 72, (200,), 32, 6), (9000, 72, (72,), 56, 5), (16000, 40, (136, 8), 32, 4), (20000, 40, (72,), 32, 4),
    (2048, 8, (8,), 32, 1), (3000, 3000, (1000,), 64, 24), (2300, 30000, (104, 72), 64, 3)]


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
                                             (torch.float16, torch.float32)])
@pytest.mark.parametrize("tokens,inputs,shards,rank,n", MANY)
def test_many_tokens(tokens, inputs, shards, rank, n, dtype, out_dtype):
    x, y, a, b, s, which = make(tokens, inputs, shards, rank, n, dtype, out_dtype, seed=tokens + rank)
    ad = tl.Adapters(a, b, s, shards=shards)
    z, off = exact(x, y, a, b, s, which, shards)
    got = tl.lora_add(x, ad, which, y)
    close(got, z, off)
    assert torch.equal(got[which < 0], y[which < 0])
    wide = torch.full((tokens, y.shape[1] + 24), 3.0, dtype=out_dtype, device=DEV)  # rows of a larger tensor, in place
    part = wide[:, 8:-16]
    part.copy_(y)
    tl.lora_add(x, ad, which, part, out=part)
    assert torch.equal(part, got) and bool((wide[:, :8] == 3).all()) and bool((wide[:, -16:] == 3).all())


def test_values_that_are_no_numbers_stay_in_their_rows_of_large_tiles():
    tokens, k = 2304, 264
    x, y, a, b, s, which = make(tokens, k, (136,), 40, 3, torch.float16, torch.float16, seed=33)
    clean = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    x[7, 3], x[300, 5], y[11, 4] = float("inf"), float("nan"), float("nan")
    got = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    odd = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    odd[7], odd[300], odd[11] = True, True, True
    assert torch.equal(got[~odd], clean[~odd])
    for row in (7, 300):
        if int(which[row]) >= 0:
            assert not torch.isfinite(got[row]).all()
    assert torch.isnan(got[11, 4]) and torch.equal(got[11, 5:], clean[11, 5:])


@pytest.mark.parametrize("share", [0.0, 0.1, 0.45, 0.55, 0.95, 1.0])
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
def test_tokens_without_an_adapter_among_many(share, out_dtype):
    """From none of them to all: their rows are copied, beside the others' or by themselves, or left as they are."""
    tokens, shards = 3100, (136, 48)
    x, y, a, b, s, which = make(tokens, 72, shards, 48, 3, torch.float16, out_dtype, seed=77)
    gen = torch.Generator(device=DEV).manual_seed(5)
    which = torch.randint(0, 3, (tokens,), generator=gen, device=DEV).int()
    which[torch.rand(tokens, generator=gen, device=DEV) < share] = -1
    ad = tl.Adapters(a, b, s, shards=shards)
    got = tl.lora_add(x, ad, which, y, out=torch.full_like(y, float("nan")))
    close(got, *exact(x, y, a, b, s, which, shards))
    assert torch.equal(got[which < 0], y[which < 0])
    tl.lora_add(x, ad, which, y, out=y)
    assert torch.equal(y, got)
