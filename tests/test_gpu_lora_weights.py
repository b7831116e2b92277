"""Infinities and NaN in an adapter's matrices: they stay with the tokens of that adapter, those of b in their column."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from test_gpu_lora import make

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")

# tokens, inputs, columns, rank, types: tiles of 16 by whole blocks of columns and by any, and tiles of 128
SIZES = [(40, 256, 128, 16, "bf", "bf"), (40, 256, 100, 16, "h", "h"), (40, 256, 128, 40, "bf", "f"), (300, 64, 128, 32, "h", "f"),
         (2304, 264, 136, 40, "bf", "bf"), (2304, 264, 136, 40, "h", "h"), (2304, 9600, 136, 40, "bf", "f"), (2304, 9600, 136, 40, "h", "f")]
KIND = {"bf": torch.bfloat16, "h": torch.float16, "f": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def case(tokens, inputs, columns, rank, kind, out):
    x, y, a, b, s, which = make(tokens, inputs, (columns,), rank, 3, KIND[kind], KIND[out], seed=tokens + columns)
    which[0], which[1], which[2] = 0, 1, -1
    return x, y, a, b, s, which, tl.lora_add(x, tl.Adapters(a, b, s), which, y)


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("size", SIZES)
def test_b(size, value):
    x, y, a, b, s, which, clean = case(*size)
    b[1, 7, 3] = value
    got = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[which == 1, 7] = True
    assert torch.equal(got[~hit], clean[~hit]) and not torch.isfinite(got[hit]).any()


@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("size", SIZES)
def test_a(size, value):
    x, y, a, b, s, which, clean = case(*size)
    a[1, 5, 11] = value
    got = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    assert torch.equal(got[which != 1], clean[which != 1])
    assert not torch.isfinite(got[which == 1]).all(1).any()


@pytest.mark.parametrize("size", SIZES)
def test_scales(size):
    """A scale of 0, and one that is no number."""
    x, y, a, b, s, which, clean = case(*size)
    s[1], s[2] = 0.0, NAN
    got = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    assert torch.equal(got[which <= 0], clean[which <= 0]) and torch.equal(got[which == 1], y[which == 1])
    assert torch.isnan(got[which == 2]).all()


@pytest.mark.parametrize("rank", [16, 24])
def test_b_of_a_gated_layer(rank):
    x, y, a, b, s, which = make(60, 256, (96, 96), rank, 3, torch.bfloat16, torch.bfloat16, seed=1)
    which[0] = 1
    clean = tl.lora_silu_mul(x, tl.Adapters(a, b, s, shards=(96, 96)), which, y)
    b[1, 96 + 7, 3] = INF
    got = tl.lora_silu_mul(x, tl.Adapters(a, b, s, shards=(96, 96)), which, y)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[which == 1, 7] = True
    assert torch.equal(got[~hit], clean[~hit]) and not torch.isfinite(got[hit]).any()
