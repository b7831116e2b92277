"""fp32 outputs of many tokens, in tiles of 128 (h in three numbers of bf16 or two of f16, blocks of 32 columns), against the formula in
64 bits; bounds as in test_gpu_lora.py."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from lora_forms import MANY32, tile
from test_gpu_lora import close, exact, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,inputs,shards,rank,n", MANY32)
def test_many_tokens(tokens, inputs, shards, rank, n, dtype):
    assert tile(tokens, inputs, shards, rank, n, dtype, torch.float32) == 128
    x, y, a, b, s, which = make(tokens, inputs, shards, rank, n, dtype, torch.float32, seed=tokens + rank)
    ad = tl.Adapters(a, b, s, shards=shards)
    got = tl.lora_add(x, ad, which, y, out=torch.full_like(y, float("nan")))
    close(got, *exact(x, y, a, b, s, which, shards))
    assert torch.equal(got[which < 0], y[which < 0])
    wide = torch.full((tokens, y.shape[1] + 24), 3.0, device=DEV)  # rows of a larger tensor, in place
    part = wide[:, 8:-16]
    part.copy_(y)
    tl.lora_add(x, ad, which, part, out=part)
    assert torch.equal(part, got) and bool((wide[:, :8] == 3).all()) and bool((wide[:, -16:] == 3).all())


@pytest.mark.parametrize("share", [0.0, 0.1, 0.5, 0.95, 1.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tokens_without_an_adapter_among_many(share, dtype):
    """From none of them to all, the last as tiles that have no adapter at all."""
    tokens, inputs, shards = 3100, 3008, (136, 48)
    assert tile(tokens, inputs, shards, 48, 3, dtype, torch.float32) == 128
    x, y, a, b, s, which = make(tokens, inputs, shards, 48, 3, dtype, torch.float32, seed=77)
    gen = torch.Generator(device=DEV).manual_seed(5)
    which = torch.randint(0, 3, (tokens,), generator=gen, device=DEV).int()
    which[torch.rand(tokens, generator=gen, device=DEV) < share] = -1
    ad = tl.Adapters(a, b, s, shards=shards)
    got = tl.lora_add(x, ad, which, y, out=torch.full_like(y, float("nan")))
    close(got, *exact(x, y, a, b, s, which, shards))
    assert torch.equal(got[which < 0], y[which < 0])
    tl.lora_add(x, ad, which, y, out=y)
    assert torch.equal(y, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_that_are_no_numbers_stay_in_their_rows(dtype):
    tokens, inputs, shards, rank = 2304, 9552, (136,), 40
    assert tile(tokens, inputs, shards, rank, 3, dtype, torch.float32) == 128
    x, y, a, b, s, which = make(tokens, inputs, shards, rank, 3, dtype, torch.float32, seed=33)
    which[7] = which[300] = 1
    clean = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    x[7, 3], x[300, 9000], y[11, 4] = float("inf"), float("nan"), float("nan")
    got = tl.lora_add(x, tl.Adapters(a, b, s), which, y)
    odd = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    odd[7], odd[300], odd[11] = True, True, True
    assert torch.equal(got[~odd], clean[~odd])
    assert not torch.isfinite(got[7]).any() and torch.isnan(got[300]).all()
    assert torch.isnan(got[11, 4]) and torch.equal(got[11, 5:], clean[11, 5:])


def test_replayed():
    tokens, inputs, n = 2048, 30000, 6
    assert tile(tokens, inputs, (96,), 16, n, torch.bfloat16, torch.float32) == 128
    x, y, a, b, s, which = make(tokens, inputs, (96,), 16, n, torch.bfloat16, torch.float32, seed=5)
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
    for i in range(3):
        which.copy_(torch.randint(-1, n, (tokens,), generator=gen, device=DEV) if i else torch.full((tokens,), 2))
        graph.replay()
        close(got, *exact(x, y, a, b, s, which, (96,)))
