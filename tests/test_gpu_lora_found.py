"""Tiles of 128 that each block finds by itself: up to 1024 tokens of few adapters over many inputs need no plan."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from lora_forms import tile
from test_gpu_lora import close, exact, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
                                             (torch.float16, torch.float32)])
@pytest.mark.parametrize("tokens,inputs,shards,rank,n", [(512, 110016, (72,), 16, 1), (1024, 72000, (40, 24), 16, 2), (777, 80000, (136,), 24, 1),
                                                         (1000, 60008, (8, 0, 48), 24, 1)])
def test_few_tokens_of_many_inputs(tokens, inputs, shards, rank, n, dtype, out_dtype):
    assert tile(tokens, inputs, shards, rank, n, dtype, out_dtype) == 128
    x, y, a, b, s, which = make(tokens, inputs, shards, rank, n, dtype, out_dtype, seed=tokens)
    ad = tl.Adapters(a, b, s, shards=shards)
    for _ in range(2):
        got = tl.lora_add(x, ad, which, y, out=torch.full_like(y, float("nan")))
        close(got, *exact(x, y, a, b, s, which, shards))
        assert torch.equal(got[which < 0], y[which < 0])
        which = which.sort().values                     # runs, in which a tile ends inside a warp's tokens
    which = torch.full_like(which, -1)
    assert torch.equal(tl.lora_add(x, ad, which, y, out=torch.full_like(y, float("nan"))), y)
    which[tokens - 1] = n                              # beyond the adapters: none, and said so
    assert torch.equal(tl.lora_add(x, ad, which, y), y) and tl.device_status() == 5


def test_one_token():
    """No leading dimension at all, and one."""
    x, y, a, b, s, which = make(1, 256, (96,), 16, 2, torch.bfloat16, torch.bfloat16, seed=1)
    ad = tl.Adapters(a, b, s)
    which[0] = 1
    want = tl.lora_add(x, ad, which, y)
    close(want, *exact(x, y, a, b, s, which, (96,)))
    got = tl.lora_add(x[0], ad, which[0], y[0])
    assert got.shape == (96,) and torch.equal(got, want[0])
    again = y[0].clone()
    assert tl.lora_add(x[0], ad, which[0], again, out=again) is again and torch.equal(again, want[0])
