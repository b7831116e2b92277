"""Adapters whose numbers are written by another stream during the call: the answers are then of no use, but nothing outside of
the call's own tensors is touched, the call returns, and the next one is right."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import attention, lora

from test_gpu_lora import close, exact, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("tokens", [9000, 60000])
def test_the_plan_stays_in_its_workspace(tokens):
    """More tokens than the plan keeps from its first look (8192): counted under one number, placed under another, they would
    lie behind the last token's place."""
    n, guard = 5, 4 * tokens + 4096
    x, y, a, b, s, which = make(tokens, 64, (40,), 16, n, torch.bfloat16, torch.bfloat16, seed=1)
    ad, lib = tl.Adapters(a, b, s), lora._lib()
    need = lib.ternary_lora_workspace(tokens, n)
    ws = torch.full((need + guard,), 0x5A, dtype=torch.uint8, device=DEV)
    out, other, calm = torch.empty_like(y), torch.cuda.Stream(), which.clone()
    torch.cuda.synchronize()
    for _ in range(30):
        with torch.cuda.stream(other):
            for _ in range(10):
                which.fill_(0)
                which.fill_(n - 1)
                which.fill_(-1)
        for _ in range(5):
            rc = lib.ternary_lora_add(x.data_ptr(), 64, ad._ref, which.data_ptr(), y.data_ptr(), 40, out.data_ptr(), 40, 1, tokens, ws.data_ptr(),
                                      need, attention._stream(ad.device))
            assert rc == 0
        torch.cuda.synchronize()
    assert bool((ws[need:] == 0x5A).all())
    assert tl.device_status() == 0
    close(tl.lora_add(x, ad, calm, y), *exact(x, y, a, b, s, calm, (40,)))
