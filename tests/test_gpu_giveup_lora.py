"""The waits of the adapters' tcgen05 form run out: the call returns, says so, gives NaN, and leaves the device usable."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tokens,inputs,n", [(1100, 92000, 2), (3000, 37000, 5)])
def test_a_wait_that_runs_out(tokens, inputs, n):
    tl.build()
    lib = tl.load()
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(tokens, inputs, generator=gen, device=DEV).bfloat16()
    y = torch.randn(tokens, 96, generator=gen, device=DEV).bfloat16()
    a = (0.01 * torch.randn(n, 16, inputs, generator=gen, device=DEV)).bfloat16()
    b = torch.randn(n, 96, 16, generator=gen, device=DEV).bfloat16()
    which = torch.randint(-1, n, (tokens,), generator=gen, device=DEV).int()
    ad = tl.Adapters(a, b)
    want = tl.lora_add(x, ad, which, y)
    torch.cuda.synchronize()
    try:
        lib.ternary_test_set_wait_limit(100000, 1)
        got = tl.lora_add(x, ad, which, y)
        torch.cuda.synchronize()
    finally:
        lib.ternary_test_set_wait_limit(0, 0)
    assert tl.device_status() == 7  # TL_ERR_TIMEOUT
    assert torch.isnan(got[which >= 0]).all() and torch.equal(got[which < 0], y[which < 0])
    assert torch.equal(tl.lora_add(x, ad, which, y), want)
    torch.cuda.synchronize()
    assert tl.device_status() == 0
