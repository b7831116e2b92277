"""The tcgen05 attention kernel's bounded waits give up cleanly.

ternary_test_set_wait_limit makes the softmax warps of the next launches first wait on a barrier
that nothing arrives on, with a short give-up time, while copies, decoded tiles and products of
the first tiles are under way.  The wait runs out (no fault, no hang): the call returns, the
status word reads TL_ERR_TIMEOUT, no output is written (NaN where partial results were to be
joined), and the next normal call on the same device is correct with the status clear.
"""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

pytestmark = pytest.mark.gpu
DEV = "cuda"
TL_ERR_TIMEOUT = 7


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()
    yield
    tl.load().ternary_test_set_wait_limit(0, 0)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,t,context,wide", [(1, 17, 0, 8),        # one tile, a block per unit
                                                  (160, 20, 300, 32),   # more blocks than fit at once
                                                  (3, 40, 3000, 256),   # dealt to blocks and joined
                                                  (2, 300, 900, 256)])  # several row blocks
def test_wait_gives_up_then_recovers(fmt, d, batch, t, context, wide):
    lib = tl.load()
    g = torch.Generator(device=DEV).manual_seed(t)
    cache = tl.KVCache.empty(fmt, wide, 16, 2, d)
    n = wide * 16
    y = torch.randn(2, n, 2, d, generator=g, device=DEV).half()
    tl.kv_append(cache, y[0], y[1], torch.arange(n, device=DEV))
    q = torch.randn(batch, t, 2, d, generator=g, device=DEV).half()
    table = torch.randint(0, wide, (batch, wide), generator=g, device=DEV).int()
    lens = torch.full((batch,), context, dtype=torch.int32, device=DEV)
    want = tl.tree_attention(q, cache, table, lens)
    out = torch.full_like(want, 123.0)
    torch.cuda.synchronize()
    assert tl.device_status(clear=True) == 0
    lib.ternary_test_set_wait_limit(1 << 16, 1)  # ~30 us, and a wait that nothing satisfies
    try:
        tl.tree_attention(q, cache, table, lens, out=out)
        torch.cuda.synchronize()
    finally:
        lib.ternary_test_set_wait_limit(0, 0)
    assert tl.device_status(clear=True) == TL_ERR_TIMEOUT
    assert (torch.isnan(out) | (out == 123.0)).all()
    got = tl.tree_attention(q, cache, table, lens, out=out)
    torch.cuda.synchronize()
    assert tl.device_status(clear=True) == 0
    assert torch.equal(got, want)
