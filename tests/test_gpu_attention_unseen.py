"""A new token that a row does not see changes no bit of it, whatever its scales hold."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("t,share", [(4, 2), (16, 1), (24, 1), (40, 4)])
@pytest.mark.parametrize("n", [0, 37, 200])
@pytest.mark.parametrize("bad", [float("inf"), 1e30, 3e3, 1e-30, 0.0, float("nan")])
def test_unseen_scales_change_no_bit(t, share, n, bad):
    """A new token's scales, which only itself sees, beside keys of scales of every size: all other rows
    are the same, bit for bit."""
    g = torch.Generator().manual_seed(n + t)
    d, pages = 64, -(-(n + t) // 16)
    cache = tl.KVCache.empty("int8", pages, 16, 1, d)
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        codes.copy_(torch.randint(-127, 128, codes.shape, generator=g).to(torch.int8))
        scale.copy_(0.01 * torch.exp2(torch.randint(-2, 2, scale.shape, generator=g).float() + torch.rand(scale.shape, generator=g)))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    q = torch.randn(1, t, share, d, generator=g).to(torch.bfloat16).to(DEV)
    tree = torch.eye(t, dtype=torch.bool, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    want = tl.tree_attention(q, cache, table, lens, tree)
    cache.v_scale[(n + 1) // 16, :, (n + 1) % 16] = bad
    got = tl.tree_attention(q, cache, table, lens, tree)
    rest = [i for i in range(t) if i != 1]
    assert torch.equal(got[0, rest], want[0, rest])
