"""Scores so large that fp32 holds them to whole numbers only: one key takes all of a row's weight, and
the answer is its value."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = [(1, 7), (4, 2), (16, 1), (24, 1), (70, 2)]   # streaming with 8 and 16 rows, tcgen05


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def run(z, vz, vs, n, t, share, wide):
    """Scores z [pages * 16] (natural units) from a query of (1, 0, 0 ..), values vz vs."""
    d, pages = vz.shape[1], len(z) // 16
    cache = tl.KVCache.empty("int8", pages, 16, 1, d)
    kz = torch.zeros(pages * 16, d, dtype=torch.int8)
    kz[:, 0] = 64
    for codes, scale, c, s in ((cache.k_codes, cache.k_scale, kz, z / (64 * 0.125)), (cache.v_codes, cache.v_scale, vz, vs)):
        codes.copy_(c.view(pages, 1, 16, d))
        scale.copy_(s.float().view(pages, 1, 16))
    table = torch.zeros(1, wide or pages, dtype=torch.int32, device=DEV)
    table[0, :pages] = torch.arange(pages)
    q = torch.zeros(1, t, share, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    out, lse = tl.tree_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), return_lse=True)
    return out.double().cpu(), lse.double().cpu()


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("wide", [None, 1024])
@pytest.mark.parametrize("size", [1e3, 1e5, 1.3e6, 3e6, 7e6, 1.1e7, 1.7e7, 2.3e7, 3.3e7, 4.1e7])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_score_takes_all(t, share, wide, size, sign):
    """Scores of `size` (natural units) with steps that fp32 resolves: 2^-18 of it and 200 more. One
    step down is a weight of e^-200."""
    n, d = 500, 64
    g = torch.Generator().manual_seed(int(size) + t)
    pages = -(-(n + t) // 16)
    vz = torch.randint(-100, 101, (pages * 16, d), generator=g).to(torch.int8)
    step = size * 2.0 ** -18 + 200
    z = sign * size - step * torch.randint(1, 40, (pages * 16,), generator=g)
    order = torch.randperm(n, generator=g)
    best = int(order[0])
    z[best] = sign * size
    z[n:] = sign * size - 50 * step        # the new tokens' own keys
    vs = 0.5 + torch.rand(pages * 16, generator=g)
    got, lse = run(z, vz, vs, n, t, share, wide)
    want = (vz[best].double() * vs[best].float().double())
    assert torch.isfinite(got).all()
    # the weight's rounding to f16 and the output's to bf16
    assert ((got - want).abs() <= (2.0 ** -11 + 2.0 ** -8) * want.abs()).all()
    # a product and a sum of fp32 numbers of this size, then ln 2
    assert ((lse - sign * size).abs() <= 2.0 ** -21 * size + 2.0 ** -13).all()


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("wide", [None, 1024])
@pytest.mark.parametrize("size", [1.3e6, 3e6, 5e6, 7e6, 1.1e7, 1.7e7, 2.3e7, 3.3e7, 4.1e7, 9e7, 2.6e8])
@pytest.mark.parametrize("sign", [1, -1])
def test_equal_scores_within_their_rounding(t, share, wide, size, sign):
    """Scores that differ by no more than a few roundings of their size: any weights are an answer, but the
    output lies between the values and the sum is finite."""
    n, d = 700, 64
    g = torch.Generator().manual_seed(int(size) % 1000 + t)
    pages = -(-(n + t) // 16)
    step = max(size * 2.0 ** -23, 0.7)
    z = sign * size + step * torch.randint(-4, 5, (pages * 16,), generator=g)
    vz = torch.randint(20, 101, (pages * 16, d), generator=g).to(torch.int8)
    vs = torch.exp2(torch.randint(-3, 1, (pages * 16,), generator=g).double())
    got, lse = run(z, vz, vs, n, t, share, wide)
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    if size < 5e7:  # beyond, a weight may leave f16 at its lower end
        assert (got >= 20 / 8 * (1 - 2.0 ** -7)).all() and (got <= 100 * (1 + 2.0 ** -7)).all()
