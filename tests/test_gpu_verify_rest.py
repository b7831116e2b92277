"""A rest that is small beside p and A q: what is left of a token after many rejections is still drawn."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

import verify_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("vocab", [2, 7, 8, 5000, 40001])
@pytest.mark.parametrize("children", [1, 23, 24, 25, 30, 45])
def test_the_only_token_that_is_left(vocab, children):
    """p all on token 1, q half on it and half on token 0, which is drafted again and again: after k rejections W = 2^-k, A = 2 - 2^(1-k) and
    w(1) = 1 - A / 2 = 2^-k, all exact in 64 bits and in pairs of fp32.  From 25 rejections on A q rounds to p in fp32."""
    p = torch.zeros(2, children + 1, vocab, device=DEV)
    p[:, :, 1] = 1
    q = torch.zeros(2, children, vocab, device=DEV)
    q[:, :, :2] = 0.5
    parent = torch.full((children,), -1, dtype=torch.int32, device=DEV)
    u = torch.full((2, children + 1), 0.75, device=DEV)
    u[1] = 0.0
    u[1, :children] = 2.0 ** -20                      # u W q < w(0) = 0 is false for any u
    got = tl.verify_drafts(p, torch.zeros(2, children, dtype=torch.int64, device=DEV), u, draft=q, parent=parent)
    assert got[1].tolist() == [0, 0]
    assert got[2][:, 0].tolist() == [1, 1]
    want = ref.verify(p.cpu(), torch.zeros(2, children, dtype=torch.int64), u.cpu(), q.cpu(), parent.cpu())
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)


def test_rests_of_a_few_units():
    """Rests of p(v) = 1/2 on two tokens each, whose A q lies within a few units of p: either may be drawn, none is lost.  The border
    between them is looked at from both sides, 2^-10 away, where the sums differ by less than 2^-15."""
    children, vocab = 26, 3
    p = torch.tensor([0.5, 0.5, 0.0], device=DEV).expand(4, children + 1, vocab).contiguous()
    q = torch.tensor([0.25, 0.25, 0.5], device=DEV).expand(4, children, vocab).contiguous()
    parent = torch.full((children,), -1, dtype=torch.int32, device=DEV)
    u = torch.full((4, children + 1), 0.5, device=DEV)
    u[:, children] = torch.tensor([0.0, 0.5 - 2.0 ** -10, 0.5 + 2.0 ** -10, 1 - 2.0 ** -10], device=DEV)
    out = tl.verify_drafts(p, torch.full((4, children), 2, device=DEV), u, draft=q, parent=parent)[2]
    assert out[:, 0].tolist() == [0, 0, 1, 1]
