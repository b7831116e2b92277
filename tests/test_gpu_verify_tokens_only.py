"""Chains and trees from a drafter that gives tokens only: the tokens are distributed as the target's own, whatever was drafted."""
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


def within(freq, p, n):
    sd = (p * (1 - p) / n).sqrt()
    return bool(((freq - p).abs() <= 6 * sd + 1e-9).all())


@pytest.mark.parametrize("drafted", [[3], [3, 9, 0, 3, 21], list(range(12)), [39] * 4])
def test_first_token(drafted):
    """Children of one node, some twice: frequencies of the first token within six standard deviations of the target."""
    batch, vocab, n = 1 << 16, 40, len(drafted)
    gen = torch.Generator(device=DEV).manual_seed(n)
    p = (1.5 * torch.randn(vocab, generator=gen, device=DEV)).softmax(0)
    tokens = torch.tensor(drafted, device=DEV).expand(batch, n).contiguous()
    u = torch.rand(batch, n + 1, generator=gen, device=DEV)
    parent = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    t = p.expand(batch, n + 1, vocab)
    path, count, out = tl.verify_drafts(t, tokens, u, parent=parent if n > 1 else None)
    assert within(torch.bincount(out[:, 0], minlength=vocab).double() / batch, p.double(), batch)
    # a drafted token is accepted as often as the target has one of them
    own = p[torch.tensor(sorted(set(drafted)), device=DEV)].double().sum()
    assert within((count == 1).double().mean()[None], own[None], batch)


def test_first_two_tokens_of_a_tree():
    """Two levels: after an accepted child its own row decides.  Frequencies of (first, second) where the first was accepted."""
    batch, vocab = 1 << 16, 6
    gen = torch.Generator(device=DEV).manual_seed(9)
    rows = torch.randn(6, vocab, generator=gen, device=DEV).softmax(1)   # after the root and after each drafted token
    drafted, parent = [4, 1, 2, 0, 5], [-1, -1, 0, 0, 1]
    tokens = torch.tensor(drafted, device=DEV).expand(batch, 5).contiguous()
    u = torch.rand(batch, 6, generator=gen, device=DEV)
    path, count, out = tl.verify_drafts(rows.expand(batch, 6, vocab), tokens, u, parent=torch.tensor(parent, dtype=torch.int32, device=DEV))
    first = torch.bincount(out[:, 0], minlength=vocab).double()
    assert within(first / batch, rows[0].double(), batch)
    for node, token in ((1, 4), (2, 1)):
        mine = out[:, 0] == token
        assert torch.equal(path[mine, 0], torch.full_like(path[mine, 0], node - 1)) and bool((count[mine] >= 1).all())
        n = int(mine.sum())
        assert within(torch.bincount(out[mine, 1], minlength=vocab).double() / n, rows[node].double(), n)
