"""Verification of drafted tokens on the GPU against the plain form in 64 bits: paths, counts and tokens are equal.

Random numbers of 24 bits fall on a border of a sum only by construction.  Between borders the two sides can
differ where a number lies within the sums' errors of one: with fewer than 2^17 tokens, and errors of about
2^-44, that is a chance below 2^-27 a draw -- the cases here draw a few thousand times.  The tests on borders
use probabilities whose sums are exact in either arithmetic."""
import random

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

import verify_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
VALUE = 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def check(target, tokens, uniform, draft=None, parent=None, flags=False):
    got = tl.verify_drafts(target, tokens, uniform, draft=draft, parent=parent)
    cpu = [None if t is None else t.cpu() for t in (target, tokens, uniform, draft, parent)]
    want = ref.verify(*cpu)
    for g, w in zip(got, want):
        assert g.dtype == w.dtype and torch.equal(g.cpu(), w)
    assert want[3] == flags
    assert tl.device_status() == (VALUE if flags else 0)
    return want


def trees(rng, batch, n, width):
    """Parents of random trees with up to about `width` children a node."""
    return torch.tensor([[rng.randrange(max(-1, i // width - 1), max(0, (i + 1) // 2)) if i else -1 for i in range(n)] for _ in range(batch)],
                        dtype=torch.int32).reshape(batch, n)


def inputs(batch, n, vocab, dtype, parent, seed, spread=2.5, off=0.7):
    gen = torch.Generator().manual_seed(seed)
    z = spread * torch.randn(batch, n + 1, vocab, generator=gen)
    p = z.softmax(-1)
    p = torch.where(p < 0.02 / vocab, torch.zeros_like(p), p)
    p = (p / p.sum(-1, keepdim=True)).to(dtype)
    q = (z[:, :n] + off * torch.randn(batch, n, vocab, generator=gen)).softmax(-1).to(dtype)
    node = torch.arange(n).expand(batch, n) if parent is None else parent.expand(batch, n).long() + 1
    tokens = torch.zeros(batch, n, dtype=torch.int64)
    for b in range(batch):
        for i in range(n):
            tokens[b, i] = torch.multinomial(q[b, node[b, i]].float(), 1, generator=gen)
    u = torch.rand(batch, n + 1, generator=gen)
    return [t.to(DEV) for t in (p, q, tokens, u)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("batch,n,vocab", [(1, 1, 1), (3, 0, 17), (2, 4, 1000), (9, 7, 4097), (33, 3, 32000), (2, 12, 50021), (1, 5, 131072)])
@pytest.mark.parametrize("has_q", [True, False])
def test_chains(batch, n, vocab, dtype, has_q):
    p, q, tokens, u = inputs(batch, n, vocab, dtype, None, seed=batch * vocab + n)
    check(p, tokens, u, q if has_q else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,n,vocab,width", [(2, 2, 64, 4), (7, 15, 999, 3), (5, 31, 4096, 8), (3, 64, 8200, 2), (2, 200, 512, 40)])
@pytest.mark.parametrize("has_q", [True, False])
def test_trees(batch, n, vocab, width, dtype, has_q):
    parent = trees(random.Random(n * width), batch, n, width)
    p, q, tokens, u = inputs(batch, n, vocab, dtype, parent, seed=n + vocab, off=1.5)
    check(p, tokens, u, q if has_q else None, parent.to(DEV))
    check(p, tokens, u, q if has_q else None, parent[0].to(DEV))     # one tree for all


def test_many_children_rejected():
    """A node with 60 children whose numbers are near 1, some tokens among them twice: sums of many rejections."""
    n, vocab = 60, 300
    parent = torch.full((2, n), -1, dtype=torch.int32)
    p, q, tokens, u = inputs(2, n, vocab, torch.float32, parent, seed=8, spread=1.0, off=2.0)
    u[:, :n] = 1 - 2.0 ** -24
    for has_q in (True, False):
        want = check(p, tokens, u, q if has_q else None, parent.to(DEV))
        assert int(want[1].max()) <= 1


def test_numbers_on_borders():
    """Probabilities of a multiple of 2^-9: running sums, and u times them, are exact.  A number on the border of
    two tokens belongs to the second; u q = p rejects."""
    gen = torch.Generator().manual_seed(1)
    vocab, n = 300, 3
    for trial in range(20):
        cuts = torch.randint(0, 513, (64, n + 1, vocab - 1), generator=gen).sort(-1).values
        p = torch.diff(cuts, dim=-1, prepend=torch.zeros(64, n + 1, 1, dtype=torch.int64),
                       append=torch.full((64, n + 1, 1), 512)).float() / 512
        q = p[:, torch.randperm(n, generator=gen)].roll(trial, -1).contiguous()
        tokens = torch.stack([torch.multinomial(q[:, i], 1, generator=gen)[:, 0] for i in range(n)], 1)
        u = torch.randint(0, 512, (64, n + 1), generator=gen).float() / 512
        u[::2, :n] = 0.5
        for has_q in (True, False):
            check(p.to(DEV), tokens.to(DEV), u.to(DEV), q.to(DEV) if has_q else None)


def test_equal_distributions_accept_everything():
    p, _, _, u = inputs(5, 6, 1234, torch.float32, None, seed=3)
    q = p[:, :6].contiguous()
    gen = torch.Generator().manual_seed(2)
    tokens = torch.stack([torch.multinomial(q[:, i].cpu(), 1, generator=gen)[:, 0] for i in range(6)], 1).to(DEV)
    assert check(p, tokens, u, q)[1].tolist() == [6] * 5


def test_nothing_left_of_the_target():
    """q covers p: after the rejection the target's own row serves; with one token in p, and the only one."""
    vocab = 100
    p = torch.zeros(3, 2, vocab, device=DEV)
    p[:, 0, 7] = 0.25
    p[:, 0, 60] = 0.5
    p[:, 1] = 1 / vocab
    q = torch.zeros(3, 1, vocab, device=DEV)
    q[:, 0, 7] = 0.5
    q[:, 0, 60] = 0.5
    tokens = torch.full((3, 1), 7, device=DEV)
    u = torch.tensor([[0.5, 0.0], [0.75, 0.4], [0.25, 0.99]], device=DEV)
    want = check(p, tokens, u, q)
    assert want[1].tolist() == [0, 0, 1] and want[2][:2, 0].tolist() == [7, 60]
    one = torch.zeros(2, 2, vocab, device=DEV)
    one[:, :, 42] = 1
    check(one, torch.full((2, 1), 41, device=DEV), torch.tensor([[0.0, 0.999], [0.5, 0.0]], device=DEV))
    half = one * 0.5
    check(half, torch.full((2, 1), 42, device=DEV), torch.tensor([[0.5, 0.7], [0.25, 0.0]], device=DEV))


def test_entries_that_are_no_probabilities():
    """NaN and negative entries count as 0; a row of nothing gives -1 and sets the status word."""
    p, q, tokens, u = inputs(4, 3, 777, torch.float32, None, seed=11)
    p[:, :, 5] = float("nan")
    p[1, :, 100:200] *= -1
    q[:, :, 9] = float("nan")
    q[2, :, 300:] *= -1
    check(p, tokens, u, q)
    p[3] = -1
    check(p, tokens, u, q, flags=True)
    check(p, tokens, u, flags=True)


def test_numbers_out_of_range_follow_nothing_out_of_bounds():
    p, q, tokens, u = inputs(3, 2, 500, torch.bfloat16, None, seed=12)
    u[0, 2], u[1, 2], u[2, 2] = 1.0, 7.0, float("nan")
    u[2, 0] = float("nan")
    path, count, out = tl.verify_drafts(p, tokens, u, draft=q)
    for b in range(3):
        assert 0 <= int(out[b, int(count[b])]) < 500


@pytest.mark.parametrize("what", ["token", "parent", "self"])
def test_drafted_tokens_refused(what):
    parent = torch.tensor([[-1, 0, 0, 2, 3], [-1, -1, 1, 1, 2]], dtype=torch.int32)
    p, q, tokens, u = inputs(2, 5, 640, torch.float32, parent, seed=5)
    u[:, :5] *= 0.1
    if what == "token":
        tokens[0, 2], tokens[1, 0], tokens[1, 1] = 640, -1, 1 << 40
    else:
        parent[0, 2], parent[1, 0] = (7, -2) if what == "parent" else (2, 0)
    check(p, tokens, u, q, parent.to(DEV), flags=True)
    check(p, tokens, u, None, parent.to(DEV), flags=True)


def test_strided_inputs():
    """Rows in larger tensors, a vocabulary that does not fill its rows, more draft rows than needed, int strides."""
    p, q, tokens, u = inputs(4, 5, 2000, torch.float16, None, seed=21)
    wide = torch.full((4, 9, 2048), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, 1:7, :2000] = p
    wq = torch.full((4, 6, 2001), float("nan"), dtype=torch.float16, device=DEV)
    wq[:, :5, 1:] = q
    many = torch.zeros(4, 11, dtype=torch.int64, device=DEV)
    many[:, 3:8] = tokens
    uu = torch.zeros(12, 4, device=DEV)
    uu[2:8] = u.t()
    want = check(p, tokens, u, q)
    got = tl.verify_drafts(wide[:, 1:7, :2000], many[:, 3:8], uu[2:8].t(), draft=wq[:, :, 1:])
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)
    back = tl.verify_drafts(p.flip(0), tokens.flip(0), u.flip(0), draft=q.flip(0))
    for g, w in zip(back, want):
        assert torch.equal(g.flip(0).cpu(), w)


def test_tokens_are_distributed_as_the_target():
    """One node, 40 tokens, 2^16 sequences: the first token's frequencies against the target's, within six standard
    deviations (a wrong rest after a rejection is off by tens)."""
    batch, vocab = 1 << 16, 40
    gen = torch.Generator(device=DEV).manual_seed(4)
    p = torch.randn(vocab, generator=gen, device=DEV).softmax(0)
    q = (2 * torch.randn(vocab, generator=gen, device=DEV)).softmax(0)
    for tree in (False, True):
        n = 3 if tree else 1
        parent = torch.full((n,), -1, dtype=torch.int32, device=DEV) if tree else None
        tokens = torch.multinomial(q, batch * n, replacement=True, generator=gen).view(batch, n)
        u = torch.rand(batch, n + 1, generator=gen, device=DEV)
        t = p.expand(batch, n + 1, vocab).contiguous()
        out = tl.verify_drafts(t, tokens, u, draft=q.expand(batch, n, vocab).contiguous(), parent=parent)[2][:, 0]
        freq = torch.bincount(out, minlength=vocab).double() / batch
        sd = (p.double() * (1 - p.double()) / batch).sqrt()
        assert ((freq - p.double()).abs() <= 6 * sd + 1e-9).all()


def test_replayed():
    """Captured once, replayed on other numbers; the same inputs give the same answers every time."""
    p, q, tokens, u = inputs(6, 4, 3000, torch.float32, None, seed=31)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tl.verify_drafts(p, tokens, u, draft=q)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tl.verify_drafts(p, tokens, u, draft=q)
    gen = torch.Generator(device=DEV).manual_seed(6)
    for _ in range(10):
        u.uniform_(generator=gen)
        graph.replay()
        want = ref.verify(p.cpu(), tokens.cpu(), u.cpu(), q.cpu())
        for g, w in zip(got, want):
            assert torch.equal(g.cpu(), w)
