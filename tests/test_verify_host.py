"""Host-side refusals of the verification of drafted tokens (no GPU, nothing is launched), and its plain form."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import verify

import verify_ref as ref

OK, NULL, SHAPE, DTYPE, ALIGN, VALUE, CUDA = 0, 1, 2, 3, 4, 5, 6
A, B, C, D, E, F, G, H = (0x10000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    tl.build()
    tl.load()
    return verify._lib()


def test_refusals(lib):
    def call(target=A, tb=900, tn=300, q=B, qb=600, qn=300, dt=2, tokens=C, parent=D, u=E, b=2, n=2, v=300, path=F, count=G, out=H):
        return lib.ternary_verify_drafts(target, tb, tn, q, qb, qn, dt, tokens, 2, parent, 2, u, 3, b, n, v, path, count, out, None)

    assert call(dt=3) == DTYPE and call(dt=-1) == DTYPE
    for bad in (dict(b=-1), dict(b=(1 << 16) + 1), dict(n=-1), dict(n=1025), dict(v=0), dict(v=1 << 31), dict(tb=1 << 41), dict(qn=1 << 41)):
        assert call(**bad) == SHAPE
    for name in ("target", "tokens", "u", "path", "count", "out"):
        assert call(**{name: None}) == NULL
    for bad in (dict(target=A + 2), dict(q=B + 1), dict(tokens=C + 4), dict(parent=D + 2), dict(u=E + 2), dict(path=F + 1), dict(count=G + 2),
                dict(out=H + 4)):
        assert call(**bad) == ALIGN
    assert call(b=0, target=None) == OK
    lib.ternary_test_inject_launch_failures(2)
    try:
        assert call() == CUDA and call(n=0, tokens=None, path=None, q=None, parent=None) == CUDA
    finally:
        lib.ternary_test_inject_launch_failures(0)


def test_binding_refuses():
    p, t, u = torch.zeros(2, 3, 10), torch.zeros(2, 2, dtype=torch.int64), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        tl.verify_drafts(p, t, u)
    with pytest.raises(ValueError, match="target"):
        tl.verify_drafts(p.double(), t, u)
    with pytest.raises(ValueError, match="target"):
        tl.verify_drafts(p[0], t, u)


def test_plain_form_of_two_tokens_by_hand():
    """p = (1/2, 1/2), q = (3/4, 1/4).  Token 0 is accepted below u = 2/3; rejected, token 1 follows."""
    p, q = torch.tensor([[[0.5, 0.5], [0.25, 0.75]]]), torch.tensor([[[0.75, 0.25]]])
    x = torch.zeros(1, 1, dtype=torch.int64)
    for u, v, want in ((0.66, 0.2, [0, 0]), (0.66, 0.25, [0, 1]), (0.67, 0.9, [1, -1]), (0.67, 0.0, [1, -1])):
        assert ref.verify(p, x, torch.tensor([[u, v]]), q)[2].tolist() == [want]


def test_plain_form_rejections_unroll():
    """w after k rejections is max(p - A_k q, 0), A_k the sum of the W before: what the kernel computes."""
    gen = torch.Generator().manual_seed(0)
    p, q = (torch.randn(50, generator=gen, dtype=torch.float64).softmax(0) for _ in "pq")
    w, total, a = p, 1.0, 0.0
    for _ in range(6):
        a += total
        w = (w - total * q).clamp(min=0)
        total = float(w.sum())
        assert torch.allclose(w, (p - a * q).clamp(min=0), rtol=0, atol=1e-15)
