"""Sums over a large vocabulary whose entries are not exact in fp32: one entry beside thousands that are small against it."""
from fractions import Fraction

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


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("side", [-1, 1])
def test_a_border_between_two_halves(side, dtype, aligned):
    """2^22 tokens.  In the first half every lane's first entry is 2^-10 and the others are s = 2^-35 + 2^-49 - 2^-58 (bf16: 2^-35), whose sums in plain
    fp32 drop the 2^-49: 2^-29 of the half's sum S1 in all.  The second half holds S1 (1 + side 2^-31) on its last five tokens.
    u = 1/2 then falls just before the end of the first half (side -1) or just behind it (+1), 2^-32 of the total away.  The
    sums' errors, V (W + 2) 2^-59 with the W = 4 (8, and where rows start anywhere) entries between two renormalisations, are 2^-34.4
    (2^-33.6) at most."""
    vocab, run = 1 << 22, 1 << 16                       # 8 blocks of 8 warps
    width = 4 if dtype is torch.float32 and aligned else 8
    small = 2.0 ** -35 + (2.0 ** -49 - 2.0 ** -58 if dtype is torch.float32 else 0.0)
    p = torch.zeros(vocab, dtype=torch.float64)
    at = torch.arange(vocab // 2)
    p[:vocab // 2] = small
    first = (at % run < 32 * width) & (at % width == 0) if aligned else at % run < 32
    p[:vocab // 2][first] = 2.0 ** -10
    assert torch.equal(p.to(dtype).double(), p)
    n = int(first.sum())
    half = Fraction(n, 1 << 10) + (vocab // 2 - n) * Fraction(small)
    rest, tail = half * (1 + side * Fraction(1, 1 << 31)), []
    for _ in range(5):                                 # the other half's sum, to 2^-40 or better, in few entries
        v = float(torch.tensor(float(rest), dtype=torch.float64).to(dtype))
        if Fraction(v) > rest:                         # (rounded down, so that what is left is positive)
            v = float(torch.nextafter(torch.tensor(v, dtype=dtype), torch.tensor(0.0, dtype=dtype)))
        tail.append(v)
        rest -= Fraction(v)
    assert 0 <= rest < Fraction(1, 1 << 38)
    p[-len(tail):] = torch.tensor(tail, dtype=torch.float64)
    wide = torch.zeros(vocab + 1, dtype=dtype, device=DEV)
    target = wide[(0 if aligned else 1):][None, None, :vocab]
    target.copy_(p)
    assert torch.equal(target.cpu().double()[0, 0], p)
    out = tl.verify_drafts(target, torch.zeros(1, 0, dtype=torch.int64, device=DEV), torch.full((1, 1), 0.5, device=DEV))[2]
    token = int(out[0, 0])
    if side > 0:
        assert token == vocab - len(tail)
        return
    # running sums pass u total = half (1 - 2^-32) this many small tokens before the end of the first half
    behind = half / (1 << 32) / Fraction(small)
    off = half * Fraction(vocab * (width + 2), 1 << 59) / Fraction(small)
    assert vocab // 2 - 1 - behind - off - 1 <= token <= vocab // 2 - 1 - behind + off + 1
