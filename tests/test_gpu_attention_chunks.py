"""A causal chunk of a prompt: some hundred new tokens, whose rows fill several blocks, over no
context and over one, and beside an explicit lower-triangular tree."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("fmt,dtype,d,share,page", [("int8", torch.bfloat16, 128, 7, 64), ("fp8", torch.float16, 64, 1, 16),
                                                    ("int4", torch.bfloat16, 128, 2, 48)])
@pytest.mark.parametrize("t", [128, 129, 257, 400])
def test_chunk(fmt, dtype, d, share, page, t):
    c = Case(fmt, [0, 5, 300], t, 1, d, page, seed=t)
    q = c.q(share, dtype, 2.0)
    out, lse = c.check(q, None, what="chunk")
    tree = torch.tril(torch.ones(t, t, dtype=torch.bool))
    assert torch.equal(c.run(q, tree), out)


@pytest.mark.parametrize("share", [1, 4])
def test_chunk_equals_its_tokens_one_by_one(share):
    """Rows of a chunk against single tokens over the same keys: two kernels, the bound of either twice
    (2^-10 of the mean of |v|, here below 6, and one rounding to f16)."""
    t = 300
    c = Case("int8", [40], t, 1, 64, 16)
    q = c.q(share, torch.float16)
    out = c.run(q, None)
    table = c.table.to(DEV)
    mag = max(float(v.abs().max()) for v in c.v)
    for i in (0, 1, 63, 64, 127, 128, 200, t - 1):
        one = tl.tree_attention(q[:, i:i + 1].to(DEV), c.cache, table, torch.tensor([40 + i], dtype=torch.int32, device=DEV))
        assert float((one.float() - out[:, i:i + 1].float()).abs().max()) <= 2 * (2.0 ** -10 + 2.0 ** -11) * mag
