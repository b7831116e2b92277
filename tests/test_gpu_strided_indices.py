"""Index arrays that are views (columns of a table, every other entry) give what dense ones give: a
copy that a call makes of them lives until the call's work is enqueued."""
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


def column(t):
    """The same numbers as one column of a table."""
    wide = torch.full((t.shape[0], 3), 1 << 20, dtype=t.dtype, device=DEV)
    wide[:, 1] = t
    return wide[:, 1]


@pytest.mark.parametrize("n", [2, 3, 4, 8, 63, 64, 500])
@pytest.mark.parametrize("heads,dim", [(1, 64), (4, 128)])
def test_append_read_and_rope(n, heads, dim):
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randn(n, heads + 2, dim, generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.randint(0, 1000, (n,), generator=g, device=DEV)
    slots = torch.randperm(n + 40, generator=g, device=DEV)[:n]
    table = tl.rope_table(1000, dim)
    got = []
    for p, s in ((pos, slots), (column(pos), column(slots))):
        cache = tl.KVCache.empty("int8", -(-(n + 40) // 16), 16, 1, dim)
        for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale):
            t.zero_()
        torch.cuda.synchronize()
        q = tl.kv_append(cache, x[:, heads:heads + 1], x[:, heads + 1:], s, q=x[:, :heads], positions=p, table=table)
        got.append((q, cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, *tl.kv_read(cache, s),
                    tl.rope(x, p, table)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("t,share", [(1, 2), (20, 1)])
def test_attention(t, share):
    b, page, d = 5, 16, 64
    g = torch.Generator(device=DEV).manual_seed(t)
    cache = tl.KVCache.empty("fp8", 40, page, 1, d)
    y = torch.randn(40 * page, 1, d, generator=g, device=DEV).half()
    tl.kv_append(cache, y, y.flip(0), torch.arange(40 * page, device=DEV))
    q = torch.randn(b, t, share, d, generator=g, device=DEV).half()
    lens = torch.tensor([3, 0, 50, 77, 16], dtype=torch.int32, device=DEV)
    table = torch.randint(0, 40, (b, 7), generator=g, device=DEV).int()
    tree = torch.rand(b, t, t, generator=g, device=DEV) < 0.5
    want = tl.tree_attention(q, cache, table, lens, tree)
    got = tl.tree_attention(q, cache, table.t().contiguous().t(), column(lens), tree.transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.equal(got, want)
