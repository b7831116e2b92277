"""The calls together, as a user runs them: a stack of ternary layers whose drafted tree gives,
for every path, what the same tokens give one by one; and accepted entries moved in the cache."""
import os
import sys

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import verify_step as vs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("fmt,draft,context", [("int8", 6, 150), ("fp8", 20, 70), ("int4", 12, 33)])
def test_tree_and_chain_agree(fmt, draft, context):
    """bf16 hidden states of two layers pass through about ten roundings of 2^-9 each on either
    side, and a key or value next to a rounding boundary of its format may take the other code
    (one step of 1/127, 2^-4 or 1/7 of the row's largest, in a weighted mean of `context` keys):
    2% (int4: 5%) covers both, where a wrong mask, slot or position gives differences of order 1."""
    gen, cpu = torch.Generator(device=DEV).manual_seed(5), torch.Generator().manual_seed(5)
    batch, per = 3, -(-(context + draft) // 16)
    st = vs.Stack(layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, ffn=768, fmt=fmt, page_size=16,
                  pages=batch * per + 2, positions=1024)
    table = torch.randperm(batch * per + 2, generator=gen, device=DEV)[:batch * per].int().view(batch, per)
    ctx = vs.prefill(st, context, table, gen, DEV)
    parent, depth, sees = vs.random_trees(batch, draft, cpu)
    x = torch.randn(batch, draft, 512, generator=gen, device=DEV).to(torch.bfloat16)
    places = (ctx[:, None] + torch.arange(draft, device=DEV)).long()
    tree = st.step(x, (ctx[:, None] + depth.to(DEV)).flatten().long(), vs.slots_of(table, places, 16).flatten(), table, ctx,
                   sees.to(DEV))
    # accept the path to the deepest token of each tree, as far as the shallowest reaches
    paths = []
    for b in range(batch):
        path, i = [], int(depth[b].argmax())
        while i >= 0:
            path.insert(0, i)
            i = int(parent[b, i])
        paths.append(path)
    n = min(len(p) for p in paths)
    path = torch.tensor([p[:n] for p in paths], device=DEV)
    before = [[t.clone() for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)] for _, c in st.layers]
    count = torch.full((batch,), n, device=DEV)
    after = st.accept(table, ctx, path, count)
    assert torch.equal(after, ctx + n)
    for (_, c), old in zip(st.layers, before):
        for new, was in zip((c.k_codes, c.v_codes, c.k_scale, c.v_scale), old):
            if new.dtype == torch.float8_e4m3fn:
                new, was = new.view(torch.uint8), was.view(torch.uint8)
            for b in range(batch):
                for i in range(n):
                    d, s = int(places[b, i]), int(places[b, int(path[b, i])])
                    assert torch.equal(new[table[b, d // 16], :, d % 16], was[table[b, s // 16], :, s % 16])
    # the same tokens one by one
    lim = 0.05 if fmt == "int4" else 0.02
    for i in range(n):
        now = ctx + i
        tok = path[:, i, None, None].expand(-1, 1, 512)
        y = st.step(x.gather(1, tok), now.long(), vs.slots_of(table, now[:, None].long(), 16).flatten(), table, now)
        want = tree.gather(1, tok)
        off = float((y.float() - want.float()).norm() / want.float().norm())
        assert off <= lim, (i, off)
