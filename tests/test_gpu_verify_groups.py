"""The calls of a step one after the other with group-scaled layers: the layers that follow the
attention are launched while it runs, in every form it takes (with and without a join, few rows and
many), and give what they give when each call is waited for."""
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


class Waiting:
    """The calls, each followed by a wait for the device."""

    def __getattr__(self, name):
        f = getattr(tl, name)

        def call(*args, **kw):
            r = f(*args, **kw)
            torch.cuda.synchronize()
            return r
        return call


# M = batch * draft tokens: the decode, the skinny and the tile kernels, split over a cluster or not
@pytest.mark.parametrize("group", [0, 64, 128])
@pytest.mark.parametrize("batch,draft,wide", [(1, 1, 4), (4, 3, 4), (5, 23, 8), (5, 23, 400), (20, 6, 400), (32, 17, 8), (2, 150, 20)])
def test_overlapped_steps_give_the_same(group, batch, draft, wide, monkeypatch):
    gen = torch.Generator(device=DEV).manual_seed(7)
    context = 30
    st = vs.Stack(layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, ffn=768, fmt="int8", page_size=16,
                  pages=batch * wide, positions=1024, group=group)
    table = torch.randperm(batch * wide, generator=gen, device=DEV).int().view(batch, wide)
    done = torch.zeros(batch, dtype=torch.int32, device=DEV)
    y = torch.randn(batch, context, 512, generator=gen, device=DEV).to(torch.bfloat16)
    places = torch.arange(context, device=DEV).expand(batch, -1)
    st.step(y, places.flatten(), vs.slots_of(table, places, 16).flatten(), table, done)
    ctx = done + context
    x = torch.randn(batch, draft, 512, generator=gen, device=DEV).to(torch.bfloat16)
    places = (ctx[:, None] + torch.arange(draft, device=DEV)).long()
    if int(places.max()) >= wide * 16:
        pytest.skip("the page table's row is too short for these tokens")
    args = (x, places.flatten(), vs.slots_of(table, places, 16).flatten(), table, ctx)
    with monkeypatch.context() as m:
        m.setattr(vs, "tl", Waiting())
        want = st.step(*args)
    for _ in range(10):
        assert torch.equal(st.step(*args), want)
    graph, warm = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        st.step(*args)
    torch.cuda.current_stream().wait_stream(warm)
    with torch.cuda.graph(graph):
        got = st.step(*args)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("group", [64, 128])
def test_chain_and_single_tokens_agree(group):
    """As in the tree test with channel scales, for group scales: 2%."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    st = vs.Stack(layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, ffn=768, fmt="int8", page_size=16, pages=30,
                  positions=1024, group=group)
    table = torch.randperm(30, generator=gen, device=DEV).int().view(3, 10)
    ctx = vs.prefill(st, 100, table, gen, DEV)
    x = torch.randn(3, 24, 512, generator=gen, device=DEV).to(torch.bfloat16)
    places = (ctx[:, None] + torch.arange(24, device=DEV)).long()
    chain = st.step(x, places.flatten(), vs.slots_of(table, places, 16).flatten(), table, ctx)
    for i in range(0, 24):
        now = ctx + i
        y = st.step(x[:, i:i + 1], now.long(), vs.slots_of(table, now[:, None].long(), 16).flatten(), table, now)
        off = float((y.float() - chain[:, i:i + 1].float()).norm() / chain[:, i:i + 1].float().norm())
        assert off <= 0.02, (i, off)
