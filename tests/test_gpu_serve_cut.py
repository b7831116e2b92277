"""A sequence cut inside a page that a fork shares: it is refused room until it is forked itself, and goes on from there."""
import os
import sys

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

import pages_ref as ref
from conftest import ROOT
from test_gpu_serve_short import images, short_server, slots_changed

sys.path.insert(0, os.path.join(ROOT, "examples"))
import verify_step as vs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV, VALUE = "cuda", 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("fmt", ["int8", "int4"])
def test_cut_refused_forked_and_on(fmt):
    s = short_server(4, 24, fmt)
    gen, cpu = torch.Generator(device=DEV).manual_seed(3), torch.Generator().manual_seed(4)
    assert s.prompt(0, torch.randint(0, s.vocab, (40,), generator=gen, device=DEV))
    assert s.fork(i32([-1, 0, -1, -1])).tolist() == [True] * 4
    table = s.pages.table.tolist()
    assert table[1][:2] == table[0][:2]
    tl.pages_free(s.pages, i32([25, -1, -1, -1]))          # row 0 goes back into the second page, which row 1 holds too
    assert s.pages.refs.tolist()[table[0][1]] == 2
    draft = 6
    tree, depth, sees = (v.to(DEV) for v in vs.random_trees(4, draft, cpu))
    before, lens, last = images(s), s.pages.lens.tolist(), s.last.tolist()
    got = s.step(tree.int(), depth, sees)
    assert got["ok"].tolist() == [False, True, False, False] and tl.device_status() == VALUE
    assert s.pages.lens.tolist()[0] == lens[0] == 25 and s.last.tolist()[0] == last[0]
    mine = {p * 16 + i for p in s.pages.table.tolist()[1][2:s.pages.held.tolist()[1]] for i in range(16)}
    mine |= set(got["slots"][1][got["slots"][1] >= 0].tolist())
    assert slots_changed(before, images(s)) <= mine        # row 1's own pages alone; the shared ones are as they were
    # row 2 continues row 0 with a page of its own for the cut one's first nine places; row 0 ends
    assert s.fork(i32([-1, -1, 0, -1])).tolist() == [True] * 4
    tl.pages_free(s.pages, i32([0, -1, -1, -1]))
    now = s.pages.table.tolist()
    assert now[2][0] == table[0][0] and now[2][1] != table[0][1]
    assert s.pages.refs.tolist()[table[0][0]] == 2 and s.pages.refs.tolist()[table[0][1]] == 1
    for raw in images(s):
        for t in raw:
            assert torch.equal(t[now[2][1], :, :9], t[table[0][1], :, :9])
    shared = [[t[table[0][:2]].clone() for t in raw] for raw in images(s)]
    for _ in range(3):
        got = s.step(tree.int(), depth, sees)
        assert got["ok"].tolist() == [False, True, True, False]
    for raw, old in zip(images(s), shared):
        for t, o in zip(raw, old):
            assert torch.equal(t[table[0][:2]], o)
    held = s.pages.held.tolist()
    used = [p for r in range(4) for p in s.pages.table.tolist()[r][:held[r]]]
    assert all(n == used.count(p) for p, n in enumerate(s.pages.refs.tolist()))
    assert tl.device_status() == 0
