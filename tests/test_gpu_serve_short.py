"""A server whose pages run out: rows that find none keep what they have, and nothing of the other rows' pages changes."""
import os
import sys

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

import pages_ref as ref
import verify_ref
from conftest import ROOT
from test_gpu_pages import filled

sys.path.insert(0, os.path.join(ROOT, "examples"))
import serve_step as ss  # noqa: E402
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


def short_server(rows, pages, fmt="int8", wide=20):
    stack = vs.Stack(layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, ffn=768, fmt=fmt, page_size=16, pages=pages, positions=1024)
    return ss.Server(stack, rows, wide, vocab=600)


def images(s):
    return [ref.raw(c) for c in s.stack.caches.caches]


def slots_changed(old, new, page=16):
    """Slots of which any byte of any layer differs."""
    out = set()
    for a, b in zip(old, new):
        for x, y in zip(a, b):
            diff = (x != y).flatten(3).any(-1) if x.dim() == 4 else x != y   # [pages, heads, places]
            out |= {int(p) * page + int(i) for p, i in diff.any(1).nonzero().tolist()}
    return out


@pytest.mark.parametrize("rows,pages,prompt,draft,fmt", [(5, 13, 37, 9, "int8"), (7, 12, 16, 12, "fp8"), (4, 9, 30, 15, "int4"), (6, 20, 47, 7, "int8")])
def test_steps_with_too_few_pages(rows, pages, prompt, draft, fmt):
    """After every step: what was written lies in the served rows' own places, accepted entries moved there alone; tables, lengths
    and last tokens of the other rows are as before."""
    s = short_server(rows, pages, fmt)
    gen, cpu = torch.Generator(device=DEV).manual_seed(3), torch.Generator().manual_seed(rows)
    want = ref.Pages(16, s.pages.refs, s.pages.table, s.pages.lens, s.pages.held)
    assert s.prompt(0, torch.randint(0, s.vocab, (prompt,), generator=gen, device=DEV))
    want.reserve([prompt] + [-1] * (rows - 1), prompt)
    want.free([prompt] + [-1] * (rows - 1))
    parent = [-1] + [0] * (rows - 1)
    forked = s.fork(i32(parent))
    assert torch.equal(forked.cpu(), want.fork(parent)[0])
    refused = moved = 0
    for _ in range(30):
        tree, depth, sees = vs.random_trees(rows, draft, cpu)
        lens, last, before = s.pages.lens.tolist(), s.last.tolist(), images(s)
        live = [n > 0 for n in lens]
        slots64, ok64 = want.reserve([draft + 1 if n else -1 for n in live], draft + 1)
        ok64 = ok64 & torch.tensor(live)
        kept = {}

        def keep(caches, *args):
            kept["raw"] = images(s)
            return compact(caches, *args)

        compact = tl.kv_compact
        tl.kv_compact = keep
        try:
            got = s.step(tree.to(DEV, torch.int32), depth.to(DEV), sees.to(DEV))
        finally:
            tl.kv_compact = compact
        assert torch.equal(got["ok"].cpu(), ok64) and torch.equal(got["slots"].cpu(), slots64)
        path, count, tokens, _ = verify_ref.verify(got["target"].cpu(), got["drafted"].cpu(), got["uniform"].cpu(), got["q"].cpu(), tree.int())
        path, count, tokens = torch.where(ok64[:, None], path, -1), torch.where(ok64, count, 0), torch.where(ok64[:, None], tokens, -1)
        assert torch.equal(got["path"].cpu(), path.int()) and torch.equal(got["count"].cpu(), count.int()) and torch.equal(got["tokens"].cpu(), tokens)
        # written before the entries are closed up: the served rows' slots alone
        assert slots_changed(before, kept["raw"]) <= set(slots64[slots64 >= 0].tolist())
        moves, bad = ref.compact(want.table, 16, [n + 1 for n in lens], path.tolist(), count.tolist(), 20 * 16)
        assert not bad
        moved += sum(a != b for a, b in moves)
        for now, old in zip(images(s), kept["raw"]):
            ref.move(old, [a for a, _ in moves], [b for _, b in moves], 16)
            for x, y in zip(now, old):
                assert torch.equal(x, y)
        want.free([n + 1 + c if k else -1 for n, c, k in zip(lens, count.tolist(), ok64.tolist())])
        for name, w in zip(("refs", "table", "lens", "held"), want.tensors()):
            assert torch.equal(getattr(s.pages, name).cpu(), w), name
        assert s.last.tolist() == [int(tokens[r, int(count[r])]) if ok64[r] else last[r] for r in range(rows)]
        refused += int((torch.tensor(live) & ~ok64).sum())
    assert refused > 0 and moved > 0 and not want.flags  # (pages run out within 30 steps)
    assert tl.device_status() == 0


def test_a_prompt_without_pages_leaves_its_row_empty():
    s = short_server(3, 4)
    gen = torch.Generator(device=DEV).manual_seed(1)
    assert s.prompt(1, torch.randint(0, s.vocab, (40,), generator=gen, device=DEV))
    before, last = images(s), s.last.clone()
    assert not s.prompt(2, torch.randint(0, s.vocab, (33,), generator=gen, device=DEV))
    assert not slots_changed(before, images(s))
    assert s.pages.lens.tolist() == [0, 40, 0] and s.pages.held.tolist() == [0, 3, 0] and torch.equal(s.last, last)
    assert tl.device_status() == 0


@pytest.mark.parametrize("n", [6, 300])
def test_entries_behind_the_held_pages_stay(n):
    """Closing up rows of a pool: a row's moves end where its pages end, whatever its table says behind them."""
    page, wide = 16, 2 * n // 16 + 3
    pages = 3 * wide
    caches = filled("int8", pages, page, 2, 64, 2, seed=n)
    table = torch.zeros(4, wide, dtype=torch.int32)
    table[0] = torch.arange(wide)
    table[1, :3] = torch.arange(wide, wide + 3)
    table[3] = torch.arange(2 * wide, 3 * wide)
    held = [wide, 3, 0, wide + 1]                       # row 2 holds nothing, row 3 more than its table
    keep = [[2 * i + 1 for i in range(n)]] * 4
    pool = tl.KVPages(page, torch.ones(pages, dtype=torch.int32, device=DEV), table.to(DEV), i32([0] * 4), i32(held))
    old = [ref.raw(c) for c in caches]
    tl.kv_compact(caches, pool, i32([3, 41, 0, 0]), i32(keep), i32([n] * 4))
    moves = ref.compact(table.tolist(), page, [3], keep, [n], wide * page)[0]
    moves += ref.compact(table[1:2].tolist(), page, [41], keep, [n], 48)[0]
    for c, o in zip(caches, old):
        ref.move(o, [a for a, _ in moves], [b for _, b in moves], page)
        for x, y in zip(ref.raw(c), o):
            assert torch.equal(x, y)
    assert tl.device_status() == VALUE
