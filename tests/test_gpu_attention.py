"""Attention over the quantised cache against fp64: head sharing, formats, lengths around every
tile edge, trees and rows that see nothing, whatever lies in unseen places, long contexts split
over many blocks, strides, streams, graphs and indices out of range."""
import math

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from attn_ref import attention64, check_attention, codes_of, numbers, quantise

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


class Case:
    """A cache of random rows, a shuffled page table, and the fp64 answer of any call on it.
    Everything that no row may read -- places beyond a length, pages of nobody -- holds the
    worst there is: scales NaN and infinite, codes of every bit pattern (0x7F included)."""

    def __init__(self, fmt, lens, t, hk, d, page, seed=0, spread=1.0):
        g = torch.Generator().manual_seed(seed + 7 * t + d + page)
        self.g, self.fmt, self.lens, self.t, self.hk, self.d, self.page = g, fmt, lens, t, hk, d, page
        used = [-(-(n + t) // page) for n in lens]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=g)
        wide = max(used) + 2
        self.table = torch.full((len(lens), wide), pages - 1, dtype=torch.int32)
        self.cache = tl.KVCache.empty(fmt, pages, page, hk, d)
        junk = [torch.randint(0, 256, self.cache.k_codes.shape, generator=g, dtype=torch.uint8) for _ in "kv"]
        for j in junk:
            j[::2] = 0x7F
        bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).max])
        scales = [bad[torch.randint(0, 4, self.cache.k_scale.shape, generator=g)] for _ in "kv"]
        self.k, self.v, at = [], [], 0
        for b, n in enumerate(lens):
            mine = order[at:at + used[b]]
            at += used[b]
            self.table[b, :used[b]] = mine.int()
            for side, keep in ((0, self.k), (1, self.v)):
                y = torch.randn(n + t, hk, d, generator=g) * torch.exp(spread * torch.randn(n + t, hk, 1, generator=g))
                z, s = quantise(y, fmt)
                j = torch.arange(n + t)
                junk[side][mine[j // page], :, j % page] = codes_of(z, fmt).view(torch.uint8)
                scales[side][mine[j // page], :, j % page] = s
                keep.append((z.double() * s.double()[..., None]))
        self.cache.k_codes.view(torch.uint8).copy_(junk[0])
        self.cache.v_codes.view(torch.uint8).copy_(junk[1])
        self.cache.k_scale.copy_(scales[0])
        self.cache.v_scale.copy_(scales[1])

    def q(self, heads, dtype, size=1.0):
        return (size * torch.randn(len(self.lens), self.t, heads, self.d, generator=self.g)).to(dtype)

    def sees(self, b, tree):
        n, t = self.lens[b], self.t
        own = torch.tril(torch.ones(t, t, dtype=torch.bool)) if tree is None else (tree if tree.dim() == 2 else tree[b]) != 0
        return torch.cat([torch.ones(t, n, dtype=torch.bool), own], 1)

    def run(self, q, tree=None, **kw):
        return tl.tree_attention(q.to(DEV), self.cache, self.table.to(DEV),
                                 torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                                 None if tree is None else tree.to(DEV), **kw)

    def check(self, q, tree=None, scale=None, what=""):
        out, lse = self.run(q, tree, scale=scale, return_lse=True)
        for b in range(len(self.lens)):
            ref = attention64(q[b], self.k[b], self.v[b], self.sees(b, tree), self.d ** -0.5 if scale is None else scale)
            check_attention(out[b], lse[b], ref, q.dtype, f"{what} sequence {b}")
        return out, lse


def random_tree(g, b, t):
    sees = torch.zeros(b, t, t, dtype=torch.bool)
    for i in range(b):
        for j in range(t):
            if j:
                sees[i, j] = sees[i, int(torch.randint(0, j, (1,), generator=g))]
            sees[i, j, j] = True
    return sees


EDGES = [0, 1, 14, 15, 16, 17, 47, 62, 63, 64, 65, 126, 127, 128, 129, 200, 255, 256, 257, 500]


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_single_tokens_at_every_edge(fmt, d, dtype):
    c = Case(fmt, EDGES, 1, 2, d, 16)
    for share in (1, 7, 16):
        c.check(c.q(2 * share, dtype, 2.0), what=f"{fmt} share {share}")


@pytest.mark.parametrize("fmt,dtype,d,share,page", [
    ("int8", torch.bfloat16, 128, 7, 48), ("fp8", torch.float16, 128, 1, 16), ("int4", torch.bfloat16, 64, 4, 64),
    ("fp8", torch.bfloat16, 64, 1, 80), ("int4", torch.float16, 128, 7, 16), ("int8", torch.float16, 64, 3, 128)])
@pytest.mark.parametrize("t", [2, 3, 9, 16, 17, 33, 64, 100])
def test_trees(fmt, dtype, d, share, page, t):
    c = Case(fmt, [0, 1, 63, 130, 333], t, 2, d, page, seed=t)
    tree = random_tree(c.g, 5, t)
    q = c.q(2 * share, dtype, 2.0)
    c.check(q, tree, what="tree")
    c.check(q, None, what="chain")
    tree[:, 1] = False              # token 1 sees no new token,
    tree[2, :, :] = False           # and in sequence 2 nobody does
    tree[4, 0] = True               # a row that sees all of them
    out, lse = c.check(q, tree, what="holes")
    assert (out[0, 1] == 0).all() and torch.isinf(lse[0, 1]).all()  # no context either: a row of nothing
    c.check(q, tree[4].to(torch.uint8) * 255, what="one tree for all")


def test_masked_drafts_may_hold_anything():
    """New tokens that nobody sees are padding: their codes and scales may be junk."""
    c = Case("fp8", [0, 40, 130], 20, 2, 128, 16)
    tree = random_tree(c.g, 3, 20)
    tree[:, :, 7] = False
    tree[:, :, 19] = False
    q = c.q(14, torch.bfloat16)
    want = c.run(q, tree)
    for b, n in enumerate(c.lens):
        for j in (7, 19):
            page, off = int(c.table[b, (n + j) // 16]), (n + j) % 16
            for s in (c.cache.k_scale, c.cache.v_scale):
                s[page, :, off] = float("nan")
            for s in (c.cache.k_codes, c.cache.v_codes):
                s.view(torch.uint8)[page, :, off] = 0x7F
    got, lse = c.check(q, tree)
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("t,share", [(1, 7), (1, 1), (12, 7), (40, 1)])
def test_long_contexts(fmt, t, share):
    """One sequence over many blocks, joined; and a ragged batch."""
    c = Case(fmt, [7001], t, 1, 128, 64)
    c.check(c.q(share, torch.bfloat16, 3.0), random_tree(c.g, 1, t), what="long")
    c = Case(fmt, [3000, 5, 0, 900, 1777], t, 2, 64, 32)
    c.check(c.q(2 * share, torch.float16, 3.0), random_tree(c.g, 5, t), what="ragged")


@pytest.mark.parametrize("t", [1, 24])
def test_large_scores_and_unequal_rows(t):
    """Scores of hundreds (one key takes all), value rows of very unequal size, scores all equal."""
    c = Case("int8", [300, 77], t, 2, 128, 16, spread=3.0)
    c.check(c.q(14, torch.float16, 20.0), what="sharp")
    c.check(c.q(14, torch.bfloat16, 1e-4), what="flat")
    c.check(c.q(14, torch.bfloat16, 3000.0), scale=1e-3, what="scaled")


@pytest.mark.parametrize("t,share,batch", [(1, 1, 129), (1, 3, 300), (20, 1, 257), (3, 3, 128)])
def test_large_ragged_batches(t, share, batch):
    """More sequences than one chunk of the length scan holds, many of them without a context."""
    g = torch.Generator().manual_seed(batch)
    lens = (torch.rand(batch, generator=g) ** 4 * 300).int().tolist()
    c = Case("int8", lens, t, 1, 64, 16, seed=batch)
    c.check(c.q(share, torch.float16), what="batch")


@pytest.mark.parametrize("t,share", [(1, 4), (10, 4)])
def test_values_far_apart_in_size(t, share):
    """Value scales that grow by 2^40 along the context, and ones that fall; rows of zeros."""
    for sign in (1, -1):
        c = Case("int8", [400], t, 1, 64, 16)
        j = torch.arange(400 + t)
        factor = torch.exp2(sign * (j.double() / (400 + t) * 40 - 20))
        page, off = c.table[0].long()[j // 16], j % 16
        c.cache.v_scale[page.to(DEV), :, off.to(DEV)] *= factor.float().to(DEV)[:, None]
        s = c.cache.v_scale.cpu()[page, :, off].double()
        c.v[0] = numbers(c.cache.v_codes, "int8")[page, :, off].double() * s[..., None]
        c.check(c.q(share, torch.float16), what=f"factor {sign}")
    c = Case("int8", [100], t, 1, 64, 16)
    c.cache.v_scale.fill_(0.0)
    c.v[0] = c.v[0] * 0
    out, _ = c.check(c.q(share, torch.float16), what="zero values")
    assert (out == 0).all()


@pytest.mark.parametrize("t,share", [(1, 7), (5, 7), (30, 2)])
def test_strides_and_alignment(t, share):
    c = Case("int8", [100, 33, 0], t, 2, 128, 16)
    tree = random_tree(c.g, 3, t)
    q = c.q(2 * share, torch.bfloat16)
    want = c.run(q, tree)
    n = q.numel()
    flat = torch.zeros(n + 8, dtype=torch.bfloat16)
    for shift in (1, 4):
        x = flat.to(DEV)
        x[shift:shift + n] = q.to(DEV).flatten()
        assert torch.equal(c.run(x[shift:shift + n].view(q.shape), tree), want)
    wide = torch.zeros(3, t, 4 * share, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, :, 1::2] = q.to(DEV)
    assert torch.equal(c.run(wide[:, :, 1::2], tree), want)
    byhead = q.to(DEV).permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    assert torch.equal(c.run(byhead, tree), want)
    big = torch.zeros(3, t, t + 3, dtype=torch.bool)
    big[:, :, 3:] = tree
    assert torch.equal(c.run(q, big.to(DEV)[:, :, 3:]), want)
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    assert c.run(q, tree, out=out) is out and torch.equal(out, want)
    table = torch.zeros(3, 2 * c.table.shape[1], dtype=torch.int32, device=DEV)
    table[:, ::2] = c.table.to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    assert torch.equal(tl.tree_attention(q.to(DEV), c.cache, table[:, ::2], lens, tree.to(DEV)), want)


@pytest.mark.parametrize("t,share", [(1, 7), (20, 4)])
def test_streams_graphs_and_repeats(t, share):
    c = Case("fp8", [2500, 10, 700], t, 2, 128, 64)
    tree = random_tree(c.g, 3, t).to(DEV)
    q = c.q(2 * share, torch.bfloat16).to(DEV)
    table, lens = c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV)

    def call(**kw):
        return tl.tree_attention(q, c.cache, table, lens, tree, **kw)

    want = call()
    for _ in range(5):
        assert torch.equal(call(), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = call()
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens.sub_(5).clamp_(min=0)  # a graph's lengths are read on the device
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call()) and not torch.equal(out, want)


def test_empty():
    c = Case("int8", [5, 6], 3, 1, 64, 16)
    q = c.q(2, torch.float16).to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    assert tl.tree_attention(q[:0], c.cache, c.table.to(DEV)[:0], lens[:0]).shape == (0, 3, 2, 64)
    out, lse = tl.tree_attention(q[:, :0], c.cache, c.table.to(DEV), lens, return_lse=True)
    assert out.shape == (2, 0, 2, 64) and lse.shape == (2, 0, 2)


@pytest.mark.parametrize("t,share", [(1, 2), (20, 2)])
def test_indices_out_of_range(t, share):
    c = Case("int8", [40, 9], t, 1, 64, 16)
    c.cache.k_scale.nan_to_num_(nan=1.0, posinf=1.0, neginf=1.0).clamp_(max=10.0)
    c.cache.v_scale.nan_to_num_(nan=1.0, posinf=1.0, neginf=1.0).clamp_(max=10.0)
    q = c.q(share, torch.float16).to(DEV)
    good = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    want = tl.tree_attention(q, c.cache, c.table.to(DEV), good)
    for bad_len in (-3, 1 << 30):
        lens = good.clone()
        lens[0] = bad_len
        got = tl.tree_attention(q, c.cache, c.table.to(DEV), lens)
        torch.cuda.synchronize()
        assert tl.device_status(clear=True) == 5
        assert torch.equal(got[1], want[1]) and torch.isfinite(got).all()
    for bad_page in (-1, c.cache.pages, 2 ** 31 - 1):
        table = c.table.to(DEV).clone()
        table[0, 1] = bad_page
        got = tl.tree_attention(q, c.cache, table, good)
        torch.cuda.synchronize()
        assert tl.device_status(clear=True) == 5
        assert torch.equal(got[1], want[1]) and torch.isfinite(got).all()


@pytest.mark.parametrize("t", [1, 20])
def test_offsets_beyond_32_bits(t):
    """Pages whose rows start past 2^32 bytes of codes."""
    page, hk, d = 64, 4, 128
    pages = (1 << 32) // (page * hk * d) + 3
    cache = tl.KVCache.empty("int8", pages, page, hk, d)
    n = 150
    table = torch.tensor([[pages - 1, 0, pages - 2, 1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    y = torch.randn(2, n + t, hk, d, generator=g)
    j = torch.arange(n + t)
    slots = (table[0].long()[j // page] * page + j % page).to(DEV)
    tl.kv_append(cache, y[0].to(torch.float16).to(DEV), y[1].to(torch.float16).to(DEV), slots)
    k, v = tl.kv_read(cache, slots, torch.float32)
    q = torch.randn(1, t, 8, d, generator=g).to(torch.float16)
    out, lse = tl.tree_attention(q.to(DEV), cache, table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                                 return_lse=True)
    sees = torch.cat([torch.ones(t, n, dtype=torch.bool), torch.tril(torch.ones(t, t, dtype=torch.bool))], 1)
    # fp32 values of the cache are its products rounded once: inside the score's bound
    check_attention(out[0], lse[0], attention64(q[0], k.double().cpu(), v.double().cpu(), sees, d ** -0.5), q.dtype)


def test_scores_with_nan_stay_in_their_rows():
    """A NaN in a key that one token sees reaches that token alone."""
    c = Case("int8", [0], 4, 1, 64, 16)
    page = int(c.table[0, 0])
    c.cache.k_scale[page, :, 2] = float("nan")
    q = c.q(1, torch.float16)
    tree = torch.eye(4, dtype=torch.bool)
    out = c.run(q, tree)
    bad = torch.isnan(out).flatten(2).any(-1)[0].tolist()
    assert bad == [False, False, True, False]
    assert math.isfinite(float(out[0, 0].abs().sum()))
