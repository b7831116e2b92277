"""Pages and entries of the cache on the GPU: every integer and every byte equals the plain form's."""
import random

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

import pages_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
VALUE = 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def filled(fmt, pages, page, heads, dim, layers, seed=0):
    """Layers of caches with every byte set at random."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for _ in range(layers):
        c = tl.KVCache.empty(fmt, pages, page, heads, dim)
        for t in (c.k_codes, c.v_codes):
            t.view(torch.uint8).random_(0, 256, generator=gen)
        for t in (c.k_scale, c.v_scale):
            t.view(torch.int32).random_(0, 1 << 31, generator=gen)
        out.append(c)
    return out


def pool(rng, rows, pages, wide, page, fill=0.6, share=True):
    """A pool in use: rows of random lengths, some with pages ahead, some that share their first pages."""
    table = torch.zeros(rows, wide, dtype=torch.int32)
    lens, held, refs = torch.zeros(rows, dtype=torch.int32), torch.zeros(rows, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32)
    free = list(range(pages))
    rng.shuffle(free)
    free = free[:int(fill * pages)]
    for r in range(rows):
        n = rng.randrange(0, min(wide, max(1, 2 * int(fill * pages) // rows)) + 1)
        n = min(n, len(free))
        mine = [free.pop() for _ in range(n)]
        if share and r % 3 == 1 and n > 1:
            both = min(n, int(held[r - 1])) // 2
            mine[:both] = table[r - 1, :both].tolist()
            lens[r - 1] = max(int(lens[r - 1]), both * page)
        table[r, :n] = torch.tensor(mine, dtype=torch.int32)
        held[r] = n
        low = (n // 2) * page
        lens[r] = rng.randrange(low, n * page + 1) if n else 0
        for p in mine:
            refs[p] += 1
    return refs, table, lens, held


def handle(page, state):
    return tl.KVPages(page, *(t.clone().to(DEV) for t in state))


def same(pages, want):
    for name, w in zip(("refs", "table", "lens", "held"), want.tensors()):
        assert torch.equal(getattr(pages, name).cpu(), w), name


SIZES = [(1, 3, 2, 16), (5, 40, 9, 16), (16, 700, 64, 48), (37, 1024, 30, 64), (1025, 9000, 11, 16), (300, 40000, 150, 32),
         (2500, 270001, 120, 16)]


@pytest.mark.parametrize("rows,pages,wide,page", SIZES)
def test_steps_of_a_server(rows, pages, wide, page):
    """Free, reserve, fork, in turn, over several rounds: tables, counts, lengths, slots and answers."""
    rng = random.Random(rows * 7 + pages)
    state = pool(rng, rows, pages, wide, page)
    got, want = handle(page, state), ref.Pages(page, *state)
    for step in range(4):
        keep = []
        for r in range(rows):
            n, top = want.lens[r], want.held[r] * page
            shared = max([i + 1 for i in range(want.held[r]) if want.refs[want.table[r][i]] > 1], default=0) * page
            what = rng.random()
            keep.append(-1 if what < 0.2 else 0 if what < 0.35 else rng.randrange(min(max(n - 9, shared), top), top + 1))
        tl.pages_free(got, torch.tensor(keep, dtype=torch.int32, device=DEV))
        want.free(keep)
        same(got, want)
        extra = [rng.choice((-1, 0, 1, 5, 17)) for _ in range(rows)]
        extra = [min(e, wide * page - want.lens[r]) for r, e in enumerate(extra)]
        slots, ok = tl.pages_reserve(got, torch.tensor(extra, dtype=torch.int32, device=DEV), 7)
        slots64, ok64 = want.reserve(extra, 7)
        assert torch.equal(ok.cpu(), ok64) and torch.equal(slots.cpu(), slots64)
        same(got, want)
        full = [r for r in range(rows) if want.lens[r] > 0 and want.lens[r] <= want.held[r] * page]
        parent = [-1] * rows
        for r in range(rows):
            if want.held[r] == 0 and full and rng.random() < 0.7:
                parent[r] = rng.choice(full)
        ok = tl.pages_fork(got, torch.tensor(parent, dtype=torch.int32, device=DEV))
        ok64, _ = want.fork(parent)
        assert torch.equal(ok.cpu(), ok64)
        same(got, want)
    assert not want.flags


def test_lowest_pages_in_order_and_nothing_beyond_the_free_ones():
    """Seven free pages; rows want 2, 0, 3, 3, 0, 1: the first two wants fit, the fourth and all later ones do not."""
    got = tl.KVPages.empty(9, 6, 4, 16)
    got.refs[2] = 1
    got.refs[5] = 4
    extra = torch.tensor([17, 0, 48, 33, -1, 16], dtype=torch.int32, device=DEV)
    slots, ok = tl.pages_reserve(got, extra, 2)
    assert ok.tolist() == [True, True, True, False, True, False]
    assert got.held.tolist() == [2, 0, 3, 0, 0, 0]
    assert got.table.tolist() == [[0, 1, 0, 0], [0] * 4, [3, 4, 6, 0], [0] * 4, [0] * 4, [0] * 4]
    assert got.refs.tolist() == [1, 1, 1, 1, 1, 4, 1, 0, 0]
    assert slots.tolist() == [[0, 1], [-1, -1], [48, 49], [-1, -1], [-1, -1], [-1, -1]]
    assert got.lens.tolist() == [0] * 6


def test_a_fresh_large_pool():
    """Needs of thousands of pages at once, from the front of the pool."""
    got = tl.KVPages.empty(60000, 700, 60, 16)
    extra = torch.full((700,), 16 * 60 - 3, dtype=torch.int32, device=DEV)
    slots, ok = tl.pages_reserve(got, extra, 3)
    assert ok.all()
    assert torch.equal(got.table.cpu(), torch.arange(700 * 60, dtype=torch.int32).view(700, 60))
    assert int(got.refs.sum()) == 42000 and torch.equal(got.refs[:42000], torch.ones_like(got.refs[:42000]))
    assert torch.equal(slots[:, 0].cpu(), torch.arange(700) * 960)


@pytest.mark.parametrize("what", ["keep", "held", "lens", "table", "extra", "parent", "chain", "busy", "cut", "twice"])
def test_rows_that_cannot_be_served(what):
    """The row is left as it is, the status word is set, the other rows are served."""
    page, rows, wide = 16, 6, 5
    state = [torch.tensor([1, 1, 2, 1, 1, 0, 0, 0, 0, 0], dtype=torch.int32),
             torch.tensor([[0, 1, 0, 0, 0], [2, 3, 0, 0, 0], [2, 4, 0, 0, 0], [0] * 5, [0] * 5, [0] * 5], dtype=torch.int32),
             torch.tensor([20, 30, 32, 0, 0, 0], dtype=torch.int32), torch.tensor([2, 2, 2, 0, 0, 0], dtype=torch.int32)]
    keep, extra, parent = [-1] * 6, [-1] * 6, [-1] * 6
    if what == "keep":
        keep = [33, 3, -1, 1, -1, -1]
    elif what == "held":
        state[3][0] = 6
        keep, extra = [3, -1, -1, -1, -1, -1], [1, -1, -1, 5, -1, -1]
    elif what == "lens":
        state[2][0] = -5
        extra, parent = [3, 3, -1, -1, 2, -1], [-1, -1, -1, 0, -1, 2]
    elif what == "table":
        state[1][0, 1] = 10
        keep, extra = [4, -1, -1, -1, -1, -1], [5, -1, -1, -1, -1, -1]
    elif what == "extra":
        extra = [61, 50, 1 << 30, 3, -1, -1]
    elif what == "parent":
        parent = [-1, -1, -1, 6, 1 << 30, 0]
    elif what == "chain":
        parent = [-1, -1, -1, 0, 3, 4]
    elif what == "busy":
        parent = [1, -1, -1, 1, -1, -1]
    elif what == "cut":           # row 1 is cut inside the page that row 2 shares
        keep, extra = [-1, 10, -1, -1, -1, -1], [3, 1, 4, -1, -1, -1]
    elif what == "twice":         # a page whose count is 0 already
        state[0][1] = 0
        keep = [0, 0, -1, -1, -1, -1]
    got, want = handle(page, state), ref.Pages(page, *state)
    dev = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (keep, extra, parent)]
    tl.pages_free(got, dev[0])
    want.free(keep)
    slots, ok = tl.pages_reserve(got, dev[1], 4)
    slots64, ok64 = want.reserve(extra, 4)
    assert torch.equal(ok.cpu(), ok64) and torch.equal(slots.cpu(), slots64)
    ok = tl.pages_fork(got, dev[2])
    ok64, _ = want.fork(parent)
    assert torch.equal(ok.cpu(), ok64)
    same(got, want)
    assert want.flags and tl.device_status() == VALUE


@pytest.mark.parametrize("fmt,page,heads,dim,layers", [("int8", 16, 2, 64, 1), ("fp8", 64, 4, 128, 3), ("int4", 48, 1, 64, 2), ("int4", 16, 3, 128, 66)])
def test_fork_copies_the_last_page(fmt, page, heads, dim, layers):
    """Only the places in use are copied; pages run out for the last rows."""
    rng, rows, pages = random.Random(page + dim), 23, 60
    state = pool(rng, rows, pages, 9, page, fill=0.75, share=False)
    for r in range(8, rows):
        for p in state[1][r, :state[3][r]].tolist():
            state[0][p] -= 1
        state[1][r], state[2][r], state[3][r] = 0, 0, 0
    caches = filled(fmt, pages, page, heads, dim, layers)
    parent = [-1] * 8 + [r % 8 for r in range(8, rows)]
    got, want = handle(page, state), ref.Pages(page, *state)
    old = [ref.raw(c) for c in caches]
    ok = tl.pages_fork(got, torch.tensor(parent, dtype=torch.int32, device=DEV), caches)
    ok64, copies = want.fork(parent)
    assert torch.equal(ok.cpu(), ok64)
    same(got, want)
    src = [s * page + i for s, _, n in copies for i in range(n)]
    dst = [d * page + i for _, d, n in copies for i in range(n)]
    assert len(src) > 0
    for c, o in zip(caches, old):
        ref.move(o, src, dst, page)
        for a, b in zip(ref.raw(c), o):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt,page,heads,dim,layers,n", [("int8", 16, 1, 64, 1, 1), ("fp8", 128, 4, 128, 2, 9), ("int4", 48, 2, 64, 65, 5),
                                                         ("int8", 512, 1, 128, 1, 3), ("int4", 64, 3, 128, 1, 400)])
def test_copy(fmt, page, heads, dim, layers, n):
    rng, pages = random.Random(n), 2 * n + 3
    caches = filled(fmt, pages, page, heads, dim, layers)
    order = list(range(pages))
    rng.shuffle(order)
    src, dst = order[:n], order[n:2 * n]
    tokens = [rng.randrange(0, page + 1) for _ in range(n)]
    if n > 4:
        src[1], dst[3] = -1, -1
        src[4] = src[0]                     # one page copied twice
    pairs = [(s, d, t) for s, d, t in zip(src, dst, tokens) if s >= 0 and d >= 0]
    as_dev = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (src, dst, tokens)]
    for counts in (as_dev[2], None):
        old = [ref.raw(c) for c in caches]
        tl.kv_copy(tl.KVLayers(caches), as_dev[0], as_dev[1], counts)
        for c, o in zip(caches, old):
            ref.move(o, [s * page + i for s, _, t in pairs for i in range(t if counts is not None else page)],
                     [d * page + i for _, d, t in pairs for i in range(t if counts is not None else page)], page)
            for a, b in zip(ref.raw(c), o):
                assert torch.equal(a, b)


def test_copy_refuses_pages_and_counts():
    caches = filled("int8", 6, 16, 1, 64, 1)
    old = ref.raw(caches[0])
    src, dst, tokens = ([6, 0, 1, 2], [1, 1 << 30, 3, 4], [16, 16, 17, 5])
    tl.kv_copy(caches[0], *(torch.tensor(v, dtype=torch.int32, device=DEV) for v in (src, dst, tokens)))
    ref.move(old, [2 * 16 + i for i in range(5)], [4 * 16 + i for i in range(5)], 16)
    for a, b in zip(ref.raw(caches[0]), old):
        assert torch.equal(a, b)
    assert tl.device_status() == VALUE


@pytest.mark.parametrize("fmt,heads,dim", [("int8", 2, 128), ("fp8", 1, 64), ("int4", 3, 128), ("int4", 1, 64)])
@pytest.mark.parametrize("batch,n,page,layers", [(40, 130, 32, 24), (1, 1, 16, 1), (5, 17, 16, 3), (33, 64, 64, 2), (3, 65, 48, 1), (4, 1000, 32, 2), (2, 5000, 64, 1)])
def test_compact(fmt, heads, dim, batch, n, page, layers):
    """Paths of drafted trees (n up to 64) and contexts of which a part is kept, in place."""
    rng = random.Random(batch * n + dim)
    start = [rng.randrange(0, 40) for _ in range(batch)]
    wide = -(-(max(start) + 2 * n) // page) + 1
    pages = batch * wide + 2
    order = list(range(pages))
    rng.shuffle(order)
    table = [order[b * wide:(b + 1) * wide] for b in range(batch)]
    keep = [sorted(rng.sample(range(2 * n), n)) for _ in range(batch)]
    count = [rng.randrange(0, n + 1) for _ in range(batch)]
    count[0] = n
    if batch > 2:
        count[1], keep[2], count[2] = 0, list(range(n)), n   # nothing, and everything where it is
    if batch > 3:
        keep[3], count[3] = list(range(1, n + 1)), n         # every entry one place on
    caches = filled(fmt, pages, page, heads, dim, layers, seed=n)
    old = [ref.raw(c) for c in caches]
    dev = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (table, start, keep, count)]
    tl.kv_compact(caches, *dev)
    moves, flags = ref.compact(table, page, start, keep, count, wide * page)
    assert not flags
    for c, o in zip(caches, old):
        ref.move(o, [s for s, _ in moves], [d for _, d in moves], page)
        for a, b in zip(ref.raw(c), o):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [20, 700])
def test_compact_stops_where_keep_is_wrong(n):
    """keep that repeats, falls, leaves the table or begins below 0; counts out of range; a start below 0."""
    batch, page, wide = 8, 16, 2 * n // 16 + 2
    table = [[b * wide + i for i in range(wide)] for b in range(batch)]
    keep = [[i + i // 3 + 1 for i in range(n)] for _ in range(batch)]
    start, count = [3] * batch, [n] * batch
    keep[0][n // 2] = keep[0][n // 2 - 1]
    keep[1][n - 3] = 1
    keep[2][n - 1] = wide * page - 3
    keep[3][0] = -1
    count[4], count[5], start[6] = n + 1, -2, -1
    keep[7] = [n + 9] + list(range(n - 1))
    caches = filled("int8", batch * wide, page, 2, 64, 1)
    old = ref.raw(caches[0])
    tl.kv_compact(caches, *(torch.tensor(v, dtype=torch.int32, device=DEV) for v in (table, start, keep, count)))
    moves, flags = ref.compact(table, page, start, keep, count, wide * page)
    ref.move(old, [s for s, _ in moves], [d for _, d in moves], page)
    for a, b in zip(ref.raw(caches[0]), old):
        assert torch.equal(a, b)
    assert flags and tl.device_status() == VALUE


def test_compact_skips_pages_that_the_cache_does_not_have():
    page, n = 16, 5
    table = [[0, 9, 1], [2, 3, 4]]
    caches = filled("int8", 6, page, 1, 64, 1)
    old = ref.raw(caches[0])
    dev = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (table, [0, 0], [[1, 17, 33, 34, 35], [1, 17, 33, 34, 35]], [n, n])]
    tl.kv_compact(caches, *dev)
    moves, _ = ref.compact([table[1]], page, [0], [[1, 17, 33, 34, 35]], [n], 48)
    keep = [(1, 0), (16 + 1, 2), (16 + 2, 3), (16 + 3, 4)]  # of the first sequence: all but the entry of page 9
    ref.move(old, [s for s, _ in moves] + [s for s, _ in keep], [d for _, d in moves] + [d for _, d in keep], page)
    for a, b in zip(ref.raw(caches[0]), old):
        assert torch.equal(a, b)
    assert tl.device_status() == VALUE


def test_captured_steps():
    """A step captured once and replayed: the arrays on the device decide each time."""
    page, rows = 16, 9
    pages = tl.KVPages.empty(64, rows, 7, page)
    caches = filled("int8", 64, page, 1, 64, 2)
    layers = tl.KVLayers(caches)
    keep, extra = (torch.zeros(rows, dtype=torch.int32, device=DEV) for _ in "ke")
    parent = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tl.pages_free(pages, keep)
        tl.pages_reserve(pages, extra, 4)
        tl.pages_fork(pages, parent, layers)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.pages_free(pages, keep)
        slots, ok = tl.pages_reserve(pages, extra, 4)
        forked = tl.pages_fork(pages, parent, layers)
    want = ref.Pages(page, pages.refs, pages.table, pages.lens, pages.held)
    rng = random.Random(3)
    for step in range(12):
        k = [rng.choice((-1, 0, min(want.lens[r] + 4, want.held[r] * page))) for r in range(rows)]
        for r in range(rows):  # no cut inside a shared page
            if 0 < k[r] and any(want.refs[p] > 1 for p in want.table[r][k[r] // page:want.held[r]]):
                k[r] = -1
        keep.copy_(torch.tensor(k))
        want.free(k)
        e = [rng.randrange(0, 20) if want.lens[r] + 20 <= 7 * page else 0 for r in range(rows)]
        extra.copy_(torch.tensor(e))
        slots64, ok64 = want.reserve(e, 4)
        p = [rng.choice([-1] + [q for q in range(rows) if want.lens[q] > 0 and want.held[q] > 0]) if want.held[r] == 0 else -1 for r in range(rows)]
        p = [-1 if q >= 0 and p[q] >= 0 else q for q in p]
        parent.copy_(torch.tensor(p))
        old = [ref.raw(c) for c in caches]
        forked64, copies = want.fork(p)
        graph.replay()
        assert torch.equal(slots.cpu(), slots64) and torch.equal(ok.cpu(), ok64) and torch.equal(forked.cpu(), forked64)
        same(pages, want)
        for c, o in zip(caches, old):
            ref.move(o, [s * page + i for s, _, n in copies for i in range(n)], [d * page + i for _, d, n in copies for i in range(n)], page)
            for a, b in zip(ref.raw(c), o):
                assert torch.equal(a, b)
    assert not want.flags
