"""Offsets beyond 32 bits, and calls on several streams at once: pages, entries, adapters, verification."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

import pages_ref as ref
import verify_ref
from test_gpu_lora import close, exact, make
from test_gpu_verify import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def free_bytes(n):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < n:
        pytest.skip("not enough device memory")


@pytest.fixture(scope="module")
def far_cache():
    """300000 pages of 16 x 8 x 128 bytes, keys and values: 4.9 GB each, the last pages beyond 2^32 bytes."""
    free_bytes(14 << 30)
    cache = tl.KVCache.empty("int8", 300000, 16, 8, 128)
    yield cache
    del cache
    torch.cuda.empty_cache()


def fill(cache, pages, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    for p in pages:
        for t in (cache.k_codes, cache.v_codes):
            t[p].view(torch.uint8).random_(0, 256, generator=gen)
        for t in (cache.k_scale, cache.v_scale):
            t[p].uniform_(generator=gen)


def page_bytes(cache, p):
    return [t[p].clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]


def test_copy_and_fork_of_far_pages(far_cache):
    last = 299999
    fill(far_cache, [3, last], 1)
    near, far = page_bytes(far_cache, 3), page_bytes(far_cache, last)
    tl.kv_copy(far_cache, i32([3, last]), i32([last - 1, 4]), i32([16, 16]))
    for got, want in ((page_bytes(far_cache, last - 1), near), (page_bytes(far_cache, 4), far)):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    refs = torch.ones(300000, dtype=torch.int32, device=DEV)
    refs[last - 7] = 0
    table = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    table[0, 0], table[0, 1] = 3, last
    pages = tl.KVPages(16, refs, table, i32([16 + 9, 0]), i32([2, 0]))
    blank = page_bytes(far_cache, last - 7)
    assert tl.pages_fork(pages, i32([-1, 0]), far_cache).tolist() == [True, True]
    assert table[1, :2].tolist() == [3, last - 7] and pages.lens.tolist() == [25, 25]
    # codes and scales are [page, head, place, ..]
    for got, want, old in zip(page_bytes(far_cache, last - 7), far, blank):
        assert torch.equal(got[:, :9], want[:, :9]) and torch.equal(got[:, 9:], old[:, 9:])
    assert tl.device_status() == 0


@pytest.mark.parametrize("n", [20, 500])
def test_compact_of_far_pages(far_cache, n):
    """A few moves (a warp each) and many (a block): from pages at the end of the pool to others there and at its beginning."""
    last, wide = 299999, 2 * n // 16 + 2
    table = [[last - 2 * i if i % 2 else i for i in range(wide)]]
    fill(far_cache, table[0], n)
    old = [page_bytes(far_cache, p) for p in table[0]]
    keep = [2 * i + 1 for i in range(n)]
    tl.kv_compact(far_cache, i32(table), i32([5]), i32([keep]), i32([n]))
    want = [[t.clone() for t in page] for page in old]
    for i, k in enumerate(keep):
        for to, frm in zip(want[(5 + i) // 16], old[(5 + k) // 16]):
            to[:, (5 + i) % 16] = frm[:, (5 + k) % 16]
    for p, w in zip(table[0], want):
        for a, b in zip(page_bytes(far_cache, p), w):
            assert torch.equal(a, b)
    assert tl.device_status() == 0


@pytest.mark.parametrize("gated", [False, True])
def test_adapters_between_far_rows(gated):
    """Rows of x, y and out more than 2^32 bytes apart."""
    free_bytes(20 << 30)
    tokens, far = 3, (1 << 30) + 8
    x, y, a, b, s, which = make(tokens, 256, (64, 64), 16, 2, torch.bfloat16, torch.bfloat16, seed=3)
    which = i32([0, 1, 0])
    flat = torch.empty(tokens * far, dtype=torch.bfloat16, device=DEV)
    rows = [flat.as_strided((tokens, n), (far, 1), at) for n, at in ((256, 0), (128, 512), (128, 1024))]
    rows[0].copy_(x), rows[1].copy_(y)
    ad = tl.Adapters(a, b, s, shards=(64, 64))
    call, out = (tl.lora_silu_mul, rows[2][:, :64]) if gated else (tl.lora_add, rows[2])
    assert torch.equal(call(rows[0], ad, which, rows[1], out=out), call(x, ad, which, y))
    if not gated:
        close(out, *exact(x, y, a, b, s, which, (64, 64)))


def test_many_adapters_of_far_matrices():
    """B beyond 2^32 bytes (and A beyond 2^31 elements)."""
    free_bytes(30 << 30)
    n, rank, inputs_, outputs = 2048, 64, 18944, 18944
    a = torch.empty(n, rank, inputs_, dtype=torch.bfloat16, device=DEV)
    b = torch.empty(n, outputs, rank, dtype=torch.bfloat16, device=DEV)
    which = i32([2047, 0, -1, 2046, 2047])
    x, y, a2, b2, s, _ = make(5, inputs_, (outputs,), rank, 3, torch.bfloat16, torch.bfloat16, seed=4)
    for to, i in ((2047, 0), (0, 1), (2046, 2)):
        a[to], b[to] = a2[i], b2[i]
    got = tl.lora_add(x, tl.Adapters(a, b), which, y)
    close(got, *exact(x, y, a2, b2, None, i32([0, 1, -1, 2, 0]), (outputs,)))


def test_verification_between_far_rows():
    free_bytes(20 << 30)
    p, q, tokens, u = inputs(2, 3, 5000, torch.bfloat16, None, seed=8)
    far, node = (1 << 31) + 4096, 1 << 29
    flat = torch.empty(far + 3 * node + 16384, dtype=torch.bfloat16, device=DEV)
    wide = flat.as_strided((2, 4, 5000), (far, node, 1), 0)
    draft = flat.as_strided((2, 3, 5000), (far, node, 1), 8192)
    wide.copy_(p), draft.copy_(q)
    want = verify_ref.verify(p.cpu(), tokens.cpu(), u.cpu(), q.cpu())
    for g, w in zip(tl.verify_drafts(wide, tokens, u, draft=draft), want):
        assert torch.equal(g.cpu(), w)


@pytest.mark.parametrize("vocab", [1 << 20, (1 << 21) + 3])
def test_large_vocabulary(vocab):
    """More than 2^17 tokens: probabilities whose sums are exact in either arithmetic."""
    gen = torch.Generator(device=DEV).manual_seed(vocab)
    p = torch.randint(0, 3, (2, 2, vocab), generator=gen, device=DEV).float() * 2.0 ** -21
    q = torch.randint(0, 3, (2, 1, vocab), generator=gen, device=DEV).float() * 2.0 ** -21
    tokens = torch.tensor([[7], [vocab - 1]], device=DEV)
    q[0, 0, 7], q[1, 0, vocab - 1] = 2.0 ** -20, 2.0 ** -21
    p[0, 0, 7] = 0.0
    u = torch.tensor([[0.5, 0.25], [0.75, 0.999]], device=DEV)
    want = verify_ref.verify(p.cpu(), tokens.cpu(), u.cpu(), q.cpu())
    for g, w in zip(tl.verify_drafts(p, tokens, u, draft=q), want):
        assert torch.equal(g.cpu(), w)


def test_two_streams_at_once():
    """Calls in flight on two streams answer as one after the other: nothing is shared but the status word."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    lo, ve, co = [], [], []
    for i in range(2):
        lo.append(make(1500, 512, (96, 32), 16, 6, torch.bfloat16, torch.bfloat16, seed=20 + i))
        ve.append(inputs(6, 4, 20000, torch.float32, None, seed=30 + i))
        caches = [tl.KVCache.empty("int8", 64, 16, 2, 64) for _ in range(3)]
        for c in caches:
            fill(c, range(64), 40 + i)
        co.append((tl.KVLayers(caches), tl.KVPages.empty(64, 5, 12, 16)))
    ads = [tl.Adapters(v[2], v[3], v[4], shards=(96, 32)) for v in lo]
    extra = [i32([40, 3, 0, 100, 17]), i32([5, 60, 31, 1, 90])]
    keep, zeros, count = i32([[1, 2, 5, 8]] * 5), i32([0] * 5), i32([4, 3, 0, 4, 1])
    want = [(tl.lora_add(lo[i][0], ads[i], lo[i][5], lo[i][1]), *tl.verify_drafts(ve[i][0], ve[i][2], ve[i][3], draft=ve[i][1])) for i in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for step in range(10):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                layers, pages = co[i]
                slots, ok = tl.pages_reserve(pages, extra[i], 4)
                tl.kv_compact(layers, pages.table, zeros, keep, count)
                got[i] = (tl.lora_add(lo[i][0], ads[i], lo[i][5], lo[i][1]), *tl.verify_drafts(ve[i][0], ve[i][2], ve[i][3], draft=ve[i][1]), ok)
                tl.pages_free(pages, zeros)
        torch.cuda.synchronize()
        for i in range(2):
            for g, w in zip(got[i], want[i]):
                assert torch.equal(g, w)
            assert bool(got[i][-1].all()) and int(co[i][1].refs.sum()) == 0
    assert tl.device_status() == 0
