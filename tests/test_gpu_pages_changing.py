"""Pages taken while another stream writes what rows want: the answers are then of no use, but the call returns, no page is given
to two rows by one call, and the next call is right."""
import random

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

import pages_ref as ref

pytestmark = pytest.mark.gpu
DEV, VALUE = "cuda", 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("fork", [False, True])
def test_blocks_of_a_cluster_return(fork):
    """A pool of eight blocks' runs of pages, wants that go from nothing to something and back."""
    rows, pages, page = 300, 270001, 16
    want = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    other = torch.cuda.Stream()
    pool = tl.KVPages.empty(pages, rows, 8, page)
    zero = torch.zeros(rows, dtype=torch.int32, device=DEV)
    parent = zero.clone()
    parent[0] = -1
    torch.cuda.synchronize()
    for step in range(40):
        if fork:  # row 0 holds a page in part, the others none
            first = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
            first[0] = 5
            tl.pages_free(pool, zero)
            tl.pages_reserve(pool, first, 0)
            tl.pages_free(pool, first)
        else:
            tl.pages_free(pool, zero)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(15):
                want.fill_(-1)
                want.copy_(parent if fork else zero + 20)
        for _ in range(3 if not fork else 1):
            if fork:
                tl.pages_fork(pool, want)
            else:
                tl.pages_reserve(pool, want, 2)
        torch.cuda.synchronize()
        assert int(pool.refs.min()) >= 0 and int(pool.refs.max()) <= 1
    tl.device_status()
    state = [t.zero_().cpu() for t in (pool.refs, pool.table, pool.lens, pool.held)]
    plain, rng = ref.Pages(page, *state), random.Random(1)
    extra = [rng.choice((0, 5, 40, -1)) for _ in range(rows)]
    slots, ok = tl.pages_reserve(pool, torch.tensor(extra, dtype=torch.int32, device=DEV), 3)
    slots64, ok64 = plain.reserve(extra, 3)
    assert torch.equal(slots.cpu(), slots64) and torch.equal(ok.cpu(), ok64)
    for name, w in zip(("refs", "table", "lens", "held"), plain.tensors()):
        assert torch.equal(getattr(pool, name).cpu(), w), name
