"""A table entry that names no page of the pool gives no slots."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

pytestmark = pytest.mark.gpu
DEV, VALUE = "cuda", 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("page", [-1, -(1 << 31), 8, 1 << 28, (1 << 31) - 1])
def test_reserve_gives_no_slots_of_pages_that_are_not_there(page):
    """Row 0's next tokens lie in a page held ahead that the pool does not have, then in one that it has; row 1 is served."""
    refs = torch.tensor([1, 0, 1, 1, 0, 0, 0, 0], dtype=torch.int32, device=DEV)
    table = torch.tensor([[0, page, 2, 0], [3, 0, 0, 0]], dtype=torch.int32, device=DEV)
    lens, held = torch.tensor([16, 5], dtype=torch.int32, device=DEV), torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    pool = tl.KVPages(16, refs, table, lens, held)
    slots, ok = tl.pages_reserve(pool, torch.tensor([18, 3], dtype=torch.int32, device=DEV), 18)
    assert ok.tolist() == [True, True]
    assert slots[0].tolist() == [-1] * 16 + [32, 33] and slots[1].tolist() == [53, 54, 55] + [-1] * 15
    assert tl.device_status() == VALUE
    assert table.tolist() == [[0, page, 2, 0], [3, 0, 0, 0]] and refs.tolist() == [1, 0, 1, 1, 0, 0, 0, 0]
