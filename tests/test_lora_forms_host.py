"""Which form the cases of the adapters' tests run (no GPU, nothing is launched): a rule that moves must not leave one untested."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from lora_forms import MANY32, tile
from test_gpu_lora import CASES, MANY

BF, H, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tl.build()
    tl.load()


@pytest.mark.parametrize("dtype", [BF, H])
def test_tiles_of_128(dtype):
    for case in MANY:
        assert tile(*case, dtype, dtype) == 128, case
    for case in MANY32:
        assert tile(*case, dtype, F) == 128, case
    assert tile(3100, 72, (136, 48), 48, 3, dtype, dtype) == 128          # tokens without an adapter among many
    assert tile(3100, 3008, (136, 48), 48, 3, dtype, F) == 128
    assert tile(2304, 264, (136,), 40, 3, dtype, dtype) == 128            # values that are no numbers
    assert tile(4100, 14000, (96,), 16, 3, dtype, dtype) == 128           # runs and orders
    assert tile(2000, 30000, (96,), 16, 6, dtype, dtype) == 128           # replayed
    for tokens, inputs, n in ((1100, 92000, 2), (3000, 37000, 5)):        # waits that run out
        assert tile(tokens, inputs, (96,), 16, n, dtype, dtype) == 128


@pytest.mark.parametrize("dtype", [BF, H])
def test_tiles_of_16(dtype):
    small = [c for c in CASES if c[0] < 1000]
    assert len(small) > 10 and all(tile(*c, dtype, out) == 16 for c in small for out in (dtype, F))
    assert tile(8192, 3584, (18944, 18944), 16, 6, dtype, dtype, gated=True) == 16
    assert tile(8192, 3584, (3584,), 72, 6, dtype, dtype) == 16           # ranks above 64
    assert tile(8192, 3588, (3584,), 64, 6, dtype, dtype) == 16           # rows that do not start on 16 bytes


def test_nothing_to_do_and_refused():
    assert tile(0, 64, (32,), 16, 2, BF, BF) == 0 and tile(5, 64, (0,), 16, 2, BF, BF) == 0
    assert tile(5, 64, (32,), 12, 2, BF, BF) == -1 and tile(5, 64, (32,), 16, 2, BF, H) == -1
