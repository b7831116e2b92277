"""Sizes at the edge of 32-bit key counts (no GPU): a call whose tile arithmetic would not fit is refused."""
import ctypes

import pytest

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import attention

SHAPE, CUDA = 2, 6
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    tl.build()
    tl.load()
    return attention._lib()


@pytest.mark.parametrize("page", [16, 64, 80, 1 << 20])
def test_keys_of_a_sequence_leave_room_for_a_tile(lib, page):
    """Tiles of up to 128 keys are counted with (keys + 127) / 128 and addressed by their first key
    plus a place within, all in 31 bits."""
    cache = ctypes.byref(attention._Cache(A, B, C, D, 4, page, 2, 64, 0))

    def call(wide):
        lib.ternary_test_inject_launch_failures(1)  # nothing is launched, whatever the answer
        try:
            return lib.ternary_tree_attention(A, 768, 256, 64, 1, 2, 3, 4, cache, B, wide, wide, C, None, 0, 0, 0.125, D, None, A,
                                              1 << 40, None)
        finally:
            lib.ternary_test_inject_launch_failures(0)

    most = ((1 << 31) - 256) // page
    assert call(most) == CUDA            # accepted (and stopped by the injected failure)
    assert call(most + 1) == SHAPE
    w = lib.ternary_tree_attention_workspace
    assert w(2, 3, 4, 2, 64, most * page) > 0 and w(2, 3, 4, 2, 64, (1 << 31) - 255) == -1
