"""Blocks of kernels that hold tensor memory while they wait for their cluster, side by side on one SM (no GPU).

`tcgen05.alloc` waits without a limit.  Two clusters of different kernels, launched on two streams, may share two SMs: if an SM
takes blocks of both for more than its 512 columns, one cluster can hold on one SM what the other waits for, and the other way
round.  Shared memory decides what fits: every set of blocks that does has to find its columns."""
import itertools
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "ternary_weight_linear_02_gb300", "csrc")
KB, SM, COLUMNS = 1024, 228 * 1024, 512


def text(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def value(expr):
    """A constant expression of literals and of tc.cuh's constants."""
    consts = dict(re.findall(r"(kSmem\w+) = ([^,;]+)", text("tc.cuh")))
    expr = re.sub(r"(?:tc::)?(kSmem\w+)", lambda m: "(" + consts[m.group(1)] + ")", expr)
    assert re.fullmatch(r"[\d\s*+()]+", expr), expr
    return eval(expr)


def holders():
    """(kernel, columns, least bytes of shared memory of a block)."""
    tile, skinny, lora = text("tile.cuh"), text("skinny_tc.cuh"), text("kern_lora.cuh")
    two, one = re.search(r"SMEM_FLOOR = TMEM_CPS >= 2 \? ([^:]+(?:::\w+)?) : ([^;]+);", tile).groups()
    stages = int(re.search(r"STAGES = (\d+), LAG", lora).group(1))
    assert "stage = (128 + npad) * 128;" in lora and "ring + 1024" not in lora and "const int ring = Form<true>::STAGES * stage;" in lora
    return [("tile, 256 columns", 256, value(two)), ("tile, 512 columns", 512, value(one)),
            ("skinny", int(re.search(r"kTmemCols = (\d+)", skinny).group(1)), value(re.search(r"kSmemFloor = ([^;]+);", skinny).group(1))),
            ("adapters, tiles of 128", int(re.search(r"kTmemCols = (\d+)", lora).group(1)), stages * (128 + 16) * 128 + 1024)]


def test_what_shares_an_sm_finds_its_columns():
    kinds = holders()
    for n in range(1, 5):
        for blocks in itertools.combinations_with_replacement(kinds, n):
            if sum(b[2] + KB for b in blocks) <= SM:
                assert sum(b[1] for b in blocks) <= COLUMNS, [b[0] for b in blocks]
