"""Order of tensor-memory allocation and dependent launch in the kernels' sources (no GPU).

A kernel launched with programmatic serialisation may allocate tensor memory before it waits for
the grid ahead of it.  That grid therefore lets dependents start only when each of its own blocks
holds its columns: otherwise a dependent can hold the columns that a block of the grid waits
for, while it waits for that block.
"""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "ternary_weight_linear_02_gb300", "csrc")
ALLOC, TRIGGER, SYNC = r"\btmem_alloc\(", r"\bpdl_launch_dependents\(\)\s*;", r"\b__syncthreads\(\)\s*;"


def kernels():
    """(file, name, body) of every __global__ function in the sources."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            brace = text.index("{", m.start())
            depth, end = 0, brace
            for end in range(brace, len(text)):
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
            name = re.findall(r"(\w+)\s*\(", text[m.start():brace])[-1]
            yield os.path.basename(path), name, text[brace:end]


WITH_TMEM = [k for k in kernels() if re.search(ALLOC, k[2])]


def test_the_kernels_are_found():
    assert {f for f, _, _ in WITH_TMEM} >= {"attn_tile.cuh", "skinny_tc.cuh", "tile.cuh", "tile_persist.cuh"}


@pytest.mark.parametrize("file,name,body", WITH_TMEM, ids=[f"{f}:{n}" for f, n, _ in WITH_TMEM])
def test_dependents_start_after_the_allocation(file, name, body):
    alloc = [m.start() for m in re.finditer(ALLOC, body)]
    for m in re.finditer(TRIGGER, body):
        assert max(alloc) < m.start(), "dependents may start before the tensor memory is allocated"
        # one warp allocates: the others have to have waited for it
        assert re.search(SYNC, body[max(alloc):m.start()]), "no barrier between the allocation and the trigger"
