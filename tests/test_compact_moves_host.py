"""The largest number of moves of a sequence (no GPU, nothing is launched)."""
import os
import re

from conftest import ROOT
from test_pages_host import B, C, D, OK, SHAPE, cache, lib, many, pool  # noqa: F401

MOST = (1 << 31) - (1 << 13)


def test_moves_are_counted_in_31_bits(lib):  # noqa: F811
    """A block is up to five groups ahead of the group that it writes: move numbers of the largest n stay below 2^31."""
    text = open(os.path.join(ROOT, "ternary_weight_linear_02_gb300", "csrc", "kern_move.cu")).read()
    movers, pieces = (int(re.search(rf"{name} = (\d+)", text).group(1)) for name in ("kMovers", "kPieces"))
    group = max(movers // 32 * 32 * pieces // p for p in (2, 4, 8))
    ahead = max(int(n or 1) for n in re.findall(r"i0 \+ (?:(\d+) \* )?ROWS", text))
    assert MOST - 1 + (ahead + 1) * group < 1 << 31
    for n, want in ((MOST + 1, SHAPE), ((1 << 31) - 1, SHAPE)):
        assert lib.ternary_kv_compact(many(cache()), 1, B, 4, 4, B, C, n, D, 2, n, None) == want
        assert lib.ternary_pages_compact(pool(), many(cache()), 1, B, C, n, D, n, None) == want
    assert lib.ternary_kv_compact(many(cache()), 1, B, 4, 4, B, C, MOST, D, 0, MOST, None) == OK
    assert lib.ternary_pages_compact(pool(rows=0), many(cache()), 1, B, C, MOST, D, MOST, None) == OK
