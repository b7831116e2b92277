"""The two NaN codes of an fp8 cache, which no append writes but a caller's own conversion may: they
read back as NaN, reach what sees them element by element, and nothing else."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_every_pattern_reads_back(dtype):
    """All 256 bytes at every place of a row, as torch converts them."""
    cache = tl.KVCache.empty("fp8", 16, 16, 1, 64)
    u = (torch.arange(16 * 16 * 64) + 37 * (torch.arange(16 * 16 * 64) // 256)).to(torch.uint8).view(16, 1, 16, 64)
    for c in (cache.k_codes, cache.v_codes):
        c.view(torch.uint8).copy_(u)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(0.5)
    want = u.view(torch.float8_e4m3fn).float().view(256, 1, 64)
    assert int(torch.isnan(want).sum()) == 128
    for got, scale in zip(tl.kv_read(cache, torch.arange(256, device=DEV), dtype), (1.0, 0.5)):
        assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want))
        assert torch.equal(got.cpu().float().nan_to_num(0.0), (want * scale).to(dtype).float().nan_to_num(0.0))


class Run:
    def __init__(self, n, t, share, d, wide, seed=0):
        g = torch.Generator().manual_seed(100 * n + t + d + seed)
        self.n, self.t, self.share = n, t, share
        pages = -(-(n + t) // 16)
        self.cache = tl.KVCache.empty("fp8", pages, 16, 2, d)
        y = torch.randn(2, n + t, 2, d, generator=g).to(torch.float16).to(DEV)
        self.table = torch.zeros(1, wide or pages, dtype=torch.int32, device=DEV)
        self.table[0, :pages] = torch.randperm(pages, generator=g).int()
        key = torch.arange(n + t, device=DEV)
        tl.kv_append(self.cache, y[0], y[1], self.table[0].long()[key // 16] * 16 + key % 16)
        self.q = torch.randn(1, t, 2 * share, d, generator=g).to(torch.bfloat16).to(DEV)
        self.tree = torch.zeros(t, t, dtype=torch.bool)
        for i in range(t):                   # a path 0-1-2-.., and every third token beside it
            self.tree[i, i] = True
            self.tree[i, [j for j in range(i) if j % 3 != 1 or j < 1]] = True
        self.g = g

    def put(self, side, key, head, d, code):
        c = self.cache.k_codes if side == "k" else self.cache.v_codes
        c.view(torch.uint8)[int(self.table[0, key // 16]), head, key % 16, d] = code

    def __call__(self):
        out, lse = tl.tree_attention(self.q, self.cache, self.table, torch.tensor([self.n], dtype=torch.int32, device=DEV),
                                     self.tree.to(DEV), return_lse=True)
        return out[0].cpu(), lse[0].cpu()


FORMS = [(4, 2), (3, 1), (8, 2), (16, 1), (20, 1), (70, 2)]   # streaming with 8 and 16 rows, tcgen05


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("d,n,wide", [(64, 0, None), (128, 37, None), (64, 700, 1024), (128, 1500, 1024)])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_attention(t, share, d, n, wide, code):
    x = Run(n, t, share, d, wide)
    spots = [(n + 1, d // 2 + 3), (n + 2, 0), (n + t - 1, d - 1)] + ([(0, 5), (n - 1, 17), (n // 2, 33)] if n else [])
    for key, e in spots:                       # the largest value there: what unseen NaN codes may not differ from
        x.put("v", key, 1, e, 0x7E)
        x.put("k", key, 1, e, 0x7E)
    want, want_lse = x()
    sees = torch.cat([torch.ones(t, n, dtype=torch.bool), x.tree], 1)
    for key, e in spots:
        # a value: that element of the tokens that see it, in the heads of its kv head
        x.put("v", key, 1, e, code)
        out, lse = x()
        hit = torch.zeros_like(want, dtype=torch.bool)
        hit[:, share:, e] = sees[:, key][:, None]
        assert torch.equal(torch.isnan(out), hit), f"value {key}"
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse, want_lse), f"value {key}"
        x.put("v", key, 1, e, 0x7E)
        # a key: every element of the tokens that see it
        x.put("k", key, 1, e, code)
        out, lse = x()
        hit = torch.zeros_like(want, dtype=torch.bool)
        hit[:, share:] = sees[:, key][:, None, None]
        assert torch.equal(torch.isnan(out), hit), f"key {key}"
        assert torch.equal(out[~hit], want[~hit]), f"key {key}"
        assert torch.equal(torch.isnan(lse), hit[..., 0]) and torch.equal(lse[~hit[..., 0]], want_lse[~hit[..., 0]])
        x.put("k", key, 1, e, 0x7E)


def test_several_at_once():
    """NaN codes of several drafted tokens, in tiles of their own and in several units."""
    x = Run(200, 150, 1, 128, 1024)
    gone = [(205, 3), (290, 3), (290, 64), (340, 127), (100, 9)]
    for key, e in gone:
        x.put("v", key, 0, e, 0x7E)
    want, _ = x()
    sees = torch.cat([torch.ones(150, 200, dtype=torch.bool), x.tree], 1)
    hit = torch.zeros_like(want, dtype=torch.bool)
    for key, e in gone:
        x.put("v", key, 0, e, 0x7F)
        hit[:, 0, e] |= sees[:, key]
    out, _ = x()
    assert torch.equal(torch.isnan(out), hit)
    assert torch.equal(out[~hit], want[~hit])
