"""Attention where scales are far apart: a token's scale stays its own affair, whatever it holds;
small values that the softmax picks beside large ones that it leaves out; scales at the edge of
the reference of the weights; negative scales."""
import math

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from attn_ref import U, attention64, check_attention, codes_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


class Pool:
    """One sequence of n + t keys in pages 0, 1, .. in order; codes random, scales given by the test.

    Every key's codes are small whole numbers in all formats.  Scores are steered: element 0 of
    every query is 1 and of key j its own scale's worth, the others of the queries are 0 unless
    the test sets them, so that score j = scale * k_scale[j] * code[j, 0]."""

    def __init__(self, fmt, n, t, hk, d, page=16, seed=0):
        g = torch.Generator().manual_seed(1000 * n + 10 * t + d + seed)
        self.fmt, self.n, self.t, self.hk, self.d, self.page, self.g = fmt, n, t, hk, d, page, g
        self.pages = -(-(n + t) // page)
        self.cache = tl.KVCache.empty(fmt, self.pages, page, hk, d)
        shape = (self.pages, hk, page, d)
        self.kz = torch.randint(-7, 8, shape, generator=g).float()
        self.kz[..., 0] = 4.0
        self.vz = torch.randint(1, 8, shape, generator=g).float() * (1 - 2 * torch.randint(0, 2, shape, generator=g))
        self.ks = torch.ones(shape[:3])
        self.vs = torch.ones(shape[:3])

    def scores(self, z, scale):
        """Key j of every head gets the score z[j] (natural units) from a query of (1, 0, 0 ..)."""
        j = torch.arange(len(z))
        self.ks[j // self.page, :, j % self.page] = (z / (4.0 * scale)).float()[:, None]

    def values(self, s):
        j = torch.arange(len(s))
        self.vs[j // self.page, :, j % self.page] = s.float()[:, None]

    def upload(self):
        c = self.cache
        c.k_codes.view(torch.uint8).copy_(codes_of(self.kz, self.fmt).view(torch.uint8))
        c.v_codes.view(torch.uint8).copy_(codes_of(self.vz, self.fmt).view(torch.uint8))
        c.k_scale.copy_(self.ks)
        c.v_scale.copy_(self.vs)

    def query(self, heads, dtype):
        q = torch.zeros(1, self.t, heads, self.d)
        q[..., 0] = 1.0
        return q.to(dtype)

    def run(self, q, tree=None, wide=None, **kw):
        self.upload()
        table = torch.zeros(1, wide or self.pages, dtype=torch.int32, device=DEV)  # wide: a row with more room
        table[0, :self.pages] = torch.arange(self.pages)
        return tl.tree_attention(q.to(DEV), self.cache, table, torch.tensor([self.n], dtype=torch.int32, device=DEV),
                                 None if tree is None else tree.to(DEV), **kw)

    def answer(self, q, tree=None, scale=None):
        m = self.n + self.t
        k, v = ((z.double() * s.double()[..., None]).transpose(1, 2).reshape(-1, self.hk, self.d)[:m]
                for z, s in ((self.kz, self.ks), (self.vz, self.vs)))
        own = torch.tril(torch.ones(self.t, self.t, dtype=torch.bool)) if tree is None else tree.bool()
        sees = torch.cat([torch.ones(self.t, self.n, dtype=torch.bool), own], 1)
        return attention64(q[0], k, v, sees, self.d ** -0.5 if scale is None else scale)

    def check(self, q, tree=None, scale=None, wide=None, what=""):
        out, lse = self.run(q, tree, wide, scale=scale, return_lse=True)
        check_attention(out[0], lse[0], self.answer(q, tree, scale), q.dtype, what)
        return out, lse

    def check_relative(self, q, wide=None, what=""):
        """The bound of check_attention without its absolute part: for bf16 answers of any size."""
        out, lse = self.run(q, None, wide, return_lse=True)
        o, l64, mag, top = self.answer(q)
        delta = (self.d + 4) * 2.0 ** -24 * top
        bound = (2.0 ** -10 + 2 * delta)[..., None] * mag * (1 + 2 * U[q.dtype]) + U[q.dtype] * o.abs()
        err = (out[0].double().cpu() - o).abs()
        assert (err <= bound).all(), f"{what}: error {float((err / bound).max()):.3g} of its bound"
        lim = delta + 2.0 ** -14 + 2.0 ** -22 * l64.abs()
        assert ((lse[0].double().cpu() - l64).abs() <= lim).all(), f"{what}: lse"


# 8 and 16 rows per kv head and the streaming kernel's single head; the tcgen05 kernel
FORMS = [(4, 2), (4, 1), (8, 2), (16, 1), (10, 2), (24, 1), (40, 4)]


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("fmt,dtype", [("int8", torch.float16), ("fp8", torch.bfloat16), ("int4", torch.bfloat16)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, torch.finfo(torch.float32).max, 1e30, -1e30, math.nan])
def test_a_value_scale_stays_with_the_tokens_that_see_it(t, share, fmt, dtype, bad):
    """New token 2 holds a place that nothing was written to; only itself sees it."""
    p = Pool(fmt, 37, t, 2, 64)
    q = torch.randn(1, t, 2 * share, 64, generator=p.g).to(dtype)
    tree = torch.eye(t, dtype=torch.bool)
    tree[t - 1, 0] = True
    want, want_lse = p.run(q, tree, return_lse=True)
    page, off = (p.n + 2) // p.page, (p.n + 2) % p.page
    p.vs[page, :, off] = bad
    got, lse = p.run(q, tree, return_lse=True)
    rest = [i for i in range(t) if i != 2]
    assert torch.equal(got[0, rest], want[0, rest])
    assert torch.equal(lse[0, rest], want_lse[0, rest])
    # its own sum of weights does not hold the value scale; each of the two is off by the bound of an lse
    assert ((lse - want_lse).abs() <= 2 * (2.0 ** -14 + 2.0 ** -22 * want_lse.abs())).all()


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("d,wide", [(64, None), (128, 4096)])
@pytest.mark.parametrize("weight,size", [(-58, 30), (-45, 16), (-90, 60), (-130, 100)])
def test_small_values_that_the_softmax_picks(t, share, d, wide, weight, size):
    """Keys with scores near 0 and values near 1 beside ones of weight 2^weight and scale 2^size: the
    answer is the first ones', to the same bound, wherever the others lie."""
    p = Pool("int8", 700, t, 1, d)
    g = p.g
    m = 700 + t
    far = torch.rand(m, generator=g) < 0.3
    far[:40] = False                     # ordinary keys first, later ones of the other kind between
    z = torch.where(far, weight * math.log(2.0), 0.0) + 0.5 * torch.randn(m, generator=g).clamp(-2, 2)
    p.scores(z.double(), d ** -0.5)
    p.values(torch.where(far, 2.0 ** size, 1.0).double() * (1 + torch.rand(m, generator=g)))
    p.check(p.query(share, torch.float16), what=f"weight 2^{weight}, scale 2^{size}", wide=wide)
    down = min(size, 70)                 # the same with small values in the answer
    p.vs = p.vs * 2.0 ** -down
    p.check_relative(p.query(share, torch.bfloat16), what="small", wide=wide)


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("first,then", [(0.5, 1.0), (0.3, 1.0), (0.3, 0.6), (0.5, 0.5), (0.25, 1.0)])
@pytest.mark.parametrize("above", [1.0, 2.0, 4.9999, 5.0, 5.1, 7.0])
def test_weights_at_the_edge_of_their_reference(t, share, first, then, above):
    """Scores and value scales that rise by just as much as a reference tolerates."""
    n = 420
    p = Pool("int8", n, t, 1, 64)
    late = torch.arange(n + t) >= 256
    p.scores(torch.where(late, above * math.log(2.0), 0.0).double(), 0.125)
    p.values(torch.where(late, then, first).double())
    out, _ = p.check(p.query(share, torch.float16), what="edge")
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("size", [1.0, 1e3, 1e-3])
def test_negative_value_scales(t, share, size):
    """value = code * scale, whatever the scale's sign."""
    p = Pool("int4", 300, t, 2, 128)
    sign = 1.0 - 2.0 * torch.randint(0, 2, p.vs.shape, generator=p.g)
    p.vs = sign * size * (1 + torch.rand(p.vs.shape, generator=p.g))
    q = torch.randn(1, t, 2 * share, 128, generator=p.g).to(torch.bfloat16)
    p.ks.fill_(0.1)
    p.check(q, what="mixed")
    p.vs = -p.vs.abs()
    p.check(q, what="all negative")


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("low,high,weight", [(-60, 90, -20), (-70, 100, -30), (-60, 100, -150)])
def test_scales_from_one_end_of_fp32_to_the_other(t, share, low, high, weight):
    """The sum of the weights comes from keys whose values are 2^low, the answer from keys of a small
    weight and values of 2^high: their references lie up to 2^140 apart, in a tile, between
    warps and between blocks."""
    for wide in (None, 4096):
        p = Pool("int8", 900, t, 1, 64)
        m = 900 + t
        far = torch.arange(m) % 97 == 55
        far[:200] = False
        p.scores(torch.where(far, weight * math.log(2.0), 0.0).double() + 0.2 * torch.rand(m, generator=p.g), 0.125)
        p.values(torch.where(far, 2.0 ** high, 2.0 ** low).double())
        p.check_relative(p.query(share, torch.bfloat16), wide, f"wide {wide}")
        p.vs.fill_(0.0)                  # and values of nothing
        out, _ = p.check(p.query(share, torch.bfloat16), wide=wide, what="zero")
        assert (out == 0).all()
