"""The quantised cache against the formulas: codes and scales bit for bit (the formula in fp32,
operation by operation), the values read back, padding, odd rows, and indices out of range."""
import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from attn_ref import codes_of, numbers, quantise, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def filled(fmt, pages, page, hk, d):
    c = tl.KVCache.empty(fmt, pages, page, hk, d)
    for t in (c.k_codes, c.v_codes):
        t.view(torch.uint8).fill_(0x5A)
    for t in (c.k_scale, c.v_scale):
        t.fill_(7.0)
    return c


def at(t, slots, page):
    """Rows of a cache tensor at slots (CPU): [n, heads, ...]."""
    t = t.view(torch.uint8) if t.dtype != torch.float32 else t
    t = t.cpu()
    return t[slots // page, :, slots % page]


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,hq,hk,d,r,inter,page", [
    (1, 28, 4, 128, 128, False, 64), (33, 7, 1, 128, 64, True, 16), (70, 2, 2, 64, 64, False, 48),
    (5, 3, 3, 64, 16, True, 16), (19, 0, 2, 128, 0, False, 16), (260, 4, 1, 64, 32, False, 80)])
def test_append_and_read(fmt, dtype, n, hq, hk, d, r, inter, page):
    g = torch.Generator().manual_seed(n + d + page)
    pages = -(-n // page) + 3
    cache = filled(fmt, pages, page, hk, d)
    spread = torch.exp(2 * torch.randn(d, generator=g))
    qkv = (torch.randn(n, hq + 2 * hk, d, generator=g) * spread).to(dtype)
    if n > 4:
        qkv[2, hq] = 0                       # a zero row of k
        qkv[3, hq + hk] = 2.0 ** -24 if dtype == torch.float16 else 1e-39  # a subnormal row of v
    slots = torch.randperm(pages * page, generator=g)[:n]
    if n > 6:
        slots[5] = -1
    dev = qkv.to(DEV)
    k, v, q = dev[:, hq:hq + hk], dev[:, hq + hk:], dev[:, :hq]
    kf, vf = qkv[:, hq:hq + hk].float(), qkv[:, hq + hk:].float()
    if r:
        table = tl.rope_table(4000, r)
        pos = torch.randint(0, 4000, (n,), generator=g)
        got_q = tl.kv_append(cache, k, v, slots.to(DEV), q=q, positions=pos.to(DEV), table=table, interleaved=inter)
        rows = table.cpu()[pos]
        assert torch.equal(got_q.cpu(), rotate(qkv[:, :hq].float(), rows, inter).to(dtype))
        kf = rotate(kf, rows, inter)
    else:
        assert tl.kv_append(cache, k, v, slots.to(DEV)) is None
    put = slots >= 0
    for y, codes, scale in ((kf, cache.k_codes, cache.k_scale), (vf, cache.v_codes, cache.v_scale)):
        z, s = quantise(y, fmt)
        assert torch.equal(at(scale, slots[put], page), s[put])
        assert torch.equal(at(codes, slots[put], page), codes_of(z, fmt).view(torch.uint8)[put])
        other = torch.ones(pages * page, dtype=torch.bool)  # no other place was touched
        other[slots[put]] = False
        rest = other.nonzero()[:, 0]
        assert (at(codes, rest, page) == 0x5A).all() and (at(scale, rest, page) == 7.0).all()
    for out in (torch.bfloat16, torch.float16, torch.float32):
        got = tl.kv_read(cache, slots.to(DEV), out)
        for y, t in zip((kf, vf), got):
            z, s = quantise(y, fmt)
            want = (z * s[..., None] * put[:, None, None]).to(out)
            assert torch.equal(t.cpu(), want)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
def test_every_code_reads_back(fmt):
    """All bit patterns that an append can write, at both ends of a row."""
    page, hk, d = 16, 1, 64
    cache = filled(fmt, 16, page, hk, d)
    u = torch.arange(256, dtype=torch.uint8).repeat(64).reshape(16, 1, 16, 64)[..., :cache.k_codes.shape[-1]]
    u = (u.int() + 37 * torch.arange(16)[:, None, None, None]).to(torch.uint8)
    if fmt == "fp8":
        u[(u & 0x7F) == 0x7F] = 0
    for c in (cache.k_codes, cache.v_codes):
        c.view(torch.uint8).copy_(u)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(0.5)
    slots = torch.arange(16 * page)
    k, v = tl.kv_read(cache, slots.to(DEV), torch.float32)
    z = numbers(at(cache.k_codes, slots, page).view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn
                                                   if fmt == "fp8" else torch.uint8), fmt)
    assert torch.equal(k.cpu(), z) and torch.equal(v.cpu(), z * 0.5)


@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (0, 5)])
def test_alignment_and_in_place(shift, pad):
    n, hq, hk, d, page = 21, 3, 2, 64, 16
    row = (hq + 2 * hk) * d + pad
    flat = torch.randn(shift + n * row, device=DEV).to(torch.float16)
    qkv = flat[shift:].view(n, row)[:, :(hq + 2 * hk) * d].unflatten(1, (hq + 2 * hk, d))
    table, pos = tl.rope_table(50, 32), torch.arange(n, device=DEV)
    slots = torch.arange(n, device=DEV)
    got = []
    for src in (qkv.clone(memory_format=torch.contiguous_format), qkv):
        cache = filled("int8", 4, page, hk, d)
        q = src[:, :hq]
        out = tl.kv_append(cache, src[:, hq:hq + hk], src[:, hq + hk:], slots, q=q, positions=pos, table=table,
                           q_out=q if src is qkv else None)
        got.append((out.clone(), cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert torch.equal(qkv[:, :hq], got[0][0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite(bad):
    cache = filled("fp8", 2, 16, 2, 64)
    k = torch.randn(3, 2, 64, device=DEV).to(torch.bfloat16)
    v = torch.randn(3, 2, 64, device=DEV).to(torch.bfloat16)
    k[1, 0, 5] = bad
    tl.kv_append(cache, k, v, torch.tensor([0, 1, 2], device=DEV))
    assert torch.isnan(cache.k_scale[0, 0, 1]) and (cache.k_codes.view(torch.uint8)[0, 0, 1] == 0).all()
    rest = torch.isfinite(cache.k_scale[0, :, :3])
    assert int(rest.sum()) == 5 and torch.isfinite(cache.v_scale[0, :, :3]).all()
    back, _ = tl.kv_read(cache, torch.tensor([1, 2], device=DEV), torch.float32)
    assert torch.isnan(back[0, 0]).all() and torch.isfinite(back[0, 1]).all() and torch.isfinite(back[1]).all()


def test_indices_out_of_range():
    cache = filled("int4", 2, 16, 1, 64)
    x = torch.randn(3, 1, 64, device=DEV).to(torch.float16)
    tl.kv_append(cache, x, x, torch.tensor([4, 32, 1 << 40], device=DEV))
    torch.cuda.synchronize()
    assert tl.device_status(clear=True) == 5
    assert int((cache.k_scale != 7.0).sum()) == 1
    table = tl.rope_table(8, 32)
    out = torch.full_like(x, 3.0)
    tl.kv_append(cache, x, x, torch.tensor([8, 9, 10], device=DEV), q=x, q_out=out, table=table,
                 positions=torch.tensor([8, 7, -1], device=DEV))
    torch.cuda.synchronize()
    assert tl.device_status(clear=True) == 5
    assert (out[0] == 3.0).all() and (out[2] == 3.0).all() and not (out[1] == 3.0).all()
    assert cache.k_scale[0, 0, 8:11].tolist().count(7.0) == 2
    k, v = tl.kv_read(cache, torch.tensor([-5, 32, 9], device=DEV), torch.float32)
    torch.cuda.synchronize()
    assert tl.device_status(clear=True) == 5
    assert (k[:2] == 0).all() and (v[:2] == 0).all() and (k[2] != 0).any()


def test_empty():
    cache = filled("int8", 1, 16, 1, 64)
    x = torch.empty(0, 1, 64, dtype=torch.float16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    assert tl.kv_append(cache, x, x, none) is None
    k, v = tl.kv_read(cache, none)
    assert k.shape == v.shape == (0, 1, 64)


def test_offsets_beyond_32_bits():
    """Slots whose rows start past 2^32 bytes of codes."""
    page, hk, d = 64, 4, 128
    pages = (1 << 32) // (page * hk * d) + 5
    cache = tl.KVCache.empty("int8", pages, page, hk, d)
    x = torch.randn(3, 2 * hk, d, device=DEV).to(torch.bfloat16)
    slots = torch.tensor([pages * page - 1, (pages - 3) * page + 7, 5], device=DEV)
    tl.kv_append(cache, x[:, :hk], x[:, hk:], slots)
    k, v = tl.kv_read(cache, slots, torch.float32)
    for y, got in ((x[:, :hk], k), (x[:, hk:], v)):
        z, s = quantise(y.float().cpu(), "int8")
        assert torch.equal(got.cpu(), z * s[..., None])
