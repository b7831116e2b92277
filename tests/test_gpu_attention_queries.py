"""Queries in bf16 over their whole range: rows of any size, elements far below the row's largest."""
import math

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl

from attn_ref import attention64, check_attention, codes_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = [(1, 7), (4, 2), (16, 1), (24, 1), (70, 2)]   # streaming with 8 and 16 rows, tcgen05


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


def check(q, kz, ks, scale, fmt, what):
    """q [1, t, h, d] over n keys with codes kz [n, hk, d] of scale ks, all values 1..7 of scale 1."""
    t, n = q.shape[1], kz.shape[0] - q.shape[1]
    hk, d = kz.shape[1:]
    pages = -(-kz.shape[0] // 16)
    g = torch.Generator().manual_seed(n)
    vz = torch.randint(1, 8, kz.shape, generator=g).float()
    cache = tl.KVCache.empty(fmt, pages, 16, hk, d)
    j = torch.arange(kz.shape[0])
    for codes, scales, z, s in ((cache.k_codes, cache.k_scale, kz, ks), (cache.v_codes, cache.v_scale, vz, 1.0)):
        codes.view(torch.uint8).zero_()
        scales.fill_(s)
        codes.view(torch.uint8)[(j // 16).to(DEV), :, (j % 16).to(DEV)] = codes_of(z, fmt).view(torch.uint8).to(DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    out, lse = tl.tree_attention(q.to(DEV), cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale=scale,
                                 return_lse=True)
    sees = torch.cat([torch.ones(t, n, dtype=torch.bool), torch.tril(torch.ones(t, t, dtype=torch.bool))], 1)
    scale32 = float(torch.tensor(scale, dtype=torch.float32))
    ref = attention64(q[0], kz.double() * float(torch.tensor(ks, dtype=torch.float32)), vz.double(), sees, scale32)
    check_attention(out[0], lse[0], ref, q.dtype, what)


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("e", [127, 126, 100, 40, 16, 15, 0, -17, -60, -100])
def test_rows_of_every_size(t, share, e):
    """Largest elements in [2^e, 2^(e+1)), keys of 2^-e: scores of order 1."""
    g = torch.Generator().manual_seed(e + 200)
    q = torch.randn(1, t, 2 * share, 64, generator=g).clamp(-1.9, 1.9)
    q[..., 5] = 1.9921875
    q = (q.double() * 2.0 ** e).to(torch.bfloat16)
    kz = torch.randint(-127, 128, (90 + t, 2, 64), generator=g).float()
    half = -e / 2                      # the scale takes a part: scales of keys stay normal numbers
    check(q, kz, 2.0 ** (half - 6), 2.0 ** (half - 3) if abs(e) != 127 else 2.0 ** (math.floor(half) - 3), "int8", f"2^{e}")


@pytest.mark.parametrize("t,share", FORMS)
def test_rows_of_unequal_size_and_rows_of_nothing(t, share):
    """Neighbouring rows 2^100 apart, zero rows, rows of subnormal numbers."""
    g = torch.Generator().manual_seed(t)
    q = torch.randn(1, t, 2 * share, 128, generator=g)
    q[:, :, 0] *= 2.0 ** 60
    q[:, :, 1] *= 2.0 ** -40
    q[:, 0] = 0.0
    q[:, -1, 1] = 2.0 ** -130
    kz = torch.randint(-7, 8, (200 + t, 2, 128), generator=g).float()
    check(q.to(torch.bfloat16), kz, 2.0 ** -20, 2.0 ** -44, "int4", "unequal")


@pytest.mark.parametrize("t,share", FORMS)
@pytest.mark.parametrize("big", [14, 18, 20, 24, 31])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_small_elements_beside_a_large_one(t, share, big, fmt):
    """One element of 2^big where every key is 0; the scores come from the others, which have to
    enter with all their bits: those down to 2^-32 of the largest are exact (at 2^31, 0.5)."""
    g = torch.Generator().manual_seed(big)
    q = torch.randn(1, t, 2 * share, 64, generator=g)
    if big > 24:
        q = torch.copysign(q.abs().clamp(min=0.5), q)
    q[..., 9] = 2.0 ** big
    kz = torch.randint(-15, 16, (150 + t, 2, 64), generator=g).float()
    kz[..., 9] = 0.0
    check(q.to(torch.bfloat16), kz, 1.0, 0.125, fmt, f"2^{big}")
