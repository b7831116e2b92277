"""Gate and up reach the product of an adapted layer in fp32, as they do in linear_silu_mul: a row without an adapter loses nothing
by another row's having one."""
import os
import sys

import pytest
import torch

import ternary_weight_linear_02_gb300 as tl
from ternary_weight_linear_02_gb300 import synth

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import verify_step as vs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tl.build()
    tl.load()


@pytest.mark.parametrize("m", [3, 24, 150])
def test_a_row_without_an_adapter_is_rounded_once(m):
    """Against 64 bits: half a step of bf16 (2^-8) and what fp32 sums of K terms may lose on the way, for the call that knows no adapters and
    for rows without one in a call of the example's form."""
    k, n = 512, 768
    gen = torch.Generator(device=DEV).manual_seed(m)
    x = torch.randn(m, k, generator=gen, device=DEV).to(torch.bfloat16)
    w = synth.packed_codes(2 * n, k, 5, DEV)
    sc = synth.scales(2 * n, 0, 0.02, 0.2, 6, DEV)
    t = tl.unpack(w, k)[0].double() * sc.double()[:, None]
    z, mag = x.double() @ t.T, x.double().abs() @ t.abs().T
    g, u = z.chunk(2, 1)
    dg, du = ((k + 4) * 2.0 ** -23 * mag).chunk(2, 1)
    want = g * torch.sigmoid(g) * u
    off = 1.1 * dg * (u.abs() + du) + (g * torch.sigmoid(g)).abs() * du + 2.0 ** -21 * want.abs()
    off = off * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    a, b = (torch.randn(s, generator=gen, device=DEV).to(torch.bfloat16) for s in ((2, 32, k), (2, 2 * n, 16)))
    which = (torch.arange(m, device=DEV) % 3 - 1).int()
    y = tl.linear(x, w, sc, 0, out_dtype=torch.float32)
    got = tl.lora_silu_mul(x, tl.Adapters(a, b, shards=(n, n)), which, y).to(x.dtype)
    none = which < 0
    assert bool(((got.double() - want).abs() <= off)[none].all())
    assert bool(((tl.linear_silu_mul(x, w, sc, 0).double() - want).abs() <= off).all())


def test_the_example_keeps_them_in_fp32(monkeypatch):
    stack = vs.Stack(layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, ffn=768, fmt="int8", page_size=16, pages=4, positions=64)
    seen, call = [], tl.lora_silu_mul

    def watch(x, ad, which, y, **kw):
        seen.append(y.dtype)
        return call(x, ad, which, y, **kw)

    monkeypatch.setattr(tl, "lora_silu_mul", watch)
    x = torch.randn(1, 5, 512, device=DEV).to(torch.bfloat16)
    at = torch.arange(5, device=DEV)
    table, ctx = torch.arange(4, device=DEV).int()[None], torch.zeros(1, dtype=torch.int32, device=DEV)
    out = stack.step(x, at, at, table, ctx, adapters=stack.adapt(2, 16), which=torch.tensor([0, 1, -1, 0, -1], dtype=torch.int32, device=DEV))
    assert seen == [torch.float32] * 2 and out.dtype is torch.bfloat16 and bool(torch.isfinite(out).all())
