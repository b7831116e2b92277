"""Plain forms of the rotary, cache and attention calls for the tests, written from the
formulas: fp32 operation by operation where the codes of a cache have to be equal,
fp64 elsewhere."""
import math

import torch

QMAX = {"int8": 127.0, "fp8": 448.0, "int4": 7.0}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # unit roundoff


def table64(n, r, base=10000.0, factor=1.0, original_len=0.0, ramp=(1.0, 32.0), magnitude=1.0):
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    keep = torch.zeros_like(f)
    if original_len > 0 and ramp[1] > ramp[0]:
        turns = original_len * f / (2 * math.pi)
        keep = ((turns - ramp[0]) / (ramp[1] - ramp[0])).clamp(0, 1)
    f = f * (keep + (1 - keep) / factor)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return magnitude * torch.cat([a.cos(), a.sin()], 1)


def rotate(x, rows, interleaved, inverse=False):
    """x [n, h, d] rotated by table rows [n, r], in x's own precision, each operation rounded."""
    r = rows.shape[1]
    c, s = rows[:, None, :r // 2].to(x.dtype), rows[:, None, r // 2:].to(x.dtype)
    s = -s if inverse else s
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = u, w
    else:
        y[..., :r // 2], y[..., r // 2:r] = u, w
    return y


def quantise(y, fmt):
    """fp32 rows -> (numbers on the format's grid, fp32 scales)."""
    rq = (torch.ones((), dtype=torch.float32) / torch.tensor(QMAX[fmt], dtype=torch.float32))
    s = y.abs().amax(-1) * rq
    bad = ~torch.isfinite(y).all(-1)
    z = y / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    z = torch.where((bad | (s == 0))[..., None], torch.zeros_like(z), z)
    z = z.to(torch.float8_e4m3fn).float() if fmt == "fp8" else z.round()
    return z, torch.where(bad, torch.full_like(s, float("nan")), s)


def numbers(codes, fmt):
    """The numbers that codes stand for before their scale (fp32, exact)."""
    codes = codes.cpu()
    if fmt == "int4":
        return torch.stack([(codes & 15).float() - 8, (codes >> 4).float() - 8], -1).flatten(-2)
    return codes.float()


def codes_of(z, fmt):
    """Numbers on the grid as the cache stores them."""
    if fmt == "fp8":
        return z.to(torch.float8_e4m3fn)
    if fmt == "int8":
        return z.to(torch.int8)
    u = (z + 8).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def attention64(q, k, v, sees, scale):
    """One sequence: q [t, h, d], k and v [n, hk, d] (fp64), sees [t, n] bool -> o, lse, and per
    row sum p |v| (fp64 [t, h, d]) and the largest scale sum |q||k| over seen keys [t, h]."""
    t, h, d = q.shape
    hk = k.shape[1]
    q, g = q.double(), h // hk
    o, mag = torch.zeros(t, h, d, dtype=torch.float64), torch.zeros(t, h, d, dtype=torch.float64)
    lse, top = torch.full((t, h), -math.inf, dtype=torch.float64), torch.zeros(t, h, dtype=torch.float64)
    for i in range(t):
        j = sees[i].nonzero()[:, 0]
        if len(j) == 0:
            continue
        for a in range(hk):
            kk, vv, qq = k[j, a], v[j, a], q[i, a * g:(a + 1) * g]
            z = qq @ kk.T * scale
            w = torch.exp(z - z.max(1, keepdim=True).values)
            p = w / w.sum(1, keepdim=True)
            o[i, a * g:(a + 1) * g] = p @ vv
            mag[i, a * g:(a + 1) * g] = p @ vv.abs()
            lse[i, a * g:(a + 1) * g] = torch.logsumexp(z, 1)
            top[i, a * g:(a + 1) * g] = (qq.abs() @ kk.abs().T * scale).max(1).values
    return o, lse, mag, top


def check_attention(out, lse, ref, dtype, what=""):
    """Bound of one output element.  A score is a dot product of d exact products summed in fp32,
    then two fp32 factors: off by at most delta = (d + 4) 2^-24 scale sum |q||k|.  A weight is
    off by 2 delta relative (numerator and sum), its exponential by 2^-21, its rounding to f16
    by 2^-11, its fp32 sum by 2^-14 (thousands of terms): together below 2^-10 + 2 delta; the
    result is rounded once to dtype."""
    o, l64, mag, top = ref
    delta = (o.shape[-1] + 4) * 2.0 ** -24 * top
    bound = (2.0 ** -10 + 2 * delta)[..., None] * mag
    bound = bound * (1 + 2 * U[dtype]) + U[dtype] * o.abs() + 2.0 ** -24
    got = out.double().cpu()
    top = torch.finfo(dtype).max
    over = o.abs() - bound > top * (1 + U[dtype])   # answers beyond the output type round to infinity
    near = ~over & (o.abs() + bound > top)          # at its edge: either
    assert torch.equal(got[over], torch.sign(o[over]) * math.inf), f"{what}: overflow"
    assert torch.isfinite(got[~over & ~near]).all(), f"{what}: not finite"
    err = torch.where(over | near, 0.0, (got - o).abs())
    assert (err <= bound).all(), f"{what}: error {float((err / bound).max()):.3g} of its bound"
    if lse is not None:
        got = lse.double().cpu()
        empty = torch.isinf(l64)
        assert torch.equal(torch.isinf(got) & (got < 0), empty), f"{what}: lse of empty rows"
        lim = (delta + 2.0 ** -14 + 2.0 ** -22 * l64.abs())[~empty]
        assert ((got - l64).abs()[~empty] <= lim).all(), f"{what}: lse"
