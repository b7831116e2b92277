"""The rotary, cache and tree-attention operators as a user's program calls them, with plain forms to hold them against.

``listed()`` and ``draw()`` give the cases, ``prepare()`` what a program has in hand before the call, ``run()`` one pass, ``exact()``
the same outputs from the definitions in 64 bits, ``work()`` the bytes and operations that a pass cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
QMAX = {"int8": 127.0, "fp8": 448.0, "int4": 7.0}
CODES = {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}

# Heads as (query heads, kv heads, head size): the fused QKV layer of the 7B-shaped stack (3584 + 512 + 512), the 4096-wide and the
# 5120-wide layers without sharing, and the 1024-wide embedding model with heads of 64.
HEADS = ((28, 4, 128), (32, 32, 128), (40, 40, 128), (16, 16, 64))


def listed():
    return [
        # one decode step of a batch of 16: q and k of the stack's fused QKV output (a strided view of it) are rotated together
        dict(name="rope_decode", op="rope", tokens=16, heads=32, dim=128, rotary=128, interleaved=False, inverse=False, dtype="bf16", pad=512, span=8192),
        # a long prompt in one piece, interleaved pairs, half of the head rotated
        dict(name="rope_prompt", op="rope", tokens=16384, heads=32, dim=128, rotary=64, interleaved=True, inverse=False, dtype="bf16", pad=512, span=131072),
        # the gradient of the rotation for a batch of embedding inputs, heads of 64, an odd number of tokens
        dict(name="rope_gradient", op="rope", tokens=3001, heads=16, dim=64, rotary=64, interleaved=False, inverse=True, dtype="f16", pad=0, span=4096),
        # a single new token written to an fp8 cache: latency
        dict(name="append_token", op="append", tokens=1, q_heads=28, kv_heads=4, dim=128, rotary=128, interleaved=False, fmt="fp8", dtype="bf16", page=64, span=8192),
        # a prompt chunk written to an int8 cache and read back for the attention within the prompt
        dict(name="append_chunk", op="append", tokens=2048, q_heads=28, kv_heads=4, dim=128, rotary=128, interleaved=False, fmt="int8", dtype="bf16", page=64, span=32768),
        # many prompts at once without shared heads, four-bit cache, odd total
        dict(name="append_batch", op="append", tokens=9973, q_heads=32, kv_heads=32, dim=128, rotary=64, interleaved=True, fmt="int4", dtype="f16", page=48, span=16384),
        # a cached prefix brought back to 16 bits: a short one, and a long one
        dict(name="read_prefix", op="read", tokens=1500, kv_heads=4, dim=128, fmt="int8", dtype="bf16", page=16),
        dict(name="read_long", op="read", tokens=131072, kv_heads=4, dim=128, fmt="fp8", dtype="bf16", page=64),
        # one sequence, one token, a short context: latency
        dict(name="decode_single", op="attention", batch=1, draft=1, context=1000, q_heads=28, kv_heads=4, dim=128, fmt="fp8", dtype="bf16", page=64),
        # a full serving batch of single tokens over ragged contexts
        dict(name="decode_batch", op="attention", batch=64, draft=1, context=8192, q_heads=28, kv_heads=4, dim=128, fmt="int8", dtype="bf16", page=64),
        # drafted trees without shared heads over a four-bit cache
        dict(name="tree_heads", op="attention", batch=6, draft=23, context=4099, q_heads=32, kv_heads=32, dim=128, fmt="int4", dtype="f16", page=16),
        # large drafted trees over long contexts with shared heads: the most arithmetic
        dict(name="tree_long", op="attention", batch=8, draft=64, context=16384, q_heads=28, kv_heads=4, dim=128, fmt="fp8", dtype="bf16", page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "read", "attention", "attention"))
    hq, hk, dim = rng.choice(HEADS)
    dtype = rng.choice(("bf16", "f16"))
    fmt = rng.choice(("int8", "fp8", "int4"))
    page = rng.choice((16, 32, 48, 64, 128))
    rotary = rng.choice((dim, dim // 2))
    turn = rng.random() < 0.5
    span = _log(rng, 256, 131072)
    if op == "rope":
        tokens = min(_log(rng, 1, 16384), 16384 * 4096 // ((hq + hk) * dim))
        return dict(op=op, tokens=tokens, heads=hq + hk, dim=dim, rotary=rotary, interleaved=turn, inverse=rng.random() < 0.5, dtype=dtype,
                    pad=hk * dim * rng.choice((0, 1)), span=span)
    if op == "append":
        return dict(op=op, tokens=min(_log(rng, 1, 9973), 9973 * 12288 // ((hq + 2 * hk) * dim)), q_heads=hq, kv_heads=hk, dim=dim, rotary=rotary,
                    interleaved=turn, fmt=fmt, dtype=dtype, page=page, span=span)
    if op == "read":
        return dict(op=op, tokens=min(_log(rng, 1, 131072), 131072 * 512 // (hk * dim)), kv_heads=hk, dim=dim, fmt=fmt, dtype=dtype, page=page)
    batch, draft = _log(rng, 1, 64), rng.choice((1, 1, _log(rng, 2, 64)))
    most = min(64 * 8192 * 512 / (batch * hk * dim), 8 * 64 * 16384 * 3584 / (batch * draft * hq * dim), 131072)
    return dict(op=op, batch=batch, draft=draft, context=min(_log(rng, 16, 131072), int(most)), q_heads=hq, kv_heads=hk, dim=dim, fmt=fmt,
                dtype=dtype, page=page)


def _contexts(case):
    """The committed lengths of the batch: from half of the longest up to it, and in a batch one sequence that has none yet."""
    n, top = case["batch"], case["context"]
    lens = [max(0, top - int(0.5 * top * ((0.618034 * b) % 1.0))) for b in range(n)]
    if n > 4:
        lens[3] = 0
    return lens


def _row_bytes(case):
    return case["dim"] // 2 if case["fmt"] == "int4" else case["dim"]


def work(case):
    if case["op"] == "rope":
        values = case["tokens"] * case["heads"] * case["dim"]
        rotated = case["tokens"] * case["heads"] * case["rotary"]
        return {"bytes": 4 * values + case["tokens"] * (4 * case["rotary"] + 8), "flops": 3 * rotated}
    if case["op"] == "append":
        q, kv, n = case["q_heads"] * case["dim"], 2 * case["kv_heads"] * case["dim"], case["tokens"]
        moved = 4 * q + 2 * kv + 2 * case["kv_heads"] * (_row_bytes(case) + 4) + 4 * case["rotary"] + 16
        if case["fmt"] != "fp8":  # read back: the codes just written, and 16-bit values out
            moved += 2 * case["kv_heads"] * (_row_bytes(case) + 4) + 2 * kv + 8
        return {"bytes": n * moved, "flops": n * (3 * q + 5 * kv)}
    if case["op"] == "read":
        kv = 2 * case["kv_heads"] * case["dim"]
        return {"bytes": case["tokens"] * (2 * kv + 2 * case["kv_heads"] * (_row_bytes(case) + 4) + 8), "flops": case["tokens"] * kv}
    keys = sum(_contexts(case)) + case["batch"] * case["draft"]
    rows = case["batch"] * case["draft"] * case["q_heads"]
    held = keys * case["kv_heads"] * 2 * (_row_bytes(case) + 4)
    return {"bytes": held + 4 * rows * case["dim"], "flops": 4 * case["draft"] * case["q_heads"] * case["dim"] * keys}


# ------------------------------------------------------------------------------------------------ inputs
def _table(span, rotary, gen):
    """cos | sin of every position, f32 rounded from 64 bits, base 10000."""
    f = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=DEV) / rotary)
    a = torch.arange(span, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _pack4(c):
    """Whole numbers -7..7 as two four-bit fields a byte, value + 8, the even place in the low bits."""
    u = (c + 8).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _to_codes(y, fmt):
    """Codes and scales of rows of values (the last axis), in f32."""
    top = y.abs().amax(-1)
    s = top / QMAX[fmt]
    z = y / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    if fmt == "fp8":
        return z.to(torch.float8_e4m3fn), s
    c = z.round()
    return (_pack4(c) if fmt == "int4" else c.to(torch.int8)), s


def _values(codes, fmt, kind):
    """What codes stand for before their scale."""
    if fmt == "int4":
        lo, hi = (codes & 15).to(kind) - 8, (codes >> 4).to(kind) - 8
        return torch.stack([lo, hi], -1).flatten(-2)
    return codes.to(kind)


def _pool(gen, pages, case, spread):
    """A cache's codes and scales: rows of values with channels of unequal size, quantised row by row."""
    h, d, fmt = case["kv_heads"], case["dim"], case["fmt"]
    codes = torch.empty(pages, h, case["page"], _row_bytes(case), dtype=CODES[fmt], device=DEV)
    scales = torch.empty(pages, h, case["page"], dtype=torch.float32, device=DEV)
    size = torch.exp(spread * torch.randn(d, generator=gen, device=DEV))
    step = max(1, (1 << 27) // (h * case["page"] * d))
    for a in range(0, pages, step):
        n = min(pages, a + step) - a
        codes[a:a + n], scales[a:a + n] = _to_codes(_normal(gen, n, h, case["page"], d) * size, fmt)
    return codes, scales


def _slots(gen, case, pages):
    """Where a run of tokens lies: through a shuffled page table; in a batch every 97th token is padding and has no place."""
    n, page = case["tokens"], case["page"]
    table = torch.randperm(pages, generator=gen, device=DEV)
    at = torch.arange(n, device=DEV)
    slots = table[at // page] * page + at % page
    return torch.where(at % 97 == 96, torch.full_like(slots, -1), slots)


def _trees(case, seed):
    """Which drafted tokens each drafted token sees: itself and its ancestors, a random tree for each sequence."""
    b, t = case["batch"], case["draft"]
    gen = torch.Generator().manual_seed(seed)
    sees = torch.zeros(b, t, t, dtype=torch.bool)
    each = torch.arange(b)
    for i in range(t):
        if i:
            parent = (torch.rand(b, generator=gen) * min(i, 12)).long() + max(0, i - 12)
            sees[:, i] = sees[each, parent]
        sees[:, i, i] = True
    return sees.to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "read":
        pages = -(-case["tokens"] // case["page"]) + 3
        s["k_codes"], s["k_scale"] = _pool(gen, pages, case, 0.5)
        s["v_codes"], s["v_scale"] = _pool(gen, pages, case, 0.2)
        s["slots"] = _slots(gen, case, pages)
        return s
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "attention":
        b, t, page = case["batch"], case["draft"], case["page"]
        lens = _contexts(case)
        wide = -(-(max(lens) + t) // page)
        used = [-(-(n + t) // page) for n in lens]
        order = torch.randperm(sum(used) + 2, generator=gen, device=DEV).int()
        table, at = torch.zeros(b, wide, dtype=torch.int32, device=DEV), 0
        for i, n in enumerate(used):
            table[i, :n] = order[at:at + n]
            at += n
        s["k_codes"], s["k_scale"] = _pool(gen, sum(used) + 2, case, 0.5)
        s["v_codes"], s["v_scale"] = _pool(gen, sum(used) + 2, case, 0.2)
        s["block_table"] = table
        s["context_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["tree"] = _trees(case, int(seed))
        s["q"] = (2.0 * _normal(gen, b, t, case["q_heads"], case["dim"])).to(dtype)
        return s
    n, d = case["tokens"], case["dim"]
    s["table"] = _table(case["span"], case["rotary"], gen)
    s["positions"] = torch.randint(0, case["span"], (n,), generator=gen, device=DEV)
    if case["op"] == "rope":
        rows = _normal(gen, n, case["heads"] * d + case["pad"], dtype=dtype)
        s["x"] = rows[:, :case["heads"] * d].unflatten(1, (case["heads"], d))
        return s
    hq, hk = case["q_heads"], case["kv_heads"]
    qkv = _normal(gen, n, (hq + 2 * hk) * d, dtype=dtype).unflatten(1, (hq + 2 * hk, d))  # as the fused QKV layer leaves it
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pages = -(-n // case["page"]) + 3
    s["k_codes"], s["k_scale"] = _pool(gen, pages, case, 0.5)
    s["v_codes"], s["v_scale"] = _pool(gen, pages, case, 0.2)
    s["slots"] = _slots(gen, case, pages)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def _turned(x, s, kind=torch.float32):
    """x rotated by its tokens' positions."""
    r = s["rotary"]
    row = s["table"][s["positions"]].to(kind)[:, None]
    c, w = row[..., :r // 2], row[..., r // 2:]
    w = -w if s.get("inverse") else w
    x = x.to(kind)
    part, rest = x[..., :r], x[..., r:]
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * c - b * w, b * c + a * w], -1).flatten(-2)
    else:
        a, b = part[..., :r // 2], part[..., r // 2:]
        part = torch.cat([a * c - b * w, b * c + a * w], -1)
    return torch.cat([part, rest], -1)


def _read(s, codes, scales, kind=torch.float32):
    """The values at the slots; zeros where a token has no place."""
    at = s["slots"].clamp(min=0)
    page, off = at // s["page"], at % s["page"]
    y = _values(codes[page, :, off], s["fmt"], kind) * scales[page, :, off].to(kind)[..., None]
    return torch.where(s["slots"][:, None, None] >= 0, y, torch.zeros_like(y))


def _write(s, codes, scales, y):
    put = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"][put]
    c, w = _to_codes(y[put], s["fmt"])
    raw = torch.uint8 if s["fmt"] == "fp8" else codes.dtype
    codes.view(raw)[at // s["page"], :, at % s["page"]] = c.view(raw)
    scales[at // s["page"], :, at % s["page"]] = w


def _attend(s):
    b, t, h, d = s["q"].shape
    hk, page = s["kv_heads"], s["page"]
    table = s["block_table"].long()
    n = table.shape[1] * page
    k = (_values(s["k_codes"][table], s["fmt"], torch.float32) * s["k_scale"][table][..., None]).transpose(1, 2).reshape(b, hk, n, d)
    v = (_values(s["v_codes"][table], s["fmt"], torch.float32) * s["v_scale"][table][..., None]).transpose(1, 2).reshape(b, hk, n, d)
    q = s["q"].float().unflatten(2, (hk, h // hk)).permute(0, 2, 1, 3, 4).reshape(b, hk, t * (h // hk), d)
    score = (q @ k.transpose(2, 3)).view(b, hk, t, h // hk, n) * (d ** -0.5)
    place = torch.arange(n, device=DEV)[None] - s["context_len"][:, None]  # < 0: committed, 0..t-1: drafted
    drafted = s["tree"].gather(2, place.clamp(0, t - 1)[:, None].expand(b, t, n))
    seen = (place < 0)[:, None] | (drafted & (place < t)[:, None])
    score = score.masked_fill(~seen[:, None, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top > float("-inf"), top, torch.zeros_like(top))).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, -1, n) @ v).view(b, hk, t, h // hk, d) / total
    return o.permute(0, 2, 1, 3, 4).reshape(b, t, h, d).to(s["q"].dtype)


def _cache(s):
    """The program's handle on its cache, kept with it."""
    import ternary_weight_linear_02_gb300 as tl
    if "cache" not in s:
        s["cache"] = tl.KVCache(s["fmt"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return tl, s["cache"]


def run(s):
    if s["op"] == "rope":
        if own:
            import ternary_weight_linear_02_gb300 as tl
            return tl.rope(s["x"], s["positions"], s["table"], interleaved=s["interleaved"], inverse=s["inverse"])
        return _turned(s["x"], s).to(s["x"].dtype)
    if s["op"] == "read":
        dtype = DTYPES[s["dtype"]]
        if own:
            tl, cache = _cache(s)
            return tl.kv_read(cache, s["slots"], dtype)
        return _read(s, s["k_codes"], s["k_scale"]).to(dtype), _read(s, s["v_codes"], s["v_scale"]).to(dtype)
    if s["op"] == "attention":
        if own:
            tl, cache = _cache(s)
            return tl.tree_attention(s["q"], cache, s["block_table"], s["context_len"], s["tree"])
        return _attend(s)
    dtype = s["k"].dtype
    if own:
        tl, cache = _cache(s)
        q = tl.kv_append(cache, s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"], table=s["table"], interleaved=s["interleaved"])
    else:
        q = _turned(s["q"], s).to(dtype)
        _write(s, s["k_codes"], s["k_scale"], _turned(s["k"], s))
        _write(s, s["v_codes"], s["v_scale"], s["v"].float())
    if s["fmt"] == "fp8":  # the cache itself holds values
        return q, s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
    if own:
        k, v = tl.kv_read(cache, s["slots"], dtype)
    else:
        k, v = _read(s, s["k_codes"], s["k_scale"]).to(dtype), _read(s, s["v_codes"], s["v_scale"]).to(dtype)
    return q, k, v


# ------------------------------------------------------------------------------------------------ 64 bits
def _spin(x, s):
    """The rotation by complex numbers: each pair (a, b) is a + ib, multiplied by cos + i sin (by its conjugate for the inverse)."""
    r, half = s["rotary"], s["rotary"] // 2
    row = s["table"].double()[s["positions"]]
    turn = torch.complex(row[:, :half], row[:, half:] * (-1 if s.get("inverse") else 1))[:, None]
    y = x.double().clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if s["interleaved"] else (y[..., :half], y[..., half:r])
    z = torch.complex(a.clone(), b.clone()) * turn
    a.copy_(z.real)
    b.copy_(z.imag)
    return y


def _grid(y, fmt):
    """Rows of values on their formats' grids, in 64 bits: (numbers before the scale, scales)."""
    scale = y.abs().max(-1).values / QMAX[fmt]
    z = y / scale.clamp(min=1e-300)[..., None]
    if fmt != "fp8":
        return torch.round(z), scale
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)  # three bits of fraction, none below 2^-9
    return torch.round(z / step) * step, scale


def _number(codes, fmt):
    """Codes as 64-bit numbers, from their bits."""
    if fmt == "int8":
        return codes.double()
    u = codes.view(torch.uint8).long()
    if fmt == "int4":
        return torch.stack([u % 16 - 8, u // 16 - 8], -1).reshape(*u.shape[:-1], -1).double()
    e, m = (u >> 3) & 15, u & 7
    size = torch.where(e > 0, (8 + m).double() * torch.exp2((e - 10).double()), m.double() * 2.0 ** -9)
    return torch.where(u >= 128, -size, size)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _spin(s["x"], s)
    if case["op"] == "attention":
        b, t, h, d = s["q"].shape
        share = h // s["kv_heads"]
        out = torch.zeros(b, t, h, d, dtype=torch.float64, device=DEV)
        for i, ctx in enumerate(s["context_len"].tolist()):
            n = ctx + t
            pages = s["block_table"][i, :-(-n // s["page"])].long()
            sees = torch.cat([torch.ones(t, ctx, dtype=torch.bool, device=DEV), s["tree"][i]], 1)
            for j in range(s["kv_heads"]):
                k = (_number(s["k_codes"][pages, j], s["fmt"]) * s["k_scale"][pages, j].double()[..., None]).reshape(-1, d)[:n]
                v = (_number(s["v_codes"][pages, j], s["fmt"]) * s["v_scale"][pages, j].double()[..., None]).reshape(-1, d)[:n]
                z = torch.einsum("tgd,nd->tgn", s["q"][i, :, j * share:(j + 1) * share].double(), k) / math.sqrt(d)
                z = z.masked_fill(~sees[:, None], float("-inf"))
                out[i, :, j * share:(j + 1) * share] = torch.softmax(z, -1) @ v
        return out
    has = s["slots"] >= 0
    if case["op"] == "read":
        where = s["slots"].clamp(min=0)
        got = []
        for codes, scale in ((s["k_codes"], s["k_scale"]), (s["v_codes"], s["v_scale"])):
            rows = codes.view(torch.uint8).transpose(1, 2).flatten(0, 1)[where]
            y = _number(rows.view(codes.dtype), s["fmt"]) * scale.double().transpose(1, 2).flatten(0, 1)[where][..., None]
            got.append(y * has[:, None, None])
        return tuple(got)
    q, sides = _spin(s["q"], s), ((_spin(s["k"], s), "k"), (s["v"].double(), "v"))
    held, scales, back = [], [], []
    for y, side in sides:
        z, scale = _grid(y, s["fmt"])
        back.append(z * scale[..., None] * has[:, None, None])
        if s["fmt"] == "fp8":
            pages, heads, page, d = s[side + "_codes"].shape
            codes = _number(s[side + "_codes"], "fp8").transpose(1, 2).reshape(pages * page, heads, d)
            codes[s["slots"][has]] = z[has]
            w = s[side + "_scale"].double().transpose(1, 2).reshape(pages * page, heads)
            w[s["slots"][has]] = scale[has]
            held.append(codes.view(pages, page, heads, d).transpose(1, 2).contiguous())
            scales.append(w.view(pages, page, heads).transpose(1, 2).contiguous())
    return (q, *held, *scales) if s["fmt"] == "fp8" else (q, *back)
