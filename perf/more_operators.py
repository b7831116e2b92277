"""What a serving step does around the layers -- drafted tokens verified, cache entries and pages kept, adapters of many requests -- as a
user's program calls it, with plain forms to hold the calls against.

``listed()`` and ``draw()`` give the cases, ``prepare()`` what a program has in hand before the call, ``run()`` one pass, ``exact()``
the outputs from the definitions in 64 bits where they are computed numbers, ``work()`` the bytes and operations that a pass cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}

# Layers as (inputs, output rows of each shard): the 7B-shaped stack's fused QKV, o, fused gate/up and down, the 4096-wide and
# 5120-wide projections, and the 1024-wide embedding model's.
LAYERS = ((3584, (3584, 512, 512)), (3584, (3584,)), (18944, (3584,)), (4096, (4096,)), (5120, (5120,)), (1024, (1024,)))
GATED = ((3584, 18944), (4096, 11008), (5120, 17408))
# Caches as (kv heads, head size): the stack's, and the embedding model's heads of 64
KV = ((4, 128), (16, 64))


def listed():
    return [
        # one sequence, a short chain of drafted tokens, a small vocabulary: latency
        dict(name="verify_single", op="verify", batch=1, draft=4, vocab=32000, dtype="f32", tree=False, has_q=True),
        # a serving batch of chains over a large vocabulary
        dict(name="verify_batch", op="verify", batch=64, draft=7, vocab=131072, dtype="f32", tree=False, has_q=True),
        # drafted trees with several children drawn from one distribution; an odd vocabulary, so rows start anywhere
        dict(name="verify_trees", op="verify", batch=24, draft=31, vocab=50021, dtype="bf16", tree=True, has_q=True),
        # one prompt answered four times: its pages are shared, the last one copied in every layer
        dict(name="fork_prompt", op="fork", parents=1, children=4, context=1500, layers=28, kv_heads=4, dim=128, fmt="int8", page=64),
        # 32 prompts, seven more answers each
        dict(name="fork_batch", op="fork", parents=32, children=224, context=2048, layers=28, kv_heads=4, dim=128, fmt="fp8", page=64),
        # the accepted entries of 64 drafted trees move to the front of the drafted places, in every layer
        dict(name="compact_trees", op="compact", batch=64, places=32, most=8, context=1024, layers=28, kv_heads=4, dim=128, fmt="int8", page=64),
        # half of the entries of long contexts are dropped and the rest closed up
        dict(name="compact_long", op="compact", batch=8, places=16384, most=8192, context=0, layers=4, kv_heads=4, dim=128, fmt="int4", page=48),
        # the pages of a step: what was drafted and not accepted is given back, room for the next tokens is taken
        dict(name="pages_small", op="pages", rows=16, context=4000, width=8, page=64),
        # the same for a large server
        dict(name="pages_large", op="pages", rows=1021, context=16384, width=16, page=64),
        # one decode step of 16 requests, eight adapters, the fused QKV layer
        dict(name="lora_decode", op="lora", tokens=16, inputs=3584, shards="3584,512,512", rank=16, adapters=8, dtype="bf16", out="bf16", mixed=True, gated=False),
        # a verify step of many requests in the fused gate/up layer, with the gated product; odd number of tokens
        dict(name="lora_gated", op="lora", tokens=333, inputs=3584, shards="18944,18944", rank=16, adapters=40, dtype="bf16", out="bf16", mixed=True, gated=True),
        # several long prompts at once in the down layer
        dict(name="lora_prompts", op="lora", tokens=8192, inputs=18944, shards="3584", rank=64, adapters=6, dtype="f16", out="f16", mixed=False, gated=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("verify", "fork", "compact", "pages", "lora", "lora"))
    hk, dim = rng.choice(KV)
    fmt, page = rng.choice(("int8", "fp8", "int4")), rng.choice((16, 32, 48, 64, 128))
    layers = rng.choice((1, 4, 28))
    if op == "verify":
        tree = rng.random() < 0.5
        batch, vocab = _log(rng, 1, 64), _log(rng, 1000, 131072)
        draft = min(_log(rng, 1, 31), max(1, 64 * 8 * 131072 // (batch * vocab * (2 if tree else 1)) - 1))
        return dict(op=op, batch=batch, draft=draft, vocab=vocab, dtype=rng.choice(("f32", "f32", "f16", "bf16")), tree=tree, has_q=rng.random() < 0.7)
    if op == "fork":
        parents = _log(rng, 1, 32)
        children = _log(rng, 1, 224)
        context = min(_log(rng, 1, 16384), 32 * 2048 // parents)
        return dict(op=op, parents=parents, children=children, context=context, layers=layers if hk * dim == 512 else min(layers, 4), kv_heads=hk, dim=dim, fmt=fmt,
                    page=page)
    if op == "compact":
        if rng.random() < 0.6:
            batch, places = _log(rng, 1, 64), _log(rng, 2, 64)
            return dict(op=op, batch=batch, places=places, most=max(1, places // rng.choice((1, 2, 4))), context=_log(rng, 1, 2048), layers=layers if hk * dim == 512 else 4,
                        kv_heads=hk, dim=dim, fmt=fmt, page=page)
        batch = _log(rng, 1, 32)
        places = min(_log(rng, 65, 16384), 8 * 16384 // batch)
        return dict(op=op, batch=batch, places=places, most=max(1, int(places * rng.uniform(0.3, 0.9))), context=rng.choice((0, 100)), layers=rng.choice((1, 2)), kv_heads=hk,
                    dim=dim, fmt=fmt, page=page)
    if op == "pages":
        return dict(op=op, rows=_log(rng, 1, 1021), context=_log(rng, 1, 16384), width=_log(rng, 1, 64), page=page)
    rank = rng.choice((8, 16, 32, 64))
    adapters = _log(rng, 1, 64)
    dtype = rng.choice(("bf16", "f16"))
    if rng.random() < 0.3:
        inputs, half = rng.choice(GATED)
        tokens, shards, gated = _log(rng, 1, 1024), (half, half), True
    else:
        inputs, shards = rng.choice(LAYERS)
        tokens, gated = _log(rng, 1, 8192 * 22528 // max(22528, inputs + sum(shards))), False
    return dict(op=op, tokens=tokens, inputs=inputs, shards=",".join(str(n) for n in shards), rank=min(rank, 32) if gated else rank, adapters=adapters, dtype=dtype,
                out=rng.choice((dtype, dtype, "f32")), mixed=rng.random() < 0.5, gated=gated)


def _shards(case):
    return [int(n) for n in case["shards"].split(",")]


def _row_bytes(case):
    return case["dim"] // 2 if case["fmt"] == "int4" else case["dim"]


def _lengths(n, top):
    """Lengths of n sequences, from half of the longest up to it."""
    return [max(1, top - int(0.5 * top * ((0.618034 * b) % 1.0))) for b in range(n)]


def _kept(case):
    """How many entries each sequence of a compaction keeps: in a batch, one keeps none and one all that it may."""
    n, most = case["batch"], case["most"]
    kept = [max(1, most - int(most * ((0.618034 * b) % 1.0))) for b in range(n)]
    if n > 4:
        kept[3] = 0
    return kept


def work(case):
    if case["op"] == "verify":  # the row that the last token is drawn from, the drafter's beside it, and one entry of each a drafted token
        size = 4 if case["dtype"] == "f32" else 2
        sides = 2 if case["has_q"] else 1
        return {"bytes": case["batch"] * (sides * size * (case["vocab"] + case["draft"]) + 32 * case["draft"] + 16), "flops": case["batch"] * case["vocab"] * 3}
    if case["op"] == "fork":
        page, lens = case["page"], _lengths(case["parents"], case["context"])
        taken = [lens[i % case["parents"]] for i in range(case["children"])]
        row = 2 * case["kv_heads"] * case["layers"] * (_row_bytes(case) + 4)
        return {"bytes": sum(2 * (n % page) * row + (n // page) * 16 for n in taken), "flops": 0}
    if case["op"] == "compact":
        row = 2 * case["kv_heads"] * case["layers"] * (_row_bytes(case) + 4)
        return {"bytes": sum(_kept(case)) * (2 * row + 4) + case["batch"] * 8, "flops": 0}
    if case["op"] == "pages":  # reference counts are looked through for free pages; slots are written
        lens = _lengths(case["rows"], case["context"])
        return {"bytes": 4 * sum(-(-n // case["page"]) for n in lens) + case["rows"] * (8 * case["width"] + 40), "flops": 0}
    m, k, n, r, s = case["tokens"], case["inputs"], sum(_shards(case)), case["rank"], len(_shards(case))
    out = n // 2 if case["gated"] else n
    held = min(case["adapters"], m) * (s * r * k + n * r) * 2
    e = 4 if case["out"] == "f32" else 2
    return {"bytes": 2 * m * k + e * m * (n + out) + held + 4 * m, "flops": 2 * m * r * (s * k + n)}


# ------------------------------------------------------------------------------------------------ inputs
def _parents(case, seed):
    """Parents of drafted tokens (-1: the last committed one): a chain, or random trees of several children a node."""
    b, t = case["batch"], case["draft"]
    if not case["tree"]:
        return None
    gen = torch.Generator().manual_seed(int(seed))
    top = torch.arange(t).float()
    return ((torch.rand(b, t, generator=gen) * (top / 2).ceil()).long() - 1).clamp(max=torch.arange(t) - 1).to(DEV, torch.int32)


def _cache(gen, case, pages):
    """Codes and scales of every layer: raw codes of any value (no NaN), scales of a value's size."""
    h, page = case["kv_heads"], case["page"]
    shape = (case["layers"], pages, h, page)

    def codes():
        top = 126 if case["fmt"] == "fp8" else 256
        return torch.randint(0, top, (*shape, _row_bytes(case)), generator=gen, dtype=torch.uint8, device=DEV).view(CODES[case["fmt"]])

    return dict(k_codes=codes(), v_codes=codes(), k_scale=torch.rand(shape, generator=gen, device=DEV), v_scale=torch.rand(shape, generator=gen, device=DEV))


def _tables(gen, lens, wide, pages, page):
    """A page table of rows of given lengths over shuffled pages, and how many pages each row holds."""
    held = (torch.tensor(lens, dtype=torch.int64, device=DEV) + page - 1) // page
    table = torch.zeros(len(lens), wide, dtype=torch.int32, device=DEV)
    used = torch.arange(wide, device=DEV) < held[:, None]
    table[used] = torch.randperm(pages, generator=gen, device=DEV)[:int(held.sum())].int()
    return table, held.int(), used


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "verify":
        b, t, v, kind = case["batch"], case["draft"], case["vocab"], DTYPES[case["dtype"]]
        z = 3.0 * torch.randn(b, t + 1, v, generator=gen, device=DEV)
        p = z.softmax(-1)
        p = torch.where(p < 1e-7, torch.zeros_like(p), p)  # as a filter of unlikely tokens leaves it
        s["target"] = (p / p.sum(-1, keepdim=True)).to(kind)
        q = (z[:, :t] + 0.8 * torch.randn(b, t, v, generator=gen, device=DEV)).softmax(-1)
        parent = _parents(case, seed)
        node = torch.arange(t, device=DEV).expand(b, t) if parent is None else parent.long() + 1
        noise = -torch.empty(b, t, v, device=DEV).exponential_(generator=gen).log()
        s["tokens"] = (q.log().gather(1, node[:, :, None].expand(b, t, v)) + noise).argmax(-1)  # drawn from the drafter's distribution
        s["draft_probs"] = q.to(kind) if case["has_q"] else None
        s["parent"] = parent
        s["uniform"] = torch.rand(b, t + 1, generator=gen, device=DEV)
        return s
    if case["op"] == "fork":
        a, c, page = case["parents"], case["children"], case["page"]
        lens = _lengths(a, case["context"])
        wide = -(-case["context"] // page) + 1
        pages = sum(-(-n // page) for n in lens) + c + 2
        table, held, used = _tables(gen, lens + [0] * c, wide, pages, page)
        s.update(_cache(gen, case, pages))
        s["table"], s["held"] = table, held
        s["lens"] = torch.tensor(lens + [0] * c, dtype=torch.int32, device=DEV)
        s["refs"] = torch.bincount(table[used].long(), minlength=pages).int()
        s["parent"] = torch.cat([torch.full((a,), -1, device=DEV), torch.arange(c, device=DEV) % a]).int()
        s["keep"] = torch.cat([torch.full((a,), -1, device=DEV), torch.zeros(c, device=DEV, dtype=torch.int64)]).int()
        return s
    if case["op"] == "compact":
        n, most, page = case["places"], case["most"], case["page"]
        lens = _lengths(case["batch"], case["context"]) if case["context"] else [0] * case["batch"]
        total = [m + n for m in lens]
        pages = sum(-(-m // page) for m in total) + 2
        s["table"], _, _ = _tables(gen, total, -(-max(total) // page), pages, page)
        s.update(_cache(gen, case, pages))
        s["start"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["keep"] = torch.rand(case["batch"], n, generator=gen, device=DEV).argsort(1)[:, :most].sort(1).values.int()
        s["count"] = torch.tensor(_kept(case), dtype=torch.int32, device=DEV)
        return s
    if case["op"] == "pages":
        rows, page, width = case["rows"], case["page"], case["width"]
        lens = _lengths(rows, case["context"])
        wide = -(-(case["context"] + width) // page) + 1
        pages = sum(-(-n // page) for n in lens) + max(2, rows // 2)  # not always enough for everybody
        table, held, used = _tables(gen, lens, wide, pages, page)
        odd = torch.arange(1, rows, 4, device=DEV)  # every fourth row shares the first half of the row before it, as a fork leaves them
        both = torch.minimum(held[odd], held[odd - 1]) // 2
        first = torch.arange(wide, device=DEV) < both[:, None]
        table[odd] = torch.where(first, table[odd - 1], table[odd])
        s["table"], s["held"] = table, held
        s["refs"] = torch.bincount(table[used].long(), minlength=pages).int()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        keep = s["lens"] - torch.randint(0, width + 1, (rows,), generator=gen, device=DEV).int()
        what = torch.rand(rows, generator=gen, device=DEV)
        keep = torch.where(what < 0.05, torch.zeros_like(keep), keep.clamp(min=0))  # an answer that has ended
        s["keep"] = torch.where(what > 0.95, torch.full_like(keep, -1), keep)  # a row that this step leaves alone
        s["extra"] = torch.randint(0, width + 1, (rows,), generator=gen, device=DEV).int()
        return s
    m, k, shards, r, n = case["tokens"], case["inputs"], _shards(case), case["rank"], case["adapters"]
    kind, total = DTYPES[case["dtype"]], sum(_shards(case))
    s["x"] = torch.randn(m, k, generator=gen, device=DEV).to(kind)
    s["y"] = torch.randn(m, total, generator=gen, device=DEV).to(DTYPES[case["out"]])  # what the shared layer gave
    s["a"] = (torch.randn(n, len(shards) * r, k, generator=gen, device=DEV) * k ** -0.5).to(kind)
    s["b"] = (torch.randn(n, total, r, generator=gen, device=DEV) * r ** -0.5).to(kind)
    s["scale"] = 0.25 + 0.5 * torch.rand(n, generator=gen, device=DEV)
    if case["mixed"]:  # each token has a request of its own; some have no adapter
        s["which"] = torch.randint(-1, n, (m,), generator=gen, device=DEV).int()
    else:  # runs of tokens
        cuts = torch.randint(0, m, (n,), generator=gen, device=DEV).sort().values
        s["which"] = torch.searchsorted(cuts, torch.arange(m, device=DEV), right=True).int() - 1
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _drawn(w, p, u):
    """The token that u points at in weights w (in p where w is empty)."""
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    c = w.cumsum(1)
    last = (w > 0).long().mul(torch.arange(1, w.shape[1] + 1, device=DEV)).amax(1) - 1
    return torch.minimum((c <= u[:, None] * c[:, -1:]).sum(1), last)


def _result(s, path, count, token):
    b, t = s["tokens"].shape
    at = torch.arange(t, device=DEV)
    path = torch.where(at < count[:, None], path, torch.full_like(path, -1))
    given = torch.where(path >= 0, s["tokens"].gather(1, path.clamp(min=0)), torch.full_like(path, -1))
    out = torch.cat([given, torch.full_like(given[:, :1], -1)], 1).scatter(1, count[:, None], token[:, None])
    return path.int(), count.int(), out


def _verify_chains(s):
    b, t = s["tokens"].shape
    each = torch.arange(b, device=DEV)
    u = s["uniform"].double()
    px = s["target"][:, :t].gather(2, s["tokens"][..., None])[..., 0].double()
    qx = s["draft_probs"].gather(2, s["tokens"][..., None])[..., 0].double() if s["has_q"] else torch.ones_like(px)
    count = (u[:, :t] * qx < px).long().cumprod(1).sum(1)
    p = s["target"][each, count].double()
    stop, at = count < t, count.clamp(max=t - 1)
    if s["has_q"]:
        w = torch.where(stop[:, None], (p - s["draft_probs"][each, at].double()).clamp(min=0), p)
    else:
        x = s["tokens"][each, at][:, None]
        w = p.scatter(1, x, torch.where(stop[:, None], torch.zeros_like(p[:, :1]), p.gather(1, x)))
    path = torch.arange(t, device=DEV).expand(b, t)
    return _result(s, path, count, _drawn(w, p, u[:, t]))


def _verify_trees(s):
    """Tokens in their order, parents before children: one is looked at where its parent is the node that its sequence stands at."""
    b, t = s["tokens"].shape
    each, u = torch.arange(b, device=DEV), s["uniform"].double()
    node, count = torch.zeros(b, dtype=torch.int64, device=DEV), torch.zeros(b, dtype=torch.int64, device=DEV)
    taken, left = torch.zeros(b, dtype=torch.float64, device=DEV), torch.ones(b, dtype=torch.float64, device=DEV)
    path = torch.full((b, t), -1, dtype=torch.int64, device=DEV)
    p = s["target"][:, 0].double()
    w, q = p, (s["draft_probs"][:, 0].double() if s["has_q"] else None)
    for i in range(t):
        x = s["tokens"][:, i]
        mine = s["parent"][:, i] == node - 1
        qx = q[each, x] if s["has_q"] else torch.ones_like(left)
        yes = mine & (u[:, i] * (left * qx) < w[each, x])
        no = mine & ~yes
        if s["has_q"]:
            taken = torch.where(no, taken + left, taken)
            w = torch.where(no[:, None], (p - taken[:, None] * q).clamp(min=0), w)
            left = torch.where(no, w.sum(1), left)
        else:
            left = torch.where(no, left - w[each, x], left)
            w = w.scatter(1, x[:, None], torch.where(no, torch.zeros_like(left), w[each, x])[:, None])
        path = torch.where(yes[:, None], path.scatter(1, count.clamp(max=t - 1)[:, None], i), path)
        count = count + yes
        node = torch.where(yes, torch.full_like(node, i + 1), node)
        taken, left = torch.where(yes, torch.zeros_like(taken), taken), torch.where(yes, torch.ones_like(left), left)
        p = torch.where(yes[:, None], s["target"][:, i + 1].double(), p)
        w = torch.where(yes[:, None], p, w)
        if s["has_q"] and i + 1 < t:
            q = torch.where(yes[:, None], s["draft_probs"][:, i + 1].double(), q)
    return _result(s, path, count, _drawn(w, p, u[:, t]))


def _move(s, ps, os, pd, od):
    """Entries at (page, place) pairs to others, in every layer: all read before any is written."""
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        ten = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
        ten[:, pd, :, od] = ten[:, ps, :, os]


def _free(s):
    wide, page = s["table"].shape[1], s["page"]
    at, touch = torch.arange(wide, device=DEV), s["keep"] >= 0
    stay = torch.where(touch, (s["keep"] + page - 1) // page, s["held"])
    gone = (at >= stay[:, None]) & (at < s["held"][:, None])
    s["refs"] -= torch.bincount(s["table"][gone].long(), minlength=s["refs"].shape[0]).int()
    s["table"][gone] = 0
    s["held"].copy_(stay)
    s["lens"].copy_(torch.where(touch, s["keep"], s["lens"]))


def _take(s, need):
    """Free pages, lowest first, to rows in order as long as they suffice: who has what it needs, and each one's pages."""
    free = (s["refs"] == 0).nonzero()[:, 0]
    ok = (need == 0) | (need.cumsum(0) <= free.shape[0])
    need = torch.where(ok, need, torch.zeros_like(need))
    rows = torch.repeat_interleave(torch.arange(len(need), device=DEV), need)
    pages = free[:len(rows)]
    s["refs"][pages] = 1
    return ok, rows, torch.arange(len(rows), device=DEV) - (need.cumsum(0) - need)[rows], pages


def _fork(s):
    _free(s)
    page, wide = s["page"], s["table"].shape[1]
    child = s["parent"] >= 0
    of = s["parent"].clamp(min=0).long()
    n = torch.where(child, s["lens"][of], torch.zeros_like(s["lens"]))
    full, part = (n // page).long(), (n % page).long()
    ok, rows, _, pages = _take(s, (part > 0).long())
    full = torch.where(child & ok, full, torch.zeros_like(full))
    shared = torch.arange(wide, device=DEV) < full[:, None]
    s["table"].copy_(torch.where(shared, s["table"][of], s["table"]))
    s["refs"] += torch.bincount(s["table"][shared].long(), minlength=s["refs"].shape[0]).int()
    old = s["table"][of[rows], full[rows]].long()
    s["table"][rows, full[rows]] = pages.int()
    s["lens"].copy_(torch.where(child & ok, n, s["lens"]))
    s["held"].copy_(torch.where(child & ok, (full + (part > 0)).int(), s["held"]))
    f, o = (torch.arange(page, device=DEV) < part[rows][:, None]).nonzero(as_tuple=True)
    _move(s, old[f], o, pages[f], o)
    return ok


def _compact(s):
    page = s["page"]
    at = torch.arange(s["keep"].shape[1], device=DEV)
    b, i = (at < s["count"][:, None]).nonzero(as_tuple=True)
    src, dst = s["start"][b] + s["keep"][b, i], s["start"][b] + i
    _move(s, s["table"][b, src // page].long(), src % page, s["table"][b, dst // page].long(), dst % page)


def _reserve(s):
    page, wide, width = s["page"], s["table"].shape[1], s["width"]
    upto = (s["lens"] + s["extra"] + page - 1) // page
    ok, rows, nth, pages = _take(s, (upto - s["held"]).clamp(min=0).long())
    s["table"][rows, s["held"][rows] + nth] = pages.int()
    s["held"].copy_(torch.where(ok, torch.maximum(s["held"], upto), s["held"]))
    place = s["lens"][:, None] + torch.arange(width, device=DEV)
    slots = s["table"].long().gather(1, (place // page).clamp(max=wide - 1)) * page + place % page
    return torch.where(ok[:, None] & (torch.arange(width, device=DEV) < s["extra"][:, None]), slots, torch.full_like(slots, -1)), ok


def _lora(s):
    shards, r = _shards(s), s["rank"]
    n, cuts = s["a"].shape[0], [sum(shards[:i]) for i in range(len(shards) + 1)]
    h = (s["x"].float() @ s["a"].float().flatten(0, 1).T).view(-1, n, len(shards), r)
    mine = s["which"][:, None] == torch.arange(n, device=DEV)
    h = torch.where(mine[..., None, None], h * s["scale"][:, None, None], torch.zeros_like(h))
    z = s["y"].float() + torch.cat([h[:, :, i].flatten(1) @ s["b"][:, cuts[i]:cuts[i + 1]].float().transpose(1, 2).flatten(0, 1) for i in range(len(shards))], 1)
    if s["gated"]:
        g, u = z.chunk(2, 1)
        z = g / (1 + (-g).exp()) * u
    return z.to(s["y"].dtype)


# ------------------------------------------------------------------------------------------------ one pass
def _handles(s):
    """The program's handles on its caches and its pages, kept with them."""
    import ternary_weight_linear_02_gb300 as tl
    if "k_codes" in s and "layers_handle" not in s:
        s["layers_handle"] = tl.KVLayers([tl.KVCache(s["fmt"], s["k_codes"][i], s["v_codes"][i], s["k_scale"][i], s["v_scale"][i]) for i in range(s["layers"])])
    if "refs" in s and "pages_handle" not in s:
        s["pages_handle"] = tl.KVPages(s["page"], s["refs"], s["table"], s["lens"], s["held"])
    return tl, s.get("layers_handle"), s.get("pages_handle")


def run(s):
    if s["op"] == "verify":
        if own:
            import ternary_weight_linear_02_gb300 as tl
            return tl.verify_drafts(s["target"], s["tokens"], s["uniform"], draft=s["draft_probs"], parent=s["parent"])
        return _verify_trees(s) if s["tree"] else _verify_chains(s)
    if s["op"] == "fork":  # the children of the pass before make room, then the parents are forked again
        if own:
            tl, layers, pages = _handles(s)
            tl.pages_free(pages, s["keep"])
            ok = tl.pages_fork(pages, s["parent"], layers)
        else:
            ok = _fork(s)
        return ok, s["table"], s["refs"], s["lens"], s["held"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
    if s["op"] == "compact":
        if own:
            tl, layers, _ = _handles(s)
            tl.kv_compact(layers, s["table"], s["start"], s["keep"], s["count"])
        else:
            _compact(s)
        return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
    if s["op"] == "pages":
        if own:
            tl, _, pages = _handles(s)
            tl.pages_free(pages, s["keep"])
            slots, ok = tl.pages_reserve(pages, s["extra"], s["width"])
        else:
            _free(s)
            slots, ok = _reserve(s)
        return slots, ok, s["table"], s["refs"], s["lens"], s["held"]
    if own:
        import ternary_weight_linear_02_gb300 as tl
        if "adapters_handle" not in s:
            s["adapters_handle"] = tl.Adapters(s["a"], s["b"], s["scale"], shards=_shards(s))
        return (tl.lora_silu_mul if s["gated"] else tl.lora_add)(s["x"], s["adapters_handle"], s["which"], s["y"])
    return _lora(s)


# ------------------------------------------------------------------------------------------------ 64 bits
def _moved(case, seed):
    """The scales of a cache after a fork or a compaction, entry by entry from lists of what goes where."""
    s, page = prepare(case, seed), case["page"]
    table, moves = s["table"].tolist(), []
    if case["op"] == "fork":
        lens, free = s["lens"].tolist(), [i for i, n in enumerate(s["refs"].tolist()) if n == 0]
        for p in s["parent"].tolist():
            if p >= 0 and lens[p] % page and free:
                new = free.pop(0)
                moves += [(table[p][lens[p] // page] * page + i, new * page + i) for i in range(lens[p] % page)]
    else:
        for b, (at, n) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
            for i, j in enumerate(s["keep"][b, :n].tolist()):
                moves.append(tuple(table[b][place // page] * page + place % page for place in (at + j, at + i)))
    src, dst = torch.tensor(moves, dtype=torch.int64, device=DEV).reshape(-1, 2).T
    got = []
    for name in ("k_scale", "v_scale"):
        rows = s[name].double().transpose(2, 3).flatten(1, 2)  # [layers, slots, heads]
        rows = rows.index_copy(1, dst, rows[:, src])
        got.append(rows.unflatten(1, (-1, page)).transpose(2, 3).contiguous())
    return got


def exact(case, seed):
    if case["op"] in ("verify", "pages"):  # whole numbers
        return None
    if case["op"] == "fork":
        return (None,) * 7 + tuple(_moved(case, seed))
    if case["op"] == "compact":
        return (None, None, *_moved(case, seed))
    s, shards, r = prepare(case, seed), _shards(case), case["rank"]
    z = s["y"].double()
    for a in range(case["adapters"]):
        rows = (s["which"] == a).nonzero()[:, 0]
        if len(rows) == 0:
            continue
        x, at = s["x"][rows].double(), 0
        for i, n in enumerate(shards):
            h = torch.einsum("mk,rk->mr", x, s["a"][a, i * r:(i + 1) * r].double())
            z[rows, at:at + n] += float(s["scale"][a]) * torch.einsum("mr,nr->mn", h, s["b"][a, at:at + n].double())
            at += n
    if not case["gated"]:
        return z
    g, u = z[:, :shards[0]], z[:, shards[0]:]
    return g * torch.sigmoid(g) * u
