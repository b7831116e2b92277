#!/usr/bin/env python3
"""One decode / verify step of a ternary transformer stack: the linear layers, rotary
positions, the quantised paged cache and tree attention together.

A drafter proposes a tree of tokens for each sequence.  One pass of the stack scores
the whole tree: per layer the fused QKV call, ``kv_append`` (rotates q and k by each
token's depth and writes k and v to the cache in 8 or 4 bits), ``tree_attention`` (each
token sees the context and its own ancestors), the o call, the fused gate/up call with
the SiLU-gated product, and down.  The accepted path's entries are then moved to the
front of the drafted places (the cache's tensors take ordinary indexing), and the
next step goes on from there.

    python examples/verify_step.py [--layers 4] [--batch 4] [--draft 16] [--context 2000]

Prints the time of a step and how far a path's hidden states in the tree are from the
same tokens decoded one by one.  Synthetic weights and inputs.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ternary_weight_linear_02_gb300 as tl  # noqa: E402
from ternary_weight_linear_02_gb300 import synth  # noqa: E402


class Stack:
    """Layers of the 7B-shaped stack (sizes may be smaller), each with a cache of its own."""

    def __init__(self, layers=4, hidden=3584, q_heads=28, kv_heads=4, head_dim=128, ffn=18944, fmt="int8",
                 page_size=64, pages=256, positions=32768, seed=0, device="cuda", group=0):
        """group: columns of weights that share a scale (0: one scale per row)."""
        self.q_heads, self.kv_heads, self.page_size, self.group = q_heads, kv_heads, page_size, group
        rows = (q_heads + 2 * kv_heads) * head_dim
        self.head_dim, self.table = head_dim, tl.rope_table(positions, head_dim, base=1e6, device=device)
        self.layers = []
        for i in range(layers):
            w = {}
            for name, n, k in (("qkv", rows, hidden), ("o", hidden, q_heads * head_dim), ("gu", 2 * ffn, hidden),
                               ("down", hidden, ffn)):
                # scales that keep a unit-variance input at unit variance (60% of the weights are not 0)
                s = (0.6 * k) ** -0.5
                w[name] = (synth.packed_codes(n, k, synth.seed_for("verify", seed, i, name), device),
                           synth.scales(n, k // group if group else 0, 0.9 * s, 1.1 * s,
                                        synth.seed_for("verify", seed, i, name, "s"), device))
            self.layers.append((w, tl.KVCache.empty(fmt, pages, page_size, kv_heads, head_dim, device)))

    def step(self, x, positions, slots, page_table, context_len, tree=None):
        """x [batch, draft, hidden] through every layer; the new tokens' keys and values go to
        slots (int64 [batch * draft])."""
        b, t, hidden = x.shape
        hq, hk, g = self.q_heads, self.kv_heads, self.group
        x = x.flatten(0, 1)
        for w, cache in self.layers:
            qkv = tl.linear(norm(x), *w["qkv"], g, static_weights=True).unflatten(1, (hq + 2 * hk, self.head_dim))
            q = qkv[:, :hq]
            tl.kv_append(cache, qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, q=q, positions=positions, table=self.table,
                         q_out=q)
            a = tl.tree_attention(q.unflatten(0, (b, t)), cache, page_table, context_len, tree)
            x = x + tl.linear(a.flatten(0, 1).flatten(1), *w["o"], g, static_weights=True)
            h = tl.linear_silu_mul(norm(x), *w["gu"], g, static_weights=True)
            x = x + tl.linear(h, *w["down"], g, static_weights=True)
        return x.unflatten(0, (b, t))

    def accept(self, page_table, context_len, path, count):
        """Moves each sequence's accepted drafted entries (path int64 [batch, n], indexes of drafted
        tokens in order; the first count[b] of them are kept) to the front of the drafted places."""
        n = path.shape[1]
        at = torch.arange(n, device=path.device)
        keep = at < count[:, None]
        src = slots_of(page_table, context_len[:, None] + path, self.page_size)[keep]
        dst = slots_of(page_table, context_len[:, None] + at, self.page_size)[keep]
        for _, c in self.layers:
            for ten in (c.k_codes, c.v_codes, c.k_scale, c.v_scale):
                raw = ten.view(torch.uint8) if ten.dtype == torch.float8_e4m3fn else ten
                raw[dst // self.page_size, :, dst % self.page_size] = raw[src // self.page_size, :, src % self.page_size]
        return context_len + count.int()


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def slots_of(page_table, places, page_size):
    """Slot of each place (key index) of each sequence: [batch, n]."""
    return page_table.long().gather(1, places // page_size) * page_size + places % page_size


def random_trees(batch, draft, generator):
    """Parents (-1: the context's last token) and depths of random trees, and who sees whom."""
    parent = torch.full((batch, draft), -1)
    sees = torch.zeros(batch, draft, draft, dtype=torch.bool)
    for b in range(batch):
        for i in range(draft):
            if i:
                parent[b, i] = int(torch.randint(-1, i, (1,), generator=generator))
            if parent[b, i] >= 0:
                sees[b, i] = sees[b, parent[b, i]]
            sees[b, i, i] = True
    return parent, sees.sum(2) - 1, sees


def prefill(stack, context, page_table, generator, device):
    """Writes `context` tokens of every sequence, a chunk at a time (a chain of new tokens)."""
    batch, hidden = page_table.shape[0], stack.layers[0][0]["qkv"][0].shape[1] * 4
    done = torch.zeros(batch, dtype=torch.int32, device=device)
    for a in range(0, context, 128):
        n = min(128, context - a)
        x = torch.randn(batch, n, hidden, generator=generator, device=device).to(torch.bfloat16)
        places = (done[:, None] + torch.arange(n, device=device)).long()
        stack.step(x, places.flatten(), slots_of(page_table, places, stack.page_size).flatten(), page_table, done)
        done = done + n
    return done


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--draft", type=int, default=16)
    ap.add_argument("--context", type=int, default=2000)
    ap.add_argument("--group", type=int, default=0, choices=(0, 32, 64, 128, 256), help="columns per weight scale (0: one per row)")
    ap.add_argument("--format", choices=sorted(tl.KV_FORMATS), default="int8")
    a = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen, cpu = torch.Generator(device=dev).manual_seed(1), torch.Generator().manual_seed(1)
    per = -(-(a.context + a.draft) // 64)
    stack = Stack(layers=a.layers, fmt=a.format, pages=a.batch * per, device=dev, group=a.group)
    page_table = torch.randperm(a.batch * per, generator=gen, device=dev).int().view(a.batch, per)
    ctx = prefill(stack, a.context, page_table, gen, dev)
    parent, depth, sees = random_trees(a.batch, a.draft, cpu)
    x = torch.randn(a.batch, a.draft, 3584, generator=gen, device=dev).to(torch.bfloat16)
    places = (ctx[:, None] + torch.arange(a.draft, device=dev)).long()
    args = (x, (ctx[:, None] + depth.to(dev)).flatten().long(), slots_of(page_table, places, 64).flatten(), page_table, ctx,
            sees.to(dev))
    tree = stack.step(*args)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        stack.step(*args)
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end) / 10:.3f} ms per step: {a.layers} layers, {a.batch} trees of {a.draft} tokens "
          f"over {a.context}, {a.format} cache")
    # the deepest path of each tree, token by token
    leaf = depth.argmax(1)
    paths = []
    for b in range(a.batch):
        path, i = [], int(leaf[b])
        while i >= 0:
            path.insert(0, i)
            i = int(parent[b, i])
        paths.append(path)
    n = min(len(p) for p in paths)
    path = torch.tensor([p[:n] for p in paths], device=dev)
    for i in range(n):
        now = ctx + i
        y = stack.step(x.gather(1, path[:, i, None, None].expand(-1, 1, x.shape[2])), now.long(),
                       slots_of(page_table, now[:, None].long(), 64).flatten(), page_table, now)
    last = tree.gather(1, path[:, n - 1, None, None].expand(-1, 1, x.shape[2]))
    off = float((y.float() - last.float()).norm() / last.float().norm())
    print(f"token {n} of the deepest paths, in the tree and one by one: relative difference {off:.2e}")
    if tl.device_status() != 0:
        raise RuntimeError("a call reported " + tl.status_string(tl.device_status()))
    return off


if __name__ == "__main__":
    main()
