#!/usr/bin/env python3
"""Steps of a small server with drafted trees: pages taken, the layers with each request's own adapter, drafted tokens
verified, accepted entries closed up, pages given back -- without an answer on the host in between.

A prompt is answered several times: its row of the page table is forked, so that its full pages are shared.  Each step, a
drafter proposes a tree for every row (here: tokens drawn from a blurred copy of the target's last distribution);
``pages_reserve`` finds room for the row's last token and its tree, one pass of the stack scores them,
``verify_drafts`` accepts a path and draws the token after it, ``kv_compact`` moves the path's entries behind the
committed ones and ``pages_free`` gives back what lies behind.

    python examples/serve_step.py [--layers 2] [--rows 8] [--draft 12] [--steps 10]

Prints tokens per step and row and the time of a step.  Synthetic weights and inputs.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import ternary_weight_linear_02_gb300 as tl  # noqa: E402
import verify_step as vs  # noqa: E402


class Server:
    """A stack of layers with embeddings, adapters and the pages of its rows."""

    def __init__(self, stack, rows, max_pages, vocab=2048, adapters=4, rank=16, seed=0):
        dev = stack.table.device
        gen = torch.Generator(device=dev).manual_seed(seed)
        hidden = stack.layers[0][0]["o"][0].shape[0]
        self.stack, self.rows, self.vocab, self.gen = stack, rows, vocab, gen
        self.embed = torch.randn(vocab, hidden, generator=gen, device=dev).to(torch.bfloat16)
        self.head = (torch.randn(vocab, hidden, generator=gen, device=dev) * (2.0 * hidden ** -0.5)).to(torch.bfloat16)
        self.adapters = stack.adapt(adapters, rank, seed)
        cache = stack.caches.first
        self.pages = tl.KVPages.empty(cache.pages, rows, max_pages, cache.page_size, dev)
        self.last = torch.zeros(rows, dtype=torch.int64, device=dev)           # each row's newest token, not yet in the cache
        self.which = (torch.arange(rows, device=dev) % (adapters + 1) - 1).int()  # each row's adapter; -1: none

    def probabilities(self, x):
        return (vs.norm(x) @ self.head.T).float().softmax(-1)

    def prompt(self, row, tokens):
        """Writes a prompt into a row and draws the token after it.  Returns ok, on the device: False where it found no pages
        (the row stays as it is)."""
        n = tokens.shape[0]
        extra = torch.full((self.rows,), -1, dtype=torch.int32, device=tokens.device)
        extra[row] = n
        slots, ok = tl.pages_reserve(self.pages, extra, n)
        ctx = self.pages.lens[row:row + 1]
        x = self.stack.step(self.embed[tokens][None], torch.arange(n, device=tokens.device), slots[row], self.pages.table[row:row + 1], ctx,
                            adapters=self.adapters, which=self.which[row].expand(n))
        tl.pages_free(self.pages, torch.where(ok & (extra >= 0), self.pages.lens + extra, -1))
        drawn = torch.multinomial(self.probabilities(x[0, -1:]), 1, generator=self.gen)[0, 0]
        self.last[row] = torch.where(ok[row], drawn, self.last[row])
        return ok[row]

    def fork(self, parent):
        """Rows continue others (int32 [rows], -1: a row stays).  Returns ok: False where no page was left (the row stays empty)."""
        ok = tl.pages_fork(self.pages, parent, self.stack.caches)
        child = ok & (parent >= 0)
        self.last = torch.where(child, self.last[parent.clamp(min=0).long()], self.last)
        return ok

    def draft(self, parent, depth):
        """Tokens of a tree, drawn node by node from one distribution a node, and those distributions."""
        b, t = parent.shape
        q = torch.randn(b, t, self.vocab, generator=self.gen, device=self.last.device).mul_(2).softmax(-1)
        rows = q.gather(1, (parent + 1).long()[:, :, None].expand(b, t, self.vocab))
        return torch.multinomial(rows.flatten(0, 1), 1, generator=self.gen).view(b, t), q

    def step(self, parent, depth, sees):
        """One step: parent int32 [rows, draft], depth and sees of the trees (verify_step.random_trees) on the device.  A row that
        is empty or for which no pages are left takes no part: it keeps its tokens, entries and pages, and ok is False for it."""
        b, t = parent.shape
        dev, pages = self.last.device, self.pages
        drafted, q = self.draft(parent, depth)
        tokens = torch.cat([self.last[:, None], drafted], 1)                      # the row's newest token heads its tree
        live = pages.lens > 0
        slots, ok = tl.pages_reserve(pages, torch.where(live, t + 1, -1).int(), t + 1)
        ok = ok & live
        tree = torch.zeros(b, t + 1, t + 1, dtype=torch.bool, device=dev)
        tree[:, :, 0] = True
        tree[:, 1:, 1:] = sees
        places = pages.lens[:, None].long() + torch.cat([torch.zeros_like(depth[:, :1]), depth + 1], 1)
        x = self.stack.step(self.embed[tokens], places.flatten(), slots.flatten(), pages.table, pages.lens, tree,
                            adapters=self.adapters, which=self.which[:, None].expand(b, t + 1).flatten())
        target = self.probabilities(x)
        uniform = torch.rand(b, t + 1, generator=self.gen, device=dev)
        path, count, out = tl.verify_drafts(target, drafted, uniform, draft=q, parent=parent)
        path, count, out = torch.where(ok[:, None], path, -1), torch.where(ok, count, 0), torch.where(ok[:, None], out, -1)
        start = pages.lens + 1
        tl.kv_compact(self.stack.caches, pages, start, path, count)
        tl.pages_free(pages, torch.where(ok, start + count, -1))
        self.last = torch.where(ok, out.gather(1, count[:, None].long())[:, 0], self.last)
        return dict(target=target, q=q, drafted=drafted, uniform=uniform, path=path, count=count, tokens=out, slots=slots, ok=ok)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--rows", type=int, default=8)
    ap.add_argument("--draft", type=int, default=12)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--format", choices=sorted(tl.KV_FORMATS), default="int8")
    a = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    most = a.prompt + a.steps * (a.draft + 1) + a.draft + 1
    stack = vs.Stack(layers=a.layers, fmt=a.format, pages=a.rows * (-(-most // 64)), device=dev)
    server = Server(stack, a.rows, -(-most // 64))
    if not bool(server.prompt(0, torch.randint(0, server.vocab, (a.prompt,), generator=server.gen, device=dev))):
        raise RuntimeError("no pages were left for the prompt")
    parent = torch.zeros(a.rows, dtype=torch.int32, device=dev)
    parent[0] = -1
    if not bool(server.fork(parent).all()):
        raise RuntimeError("no page was left for a fork")
    cpu, counts, served = torch.Generator().manual_seed(1), [], []
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        tree, depth, sees = vs.random_trees(a.rows, a.draft, cpu)
        tree, depth, sees = tree.to(dev, torch.int32), depth.to(dev), sees.to(dev)
        if i == 1:
            start.record()
        got = server.step(tree, depth, sees)
        counts.append(got["count"])
        served.append(got["ok"])
    end.record()
    torch.cuda.synchronize()
    if tl.device_status() != 0 or not bool(torch.stack(served).all()):
        raise RuntimeError("a row found no pages, or a call reported an index out of range")
    mean = float(torch.stack(counts).float().mean()) + 1
    print(f"{mean:.2f} tokens a step and row, {start.elapsed_time(end) / max(a.steps - 1, 1):.3f} ms a step: {a.layers} layers, {a.rows} rows, "
          f"trees of {a.draft}, {int((server.pages.refs > 0).sum())} of {server.pages.pages} pages in use")
    return mean


if __name__ == "__main__":
    main()
