"""Tree-drafted decoding on the framework's calls: one layer's attention side of a verify step, captured once.

    python examples/tree_decoding.py [--seqs 4] [--context 2000] [--drafted 15] [--steps 20] [--cache e4m3]

Every step each request drafts a tree of tokens; the step's page tables, slots, positions and masks are built on the GPU
from the requests' lengths (`kv_assign`), keys and queries are normalised, rotated and appended in one launch
(`kv_append` with norms), each drafted token attends to its context and its ancestors (`tree_attention`), and the
accepted path's rows move next to each other (`kv_accept`), whose lengths the next step starts from.  The four calls are
one CUDA graph; lengths, trees and paths change between its replays.  Drafts and verdicts come at random: what stands
around the attention side in a model (projections, lm_head, the draft model) is not here.
"""

from __future__ import annotations

import argparse
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_w4a16_moe_skinny_gb300 import binding  # noqa: E402


class TreeDecoder:
    """A layer's cache, norms and rotary table, and the buffers of a step for a fixed batch of requests."""

    def __init__(self, lib, heads, kv_heads, dim, seqs, drafted, max_len, page=64, cache="bf16", seed=0):
        dev = torch.device("cuda", 0)
        g = torch.Generator(device=dev).manual_seed(seed)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
        self.lib, self.heads, self.kv_heads, self.seqs, self.drafted = lib, heads, kv_heads, seqs, drafted
        self.inv_freq = lib.rope_frequencies(dim, 500000.0, device=dev)
        self.q_norm, self.k_norm = ((1.0 + 0.1 * torch.randn(dim, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2))
        most = -(-(max_len + drafted) // page)
        dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
        scale = torch.full((kv_heads,), 0.02, device=dev) if cache == "e4m3" else None
        pool = torch.zeros(seqs * most, 2, kv_heads, page, dim, device=dev).to(dtype)
        self.cache = binding.KVCache(pool[:, 0], pool[:, 1], scale, scale)
        free = torch.randperm(seqs * most, generator=g, device=dev).to(torch.int32)
        self.pages = binding.PageTable(i32(seqs, most) - 1, i32(seqs), free, i32(1) + seqs * most, page)
        self.step = binding.Step(seqs, seqs * drafted, -(-drafted // 64), dev)
        self.batch = self.step.batch(self.pages.page_table, drafted)
        self.kv_len, self.new, self.parents = i32(seqs), i32(seqs), i32(seqs * drafted)
        self.paths = i32(seqs, drafted)

    def assign(self):
        """The step's tables: first, as the draft and its masks depend on nothing else."""
        return self.lib.kv_assign(self.pages, self.kv_len, self.new, self.step, self.parents)

    def attend(self, qkv):
        """Appends and attends the drafted rows qkv [rows, heads + 2 kv_heads, dim]."""
        h, kv, s = self.heads, self.kv_heads, self.step
        q = self.lib.kv_append(self.cache, qkv[:, h:h + kv], qkv[:, h + kv:], s.slots, s.positions, self.inv_freq,
                               q=qkv[:, :h], q_norm=self.q_norm, k_norm=self.k_norm)
        return self.lib.tree_attention(q, self.cache, self.batch, s.masks)

    def accept(self):
        """Keeps self.paths of the drafted rows; the next step starts from the lengths that are left."""
        self.lib.kv_accept(self.cache, self.batch, self.paths, out=self.kv_len)


def draft(rng, n):
    """A tree of n tokens: each one's parent is one of the last few, or the context."""
    return [rng.randint(max(-1, i - 4), i - 1) for i in range(n)]


def verdict(rng, parents):
    """The path to some token of the tree."""
    path, i = [], rng.randrange(len(parents))
    while i >= 0:
        path.append(i)
        i = parents[i]
    return path[::-1]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--context", type=int, default=2000)
    ap.add_argument("--drafted", type=int, default=15)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    if a.seqs < 1 or a.context < 0 or a.drafted < 1 or a.steps < 1:
        ap.error("at least one request, drafted token and step")
    heads, kv_heads, dim = 16, 8, 128
    lib = binding.load()
    dev = torch.device("cuda", 0)
    t = TreeDecoder(lib, heads, kv_heads, dim, a.seqs, a.drafted, a.context + a.steps * a.drafted, cache=a.cache)
    g = torch.Generator(device=dev).manual_seed(1)
    rows = lambda n: torch.randn(n, heads + 2 * kv_heads, dim, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    rng = random.Random(1)
    if a.context:  # the prompts, as random rows: a step of its own
        step = binding.Step(a.seqs, a.seqs * a.context, 0, dev)
        t.new.fill_(a.context)
        lib.kv_assign(t.pages, t.kv_len, t.new, step)
        qkv = rows(a.seqs * a.context)
        lib.kv_append(t.cache, qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], step.slots, step.positions,
                      t.inv_freq, k_norm=t.k_norm)
        t.kv_len.copy_(step.kv_len)
    qkv = rows(a.seqs * a.drafted)

    def plan():
        """Other trees and verdicts for every request."""
        trees = [draft(rng, a.drafted) for _ in range(a.seqs)]
        paths = [verdict(rng, tree) for tree in trees]
        t.new.fill_(a.drafted)
        t.parents.copy_(torch.tensor([p for tree in trees for p in tree], dtype=torch.int32))
        t.paths.copy_(torch.tensor([p + [-1] * (a.drafted - len(p)) for p in paths], dtype=torch.int32))
        return sum(len(p) for p in paths)

    def step_of():
        t.assign()
        out = t.attend(qkv)
        t.accept()
        return out

    accepted = plan()
    step_of()                                     # (once before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step_of()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    total = 0.0
    for _ in range(a.steps - 1):
        accepted += plan()
        begin.record()
        graph.replay()
        end.record()
        end.synchronize()
        total += begin.elapsed_time(end)
    torch.cuda.synchronize()
    assert lib.device_error() == 0 and bool(torch.isfinite(out).all())
    assert int(t.kv_len.sum()) == a.seqs * a.context + accepted
    print(f"{a.seqs} requests, {a.drafted} drafted tokens, {a.context} tokens of context, {a.cache} cache: "
          f"{total * 1e3 / max(1, a.steps - 1):.1f} us a step, {accepted} tokens accepted in {a.steps} steps")


if __name__ == "__main__":
    main()
