"""A decode loop's attention block on the framework's calls, captured once and replayed step after step.

    python examples/decode_attention.py [--seqs 8] [--context 4096] [--steps 64] [--cache e4m3]

A batch of sequences with prompts already in a paged cache decodes token by token: the fused q, k, v projection
(`gemm` on an NVFP4 weight), the rotation of q and k and the append to the cache in one launch (`kv_append`), attention
over every sequence's pages (`paged_attention`), and the output projection.  The lengths, positions and slots live in
device tensors that the graph advances by itself, so one captured step serves all steps.  Prompts come as random rows.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_w4a16_moe_skinny_gb300 import binding  # noqa: E402


class AttentionBlock:
    """Projections, rotary table and cache of one layer, for a fixed batch of sequences."""

    def __init__(self, lib, hidden, heads, kv_heads, dim, seqs, max_len, page=64, cache="bf16", seed=0):
        dev = torch.device("cuda", 0)
        g = torch.Generator(device=dev).manual_seed(seed)
        self.lib, self.heads, self.kv_heads, self.dim, self.page = lib, heads, kv_heads, dim, page
        self.w_qkv = lib.prepare(torch.randn((heads + 2 * kv_heads) * dim, hidden, generator=g, device=dev) * 0.02)
        self.w_out = lib.prepare(torch.randn(hidden, heads * dim, generator=g, device=dev) * 0.02)
        self.inv_freq = lib.rope_frequencies(dim, 500000.0, 8.0, 8192.0, device=dev)
        self.amplitude = 1.0
        per = -(-max_len // page)
        self.table = torch.randperm(seqs * per, generator=g, device=dev).to(torch.int32).view(seqs, per)
        dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
        pool = torch.zeros(seqs * per, 2, kv_heads, page, dim, device=dev).to(dtype)     # k and v in one pool
        scale = torch.full((kv_heads,), 0.02, device=dev) if cache == "e4m3" else None
        self.cache = binding.KVCache(pool[:, 0], pool[:, 1], scale, scale)

    def slots_of(self, seq, pos):
        return self.table[seq, pos // self.page].long() * self.page + pos % self.page

    def prefill(self, qkv, seq, start):
        """Appends and attends one sequence's prompt rows qkv [tokens, heads + 2 kv_heads, dim] from position start."""
        h, kv = self.heads, self.kv_heads
        n, dev = qkv.shape[0], qkv.device
        pos = torch.arange(start, start + n, dtype=torch.int32, device=dev)
        slots = self.slots_of(torch.full((n,), seq, device=dev), pos.long())
        q = self.lib.kv_append(self.cache, qkv[:, h:h + kv], qkv[:, h + kv:], slots, pos, self.inv_freq,
                               amplitude=self.amplitude, q=qkv[:, :h])
        one = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        batch = binding.Batch(one(0, n), one(start + n), self.table[seq:seq + 1], n)
        return self.lib.paged_attention(q, self.cache, batch)

    def decode(self, x, positions, batch):
        """One token of every sequence, x [seqs, hidden] at positions; batch.kv_len already counts it."""
        h, kv = self.heads, self.kv_heads
        qkv = self.lib.gemm(self.w_qkv, x).view(x.shape[0], h + 2 * kv, self.dim)
        slots = self.slots_of(torch.arange(x.shape[0], device=x.device), positions.long())
        q = self.lib.kv_append(self.cache, qkv[:, h:h + kv], qkv[:, h + kv:], slots, positions, self.inv_freq,
                               amplitude=self.amplitude, q=qkv[:, :h])
        out = self.lib.paged_attention(q, self.cache, batch)
        y = x + self.lib.gemm(self.w_out, out.view(x.shape[0], -1))
        return torch.nn.functional.rms_norm(y, y.shape[-1:])     # (what stands around the block in a model)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    if not 1 <= a.seqs <= 16 or a.context < 1 or a.steps < 1:
        ap.error("1 to 16 sequences (the projections take up to 16 tokens), a context and steps of at least 1")
    hidden, heads, kv_heads, dim = 2816, 16, 8, 128
    lib = binding.load()
    dev = torch.device("cuda", 0)
    block = AttentionBlock(lib, hidden, heads, kv_heads, dim, a.seqs, a.context + a.steps + 8, cache=a.cache)
    g = torch.Generator(device=dev).manual_seed(1)
    for s in range(a.seqs):
        block.prefill(torch.randn(a.context, heads + 2 * kv_heads, dim, generator=g, device=dev).to(torch.bfloat16), s, 0)

    x = torch.randn(a.seqs, hidden, generator=g, device=dev).to(torch.bfloat16)
    positions = torch.full((a.seqs,), a.context, dtype=torch.int32, device=dev)
    kv_len = positions + 1
    batch = binding.Batch(torch.arange(a.seqs + 1, dtype=torch.int32, device=dev), kv_len, block.table, 1)

    def step():
        x.copy_(block.decode(x, positions, batch))
        positions.add_(1)
        kv_len.add_(1)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    end.synchronize()
    assert lib.device_error() == 0 and bool(torch.isfinite(x).all())
    print(f"{a.seqs} sequences, {a.context} tokens of context, {a.cache} cache: {begin.elapsed_time(end) * 1e3 / a.steps:.1f} us"
          f" a step, ending at position {int(positions[0])}")


if __name__ == "__main__":
    main()
