"""The operators of tree-drafted decoding at the ends of what they take: offsets past 32 bits, the largest trees, calls
without tokens, captured calls beside eager ones."""

import random

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import step as OS
from tests.gpu_helpers import dev
from tests.test_gpu_head_norm import weights
from tests.test_gpu_rope import heads as rows_of
from tests.test_gpu_tree import Trees, run

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def chain_masks(n):
    return torch.tensor([OS.mask_words(range(i + 1), 1) for i in range(n)], dtype=torch.int64, device=dev())


@pytest.mark.parametrize("new,group", [(2, 2), (20, 4), (20, 8)])
def test_pools_past_32_bits(lib, new, group):
    """A pool whose last pages lie more than 2^32 elements in: attention by every kernel, append with norms, accepted
    paths; the same as on a small pool of those pages."""
    kv, page, dim = 8, 64, 128
    pages = (1 << 32) // (kv * page * dim) + 8
    pool = torch.zeros(pages, kv, page, dim, dtype=torch.bfloat16, device=dev())
    g = torch.Generator(device=dev()).manual_seed(1)
    last = torch.randn(4, kv, page, dim, generator=g, device=dev()).to(torch.bfloat16)
    pool[-4:] = last
    q = torch.randn(new, group * kv, dim, generator=g, device=dev()).to(torch.bfloat16)
    big, small = binding.KVCache(pool, pool), binding.KVCache(last, last)
    cu, kl, masks = i32([0, new]), i32([200]), chain_masks(new)
    order = [3, 1, 2, 0]
    far = binding.Batch(cu, kl, i32([[pages - 4 + x for x in order]]), new)
    near = binding.Batch(cu, kl, i32([order]), new)
    a, b = lib.tree_attention(q, big, far, masks), lib.tree_attention(q, small, near, masks)
    assert torch.equal(a, b)
    w = weights(dim, torch.bfloat16, 3)[0]
    k = torch.randn(1, kv, dim, generator=g, device=dev()).to(torch.bfloat16)
    for cache, n in ((big, pages), (small, 4)):           # (k and v are one pool: v's rows go to other slots)
        lib.kv_append(cache, k, k, torch.tensor([n * page - 1], device=dev()), k_norm=w)
    path = i32([[1] + [-1] * 3])
    lengths = lib.kv_accept(big, far, path), lib.kv_accept(small, near, path)
    torch.cuda.synchronize()
    assert lib.device_error() == 0
    assert lengths[0].tolist() == lengths[1].tolist() == [200 - new + 1]
    same = pool[-4:] == last
    same[-1, :, -1] = True                                # (two rows raced for this slot: k's and v's)
    assert same.all() and torch.count_nonzero(pool[:-4]) == 0


def test_rows_past_32_bits(lib):
    """Rows whose strides put the last ones more than 2^32 elements in, both ways."""
    tokens, n, dim, wide = 9, 2, 128, 1 << 29
    buf = torch.zeros(tokens * wide, dtype=torch.bfloat16, device=dev())
    x, dy = rows_of(tokens, n, dim, 1), rows_of(tokens, n, dim, 2)
    far = buf.as_strided((tokens, n, dim), (wide, dim, 1))
    far_dy = buf.as_strided((tokens, n, dim), (wide, dim, 1), n * dim)
    out = buf.as_strided((tokens, n, dim), (wide, dim, 1), 2 * n * dim)
    far.copy_(x), far_dy.copy_(dy)
    w = weights(dim, torch.bfloat16, 4)[0]
    pos = torch.arange(tokens, dtype=torch.int32, device=dev())
    freq = lib.rope_frequencies(dim, device=dev())
    want, _ = lib.qk_norm_rope(x, None, pos, freq, w)
    got, _ = lib.qk_norm_rope(far, None, pos, freq, w, q_out=out)
    assert got is out and torch.equal(out, want)
    back = lib.qk_norm_rope_backward(dy, None, x, None, pos, freq, w)
    there = lib.qk_norm_rope_backward(far_dy, None, far, None, pos, freq, w, dq_out=out)
    assert torch.equal(out, back[0]) and torch.equal(there[2], back[2])
    assert torch.equal(far, x) and torch.equal(far_dy, dy)


@pytest.mark.parametrize("n,back,seed", [(4096, 1, 0), (4096, 40, 1), (4001, 4096, 2)])
def test_the_largest_trees(lib, n, back, seed):
    """64 words: chains, bushes, and stars of up to 4,096 tokens through kv_assign and tree_attention."""
    rng = random.Random(seed)
    parents = [rng.randint(max(-1, i - back), i - 1) for i in range(n)]
    masks, depth = [], []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    ctx, page, heads, kv, dim = 37, 64, 2, 1, 64
    cols = -(-(ctx + n) // page)
    pages = binding.PageTable(i32([[0] + [-1] * (cols - 1)]), i32([1]), i32(list(range(1, cols + 1))), i32([cols]), page)
    step = binding.Step(1, n + 5, 64)
    lib.kv_assign(pages, i32([ctx]), i32([n]), step, i32(parents + [-1] * 5))
    torch.cuda.synchronize()
    assert lib.device_error() == 0
    assert step.positions.tolist() == [ctx + d for d in depth] + [0] * 5
    got = step.masks.cpu().numpy().view(np.uint64)
    want = np.frombuffer(b"".join(m.to_bytes(512, "little") for m in masks), np.uint64).reshape(n, 64)
    assert np.array_equal(got[:n], want) and not got[n:].any()
    g = torch.Generator(device=dev()).manual_seed(seed)
    pools = torch.randn(2, cols + 1, kv, page, dim, generator=g, device=dev()).to(torch.bfloat16)
    q = torch.randn(n + 5, heads, dim, generator=g, device=dev()).to(torch.bfloat16)
    for window in (0, 300):
        out = lib.tree_attention(q, binding.KVCache(pools[0], pools[1]), step.batch(pages.page_table, n), step.masks, window=window)
        torch.cuda.synchronize()
        assert lib.device_error() == 0
        table = pages.page_table[0].tolist()
        keys, values = (pools[x][table].transpose(1, 2).reshape(-1, kv, dim).double().cpu().numpy() for x in (0, 1))
        for i in (0, 63, 64, 1000, n - 1):
            at = [x for x in range(ctx)] + [ctx + x for x in range(i + 1) if masks[i] >> x & 1]
            at = at[-window:] if window else at
            o, _, spread, size = OS.tree_attention(q[i:i + 1].double().cpu().numpy(), keys[at], values[at], np.ones((1, 1), bool), dim ** -0.5)
            delta = dim * 2.0 ** -22 * size
            bound = 2.0 ** -8 * np.abs(o) + spread * (2.0 ** -8 + 2.0 * delta[..., None] + 2.0 ** -20 + (ctx + n) * 2.0 ** -22)
            assert np.all(np.abs(out[i].double().cpu().numpy() - o[0]) <= bound[0]), (window, i)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs", [3, 4, 7, 8, 15, 16])
@pytest.mark.parametrize("new", [8, 9, 16, 17])
def test_either_side_of_every_rule(lib, fp8, dim, seqs, new):
    """16 to 34 packed rows and 12 to 64 pairs of a sequence and a kv head: where one kernel takes over from the other."""
    c = Trees([(new, new + 90 + 13 * b) for b in range(seqs)], 8, 4, dim, 32, fp8, seed=seqs + new)
    c.check(*run(lib, c))


def test_calls_without_tokens_or_sequences(lib):
    kv, dim, page = 2, 64, 16
    pool = torch.zeros(2, 3, kv, page, dim, dtype=torch.bfloat16, device=dev())
    cache = binding.KVCache(pool[0], pool[1])
    x, none = rows_of(4, kv, dim, 1), rows_of(4, kv, dim, 1)[:0]
    w = weights(dim, torch.float32, 1)[0]
    pos, freq = i32([]), lib.rope_frequencies(dim, device=dev())
    q, k = lib.qk_norm_rope(none, none, pos, freq, w, w)
    assert q.shape == k.shape == (0, kv, dim)
    grads = lib.qk_norm_rope_backward(none, none, none, none, pos, freq, w, w)
    assert torch.equal(grads[2], torch.zeros(dim, device=dev())) and torch.equal(grads[3], grads[2])
    assert lib.kv_append(cache, none, none, torch.empty(0, dtype=torch.int64, device=dev()), pos, freq, k_norm=w) is None
    empty = binding.Batch(i32([0]), i32([]), torch.empty(0, 3, dtype=torch.int32, device=dev()), 4)
    idle = binding.Batch(i32([0, 0]), i32([20]), i32([[0, 1, 2]]), 4)
    masks = torch.zeros(4, 1, dtype=torch.int64, device=dev())
    out = torch.full((4, kv, dim), 2.0, dtype=torch.bfloat16, device=dev())
    for b in (empty, idle):
        lib.tree_attention(x, cache, b, masks, out=out)
        assert lib.tree_attention(none, cache, b, masks[:0]).shape == (0, kv, dim)
    assert torch.all(out == 2.0)
    assert lib.kv_accept(cache, empty, i32([]).view(0, 3)).shape == (0,)
    assert lib.kv_accept(cache, idle, i32([]).view(1, 0)).tolist() == [20]
    assert lib.kv_accept(cache, binding.Batch(i32([0, 6]), i32([4]), i32([[0, 1, 2]]), 6), i32([[-1]])).tolist() == [0]
    torch.cuda.synchronize()
    assert lib.device_error() == 0 and torch.count_nonzero(pool) == 0


def test_captured_beside_eager(lib):
    """Gradients, appends and accepted paths captured twice, on another stream too, and replayed between eager calls."""
    tokens, n, kv, dim, page = 700, 6, 2, 128, 16
    q, k, v = (rows_of(tokens, x, dim, 7 + i) for i, x in enumerate((n, kv, kv)))
    dq, dk = rows_of(tokens, n, dim, 5), rows_of(tokens, kv, dim, 6)
    qw, kw = weights(dim, torch.bfloat16, 1)
    pos = torch.arange(tokens, dtype=torch.int32, device=dev())
    freq = lib.rope_frequencies(dim, device=dev())
    pools = torch.zeros(2, -(-tokens // page), kv, page, dim, dtype=torch.bfloat16, device=dev())
    cache = binding.KVCache(pools[0], pools[1])
    slots = torch.arange(tokens, device=dev())
    batch = binding.Batch(i32([0, 64]), i32([tokens]), torch.arange(pools.shape[1], dtype=torch.int32, device=dev())[None], 64)
    path = i32([[3, 5, 9, 40, -1]])

    def step(stream=None):
        grads = lib.qk_norm_rope_backward(dq, dk, q, k, pos, freq, qw, kw, stream=stream)
        turned = lib.kv_append(cache, k, v, slots, pos, freq, q=q, q_norm=qw, k_norm=kw, stream=stream)
        return (*grads, turned, lib.kv_accept(cache, batch, path, stream=stream))
    want = [x.clone() for x in step()]
    cached = pools.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pools.zero_()
    torch.cuda.synchronize()
    got = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(pools, cached)
    graphs = []
    for stream in (None, side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = step()
        graphs.append((graph, outs))
    for graph, outs in graphs * 2:
        pools.zero_()
        for x in outs:
            x.zero_()
        graph.replay()
        lib.qk_norm_rope_backward(dq[:50], dk[:50], q[:50], k[:50], pos[:50], freq, qw, kw)  # (on the eager workspace)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(pools, cached)
    assert lib.device_error() == 0
