"""Attention of drafted trees over a paged cache on the GPU, against the float64 oracle on the same cache contents; the
tolerances are those of the causal calls (tests/test_gpu_attention.py): a mask changes which keys are summed, and nothing else."""

import random

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import step as OS
from tests.gpu_helpers import dev
from tests.test_gpu_attention import Case

pytestmark = pytest.mark.gpu


def tree(rng, n):
    return [rng.randint(max(-1, i - 7), i - 1) for i in range(n)]


class Trees(Case):
    """A batch of sequences whose new tokens are masked: `kind` says how."""

    def __init__(self, lens, heads, kv, dim, page, fp8, seed=0, spread=1.0, wide=0, kind="tree", words=None):
        super().__init__(lens, heads, kv, dim, page, fp8, seed, spread, wide)
        rng = random.Random(seed)
        self.words = words or max(1, -(-self.max_new // 64))
        self.seen = []                                   # [n, n] of each sequence
        for n, _ in lens:
            seen = np.zeros((n, n), bool)
            if kind == "tree":
                parents = tree(rng, n)
                for i in range(n):
                    seen[i, OS.ancestors(parents, i)] = True
            elif kind == "chain":
                seen = np.tril(np.ones((n, n), bool))
            elif kind == "any":
                seen = np.random.default_rng(seed + n).random((n, n)) < 0.4
            elif kind == "none":
                seen[1::2] = np.random.default_rng(seed + n).random((n, n))[1::2] < 0.3
            self.seen.append(seen)

    def masks(self, junk=False):
        rows = [OS.mask_words(np.flatnonzero(r).tolist() + ([x for x in range(len(r), 64 * self.words, 3)] if junk else []), self.words)
                for seen in self.seen for r in seen]
        return torch.tensor(rows, dtype=torch.int64, device=dev()).view(-1, self.words)

    def check(self, out, lse, scale=None, softcap=0.0, window=0, only=None, what=""):
        scale = self.dim ** -0.5 if scale is None else scale
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        weight = 2.0 ** (-11 if self.fp8 else -8)
        for b, (n, length) in enumerate(self.lens):
            if n == 0:
                continue
            at = slice(self.cu[b], self.cu[b + 1])
            want, wlse, spread, size = OS.tree_attention(q[at], self.keys(b, 0), self.keys(b, 1), self.seen[b], scale, softcap, window)
            delta = self.dim * 2.0 ** -22 * size + 2.0 ** -21 * softcap
            bound = 2.0 ** -8 * np.abs(want) + spread * (weight + 2.0 * delta[..., None] + 2.0 ** -20 + length * 2.0 ** -22)
            worst = np.max(np.abs(out[at] - want) / np.maximum(bound, 1e-30))
            assert worst <= 1.0, f"{what} sequence {b}: {worst} of the bound"
            assert np.array_equal(np.isneginf(lse[at]), np.isneginf(wlse)), f"{what} sequence {b}: empty rows"
            seen = np.isfinite(wlse)
            lbound = delta + 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -22 * np.abs(np.where(seen, wlse, 0.0))
            err = np.abs(np.where(seen, lse[at], 0.0) - np.where(seen, wlse, 0.0))
            assert np.all(err <= lbound), f"{what} sequence {b}: lse"


def run(lib, c, masks=None, **kw):
    out, lse = lib.tree_attention(c.q, c.cache(), c.batch(), c.masks() if masks is None else masks, with_lse=True, **kw)
    torch.cuda.synchronize()
    assert lib.device_error() == 0
    return out, lse


# every kernel and tile: 1 to 64 packed rows, more, and more than two row tiles; contexts of nothing, of one key, around
# tile borders; every head size and page size
SHAPES = [([(1, 1), (1, 2), (1, 64), (1, 129), (1, 700)], 8, 2, 128, 16), ([(1, 1), (3, 3), (7, 8), (15, 400), (2, 66)], 2, 1, 64, 32),
          ([(15, 15), (15, 400), (2, 3), (15, 131), (0, 9)], 4, 2, 128, 64), ([(15, 290), (3, 9), (9, 63)], 8, 2, 256, 16),
          ([(31, 77), (0, 50), (1, 1), (20, 20), (31, 333)], 2, 1, 64, 16), ([(64, 290), (3, 9), (40, 168)], 4, 2, 128, 128),
          ([(63, 200), (64, 64), (1, 260), (17, 145)], 8, 2, 128, 32), ([(33, 90), (64, 500), (2, 2)], 7, 1, 64, 256),
          ([(60, 300), (21, 64), (5, 69)], 6, 2, 256, 64), ([(200, 333), (90, 700), (130, 130)], 4, 1, 128, 64),
          ([(256, 400), (1, 33), (77, 900)], 3, 1, 256, 32), ([(130, 640)], 5, 1, 64, 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["tree", "chain", "any", "none"])
@pytest.mark.parametrize("lens,heads,kv,dim,page", SHAPES)
def test_masks(lib, fp8, kind, lens, heads, kv, dim, page):
    c = Trees(lens, heads, kv, dim, page, fp8, seed=dim + page + len(lens), kind=kind)
    c.check(*run(lib, c))


# two CTAs an SM: 65 to 128 rows of 64 and 128 values in any batch, fewer in large ones; pages below, at and above a tile's
# 64 keys
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens,heads,kv,dim,window", [
    ([(40, 300), (3, 70), (25, 25), (1, 129)], 2, 1, 64, 0), ([(21, 200), (32, 64), (0, 7), (9, 700)], 4, 1, 128, 0),
    ([(65, 190), (128, 128), (70, 1000)], 2, 2, 128, 100), ([(33, 2000), (30, 90)], 6, 2, 64, 31), ([(16, 150)] * 9, 8, 2, 128, 0),
    ([(8, 90 + 7 * b) for b in range(25)], 6, 2, 128, 0), ([(17, 40 + 30 * b) for b in range(16)], 2, 1, 128, 0)])
def test_two_ctas_an_sm(lib, fp8, page, lens, heads, kv, dim, window):
    c = Trees(lens, heads, kv, dim, page, fp8, seed=page + dim, kind="any" if page == 32 else "tree")
    first = run(lib, c, window=window)
    c.check(*first, window=window)
    again = run(lib, c, window=window)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_caches_without_prepared_maps(lib):
    """A C caller's cache structure without its TMA descriptors: encoded at the call, for every kernel and page size."""
    for page in (16, 128):
        for lens, heads, kv in (([(3, 50)], 4, 2), ([(40, 300), (25, 100)], 4, 2), ([(100, 300)], 4, 1)):
            c = Trees(lens, heads, kv, 128, page, False, seed=5)
            want = run(lib, c)
            cache = c.cache()
            cache.c.maps = None
            out, lse = lib.tree_attention(c.q, cache, c.batch(), c.masks(), with_lse=True)
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 2, 5, 16, 63, 200, 5000])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("lens,heads,kv,dim,page", [([(1, 1), (9, 64), (15, 65), (12, 500), (15, 15)], 4, 2, 128, 32),
                                                    ([(40, 300), (15, 15), (64, 200)], 4, 2, 64, 16), ([(100, 333), (70, 700)], 2, 1, 256, 64),
                                                    ([(150, 333), (70, 700)], 4, 1, 128, 16)])
def test_windows(lib, fp8, window, kind, lens, heads, kv, dim, page):
    c = Trees(lens, heads, kv, dim, page, fp8, seed=window, kind=kind)
    c.check(*run(lib, c, window=window), window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scale_softcap_and_strided_rows(lib, fp8, dim):
    c = Trees([(1, 200), (9, 77), (40, 90)], 6, 2, dim, 16, fp8, seed=4, spread=3.0, wide=5)
    c.check(*run(lib, c, scale=0.2, softcap=20.0), scale=0.2, softcap=20.0)
    c.check(*run(lib, c, scale=0.2, softcap=20.0, window=30), scale=0.2, softcap=20.0, window=30)
    if not fp8:
        c.check(*run(lib, c, scale=-0.1), scale=-0.1)
    buf = torch.full((c.tokens, 9, dim), 5.0, dtype=torch.bfloat16, device=dev())
    out, lse = run(lib, c, out=buf[:, 2:8])
    c.check(out, lse)
    assert torch.all(buf[:, :2] == 5.0) and torch.all(buf[:, 8:] == 5.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,heads,kv,dim", [
    ([(15, 9001), (1, 3), (15, 5200), (4, 4)], 8, 2, 128), ([(30, 20000)], 2, 1, 64), ([(40, 16000)], 4, 1, 128), ([(20, 12000)], 4, 1, 256),
    ([(100, 9000), (3, 3)], 2, 1, 128), ([(15, 3000)] * 20, 8, 2, 256)])
def test_long_contexts_over_many_ctas(lib, fp8, lens, heads, kv, dim):
    c = Trees(lens, heads, kv, dim, 64, fp8, seed=dim)
    first = run(lib, c)
    keep = [int(x) for x in (0, c.tokens // 2, c.tokens - 1)]
    q = c.q.double().cpu().numpy()
    for t in keep:                                       # the oracle walks these tokens only
        b = int(np.searchsorted(c.cu[1:], t, side="right"))
        n, length = lens[b]
        i = t - int(c.cu[b])
        keys, values = c.keys(b, 0), c.keys(b, 1)
        at = list(range(length - n)) + [length - n + x for x in np.flatnonzero(c.seen[b][i])]
        want, wlse, spread, size = OS.tree_attention(q[t:t + 1], keys[at], values[at], np.ones((1, 1), bool), dim ** -0.5)
        delta = dim * 2.0 ** -22 * size
        bound = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** (-11 if fp8 else -8) + 2.0 * delta[..., None] + 2.0 ** -20 + length * 2.0 ** -22)
        assert np.all(np.abs(first[0][t].double().cpu().numpy() - want[0]) <= bound[0]), t
        err = np.abs(first[1][t].double().cpu().numpy() - wlse[0])
        assert np.all(err <= delta[0] + 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -22 * np.abs(wlse[0]))
    again = run(lib, c)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_keys_before_the_sequence(lib):
    """kv_len below the new tokens: those before the first key are not there, whatever the masks say."""
    for window in (0, 2):
        c = Trees([(6, 4), (5, 0), (70, 66), (3, 2)], 4, 2, 64, 16, False, seed=3, kind="any")
        c.check(*run(lib, c, window=window), window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [15, 64, 70])
def test_bits_past_the_new_tokens_mean_nothing(lib, fp8, n):
    c = Trees([(n, 200), (n - 3, 90), (1, 1)], 4, 2, 128, 16, fp8, seed=n, words=3)
    for window in (0, 40):
        a, b = run(lib, c, window=window), run(lib, c, c.masks(junk=True), window=window)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,heads,kv,dim,page,window", [
    ([(15, 60), (3, 200)], 4, 2, 128, 32, 0), ([(15, 300), (9, 9)], 4, 2, 64, 16, 40), ([(50, 90)], 2, 1, 128, 64, 0), ([(20, 200)], 2, 1, 256, 16, 64),
    ([(60, 170)], 8, 2, 128, 16, 0), ([(100, 300)], 4, 1, 64, 64, 30), ([(130, 200)], 2, 1, 256, 16, 0),
    ([(40, 170)], 2, 1, 64, 16, 0), ([(32, 300)], 4, 1, 128, 128, 25)])
def test_masked_places_leave_no_trace(lib, fp8, value, lens, heads, kv, dim, page, window):
    """Infinities and NaN in K and V of a new token reach the tokens that see it and no others; those in unused slots nobody."""
    c = Trees(lens, heads, kv, dim, page, fp8, seed=12)
    clean = run(lib, c, window=window)
    junk = torch.full((1,), value, device=dev()).to(c.pools.dtype)
    raw = c.pools.view(torch.uint8 if fp8 else torch.int16)
    bits = junk.view(raw.dtype)[0]
    used = np.zeros(raw.shape[1], bool)
    for b, (_, length) in enumerate(c.lens):
        for i in range(-(-length // page)):
            used[c.table[b, i]] = True
            raw[:, c.table[b, i], :, min(page, length - i * page):] = bits
    for p in np.flatnonzero(~used):
        raw[:, p] = bits
    again = run(lib, c, window=window)
    assert torch.equal(clean[0], again[0]) and torch.equal(clean[1], again[1])
    saved = c.pools.clone()
    rng = np.random.default_rng(1)
    for which in (1, 0):                                  # V, then K
        c.pools = saved.clone()
        raw = c.pools.view(torch.uint8 if fp8 else torch.int16)
        n, length = c.lens[0]
        seen = np.zeros(n, bool)
        cols = []
        for t in sorted(rng.choice(n, 3, replace=False)):
            key, col = length - n + int(t), int(rng.integers(0, dim))
            raw[which, int(c.table[0, key // page]), 0, key % page, col] = bits
            cols.append((int(t), col))
        out, lse = run(lib, c, window=window)
        full = np.concatenate([np.ones((n, length - n), bool), c.seen[0]], 1)
        if window:
            full &= full[:, ::-1].cumsum(1)[:, ::-1] <= window
        group = heads // kv
        touched = torch.zeros_like(out, dtype=torch.bool)
        for t, col in cols:
            rows = np.zeros(c.tokens, bool)
            rows[:n] = full[:, length - n + t]
            rows = torch.from_numpy(rows).to(dev())
            if which == 1:
                touched[rows, :group, col] = True
                if not (fp8 and np.isinf(value)):         # (an infinity becomes E4M3's NaN or largest value)
                    assert not torch.isfinite(out[rows][:, :group, col]).any()
            else:
                touched[rows, :group] = True
            seen |= full[:, length - n + t]
        assert torch.equal(out[~touched], clean[0][~touched]), which
        if which == 1:
            assert torch.equal(lse, clean[1])
        else:
            keep = torch.ones_like(lse, dtype=torch.bool)
            keep[torch.from_numpy(np.flatnonzero(seen)).to(dev()), :group] = False
            assert torch.equal(lse[keep], clean[1][keep])
            if np.isnan(value):
                assert torch.isnan(lse[~keep]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [4, 20, 64])
def test_bad_pages_read_as_zeros(lib, fp8, new):
    c = Trees([(new, 400), (1, 50)], 4, 2, 128, 32, fp8, seed=3)
    good = run(lib, c)
    for bad in (-1, c.pools.shape[1], 2 ** 31 - 1):
        d = Trees(c.lens, 4, 2, 128, 32, fp8, seed=3)
        d.table[0, 12] = bad                              # the last keys'
        out, lse = lib.tree_attention(d.q, d.cache(), d.batch(), d.masks(), with_lse=True)
        torch.cuda.synchronize()
        assert lib.device_error() == 4
        assert torch.equal(out[new:], good[0][new:])
        d.table[0, 12] = d.spare
        d.pools[:, d.spare] = torch.zeros(1, device=dev()).to(d.pools.dtype)
        zeros = run(lib, d)
        assert torch.equal(out, zeros[0]) and torch.equal(lse, zeros[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 15, 60])
def test_repeats_on_other_streams_and_in_graphs(lib, fp8, new):
    c = Trees([(new, 3000), (1, 700), (new, new)], 8, 2, 128, 64, fp8, seed=21)
    ref = run(lib, c)
    cache, batch, masks = c.cache(), c.batch(), c.masks()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out, lse = lib.tree_attention(c.q, cache, batch, masks, with_lse=True, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    graphs = []
    for _ in range(2):                                    # two graphs of the same call
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.tree_attention(c.q, cache, batch, masks, out=out, lse=lse)
        graphs.append(g)
    for g in graphs * 2:
        out.zero_()
        g.replay()
        lib.paged_attention(c.q, cache, batch)            # (another call on the eager workspace)
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    # other trees: the graph reads the masks anew
    d = Trees(c.lens, 8, 2, 128, 64, fp8, seed=21, kind="any")
    masks.copy_(d.masks())
    graphs[0].replay()
    torch.cuda.synchronize()
    d.check(out, lse, what="replayed with other masks")


def test_rows_past_the_last_sequence_stay(lib):
    c = Trees([(5, 40), (9, 70)], 4, 2, 64, 16, False, seed=2)
    q = torch.cat([c.q, c.q[:3]])
    masks = torch.cat([c.masks(), torch.full((3, 1), -1, dtype=torch.int64, device=dev())])
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device=dev())
    lse = torch.full(q.shape[:2], 3.0, device=dev())
    lib.tree_attention(q, c.cache(), c.batch(), masks, out=out, lse=lse)
    want = run(lib, c)
    assert torch.equal(out[:14], want[0]) and torch.equal(lse[:14], want[1])
    assert torch.all(out[14:] == 3.0) and torch.all(lse[14:] == 3.0)


def test_a_whole_step(lib):
    """The operators as a tree-drafted decode runs them: assign, append with norms, attend, accept, and again; against
    attention over the accepted sequence from scratch."""
    heads, kv, dim, page, seqs = 4, 2, 64, 16, 3
    g = torch.Generator(device=dev()).manual_seed(5)
    rng = random.Random(2)
    w = [(1.0 + 0.2 * torch.randn(dim, generator=g, device=dev())).to(torch.bfloat16) for _ in range(2)]
    freq = lib.rope_frequencies(dim, device=dev())
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())  # noqa: E731
    pools = torch.randn(2, 30, kv, page, dim, generator=g, device=dev()).to(torch.bfloat16)
    cache = binding.KVCache(pools[0], pools[1])
    free = list(range(30))
    rng.shuffle(free)
    pages = binding.PageTable(torch.full((seqs, 9), -1, dtype=torch.int32, device=dev()), i32([0] * seqs), i32(free), i32([30]), page)
    cap = 75
    step, batch = binding.Step(seqs, cap, 1), None
    batch = step.batch(pages.page_table, 25)
    kv_len = i32([0] * seqs)
    kept = [[] for _ in range(seqs)]                      # (q, k, v, out) of each accepted token
    for turn in range(4):
        counts = [rng.randint(1, 25) for _ in range(seqs)]
        trees = [list(range(-1, n - 1)) if turn == 0 else tree(rng, n) for n in counts]   # first the prompts: chains
        parents = i32([p for t in trees for p in t] + [-1] * (cap - sum(counts)))
        row = torch.randn(cap, heads + 2 * kv, dim, generator=g, device=dev()).to(torch.bfloat16)
        lib.kv_assign(pages, kv_len, i32(counts), step, parents)
        q = lib.kv_append(cache, row[:, heads:heads + kv], row[:, heads + kv:], step.slots, step.positions, freq,
                          q=row[:, :heads], q_norm=w[0], k_norm=w[1])
        out = lib.tree_attention(q, cache, batch, step.masks)
        paths, at = [], 0
        for b, (n, t) in enumerate(zip(counts, trees)):
            path = OS.ancestors(t, rng.randrange(n))
            paths.append(path + [-1] * (26 - len(path)))
            kept[b] += [(row[at + i], out[at + i]) for i in path]
            at += n
        kv_len = lib.kv_accept(cache, batch, i32(paths))
    torch.cuda.synchronize()
    assert lib.device_error() == 0 and kv_len.tolist() == [len(x) for x in kept]
    for x in kept:
        rows, got = torch.stack([a for a, _ in x]), torch.stack([a for _, a in x]).double().cpu().numpy()
        pos = torch.arange(len(x), dtype=torch.int32, device=dev())
        q, k = lib.qk_norm_rope(rows[:, :heads], rows[:, heads:heads + kv], pos, freq, w[0], w[1])
        q, k, v = (a.double().cpu().numpy() for a in (q, k, rows[:, heads + kv:]))
        for i in range(len(x)):
            want, _, spread, size = OS.tree_attention(q[i:i + 1], k[:i + 1], v[:i + 1], np.ones((1, 1), bool), dim ** -0.5)
            delta = dim * 2.0 ** -22 * size
            bound = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2.0 * delta[..., None] + 2.0 ** -20 + 99 * 2.0 ** -22)
            assert np.all(np.abs(got[i] - want[0]) <= bound[0]), i


def test_binding_refuses(lib):
    c = Trees([(2, 30)], 4, 2, 64, 16, False)
    cache, batch, m = c.cache(), c.batch(), c.masks()
    for bad in (m[:1], m.int(), m.cpu(), m[:, 0], torch.zeros(2, 4, dtype=torch.int64, device=dev())[:, ::2]):
        with pytest.raises(ValueError):
            lib.tree_attention(c.q, cache, batch, bad)
    with pytest.raises(ValueError):
        lib.tree_attention(c.q[..., :32], cache, batch, m)
    with pytest.raises(binding.NVFP4Error):
        lib.tree_attention(c.q, cache, batch, m[:, :0].contiguous())
    with pytest.raises(binding.NVFP4Error):
        lib.tree_attention(c.q, cache, binding.Batch(batch.cu_tokens, batch.kv_len, batch.page_table, 65), m)
