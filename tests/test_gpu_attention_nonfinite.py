"""Infinities and NaN in V: right in every tile, beside other items of the same call, and paid for by the tiles that hold
them only."""

import numpy as np
import pytest
import torch

from tests.gpu_helpers import dev
from tests.test_gpu_attention import Case, run

pytestmark = pytest.mark.gpu


def put(c, seq, key, head, col, value):
    """value into V at a sequence's key."""
    raw = c.pools.view(torch.uint8 if c.fp8 else torch.int16)
    bits = torch.full((1,), value, device=dev()).to(c.pools.dtype).view(raw.dtype)[0]
    raw[1, int(c.table[seq, key // c.page]), head, key % c.page, col] = bits


# windowed calls in which most tiles are seen in part, every head size; both kernels
CALLS = [([(64, 4000)] * 48, 4, 2, 256, 1024, False), ([(64, 4000)] * 48, 4, 2, 256, 1024, True),
         ([(64, 4000)] * 48, 4, 2, 128, 1024, True), ([(300, 2000)] * 12, 8, 2, 64, 512, False),
         ([(300, 2000)] * 12, 8, 2, 64, 512, True), ([(15, 4000)] * 48, 4, 2, 128, 1024, True)]


def time_of(call, n=20):
    for _ in range(3):
        call()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)          # the host is ahead of the GPU
        a.record()
        for _ in range(n):
            call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


@pytest.mark.parametrize("lens,heads,kv,dim,window,fp8", CALLS)
def test_one_nan_does_not_slow_the_whole_call(lib, lens, heads, kv, dim, window, fp8):
    """A NaN that a few rows of one sequence see: its tile is read once more, not every tile that comes after it.  (With
    the latter these calls took 5 to 20 times as long; twice leaves room for the one tile.)"""
    c = Case(lens, heads, kv, dim, 64, fp8, seed=1)
    cache, batch = c.cache(), c.batch()
    call = lambda: lib.paged_attention(c.q, cache, batch, window=window)  # noqa: E731
    clean = time_of(call)
    put(c, 0, lens[0][1] - 2, 0, 3, float("nan"))
    one = time_of(call)
    assert one <= 2.0 * clean, f"{clean:.1f} us without, {one:.1f} us with one NaN"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,heads,kv,dim,window", [(1, 8, 2, 128, 0), (15, 4, 2, 64, 100), (20, 4, 2, 128, 0), (60, 2, 2, 256, 300),
                                                     (300, 2, 2, 128, 0), (200, 4, 2, 64, 257), (150, 2, 1, 256, 0)])
def test_each_row_sees_its_own(lib, fp8, new, heads, kv, dim, window):
    """Special values in many sequences and tiles of one call, early and late, beside sequences without any."""
    rng = np.random.default_rng(new + dim)
    lens = [(new if b % 3 else 1 + b, new + 50 + 137 * b) for b in range(12)]
    c = Case(lens, heads, kv, dim, 32, fp8, seed=new)
    clean = run(lib, c, window=window)
    special = [float("nan")] if fp8 else [float("inf"), float("-inf"), float("nan")]
    marks = []
    for b in range(0, 12, 2):
        n, length = lens[b]
        for i in range(6):
            key = length - 1 - int(rng.integers(0, min(length, n + 70)))
            e, col = int(rng.integers(0, kv)), int(rng.integers(0, dim))
            v = special[i % len(special)]
            put(c, b, key, e, col, v)
            marks.append((b, key, e, col, v))
    last = {(b, key, e, col): v for b, key, e, col, v in marks}      # a later mark replaces one in its place
    want = clean[0].float()
    g = heads // kv
    for (b, key, e, col), v in last.items():
        n, length = lens[b]
        pos = torch.arange(length - n, length, device=dev())
        sees = (pos >= key) & ((pos - window < key) if window else True)
        rows = torch.zeros(c.tokens, dtype=torch.bool, device=dev())
        rows[int(c.cu[b]):int(c.cu[b + 1])] = sees
        want[rows, e * g:(e + 1) * g, col] += v
    out, lse = run(lib, c, window=window)
    assert torch.equal(lse, clean[1])
    special_places = ~torch.isfinite(want)
    assert bool(special_places.any())
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[torch.isinf(want)].float(), want[torch.isinf(want)])
    # elsewhere only the marked value itself is missing from the clean result's sum: other columns are untouched
    touched = torch.zeros_like(special_places)
    for b, key, e, col, v in marks:
        touched[int(c.cu[b]):int(c.cu[b + 1]), e * g:(e + 1) * g, col] = True
    assert torch.equal(out[~touched], clean[0][~touched])
