"""Attention over a paged cache on the GPU, against the float64 oracle on the same cache contents.

Tolerance of an output value, with A = sum_j p_j |v_j|: its own rounding, 2^-8 of it; the weights' rounding, 2^-8 (bf16
caches) or 2^-11 (E4M3) of A; and what fp32 loses before: the logits are off by at most dim * 2^-22 of scale * sum
|q| |k| (fp32 sums of exact products, truncated by the tensor cores) and, with a softcap, 2^-21 of it, which changes
weights, sum and output by twice that factor of A; sums over n keys n * 2^-22 of A.  The log-sum-exp is off by the
logits' error and the sum's, and its own rounding."""

import math

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import attention as OA
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


class Case:
    """A batch of sequences in a shuffled pool; lens: (new tokens, kv length)."""

    def __init__(self, lens, heads, kv, dim, page, fp8, seed=0, spread=1.0, wide=0):
        g = torch.Generator(device=dev()).manual_seed(seed)
        self.lens, self.heads, self.kv, self.dim, self.page, self.fp8 = lens, heads, kv, dim, page, fp8
        counts = [-(-length // page) for _, length in lens]
        most, pool = max(1, max(counts)) + 1, sum(counts) + 2
        self.max_new = max(n for n, _ in lens)
        data = torch.randn(2, pool, kv, page, dim, generator=g, device=dev())
        self.scales = [None, None]
        if fp8:
            self.scales = [torch.rand(kv, generator=g, device=dev()) * 0.02 + 0.01 for _ in range(2)]
            self.pools = (data * 50.0).to(torch.float8_e4m3fn)
        else:
            self.pools = data.to(torch.bfloat16)
        order = torch.randperm(pool, generator=g, device=dev()).cpu().numpy()
        self.table = np.full((len(lens), most), -1, np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.spare = int(order[-1])
        tokens = sum(n for n, _ in lens)
        self.tokens = tokens
        self.q = (torch.randn(tokens, heads + wide, dim, generator=g, device=dev()) * spread).to(torch.bfloat16)[:, :heads]
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)

    def cache(self):
        return binding.KVCache(self.pools[0], self.pools[1], *self.scales)

    def batch(self):
        up = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())  # noqa: E731
        return binding.Batch(up(self.cu), up([n for _, n in self.lens]), up(self.table), self.max_new)

    def keys(self, b, which):
        length = self.lens[b][1]
        pages = self.table[b, :-(-length // self.page)]
        x = self.pools[which].float().cpu().numpy().astype(np.float64)[pages]      # [pages, kv, page, dim]
        if self.fp8:
            x = x * self.scales[which].cpu().numpy().astype(np.float64)[:, None, None]
        return x.transpose(0, 2, 1, 3).reshape(-1, self.kv, self.dim)[:length]

    def check(self, out, lse, scale=None, softcap=0.0, window=0, only=None, what=""):
        scale = 1.0 / math.sqrt(self.dim) if scale is None else scale
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        weight = 2.0 ** (-11 if self.fp8 else -8)
        for b, (n, length) in enumerate(self.lens):
            if n == 0 or (only is not None and b not in only):
                continue
            at = slice(self.cu[b], self.cu[b + 1])
            want, wlse, spread, size = OA.attention(q[at], self.keys(b, 0), self.keys(b, 1), length - n, scale, softcap,
                                                    window)
            delta = self.dim * 2.0 ** -22 * size + 2.0 ** -21 * softcap
            bound = 2.0 ** -8 * np.abs(want) + spread * (weight + 2.0 * delta[..., None] + 2.0 ** -20 + length * 2.0 ** -22)
            err = np.abs(out[at] - want)
            fine = np.isfinite(want)
            assert np.array_equal(np.isnan(out[at]), np.isnan(want)), f"{what} sequence {b}: NaN in other places"
            assert np.array_equal(out[at][~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what} {b}: infinities"
            assert np.all(err[fine] <= bound[fine]), f"{what} sequence {b}: {np.nanmax(err / np.maximum(bound, 1e-30))} of the bound"
            empty = np.isneginf(wlse)
            assert np.array_equal(np.isneginf(lse[at]), empty), f"{what} sequence {b}: empty rows"
            seen = np.isfinite(wlse)
            lbound = delta + 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -22 * np.abs(np.where(seen, wlse, 0.0))
            assert np.all(np.abs(lse[at] - wlse)[seen] <= lbound[seen]), f"{what} sequence {b}: lse"


def run(lib, c, **kw):
    out, lse = lib.paged_attention(c.q, c.cache(), c.batch(), with_lse=True, **kw)
    torch.cuda.synchronize()
    assert lib.device_error() == 0
    return out, lse


# decode steps: one token a sequence, every head size, group and page size, lengths around the tile borders
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv,dim,page", [(1, 1, 64, 16), (8, 8, 64, 32), (16, 8, 128, 16), (14, 2, 128, 64),
                                               (16, 1, 128, 128), (5, 5, 256, 32), (32, 4, 256, 256), (34, 2, 64, 64)])
def test_decode(lib, fp8, heads, kv, dim, page):
    lens = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 63), (1, 128), (1, 129), (1, 255), (1, 700), (1, 33)]
    c = Case(lens, heads, kv, dim, page, fp8, seed=heads * dim + page)
    c.check(*run(lib, c))


# verify blocks and chunks, lengths of zero and one, empty sequences, rows before the first key
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,heads,kv,dim,page", [
    ([(15, 15), (15, 400), (2, 3), (15, 131)], 4, 2, 128, 32),
    ([(15, 77), (0, 50), (1, 1), (7, 7), (0, 0), (15, 333)], 6, 2, 64, 16),
    ([(5, 0), (4, 2), (1, 0), (3, 300)], 4, 4, 128, 16),
    ([(15, 290), (3, 9)], 16, 2, 256, 64),
    ([(70, 70), (33, 190), (1, 260), (64, 64)], 3, 1, 128, 64),
    ([(130, 130), (129, 401)], 7, 1, 64, 16),
    ([(97, 240)], 10, 2, 256, 128)])
def test_chunks(lib, fp8, lens, heads, kv, dim, page):
    c = Case(lens, heads, kv, dim, page, fp8, seed=dim + page)
    c.check(*run(lib, c))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 16, 31, 64, 200, 5000])
@pytest.mark.parametrize("lens,heads,kv,dim,page", [([(1, 1), (1, 64), (1, 65), (1, 500)], 8, 4, 128, 32),
                                                    ([(15, 15), (15, 300), (40, 200)], 4, 2, 64, 16),
                                                    ([(100, 333), (1, 700)], 2, 1, 256, 64)])
def test_windows(lib, fp8, window, lens, heads, kv, dim, page):
    c = Case(lens, heads, kv, dim, page, fp8, seed=window)
    c.check(*run(lib, c, window=window), window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scale_softcap_and_strided_rows(lib, fp8, dim):
    c = Case([(1, 200), (9, 77), (40, 90)], 6, 2, dim, 16, fp8, seed=4, spread=3.0, wide=5)
    c.check(*run(lib, c, scale=0.2, softcap=20.0), scale=0.2, softcap=20.0)
    c.check(*run(lib, c, scale=-0.1), scale=-0.1) if not fp8 else None
    buf = torch.full((c.tokens, 9, dim), 5.0, dtype=torch.bfloat16, device=dev())
    out, lse = run(lib, c, out=buf[:, 2:8])
    c.check(out, lse)
    assert torch.all(buf[:, :2] == 5.0) and torch.all(buf[:, 8:] == 5.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_and_ragged_split(lib, fp8):
    """Long sequences split over many CTAs beside short ones: pieces joined in order."""
    c = Case([(1, 9001), (1, 3), (1, 5200), (1, 1), (1, 40)], 8, 2, 128, 64, fp8, seed=6)
    c.check(*run(lib, c))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,heads,kv,dim,context", [
    (1, 16, 1, 128, 60000), (1, 3, 1, 64, 90000), (2, 16, 1, 256, 21000),       # few rows: over all CTAs of the split kernel
    (100, 2, 1, 128, 41000), (200, 1, 1, 64, 45000), (70, 2, 1, 256, 22000),    # a chunk: joined in groups, three levels
    (130, 2, 2, 128, 9000), (300, 4, 2, 64, 5000)])
def test_one_item_over_many_ctas(lib, fp8, new, heads, kv, dim, context):
    c = Case([(new, new + context)], heads, kv, dim, 64, fp8, seed=new + dim)
    out, lse = run(lib, c)
    keep = sorted({0, 1, new // 2, new - 1} & set(range(new)))     # the oracle walks these tokens only
    q = c.q[keep].double().cpu().numpy()
    k, v = c.keys(0, 0), c.keys(0, 1)
    for i, tok in enumerate(keep):
        want, wlse, spread, size = OA.attention(q[i:i + 1], k, v, context + tok, dim ** -0.5)
        n = context + new
        delta = dim * 2.0 ** -22 * size
        bound = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** (-11 if fp8 else -8) + 2.0 * delta[..., None] + 2.0 ** -20 + n * 2.0 ** -22)
        assert np.all(np.abs(out[tok:tok + 1].double().cpu().numpy() - want) <= bound), tok
        err = np.abs(lse[tok].double().cpu().numpy() - wlse[0])
        assert np.all(err <= delta[0] + 2.0 ** -20 + n * 2.0 ** -22 + 2.0 ** -22 * np.abs(wlse[0]))
    again = run(lib, c)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,heads,kv,dim,context", [
    (4, 16, 1, 128, 30000), (8, 4, 1, 64, 41000), (3, 12, 1, 256, 12000), (1, 33, 1, 128, 9000), (17, 2, 1, 64, 20000)])
def test_tiles_of_32_and_64_rows_over_many_ctas(lib, fp8, new, heads, kv, dim, context):
    """Every row of one item whose shares lie in every CTA."""
    c = Case([(new, new + context)], heads, kv, dim, 32, fp8, seed=new * dim)
    c.check(*run(lib, c))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_seqs,new,heads,kv,dim", [(24, 17, 4, 2, 128), (47, 33, 1, 1, 64), (48, 33, 1, 1, 64), (12, 5, 32, 4, 256),
                                                     (11, 5, 32, 4, 256), (64, 32, 2, 1, 128), (130, 60, 1, 1, 128), (47, 33, 1, 1, 256), (48, 33, 1, 1, 256)])
def test_33_to_64_rows_in_small_and_large_batches(lib, fp8, n_seqs, new, heads, kv, dim):
    """Rows that one kernel serves in few (sequence, kv head) pairs and the other in many: both sides of the rule."""
    lens = [(new if b % 5 else 1 + b % new, new + (b * 37) % 400) for b in range(n_seqs)]
    c = Case(lens, heads, kv, dim, 64, fp8, seed=n_seqs + new)
    c.check(*run(lib, c))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("growth", [3.0, 40.0, -40.0, 600.0])
@pytest.mark.parametrize("lens,heads,kv,dim", [([(1, 700)], 4, 2, 128), ([(20, 700)], 2, 1, 64), ([(150, 900)], 2, 1, 128),
                                               ([(90, 700)], 4, 2, 64), ([(140, 600)], 1, 1, 256)])
def test_maxima_that_grow_and_fall(lib, fp8, growth, lens, heads, kv, dim):
    """Keys whose logits climb (or fall) over the sequence by hundreds: the running references move, far and often."""
    c = Case(lens, heads, kv, dim, 32, fp8, seed=77)
    length = lens[0][1]
    c.q = c.q * 0.1
    c.q[..., 0] = 8.0
    ramp = torch.linspace(0, 1, length, device=dev()) if growth > 0 else torch.linspace(1, 0, length, device=dev())
    ramp = ramp * abs(growth) * math.sqrt(dim) / 8.0               # logits 0 .. |growth| in the first value's direction
    raw = c.pools.float()
    for i in range(-(-length // 32)):
        part = ramp[i * 32:(i + 1) * 32]
        for h in range(kv):
            s = 1.0 if not fp8 else float(c.scales[0][h])
            raw[0, int(c.table[0, i]), h, :part.numel(), 0] = (part / s).clamp(max=440.0 if fp8 else 1e9)
    c.pools = raw.to(c.pools.dtype)
    out, lse = run(lib, c)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    c.check(out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 1, 100, 257])
@pytest.mark.parametrize("lens,heads,kv,dim,page", [([(300, 300), (1, 90), (257, 800)], 2, 1, 128, 16),
                                                    ([(129, 640), (5, 5)], 7, 1, 128, 128), ([(400, 1000)], 1, 1, 64, 256),
                                                    ([(130, 500), (3, 77)], 3, 1, 256, 16)])
def test_large_chunks(lib, fp8, window, lens, heads, kv, dim, page):
    c = Case(lens, heads, kv, dim, page, fp8, seed=window + dim)
    c.check(*run(lib, c, window=window), window=window)


@pytest.mark.parametrize("n_seqs", [151, 300, 700])
def test_many_sequences(lib, n_seqs):
    rng = np.random.default_rng(n_seqs)
    lens = [(int(rng.integers(0, 3)), int(rng.integers(0, 60))) for _ in range(n_seqs)]
    c = Case(lens, 2, 1, 64, 16, False, seed=n_seqs)
    c.check(*run(lib, c))


# what masked places hold leaves no trace
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,heads,kv,dim,page", [([(1, 37), (1, 130)], 4, 2, 128, 32), ([(15, 60), (20, 20)], 4, 2, 64, 16),
                                                    ([(70, 150)], 2, 1, 128, 64), ([(33, 80)], 2, 2, 256, 16),
                                                    ([(300, 500)], 4, 1, 128, 64), ([(300, 500)], 3, 1, 64, 32)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_unseen_slots_leave_no_trace(lib, fp8, lens, heads, kv, dim, page, value):
    c = Case(lens, heads, kv, dim, page, fp8, seed=12)
    before = run(lib, c)
    junk = torch.full((1,), value, device=dev()).to(c.pools.dtype)
    raw = c.pools.view(torch.uint8 if fp8 else torch.int16)
    bits = junk.view(raw.dtype)[0]
    used = np.zeros(raw.shape[1], bool)
    for b, (_, length) in enumerate(c.lens):
        for i in range(-(-length // page)):
            used[c.table[b, i]] = True
            keep = min(page, length - i * page)
            raw[:, c.table[b, i], :, keep:] = bits        # the tail of the last page
    for p in np.flatnonzero(~used):
        raw[:, p] = bits
    after = run(lib, c)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,heads,kv,dim,page,window", [
    ([(15, 60)], 4, 2, 128, 32, 0), ([(15, 300)], 4, 2, 64, 16, 40), ([(50, 90)], 2, 1, 128, 64, 0),
    ([(20, 200)], 2, 1, 256, 16, 64), ([(300, 700)], 4, 1, 128, 64, 0), ([(300, 700)], 4, 1, 64, 64, 150),
    ([(260, 300)], 2, 1, 128, 16, 0)])
def test_infinite_and_nan_keys_reach_only_the_rows_that_see_them(lib, fp8, lens, heads, kv, dim, page, window):
    """A NaN key, and values of +inf, -inf and NaN (for E4M3: NaN), late in the chunk and, with a window, early."""
    c = Case(lens, heads, kv, dim, page, fp8, seed=13)
    n, length = c.lens[0]
    raw = c.pools.float()
    special = [float("nan")] if fp8 else [float("inf"), -float("inf"), float("nan")]
    for i, v in enumerate(special):
        for j in (length - 2 - 3 * i, length - n + 1 + i, max(0, length - n - 20 - i) if window else length - 1):
            raw[1, int(c.table[0, j // page]), 0, j % page, 3 * i + (j % 5)] = v
    raw[0, int(c.table[0, (length - 4) // page]), 0, (length - 4) % page, 5] = float("nan")
    c.pools = raw.to(c.pools.dtype)
    out, lse = run(lib, c, window=window)
    q = c.q.double().cpu().numpy()
    want, wlse, spread, _ = OA.attention(q, c.keys(0, 0), c.keys(0, 1), length - n, dim ** -0.5, 0.0, window)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    # rows that see the NaN key are NaN; elsewhere each special value marks its own column
    assert np.array_equal(np.isnan(lse), np.isnan(wlse))
    assert np.array_equal(np.isfinite(out), np.isfinite(want))
    assert np.array_equal(out[np.isinf(want)], want[np.isinf(want)])
    fine = np.isfinite(want)
    finite_spread = np.where(np.isfinite(spread), spread, 0.0)
    assert np.all(np.abs(out - want)[fine] <= (2.0 ** -8 * np.abs(want) + 2.0 ** -7 * finite_spread + 1e-3)[fine])


def test_infinite_logits(lib):
    """Keys whose logit is -inf get weight 0; a row of nothing else gets zeros."""
    c = Case([(1, 40), (1, 3)], 1, 1, 64, 16, False, seed=2)
    c.q.abs_()
    for b, rows in ((0, range(0, 40, 3)), (1, range(3))):
        for j in rows:
            c.pools[0, int(c.table[b, j // 16]), 0, j % 16, 7] = -float("inf")
    out, lse = run(lib, c)
    want, wlse, _, _ = OA.attention(c.q[:1].double().cpu().numpy(), c.keys(0, 0), c.keys(0, 1), 39, 0.125)
    assert np.allclose(out[0].double().cpu().numpy(), want[0], atol=0.02) and abs(float(lse[0, 0]) - wlse[0, 0]) < 1e-4
    assert torch.all(out[1] == 0) and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 20, 300])
def test_bad_pages_read_as_zeros(lib, fp8, new):
    c = Case([(new, 400), (1, 50)], 4, 2, 128, 32, fp8, seed=3)
    good = run(lib, c)
    for bad in (-1, c.pools.shape[1], 2 ** 31 - 1, -2 ** 31):
        table = c.table.copy()
        table[0, 1] = bad
        d = Case(c.lens, 4, 2, 128, 32, fp8, seed=3)
        d.table = table
        out, lse = lib.paged_attention(d.q, d.cache(), d.batch(), with_lse=True)
        torch.cuda.synchronize()
        assert lib.device_error() == 4
        assert torch.equal(out[new:], good[0][new:])           # the other sequence
        d.table = c.table.copy()
        d.table[0, 1] = d.spare                                # a page of zeros in its place
        d.pools[:, d.spare] = torch.zeros(1, device=dev()).to(d.pools.dtype)
        zeros = run(lib, d)
        assert torch.equal(out, zeros[0]) and torch.equal(lse, zeros[1])


def test_a_window_past_every_sequence_is_no_window(lib):
    c = Case([(3, 200), (70, 100), (2, 0)], 4, 2, 128, 32, False, seed=18)
    ref = run(lib, c)
    for window in (200, 1 << 29, (1 << 30) + 5, 2 ** 31 - 1):
        out, lse = run(lib, c, window=window)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_tensors_given_away_while_another_stream_uses_them(lib):
    """A call on a stream of its own, whose inputs are dropped and whose memory is asked for again at once: the call
    still reads what it was given."""
    c = Case([(1, 4000), (40, 900)], 8, 2, 128, 64, False, seed=31)
    ref, _ = run(lib, c)
    cache, batch = c.cache(), c.batch()
    s = torch.cuda.Stream()
    big = torch.empty(1 << 28, dtype=torch.uint8, device=dev())
    for _ in range(10):
        q = c.q.clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            big.fill_(1)                       # keeps the call waiting
        out = lib.paged_attention(q, cache, batch, stream=s)
        del q
        junk = [torch.full_like(c.q, float("nan")) for _ in range(4)]
        s.synchronize()
        assert torch.equal(out, ref)
        del junk


def test_window_skips_freed_pages(lib):
    """Table entries wholly before the window may hold anything."""
    c = Case([(3, 500)], 4, 2, 128, 16, False, seed=8)
    good = run(lib, c, window=100)
    c.table[0, :(500 - 3 - 100 + 1) // 16] = -7
    again = run(lib, c, window=100)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


def test_inconsistent_lengths_stay_in_bounds(lib):
    """kv_len past the table is read as the table's size; cu_tokens past n_tokens as n_tokens."""
    c = Case([(2, 64), (3, 40)], 4, 2, 64, 16, False, seed=9)
    c.table = np.ascontiguousarray(c.table[:, :4])
    good = run(lib, c)
    b = c.batch()
    b.kv_len[0] = 1 << 20
    b.cu_tokens[2] = 900
    out, lse = lib.paged_attention(c.q, c.cache(), b, with_lse=True)
    torch.cuda.synchronize()
    assert lib.device_error() == 0
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 15, 200])
def test_repeats_bit_exact_on_other_streams_and_in_graphs(lib, fp8, new):
    c = Case([(new, 3000), (1, 700), (new, new)], 8, 2, 128, 64, fp8, seed=21)
    ref = run(lib, c)
    cache, batch = c.cache(), c.batch()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        out, lse = lib.paged_attention(c.q, cache, batch, with_lse=True, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.paged_attention(c.q, cache, batch, out=out, lse=lse)
    # other lengths and another workspace use in between; the graph reads the lengths anew
    batch.kv_len -= 1
    g.replay()
    lib.paged_attention(c.q, cache, batch)
    torch.cuda.synchronize()
    d = Case(c.lens, 8, 2, 128, 64, fp8, seed=21)
    d.lens = [(a, b - 1) for a, b in c.lens]
    d.check(out, lse, what="replayed at other lengths")
    batch.kv_len += 1
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_offsets_past_32_bits(lib):
    """A pool whose last pages lie more than 2^32 elements in."""
    kv, page, dim = 8, 64, 128
    per = kv * page * dim
    pages = (1 << 32) // per + 8
    pool = torch.zeros(pages, kv, page, dim, dtype=torch.bfloat16, device=dev())
    g = torch.Generator(device=dev()).manual_seed(1)
    last = torch.randn(4, kv, page, dim, generator=g, device=dev()).to(torch.bfloat16)
    pool[-4:] = last
    q = torch.randn(2, 16, dim, generator=g, device=dev()).to(torch.bfloat16)
    up = lambda a: torch.tensor(a, dtype=torch.int32, device=dev())  # noqa: E731
    cu, kl = up([0, 2]), up([200])
    a = lib.paged_attention(q, binding.KVCache(pool, pool), binding.Batch(cu, kl, up([[pages - 1, pages - 3, pages - 2, pages - 4]]), 2))
    b = lib.paged_attention(q, binding.KVCache(last, last), binding.Batch(cu, kl, up([[3, 1, 2, 0]]), 2))
    assert torch.equal(a, b)
    k = torch.randn(1, kv, dim, generator=g, device=dev()).to(torch.bfloat16)
    lib.kv_append(binding.KVCache(pool, pool), k, k, torch.tensor([pages * page - 1], device=dev()))
    assert torch.equal(pool[-1, :, -1], k[0]) and torch.count_nonzero(pool[:-4]) == 0
    torch.cuda.synchronize()
    assert lib.device_error() == 0


def test_append_then_attend(lib):
    """The two operators as a decode loop uses them: a prompt, then single tokens, against attention over the whole
    sequence from scratch."""
    heads, kv, dim, page, total, prompt = 8, 2, 128, 32, 90, 70
    g = torch.Generator(device=dev()).manual_seed(5)
    row = torch.randn(total, heads + 2 * kv, dim, generator=g, device=dev()).to(torch.bfloat16)
    q, k, v = row[:, :heads], row[:, heads:heads + kv], row[:, heads + kv:]
    w = lib.rope_frequencies(dim, device=dev())
    pos = torch.arange(total, dtype=torch.int32, device=dev())
    pools = torch.zeros(2, 5, kv, page, dim, dtype=torch.bfloat16, device=dev())
    cache = binding.KVCache(pools[0], pools[1])
    table = torch.tensor([[3, 0, 4]], dtype=torch.int32, device=dev())
    slots = (table[0].long()[pos.long() // page]) * page + pos.long() % page
    outs = []
    at = 0
    for n in [prompt] + [1] * (total - prompt):
        s = slice(at, at + n)
        qr = lib.kv_append(cache, k[s], v[s], slots[s], pos[s], w, q=q[s])
        b = binding.Batch(torch.tensor([0, n], dtype=torch.int32, device=dev()),
                          torch.tensor([at + n], dtype=torch.int32, device=dev()), table, n)
        outs.append(lib.paged_attention(qr, cache, b))
        at += n
    got = torch.cat(outs).double().cpu().numpy()
    rot = lambda x: lib.rope_apply(x, pos, w).double().cpu().numpy()  # noqa: E731
    want, _, spread, size = OA.attention(rot(q), rot(k), v.double().cpu().numpy(), 0, dim ** -0.5)
    delta = dim * 2.0 ** -22 * size
    bound = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2.0 * delta[..., None] + 2.0 ** -20 + total * 2.0 ** -22)
    assert np.all(np.abs(got - want) <= bound)
    assert lib.device_error() == 0


def test_binding_refuses(lib):
    c = Case([(2, 30)], 4, 2, 64, 16, False)
    cache, batch = c.cache(), c.batch()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev())  # noqa: E731
    for bad in (lambda: lib.paged_attention(c.q.float(), cache, batch), lambda: lib.paged_attention(c.q[..., :32], cache, batch),
                lambda: lib.paged_attention(c.q, cache, batch, out=torch.empty(1, 4, 64, dtype=torch.bfloat16, device=dev())),
                lambda: lib.paged_attention(c.q, cache, batch, lse=torch.empty(2, 4, device=dev()).half()),
                lambda: binding.Batch(i32(3), i32(3), i32(3, 2), 1), lambda: binding.Batch(i32(4).long(), i32(3), i32(3, 2), 1),
                lambda: binding.Batch(i32(4), i32(3), i32(2, 3).t(), 1), lambda: binding.Batch(i32(4).cpu(), i32(3), i32(3, 2), 1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.NVFP4Error):
        lib.paged_attention(c.q[:, :3].contiguous(), cache, batch)      # heads not a multiple of the kv heads


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [0.5, 20.0, 100000.0])
@pytest.mark.parametrize("lens,heads,kv,dim", [([(1, 300), (2, 40)], 4, 2, 128), ([(20, 90)], 2, 1, 64), ([(90, 200)], 2, 1, 128),
                                               ([(70, 150)], 2, 1, 256)])
def test_a_softcap_keeps_fp32_digits(lib, fp8, cap, lens, heads, kv, dim):
    """The log-sum-exp under a softcap far above the logits, around them and below: tanh is good to 2^-22 of its value
    (2^-24 of a polynomial below a half, and above it 2^-22 of 1 - 2 / (e^2x + 1) >= 0.46, hence 2^-21), the product of
    a logit 2^-23, and the rest as without one."""
    c = Case(lens, heads, kv, dim, 32, fp8, seed=11)
    _, lse = run(lib, c, softcap=cap)
    lse = lse.double().cpu().numpy()
    q = c.q.double().cpu().numpy()
    for b, (n, length) in enumerate(lens):
        at = slice(c.cu[b], c.cu[b + 1])
        _, want, _, size = OA.attention(q[at], c.keys(b, 0), c.keys(b, 1), length - n, dim ** -0.5, cap)
        capped = np.minimum(cap, size)                               # a bound on the capped logits
        bound = dim * 2.0 ** -22 * size + capped * 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22 * np.abs(want)
        assert np.all(np.abs(lse[at] - want) <= bound), f"{np.max(np.abs(lse[at] - want) / bound)} of the bound"
