"""A step's bookkeeping (kv_assign) and accepted paths (kv_accept) on the GPU: whole numbers and copies, equal to the
oracle's."""

import random

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import step as OS
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def tree(rng, n):
    return [rng.randint(max(-1, i - 9), i - 1) for i in range(n)]


class State:
    """A batch of requests in the middle of their lives, on the host and (up) on the GPU."""

    def __init__(self, kv_len, cols, page, extra=0, spare=40, seed=0, held=None):
        rng = random.Random(seed)
        self.kv_len, self.page = list(kv_len), page
        self.held = held or [min(cols, -(-n // page) + rng.randint(0, extra)) for n in kv_len]
        ids = list(range(sum(self.held) + spare))
        rng.shuffle(ids)
        self.table = [[-1] * cols for _ in kv_len]
        for row, h in zip(self.table, self.held):
            row[:h] = [ids.pop() for _ in range(h)]
        self.count = len(ids)
        self.free = ids + [-7] * sum(self.held)

    def up(self):
        return binding.PageTable(i32(self.table).view(len(self.kv_len), -1), i32(self.held), i32(self.free), i32([self.count]),
                                 self.page)

    def check(self, lib, new, rows, parents=None, words=0, pages=None, step=None, kv_len=None, error=False):
        """One step on both sides; the state moves on."""
        want = OS.assign(self.table, self.held, self.free, self.count, self.kv_len, new, rows, self.page, parents, words)
        pages = pages or self.up()
        step = step or binding.Step(len(new), rows, words)
        step.slots.fill_(99), step.positions.fill_(99), step.masks.fill_(99)
        got = lib.kv_assign(pages, i32(self.kv_len) if kv_len is None else kv_len, i32(new), step, None if parents is None else i32(parents))
        assert got is step
        torch.cuda.synchronize()
        assert lib.device_error() == (8 if error else 0) and want[-1] == (not error)
        assert step.slots.tolist() == want[0]
        assert step.positions.tolist() == want[1]
        assert step.cu_tokens.tolist() == want[2] and step.kv_len.tolist() == want[3]
        if parents is not None:
            assert step.masks.tolist() == want[4]
        assert pages.page_table.tolist() == want[5] and pages.held.tolist() == want[6]
        assert pages.free_pages.tolist() == want[7] and pages.free_count.tolist() == [want[8]]
        self.kv_len, self.table, self.held, self.free, self.count = want[3], want[5], want[6], want[7], want[8]
        return pages, step


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("kv_len,new,rows", [
    ([0], [1], 1), ([0], [0], 1), ([15, 16, 17], [1, 1, 1], 3), ([0, 255, 256, 1000], [300, 1, 0, 65], 400),
    ([5, 40, 9], [0, 0, 0], 4), ([100] * 40, [1] * 40, 64), ([16, 31, 0, 77], [-1, 2, -1, 15], 17)])
def test_decode_and_prompts(lib, page, kv_len, new, rows):
    State(kv_len, 1 + (max(kv_len) + max(new)) // 16, page, extra=1, spare=120).check(lib, new, rows)


@pytest.mark.parametrize("seqs,most,rows", [(1, 5000, 5003), (7, 300, 2100), (600, 9, 5400), (1500, 3, 4500), (2100, 20, 42000)])
def test_many_rows_and_requests(lib, seqs, most, rows):
    rng = random.Random(seqs)
    kv_len = [rng.randint(0, 200) for _ in range(seqs)]
    new = [rng.choice([-1, 0, 1, rng.randint(0, most), most]) for _ in range(seqs)]
    State(kv_len, 16 + most // 16, 16, extra=2, spare=seqs * (2 + most // 16)).check(lib, new, rows)


@pytest.mark.parametrize("words,sizes", [(1, [1, 15, 64, 0, 31, -1, 64]), (2, [65, 100, 128, 3]), (4, [256, 1, 200]), (9, [513, 576, 2])])
def test_trees(lib, words, sizes):
    rng = random.Random(words)
    parents = [p for n in sizes for p in tree(rng, n)]
    rows = len(parents) + 5
    s = State([rng.randint(0, 90) for _ in sizes], 60, 16, extra=1, spare=200)
    s.check(lib, sizes, rows, parents + [-1, 5, -9, 1 << 30, 2], words)


@pytest.mark.parametrize("seqs,rows", [(256, 512), (257, 512), (256, 513), (1, 512), (1, 513), (1024, 1100), (1025, 1100), (14336, 15000), (14337, 15000),
                                       (16384, 17000)])
def test_either_side_of_every_limit(lib, seqs, rows):
    """One CTA or eight, requests in one round of the block or more, kept in shared memory or not; rows that run out too."""
    rng = random.Random(seqs + rows)
    kv_len = [rng.randint(0, 40) for _ in range(seqs)]
    new = [rng.choice([-1, 0, 1, 1, 1]) for _ in range(seqs)]
    s = State(kv_len, 5, 16, extra=1, spare=seqs)
    s.check(lib, new, rows)
    new = [rng.choice([0, 1, 2]) for _ in range(seqs)] if seqs > 1 else [rows]
    s.check(lib, new, rows, error=sum(new) > rows or (seqs == 1 and s.kv_len[0] + rows > 80))


def test_chains_stars_and_forests(lib):
    n = 64
    for parents in (list(range(-1, n - 1)), [-1] * n, [-1] + [0] * (n - 1), [i // 2 - 1 if i > 1 else -1 for i in range(n)]):
        State([33], 10, 16, spare=12).check(lib, [n], n, parents, 1)


def test_steps_follow_each_other(lib):
    """Drafts, accepted lengths, finished requests and new ones, on one page table; kv_len in place too."""
    rng = random.Random(3)
    s = State([0] * 12, 20, 16, spare=240)
    pages, step = s.up(), binding.Step(12, 300)
    for turn in range(12):
        new = [rng.choice([0, 1, 15, 24, -1 if turn % 4 == 3 else 2]) for _ in range(12)]
        s.check(lib, new, 300, pages=pages, step=step, kv_len=step.kv_len if turn % 2 else None)
        if turn % 2 == 0:  # a verify step keeps some of the drafted tokens
            s.kv_len = [k - rng.randint(0, max(0, n - 1)) for k, n in zip(s.kv_len, new)]
            step.kv_len.copy_(i32(s.kv_len))


def test_what_cannot_be_served_is_reported(lib):
    assert lib.device_error() == 0
    State([30, 30, 30], 8, 16, spare=3).check(lib, [40, 20, 3], 64, error=True)            # pages run out
    State([30, 30], 3, 16, spare=9).check(lib, [30, 1], 64, error=True)                    # a row of the table does
    State([30, 30, 5], 8, 16, spare=9).check(lib, [7, 9, 4], 12, error=True)               # the step's rows do
    State([3], 8, 16, spare=9).check(lib, [1 << 30], 12, error=True)
    State([3, 3, 3], 8, 16, spare=9).check(lib, [1 << 30, (1 << 31) - 1, 5], 12, error=True)
    s = State([40, 40], 8, 16, spare=0)                                                    # no room for pages given back
    s.free = s.free[:2]
    s.count = 0
    s.check(lib, [-1, 0], 4, error=True)
    # parents that are none count as -1
    s, step = State([20], 8, 16, spare=9), binding.Step(1, 6, 1)
    lib.kv_assign(s.up(), i32([20]), i32([6]), step, i32([0, 0, 5, -2, 1, 1 << 30]))
    assert step.masks[:, 0].tolist() == [1, 3, 4, 8, 19, 32] and step.positions.tolist() == [20, 21, 20, 20, 22, 20]
    assert lib.device_error() == 8
    # a tree of more tokens than the words hold: the others' bits are left out
    s, step = State([20], 16, 16, spare=19), binding.Step(1, 70, 1)
    lib.kv_assign(s.up(), i32([20]), i32([70]), step, i32([-1] + [0] * 69))
    assert step.masks[63, 0].item() == 1 + (1 << 63) - (1 << 64) and step.masks[69, 0].item() == 1
    assert lib.device_error() == 8


def test_no_requests_and_no_rows(lib):
    pages = binding.PageTable(i32([[1, 2]])[:0], i32([1])[:0], i32([4, 5]), i32([2]), 16)
    step = binding.Step(0, 3)
    lib.kv_assign(pages, i32([1])[:0], i32([1])[:0], step)
    assert step.slots.tolist() == [-1] * 3 and step.cu_tokens.tolist() == [0] and pages.free_count.tolist() == [2]
    s = State([20, 3], 8, 16, spare=9)
    s.check(lib, [0, -1], 0)
    assert lib.device_error() == 0


def test_captured_steps(lib):
    """A captured step replayed with other lengths; two graphs on one page table."""
    s = State([20, 3, 50], 12, 16, spare=40)
    pages, step = s.up(), binding.Step(3, 20, 1)
    kv_len, new, parents = i32([0, 0, 0]), i32([0, 0, 0]), i32([-1] * 20)
    graphs = []
    stream = torch.cuda.Stream()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            lib.kv_assign(pages, kv_len, new, step, parents)
        graphs.append(graph)
    rng = random.Random(1)
    for turn in range(6):
        counts = [rng.randint(0, 6) for _ in range(3)]
        up = [p for n in counts for p in tree(rng, n)] + [-1] * (20 - sum(counts))
        kv_len.copy_(i32(s.kv_len)), new.copy_(i32(counts)), parents.copy_(i32(up))
        want = OS.assign(s.table, s.held, s.free, s.count, s.kv_len, counts, 20, 16, up, 1)
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        assert step.slots.tolist() == want[0] and step.positions.tolist() == want[1] and step.masks.tolist() == want[4]
        assert step.cu_tokens.tolist() == want[2] and step.kv_len.tolist() == want[3] and pages.held.tolist() == want[6]
        s.kv_len, s.table, s.held, s.free, s.count = want[3], want[5], want[6], want[7], want[8]
    assert pages.page_table.tolist() == s.table and pages.free_pages.tolist() == s.free


# ------------------------------------------------------------------ accepted paths
class Cached:
    def __init__(self, lens, kv, dim, page, fp8, one_pool=False, seed=0):
        g = torch.Generator(device=dev()).manual_seed(seed)
        counts = [-(-length // page) for _, length in lens]
        pool = sum(counts) + 2
        data = torch.randn(pool, 2, kv, page, dim, generator=g, device=dev())
        data = (data * 40).to(torch.float8_e4m3fn) if fp8 else data.to(torch.bfloat16)
        self.data = data if one_pool else data.view(torch.uint8).transpose(0, 1).contiguous().view(data.dtype)
        self.k, self.v = (data[:, 0], data[:, 1]) if one_pool else (self.data[0], self.data[1])
        order = torch.randperm(pool, generator=g, device=dev()).tolist()
        self.table = [[order.pop() for _ in range(c)] + [-1] * (max(counts) + 1 - c) for c in counts]
        self.lens, self.page, self.kv, self.dim = lens, page, kv, dim
        scale = torch.ones(kv, device=dev()) if fp8 else None
        self.cache = binding.KVCache(self.k, self.v, scale, scale)
        cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
        self.batch = binding.Batch(i32(cu.tolist()), i32([n for _, n in lens]), i32(self.table), max(n for n, _ in lens))

    def bits(self):
        return [x.contiguous().view(torch.uint8 if x.dtype == torch.float8_e4m3fn else torch.int16).cpu().numpy().copy() for x in (self.k, self.v)]

    def moved(self, before, paths):
        want = [x.copy() for x in before]
        lengths = []
        for b, path in enumerate(paths):
            n, length = self.lens[b]
            ctx = length - n
            place = lambda key: (self.table[b][key // self.page], key % self.page)  # noqa: E731
            for old, new in zip(before, want):
                for d, i in enumerate(path):
                    (fp, fo), (tp, to) = place(ctx + i), place(ctx + d)
                    new[tp, :, to] = old[fp, :, fo]
            lengths.append(ctx + len(path))
        return want, lengths


def paths_of(rng, lens):
    """Ascending indices, overlapping their own places too."""
    return [sorted(rng.sample(range(n), rng.randint(0, n))) for n, _ in lens]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,kv,dim,page,one_pool", [
    ([(15, 15)], 1, 64, 16, False), ([(15, 200)], 8, 128, 64, True), ([(1, 1), (7, 30), (64, 64), (33, 500)], 3, 256, 32, False),
    ([(200, 333), (0, 9), (2, 100)], 2, 128, 16, True), ([(21, 70)] * 40, 5, 64, 256, False), ([(700, 900)], 1, 64, 64, False)])
def test_accepted_paths_move(lib, lens, kv, dim, page, one_pool, fp8):
    c = Cached(lens, kv, dim, page, fp8, one_pool, seed=kv + dim)
    rng = random.Random(len(lens) + dim)
    for most_extra in (0, 3):
        paths = paths_of(rng, lens)
        most = max(len(p) for p in paths) + most_extra
        before = c.bits()
        want, lengths = c.moved(before, paths)
        got = lib.kv_accept(c.cache, c.batch, i32([p + [-1] * (most - len(p)) for p in paths]).view(len(lens), most))
        torch.cuda.synchronize()
        assert lib.device_error() == 0 and got.tolist() == lengths
        assert all(np.array_equal(a, b) for a, b in zip(c.bits(), want))


def test_paths_that_are_none_end_and_are_reported(lib):
    lens = [(6, 40)] * 5
    c = Cached(lens, 2, 64, 16, False)
    before = c.bits()
    paths = [[0, 3, 2, 5], [1, 1, 2, 3], [2, 6, -1, -1], [0, -1, 4, 5], [-1, 7, 7, 7]]
    want, lengths = c.moved(before, [[0, 3], [1], [2], [0], []])
    out = torch.zeros(5, dtype=torch.int32, device=dev())
    assert lib.device_error() == 0
    assert lib.kv_accept(c.cache, c.batch, i32(paths), out=out) is out
    torch.cuda.synchronize()
    assert lib.device_error() == 8 and out.tolist() == lengths
    assert all(np.array_equal(a, b) for a, b in zip(c.bits(), want))
    # a page outside the pool: that row stays, the others move
    c = Cached([(6, 22)], 2, 64, 16, False)
    before, page = c.bits(), c.table[0][1]
    c.table[0][1] = 1000
    batch = binding.Batch(i32([0, 6]), i32([22]), i32(c.table), 6)   # keys 16 .. 21: the page that is none
    assert lib.kv_accept(c.cache, batch, i32([[2, 4]])).tolist() == [18]
    torch.cuda.synchronize()
    assert lib.device_error() == 8 and page >= 0
    assert all(np.array_equal(a, b) for a, b in zip(c.bits(), before))


def test_binding_refuses(lib):
    c = Cached([(6, 40)], 2, 64, 16, False)
    pages, step = State([3, 4], 8, 16).up(), binding.Step(2, 8)
    two = i32([1, 2])
    for bad in (lambda: lib.kv_accept(c.cache, c.batch, i32([0, 1])), lambda: lib.kv_accept(c.cache, c.batch, i32([[0], [1]])),
                lambda: lib.kv_accept(c.cache, c.batch, i32([[0]]).long()), lambda: lib.kv_accept(c.cache, c.batch, i32([[0]]).cpu()),
                lambda: lib.kv_accept(c.cache, c.batch, i32([[0, 1, 2]])[:, ::2]), lambda: lib.kv_accept(c.cache, c.batch, i32([[0]]), out=two),
                lambda: lib.kv_assign(pages, two[:1], two, step), lambda: lib.kv_assign(pages, two, two.long(), step),
                lambda: lib.kv_assign(pages, two, two, binding.Step(3, 8)), lambda: lib.kv_assign(pages, two, two, step, i32([0] * 8)),
                lambda: lib.kv_assign(pages, two, two, binding.Step(2, 8, 1), i32([0] * 7)), lambda: lib.kv_assign(pages, two.cpu(), two, step),
                lambda: binding.PageTable(i32([[1]]), two, two, i32([1]), 16), lambda: binding.PageTable(i32([[1]]).long(), two[:1], two, i32([1]), 16),
                lambda: binding.PageTable(i32([[1]]).cpu(), two[:1], two, i32([1]), 16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.NVFP4Error):
        lib.kv_accept(c.cache, c.batch, i32([[0]]), out=c.batch.kv_len)
    with pytest.raises(binding.NVFP4Error):
        lib.kv_assign(binding.PageTable(i32([[1], [2]]), two, two, i32([1]), 48), two, two, step)
