"""The split of attention calls on the CPU (no GPU): paged_attention_plan_check walks the ranges, shares and joins of a
call through the kernels' own arithmetic, for batches of many shapes.

A call's key tiles, numbered item by item, are dealt to the grid in contiguous ranges.  Every tile has to be in exactly
one share, a split item's shares where its join looks for them, and no arrival counter may belong to two items: an item
whose counter another one moves is joined too early or never."""

import ctypes
import random

import numpy as np
import pytest

from nvfp4_w4a16_moe_skinny_gb300 import build as B

P = 1 << 20  # an aligned address that is never read
FIELDS = ("ok", "rows", "ranges", "items", "split", "most", "shared", "unjoined", "many")


@pytest.fixture(scope="module")
def so():
    B.build()
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    lib = ctypes.CDLL(B.LIB)
    binding._sig(lib)
    return lib


def walk(so, lens, heads, kv, dim, fp8=False, page=64, window=0, orders=4, max_new=None, status=0):
    """lens: (new tokens, kv length) of each sequence."""
    from nvfp4_w4a16_moe_skinny_gb300.binding import CBatch, CKVCache
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
    kv_len = np.array([n for _, n in lens], np.int32)
    most = max(1, max(-(-n // page) for _, n in lens))
    cache = CKVCache(P, P, None, None, kv * page * dim, 8, page, kv, dim, 1 if fp8 else 0, None)
    batch = CBatch(cu.ctypes.data, kv_len.ctypes.data, None, len(lens), most,
                   max(n for n, _ in lens) if max_new is None else max_new)
    out = (ctypes.c_int32 * 9)()
    st = so.paged_attention_plan_check(ctypes.byref(cache), ctypes.byref(batch), int(cu[-1]), heads, window, orders, out, 9)
    assert st == status
    return dict(zip(FIELDS, out))


# an item of 9, 17 or 65 shares (or so many and more in the last column) ends in the range in which another split
# item starts
NEIGHBOURS = [
    ([(32, 12832), (32, 32288), (32, 25120)], 32, 8, 128, False, 9),
    ([(64, 32320), (64, 8128)], 16, 8, 256, False, 17),
    ([(256, 30256), (512, 1536)], 8, 1, 256, False, 9),
    ([(27, 11609), (7, 255), (213, 1209), (17, 10377)], 8, 8, 64, False, 9),
    ([(162, 1603), (2, 25152), (294, 389)], 8, 8, 64, False, 17),
    ([(143, 41058), (15, 5781), (172, 1296), (274, 372)], 2, 1, 64, False, 65),
    ([(6, 14566), (136, 11187), (156, 418), (68, 200)], 8, 8, 64, True, 9),
    ([(2, 28949), (157, 369), (12, 158)], 32, 8, 64, True, 17),
    ([(104, 354), (37, 41110), (125, 208)], 2, 2, 64, True, 65),
    ([(8, 27935), (137, 1083), (9, 31671), (212, 348)], 8, 8, 128, False, 9),
    ([(106, 222), (12, 4418), (3, 24702)], 8, 8, 128, False, 17),
    ([(178, 291), (22, 1983), (77, 41165), (46, 303)], 2, 2, 128, False, 65),
    ([(31, 256), (45, 9629), (94, 551), (3, 8704)], 8, 8, 128, True, 9),
    ([(65, 15130), (3, 18137), (83, 18156)], 8, 2, 128, True, 17),
    ([(2, 32926), (52, 315), (94, 503)], 1, 1, 128, True, 65),
    ([(123, 6331), (43, 5422), (130, 3440)], 8, 2, 256, False, 9),
    ([(116, 6173), (77, 2924), (130, 11284)], 4, 2, 256, False, 17),
    ([(1, 33003), (82, 953)], 1, 1, 256, False, 65),
    ([(103, 5682), (45, 462), (132, 5316)], 8, 2, 256, True, 9),
    ([(66, 5405), (133, 10377), (44, 7622)], 4, 2, 256, True, 17),
    ([(5, 33113), (81, 10852)], 1, 1, 256, True, 65),
]


@pytest.mark.parametrize("lens,heads,kv,dim,fp8,shares", NEIGHBOURS)
def test_neighbouring_split_items_have_counters_of_their_own(so, lens, heads, kv, dim, fp8, shares):
    r = walk(so, lens, heads, kv, dim, fp8, orders=50)
    assert r["many"] == 1 and r["most"] >= shares
    assert r["ok"] == 1, r


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_drawn_batches_of_many_rows(so, dim, fp8):
    rng = random.Random(dim + fp8)
    most = split = 0
    for _ in range(600):
        kv = rng.choice([1, 1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 7, 8, 16])
        n_seqs = rng.choice([1, 2, 3, rng.randint(4, 40)])
        new = rng.choice([rng.randint(1, 80), rng.randint(65, 600), rng.randint(65, 2000)])
        context = int(2 ** rng.uniform(0, 16))
        lens = []
        for b in range(n_seqs):
            n = new if rng.random() < 0.5 else rng.randint(0, new)
            lens.append((n, n + (context if rng.random() < 0.5 else rng.randint(0, context))))
        lens[0] = (new, max(new, lens[0][1]))
        window = rng.choice([0, 0, 0, rng.randint(1, 4096)])
        r = walk(so, lens, kv * group, kv, dim, fp8, rng.choice([16, 64, 256]), window, max_new=max(new, 65))
        assert r["ok"] == 1, (r, lens, group, kv, window)
        if r["many"]:                           # (batches of few tokens go to the other kernel)
            most, split = max(most, r["most"]), split + r["split"]
    assert most > 50 and split > 1000


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_items_of_every_number_of_shares(so, dim, fp8):
    """One, two or three items over the grid, from few keys to more than 64 shares each: joins of three levels, groups
    of one at every level, and neighbours of every size."""
    seen = set()
    for n_seqs in (1, 2, 3):
        for context in list(range(0, 12000, 257)) + list(range(12000, 90000, 3001)):
            for uneven in (0, 300, 5000):
                lens = [(70, 70 + context + uneven * b) for b in range(n_seqs)]
                r = walk(so, lens, 1, 1, dim, fp8)
                assert r["many"] == 1 and r["ok"] == 1, (r, lens)
                seen.add(r["most"])
    assert {2, 8, 9, 10, 16, 17, 18} <= seen and max(seen) > 130 and any(60 < n < 70 for n in seen), sorted(seen)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_drawn_batches_of_few_rows(so, dim, fp8):
    rng = random.Random(dim + fp8 + 1)
    for _ in range(300):
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16, 33])
        new = rng.randint(1, max(1, (32 if dim == 256 else 64) // group))
        context = int(2 ** rng.uniform(0, 17))
        lens = [(rng.randint(0, new), rng.randint(0, context)) for _ in range(rng.choice([1, 2, 5, 60, 200]))]
        lens[0] = (new, context)
        window = rng.choice([0, 0, rng.randint(1, 4096)])
        r = walk(so, lens, kv * group, kv, dim, fp8, rng.choice([16, 32, 128]), window)
        assert r["ok"] == 1 and r["many"] == (1 if dim == 256 and group > 32 and len(lens) * kv >= 48 else 0), (r, lens, group, kv, window)


@pytest.mark.parametrize("lens,page", [([(0, 0)], 16), ([(1, 0)], 16), ([(0, 70), (5, 2)], 64), ([(3, 1), (0, 0), (1, 1)], 32),
                                       ([(700, 3)], 64), ([(200, 200), (0, 9), (1, 1)], 256)])
def test_lengths_of_zero_and_one(so, lens, page):
    for window in (0, 1, 64):
        for dim in (64, 128, 256):
            assert walk(so, lens, 4, 2, dim, page=page, window=window)["ok"] == 1


def test_the_check_refuses(so):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CBatch, CKVCache
    out = (ctypes.c_int32 * 9)()
    cu, kv_len = np.array([0, 1], np.int32), np.array([5], np.int32)
    cache = CKVCache(P, P, None, None, 2 * 16 * 64, 8, 16, 2, 64, 0, None)
    batch = CBatch(cu.ctypes.data, kv_len.ctypes.data, None, 1, 1, 1)
    call = lambda c=cache, b=batch, tokens=1, heads=4, window=0, orders=2, o=out, n=9: so.paged_attention_plan_check(  # noqa: E731
        ctypes.byref(c), ctypes.byref(b), tokens, heads, window, orders, o, n)
    assert call() == 0 and out[0] == 1
    assert call(heads=5) == 2 and call(window=-1) == 2 and call(orders=-1) == 2 and call(n=8) == 2 and call(tokens=-1) == 2
    assert call(b=CBatch(None, kv_len.ctypes.data, None, 1, 1, 1)) == 1
    assert call(b=CBatch(cu.ctypes.data, kv_len.ctypes.data, None, 1, 0, 1)) == 2
    assert so.paged_attention_plan_check(ctypes.byref(cache), ctypes.byref(batch), 1, 4, 0, 2, None, 9) == 1
