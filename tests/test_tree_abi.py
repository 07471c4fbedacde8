"""tree_attention without a GPU: refusals that return before any CUDA call, and the split of its calls, walked through the
kernels' own arithmetic."""

import ctypes
import random

import numpy as np
import pytest

from nvfp4_w4a16_moe_skinny_gb300 import build as B
from tests.test_attention_abi import ALIGN, LAYOUT, NULL, P, SHAPE, WORKSPACE, attention_args, batch, cache
from tests.test_attention_plan import FIELDS


@pytest.fixture(scope="module")
def so():
    B.build()
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    lib = ctypes.CDLL(B.LIB)
    binding._sig(lib)
    return lib


def call(so, c=None, b=None, masks=P, words=1, **kw):
    args = attention_args(c or cache(), b or batch(), **kw)
    return so.tree_attention(args[0], args[1], masks, words, *args[2:])


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), NULL), (dict(batch=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL), (dict(masks=None), NULL),
    (dict(words=0), SHAPE), (dict(words=-1), SHAPE), (dict(words=65), SHAPE), (dict(masks=P + 4), ALIGN),
    (dict(n_tokens=-1), SHAPE), (dict(n_heads=5), SHAPE), (dict(q_stride=248), SHAPE), (dict(out_stride=260), ALIGN),
    (dict(lse=P + 2), ALIGN), (dict(scale=float("nan")), SHAPE), (dict(softcap=-1.0), SHAPE), (dict(window=-1), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=1024), WORKSPACE), (dict(ws=P + 8), ALIGN), (dict(n_tokens=0), 0),
    (dict(n_tokens=0, masks=None), 0)])
def test_refuses(so, kw, status):
    assert call(so, **kw) == status


@pytest.mark.parametrize("kw,words,status", [
    (dict(cu_tokens=None), 1, NULL), (dict(page_table=None), 1, NULL), (dict(max_new=65), 1, SHAPE), (dict(max_new=128), 2, WORKSPACE),
    (dict(max_new=129), 2, SHAPE), (dict(n_seqs=-1), 1, SHAPE), (dict(n_seqs=0), 1, 0), (dict(max_new=0), 1, 0)])
def test_batches_are_refused(so, kw, words, status):
    b = batch(**kw)
    assert call(so, b=b, words=words, ws_bytes=1024 if status == WORKSPACE else 1 << 30) == status


def test_caches_are_refused(so):
    assert call(so, c=cache(head_dim=96)) == SHAPE and call(so, c=cache(dtype=2)) == LAYOUT and call(so, c=cache(k=None)) == NULL


def walk(so, lens, heads, kv, dim, fp8, page, window, orders=3):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CBatch, CKVCache
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
    kv_len = np.array([n for _, n in lens], np.int32)
    most = max(1, max(-(-n // page) for _, n in lens))
    c = CKVCache(P, P, None, None, kv * page * dim, 8, page, kv, dim, 1 if fp8 else 0, None)
    b = CBatch(cu.ctypes.data, kv_len.ctypes.data, None, len(lens), most, max(n for n, _ in lens))
    out = (ctypes.c_int32 * 9)()
    assert so.tree_attention_plan_check(ctypes.byref(c), ctypes.byref(b), int(cu[-1]), heads, window, orders, out, 9) == 0
    return dict(zip(FIELDS, out))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_drawn_batches(so, dim, fp8):
    rng = random.Random(dim + fp8 + 7)
    many = split = 0
    for _ in range(400):
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16])
        new = rng.choice([rng.randint(1, 16), rng.randint(1, 300)])
        context = int(2 ** rng.uniform(0, 16))
        lens = [(rng.randint(0, new), rng.randint(0, context)) for _ in range(rng.choice([1, 2, 5, 40]))]
        lens[0] = (new, new + context)
        r = walk(so, lens, kv * group, kv, dim, fp8, rng.choice([16, 32, 128]), rng.choice([0, 0, rng.randint(1, 4096)]))
        assert r["ok"] == 1, (r, lens, group, kv)
        many, split = many + r["many"], split + r["split"]
    assert many > 50 and split > 500


def test_the_check_refuses(so):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CBatch, CKVCache
    out = (ctypes.c_int32 * 9)()
    cu, kv_len = np.array([0, 1], np.int32), np.array([5], np.int32)
    c = CKVCache(P, P, None, None, 2 * 16 * 64, 8, 16, 2, 64, 0, None)
    b = CBatch(cu.ctypes.data, kv_len.ctypes.data, None, 1, 1, 1)
    run = lambda heads=4, n=9: so.tree_attention_plan_check(ctypes.byref(c), ctypes.byref(b), 1, heads, 0, 2, out, n)  # noqa: E731
    assert run() == 0 and out[0] == 1 and run(heads=5) == SHAPE and run(n=8) == SHAPE
