"""Argument checks of the attention side (no GPU): every rejected call returns before any CUDA call."""

import ctypes

import numpy as np
import pytest

from nvfp4_w4a16_moe_skinny_gb300 import build as B
from oracle import attention as OA

P = 1 << 20  # an aligned address that is never read
NULL, SHAPE, ALIGN, WORKSPACE, LAYOUT = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def so():
    B.build()
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    lib = ctypes.CDLL(B.LIB)
    binding._sig(lib)
    return lib


def cache(**kw):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CKVCache
    a = dict(k=P, v=P, k_scale=None, v_scale=None, page_stride=None, num_pages=8, page_size=16, n_kv_heads=2,
             head_dim=64, dtype=0, maps=None)
    a.update(kw)
    if a["page_stride"] is None:
        a["page_stride"] = a["n_kv_heads"] * a["page_size"] * a["head_dim"]
    return CKVCache(**a)


def batch(**kw):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CBatch
    a = dict(cu_tokens=P, kv_len=P, page_table=P, n_seqs=2, max_pages=4, max_new=3)
    a.update(kw)
    return CBatch(**a)


@pytest.mark.parametrize("args", [(16, 10000.0, 1.0, 0.0, 1.0, 32.0), (128, 500000.0, 8.0, 8192.0, 1.0, 32.0),
                                  (64, 10000.0, 4.0, 0.0, 0.0, 0.0), (512, 1e6, 2.5, 4096.0, 2.0, 16.0)])
def test_frequencies_match_the_oracle(so, args):
    out = np.empty(args[0] // 2)
    assert so.rope_frequencies(*args, out.ctypes.data) == 0
    assert np.allclose(out, OA.rope_frequencies(*args), rtol=1e-14, atol=0)


@pytest.mark.parametrize("args", [(8, 1e4, 1, 0, 1, 32), (24, 1e4, 1, 0, 1, 32), (528, 1e4, 1, 0, 1, 32),
                                  (64, 1.0, 1, 0, 1, 32), (64, 1e4, 0.5, 0, 1, 32), (64, 1e4, 2, -1, 1, 32),
                                  (64, 1e4, 2, 4096, 32, 32), (64, float("nan"), 1, 0, 1, 32),
                                  (64, 1e4, float("inf"), 0, 1, 32), (64, 1e4, 2, 4096, 1, float("inf"))])
def test_frequencies_refuse(so, args):
    out = np.full(300, 7.0)
    assert so.rope_frequencies(*args, out.ctypes.data) == SHAPE
    assert np.all(out == 7.0)
    assert so.rope_frequencies(64, 1e4, 1, 0, 1, 32, None) == NULL


def rope_args(**kw):
    a = dict(x=P, x_stride=256, n_tokens=3, n_heads=4, head_dim=64, positions=P, inv_freq=P, rot=64, amplitude=1.0,
             flags=0, y=P, y_stride=256, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(positions=None), NULL), (dict(inv_freq=None), NULL),
    (dict(n_tokens=-1), SHAPE), (dict(n_heads=0), SHAPE), (dict(head_dim=24), SHAPE), (dict(head_dim=528), SHAPE),
    (dict(rot=0), SHAPE), (dict(rot=8), SHAPE), (dict(rot=80), SHAPE), (dict(x_stride=248), SHAPE),
    (dict(y_stride=248), SHAPE), (dict(x_stride=260), ALIGN), (dict(x=P + 8), ALIGN), (dict(y=P + 2), ALIGN),
    (dict(positions=P + 2), ALIGN), (dict(inv_freq=P + 4), ALIGN), (dict(flags=4), SHAPE),
    (dict(amplitude=float("inf")), SHAPE), (dict(n_tokens=0), 0)])
def test_rope_refuses(so, kw, status):
    assert so.rope_apply(*rope_args(**kw)) == status


def append_args(c, **kw):
    a = dict(cache=ctypes.byref(c) if c is not None else None, k=P, k_stride=128, v=P, v_stride=128, n_tokens=3,
             slots=P, positions=P, inv_freq=P, rot=64, amplitude=1.0, flags=0, q=P, q_stride=256, n_heads=4, q_out=P,
             q_out_stride=256, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(page_stride=2 * 16 * 64 - 8), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=512), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(n_kv_heads=0, page_stride=4096), SHAPE), (dict(dtype=2), LAYOUT), (dict(k_scale=P), LAYOUT),
    (dict(k=P + 8), ALIGN), (dict(page_stride=2 * 16 * 64 + 4), ALIGN), (dict(dtype=1, v_scale=P + 2), ALIGN), (dict(maps=P + 64), ALIGN)])
def test_caches_are_refused(so, kw, status):
    c = cache(**kw)
    assert so.kv_append(*append_args(c)) == status
    assert so.paged_attention(*attention_args(c)) == status
    assert so.kv_cache_maps(ctypes.byref(c), P) == status


def test_maps_refuse(so):
    assert so.kv_cache_maps(None, P) == NULL
    assert so.kv_cache_maps(ctypes.byref(cache()), None) == NULL
    assert so.kv_cache_maps(ctypes.byref(cache()), P + 64) == ALIGN


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL),
    (dict(q_out=None), NULL), (dict(q=None), NULL), (dict(positions=None), NULL), (dict(n_tokens=-1), SHAPE),
    (dict(n_heads=0), SHAPE), (dict(k_stride=120), SHAPE), (dict(v_stride=132), ALIGN), (dict(q_stride=248), SHAPE),
    (dict(q_out=P + 8), ALIGN), (dict(slots=P + 4), ALIGN), (dict(rot=72), SHAPE), (dict(flags=2), SHAPE),
    (dict(amplitude=float("nan")), SHAPE), (dict(n_tokens=0), 0),
    (dict(n_tokens=0, rot=0, positions=None, inv_freq=None, q=None, q_out=None), 0)])
def test_append_refuses(so, kw, status):
    assert so.kv_append(*append_args(cache(), **kw)) == status


def attention_args(c, b=None, **kw):
    b = b or batch()
    a = dict(cache=ctypes.byref(c) if c is not None else None, batch=ctypes.byref(b), q=P, q_stride=256, n_tokens=5,
             n_heads=4, scale=0.1, softcap=0.0, window=0, out=P, out_stride=256, lse=P, ws=P, ws_bytes=1 << 30,
             stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), NULL), (dict(batch=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(n_tokens=-1), SHAPE), (dict(n_heads=5), SHAPE), (dict(n_heads=0), SHAPE), (dict(q_stride=248), SHAPE),
    (dict(out_stride=252), SHAPE), (dict(out_stride=260), ALIGN), (dict(q=P + 4), ALIGN), (dict(lse=P + 2), ALIGN),
    (dict(scale=float("nan")), SHAPE), (dict(softcap=-1.0), SHAPE), (dict(softcap=float("inf")), SHAPE),
    (dict(window=-1), SHAPE), (dict(ws=None), WORKSPACE), (dict(ws_bytes=1024), WORKSPACE), (dict(ws=P + 8), ALIGN),
    (dict(n_tokens=0), 0)])
def test_attention_refuses(so, kw, status):
    assert so.paged_attention(*attention_args(cache(), **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(cu_tokens=None), NULL), (dict(kv_len=None), NULL), (dict(page_table=None), NULL), (dict(n_seqs=-1), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 27), SHAPE), (dict(max_new=-1), SHAPE), (dict(kv_len=P + 2), ALIGN),
    (dict(n_seqs=0), 0), (dict(max_new=0), 0)])
def test_batches_are_refused(so, kw, status):
    assert so.paged_attention(*attention_args(cache(), batch(**kw))) == status


def test_workspace_sizes(so):
    f = so.paged_attention_workspace_bytes
    assert f(16, 16, 1, 32, 8, 128) > 0
    assert f(16, 16, 1, 32, 8, 128) <= f(4096, 4, 2048, 32, 8, 128)
    for bad in ((-1, 1, 1, 4, 2, 64), (1, -1, 1, 4, 2, 64), (1, 1, -1, 4, 2, 64), (1, 1, 1, 5, 2, 64), (1, 1, 1, 4, 0, 64),
                (1, 1, 1, 4, 2, 96), (1 << 30, 1, 1, 4, 2, 64), (1 << 30, 1, 1, 4, 4, 64),
                ((1 << 30) - 100, 1, 1, 4, 2, 64)):
        assert f(*bad) == 0
