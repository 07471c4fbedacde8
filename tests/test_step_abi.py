"""Argument checks of norms with the rotation, step bookkeeping and accepted paths (no GPU): every rejected call returns
before any CUDA call."""

import ctypes

import pytest

from nvfp4_w4a16_moe_skinny_gb300 import build as B
from tests.test_attention_abi import ALIGN, LAYOUT, NULL, P, SHAPE, WORKSPACE, append_args, batch, cache


@pytest.fixture(scope="module")
def so():
    B.build()
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    lib = ctypes.CDLL(B.LIB)
    binding._sig(lib)
    return lib


def norm(**kw):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CQKNorm
    a = dict(q_weight=P, k_weight=P, weight_dtype=0, eps=1e-6)
    a.update(kw)
    return CQKNorm(**a)


def forward_args(n, **kw):
    a = dict(norm=ctypes.byref(n) if n is not None else None, q=P, q_stride=256, n_heads=4, k=P, k_stride=128, kv=2,
             n_tokens=3, head_dim=64, positions=P, inv_freq=P, rot=64, amplitude=1.0, flags=0, q_out=P, q_out_stride=256,
             k_out=P, k_out_stride=128, stream=None)
    a.update(kw)
    return list(a.values())


def backward_args(n, **kw):
    a = dict(norm=ctypes.byref(n) if n is not None else None, dq=P, dq_stride=256, q=P, q_stride=256, n_heads=4, dk=P,
             dk_stride=128, k=P, k_stride=128, kv=2, n_tokens=3, head_dim=64, positions=P, inv_freq=P, rot=64,
             amplitude=1.0, flags=0, dq_out=P, dq_out_stride=256, dk_out=P, dk_out_stride=128, dq_weight=P, dk_weight=P,
             ws=P, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q_weight=None), NULL), (dict(k_weight=None), NULL), (dict(weight_dtype=2), LAYOUT), (dict(eps=-1e-6), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(q_weight=P + 1), ALIGN),
    (dict(weight_dtype=1, k_weight=P + 2), ALIGN)])
def test_weights_are_refused(so, kw, status):
    n = norm(**kw)
    assert so.qk_norm_rope(*forward_args(n)) == status
    assert so.qk_norm_rope_backward(*backward_args(n)) == status
    args = append_args(cache())
    assert so.kv_append_norm(args[0], ctypes.byref(n), *args[1:]) == status


SHARED = [
    (dict(norm=None), NULL), (dict(q=None), NULL), (dict(k=None), NULL), (dict(n_tokens=-1), SHAPE), (dict(n_heads=0), SHAPE),
    (dict(kv=-1), SHAPE), (dict(head_dim=24), SHAPE), (dict(head_dim=528), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(n_tokens=1 << 30), SHAPE), (dict(q_stride=248), SHAPE), (dict(k_stride=120), SHAPE), (dict(q_stride=260), ALIGN),
    (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(rot=72), SHAPE), (dict(rot=80), SHAPE), (dict(rot=-16), SHAPE),
    (dict(positions=None), NULL), (dict(inv_freq=None), NULL), (dict(positions=P + 2), ALIGN), (dict(inv_freq=P + 4), ALIGN),
    (dict(flags=2), SHAPE), (dict(amplitude=float("nan")), SHAPE)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(q_out=None), NULL), (dict(k_out=None), NULL), (dict(q_out_stride=248), SHAPE), (dict(k_out=P + 8), ALIGN),
    (dict(n_tokens=0), 0), (dict(n_tokens=0, kv=0, k=None, k_out=None), 0),
    (dict(n_tokens=0, rot=0, positions=None, inv_freq=None), 0)])
def test_forward_refuses(so, kw, status):
    a = dict(kw)
    n = None if "norm" in a else norm()
    a.pop("norm", None)
    assert so.qk_norm_rope(*forward_args(n, **a)) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dq_out=None), NULL), (dict(dk_out=None), NULL),
    (dict(dq_weight=None), NULL), (dict(dk_weight=None), NULL), (dict(dq_stride=248), SHAPE), (dict(dk_stride=132), ALIGN),
    (dict(dk_out_stride=64), SHAPE), (dict(dq_weight=P + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(ws=P + 8), ALIGN)])
def test_backward_refuses(so, kw, status):
    a = dict(kw)
    n = None if "norm" in a else norm()
    a.pop("norm", None)
    assert so.qk_norm_rope_backward(*backward_args(n, **a)) == status


def test_backward_workspace(so):
    f = so.qk_norm_rope_workspace_bytes
    assert f(0, 4, 2, 64) >= 16 and f(1, 4, 0, 64) >= 4 * 64
    for bad in ((-1, 4, 2, 64), (1, 0, 2, 64), (1, 4, -1, 64), (1, 4, 2, 24), (1, 4, 2, 528), (1 << 30, 4, 2, 64)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(q_out=None), NULL),
    (dict(q=None), NULL), (dict(positions=None), NULL), (dict(n_tokens=-1), SHAPE), (dict(n_heads=0), SHAPE),
    (dict(k_stride=120), SHAPE), (dict(v_stride=132), ALIGN), (dict(q_stride=248), SHAPE), (dict(q_out=P + 8), ALIGN),
    (dict(slots=P + 4), ALIGN), (dict(rot=72), SHAPE), (dict(flags=2), SHAPE), (dict(n_tokens=0), 0)])
def test_append_refuses(so, kw, status):
    args = append_args(cache(), **kw)
    assert so.kv_append_norm(args[0], ctypes.byref(norm()), *args[1:]) == status


def test_append_without_queries_needs_no_weight_of_theirs(so):
    args = append_args(cache(), n_tokens=0, q=None, q_out=None)
    assert so.kv_append_norm(args[0], ctypes.byref(norm(q_weight=None)), *args[1:]) == 0


def pages(**kw):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CPageTable
    a = dict(page_table=P, held=P, free_pages=P, free_count=P, n_seqs=2, max_pages=4, page_size=16, num_free=8)
    a.update(kw)
    return CPageTable(**a)


def step(**kw):
    from nvfp4_w4a16_moe_skinny_gb300.binding import CStep
    a = dict(slots=P, positions=P, cu_tokens=P, kv_len=P, masks=P, n_tokens=5, words=1)
    a.update(kw)
    return CStep(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(page_table=None), NULL), (dict(held=None), NULL), (dict(free_pages=None), NULL), (dict(free_count=None), NULL),
    (dict(n_seqs=-1), SHAPE), (dict(n_seqs=16385), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 26), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=512), SHAPE), (dict(num_free=-1), SHAPE), (dict(num_free=1 << 30), SHAPE),
    (dict(page_table=P + 2), ALIGN), (dict(held=P + 1), ALIGN), (dict(free_pages=P + 2), ALIGN), (dict(free_count=P + 2), ALIGN)])
def test_page_tables_are_refused(so, kw, status):
    t, s = pages(**kw), step()
    assert so.kv_assign(ctypes.byref(t), P, P, None, ctypes.byref(s), None) == status


@pytest.mark.parametrize("kw,parents,status", [
    (dict(slots=None), None, NULL), (dict(positions=None), None, NULL), (dict(cu_tokens=None), None, NULL),
    (dict(kv_len=None), None, NULL), (dict(masks=None), P, NULL), (dict(n_tokens=-1), None, SHAPE),
    (dict(n_tokens=1 << 30), None, SHAPE), (dict(words=-1), None, SHAPE), (dict(words=65), None, SHAPE),
    (dict(words=0), P, SHAPE), (dict(slots=P + 4), None, ALIGN), (dict(positions=P + 2), None, ALIGN),
    (dict(masks=P + 4), P, ALIGN), (dict(), P + 2, ALIGN)])
def test_steps_are_refused(so, kw, parents, status):
    t, s = pages(), step(**kw)
    assert so.kv_assign(ctypes.byref(t), P, P, parents, ctypes.byref(s), None) == status


def test_assign_refuses(so):
    t, s = pages(), step()
    assert so.kv_assign(None, P, P, None, ctypes.byref(s), None) == NULL
    assert so.kv_assign(ctypes.byref(t), P, P, None, None, None) == NULL
    assert so.kv_assign(ctypes.byref(t), None, P, None, ctypes.byref(s), None) == NULL
    assert so.kv_assign(ctypes.byref(t), P, None, None, ctypes.byref(s), None) == NULL
    assert so.kv_assign(ctypes.byref(t), P + 2, P, None, ctypes.byref(s), None) == ALIGN


@pytest.mark.parametrize("kw,path_len,out,status", [
    (dict(cu_tokens=None), 4, P + 64, NULL), (dict(kv_len=None), 4, P + 64, NULL), (dict(page_table=None), 4, P + 64, NULL),
    (dict(), 4, None, NULL), (dict(n_seqs=-1), 4, P + 64, SHAPE), (dict(n_seqs=65536), 4, P + 64, SHAPE),
    (dict(max_pages=0), 4, P + 64, SHAPE), (dict(max_pages=1 << 27), 4, P + 64, SHAPE), (dict(), -1, P + 64, SHAPE),
    (dict(), 1025, P + 64, SHAPE), (dict(), 4, P, SHAPE), (dict(), 4, P + 2, ALIGN), (dict(n_seqs=0), 4, P + 64, 0)])
def test_accept_refuses(so, kw, path_len, out, status):
    c, b = cache(), batch(**kw)
    assert so.kv_accept(ctypes.byref(c), ctypes.byref(b), P, path_len, out, None) == status


def test_accept_refuses_missing_arguments(so):
    c, b = cache(), batch()
    assert so.kv_accept(None, ctypes.byref(b), P, 4, P + 64, None) == NULL
    assert so.kv_accept(ctypes.byref(c), None, P, 4, P + 64, None) == NULL
    assert so.kv_accept(ctypes.byref(c), ctypes.byref(b), None, 4, P + 64, None) == NULL
    assert so.kv_accept(ctypes.byref(cache(page_size=8)), ctypes.byref(b), P, 4, P + 64, None) == SHAPE
