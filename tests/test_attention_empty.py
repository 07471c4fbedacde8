"""Calls without tokens or without sequences: nothing is launched, and rows that do not exist have no address (an empty
tensor's is NULL).  Other arguments are checked as always."""

import ctypes

import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from tests.gpu_helpers import dev
from tests.test_attention_abi import NULL, SHAPE, append_args, attention_args, batch, cache, rope_args, so  # noqa: F401


@pytest.mark.parametrize("kw,status", [
    (dict(x=None, y=None, positions=None), 0), (dict(x=None, y=None, positions=None, inv_freq=None), NULL),
    (dict(x=None, y=None, rot=80), SHAPE), (dict(x=None, y=None, head_dim=24), SHAPE)])
def test_rope_without_tokens(so, kw, status):  # noqa: F811
    assert so.rope_apply(*rope_args(n_tokens=0, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(inv_freq=None), NULL), (dict(flags=2), SHAPE), (dict(inv_freq=None, rot=0), 0), (dict(cache=None), NULL)])
def test_append_without_tokens(so, kw, status):  # noqa: F811
    args = dict(k=None, v=None, slots=None, q=None, q_out=None, positions=None, n_tokens=0)
    args.update(kw)
    assert so.kv_append(*append_args(cache(), **args)) == status


@pytest.mark.parametrize("b,kw,status", [
    (dict(), dict(q=None, out=None, n_tokens=0), 0), (dict(), dict(q=None, out=None, lse=None, n_tokens=0, n_heads=5), SHAPE),
    (dict(n_seqs=0, kv_len=None, page_table=None), dict(), 0),
    (dict(n_seqs=0, kv_len=None, page_table=None, max_pages=0, max_new=0), dict(q=None, out=None, n_tokens=0), 0),
    (dict(n_seqs=0, cu_tokens=None), dict(), NULL), (dict(n_seqs=0, max_pages=1 << 27), dict(), SHAPE),
    (dict(kv_len=None), dict(q=None, out=None, n_tokens=0), NULL)])
def test_attention_without_tokens_or_sequences(so, b, kw, status):  # noqa: F811
    assert so.paged_attention(*attention_args(cache(), batch(**b), **kw)) == status


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_empty_tensors_go_through_the_binding(lib, fp8):
    heads, kv, dim, page = 4, 2, 64, 16
    rows = lambda n, h: torch.zeros(n, h, dim, dtype=torch.bfloat16, device=dev())  # noqa: E731
    none = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device=dev())  # noqa: E731
    pools = torch.ones(2, 3, kv, page, dim, device=dev()).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
    c, w = binding.KVCache(pools[0], pools[1]), lib.rope_frequencies(dim, device=dev())
    q, k, pos = rows(0, heads), rows(0, kv), none(0)
    assert lib.rope_apply(q, pos, w).shape == (0, heads, dim)
    assert lib.kv_append(c, k, k, none(0, dtype=torch.int64), pos, w, q=q).shape == (0, heads, dim)
    assert lib.kv_append(c, k, k, none(0, dtype=torch.int64)) is None
    for b in (binding.Batch(none(4), none(3), none(3, 2), 1), binding.Batch(none(1), none(0), none(0, 2), 0),
              binding.Batch(none(1), none(0), none(0, 0), 4)):
        out, lse = lib.paged_attention(q, c, b, with_lse=True)
        assert out.shape == (0, heads, dim) and lse.shape == (0, heads)
    torch.cuda.synchronize()
    assert lib.device_error() == 0 and torch.all(pools.float() == 1)
    with pytest.raises(ValueError):
        lib.rope_apply(q.float(), pos, w)
    with pytest.raises(binding.NVFP4Error):
        lib.paged_attention(rows(0, 3), c, binding.Batch(none(1), none(0), none(0, 2), 0))
