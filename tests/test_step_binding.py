"""What the binding of norms, steps and trees refuses before it calls the library, on the CPU (stand-ins as for the rest of the
attention side)."""

import types

import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from tests.test_attention_binding import BF16, F64, I32, I64, Tensor, fake, stream  # noqa: F401

F32 = torch.float32


@pytest.fixture
def lib(fake):  # noqa: F811
    fake._tree_bytes, fake._norm_bytes = {}, {}
    return fake


def calls_on(lib, device, s):
    """One call of each operator with everything on `device`."""
    T = lambda dtype, *shape: Tensor(shape, dtype, device)  # noqa: E731
    cache = types.SimpleNamespace(device=torch.device(device), n_kv_heads=2, head_dim=64, ref=None, k=T(BF16, 1), v=T(BF16, 1),
                                  k_scale=None, v_scale=None)
    batch = types.SimpleNamespace(device=torch.device(device), n_seqs=1, max_new=4, ref=None, cu_tokens=T(I32, 2),
                                  kv_len=T(I32, 1), page_table=T(I32, 1, 1))
    pages = types.SimpleNamespace(device=torch.device(device), n_seqs=1, ref=None, page_table=T(I32, 1, 1), held=T(I32, 1),
                                  free_pages=T(I32, 1), free_count=T(I32, 1))
    step = types.SimpleNamespace(device=torch.device(device), n_seqs=1, tokens=4, words=1, ref=None, slots=T(I64, 4),
                                 positions=T(I32, 4), cu_tokens=T(I32, 2), kv_len=T(I32, 1), masks=T(I64, 4, 1))
    q, k, pos, freq, slots, w = T(BF16, 4, 8, 64), T(BF16, 4, 2, 64), T(I32, 4), T(F64, 32), T(I64, 4), T(BF16, 64)
    qo, ko, masks, one = T(BF16, 4, 8, 64), T(BF16, 4, 2, 64), T(I64, 4, 1), T(I32, 1)
    return [lambda: lib.qk_norm_rope(q, k, pos, freq, w, w, q_out=qo, k_out=ko, stream=s),
            lambda: lib.kv_append(cache, k, k, slots, pos, freq, q=q, q_out=qo, q_norm=w, k_norm=w, stream=s),
            lambda: lib.kv_assign(pages, one, one, step, parents=pos, stream=s),
            lambda: lib.kv_accept(cache, batch, T(I32, 1, 3), out=one, stream=s),
            lambda: lib.tree_attention(q, cache, batch, masks, out=qo, stream=s)]


def test_calls_on_the_current_gpu_go_through(lib):
    for call in calls_on(lib, "cuda:0", stream()):
        call()
    assert lib.lib.launches() == ["qk_norm_rope", "kv_append_norm", "kv_assign", "kv_accept", "tree_attention"]


@pytest.mark.parametrize("device,s", [("cuda:1", stream(1)), ("cuda:1", stream(0)), ("cuda:0", stream(1)), ("cpu", stream())])
def test_calls_elsewhere_are_refused(lib, device, s):
    for call in calls_on(lib, device, s):
        with pytest.raises(ValueError):
            call()
    assert lib.lib.launches() == []


@pytest.mark.parametrize("device,s", [("cuda:1", stream(1)), ("cuda:0", stream(1)), ("cpu", stream())])
def test_the_backward_pass_elsewhere_is_refused(lib, device, s):
    T = lambda dtype, *shape: Tensor(shape, dtype, device)  # noqa: E731
    q, w = T(BF16, 4, 8, 64), T(BF16, 64)
    with pytest.raises(ValueError):
        lib.qk_norm_rope_backward(q, None, q, None, T(I32, 4), T(F64, 32), w, dq_out=q, stream=s)
    assert lib.lib.launches() == []


def test_operands_of_two_gpus_are_refused(lib):
    T = lambda dtype, *shape, on="cuda:0": Tensor(shape, dtype, on)  # noqa: E731
    q, w, pos, freq = T(BF16, 4, 8, 64), T(BF16, 64), T(I32, 4), T(F64, 32)
    there = "cuda:1"
    for bad in (lambda: lib.qk_norm_rope(q, T(BF16, 4, 2, 64, on=there), pos, freq, w, w, q_out=q),
                lambda: lib.qk_norm_rope(q, None, T(I32, 4, on=there), freq, w, q_out=q),
                lambda: lib.qk_norm_rope(q, None, pos, freq, T(BF16, 64, on=there), q_out=q),
                lambda: lib.qk_norm_rope_backward(T(BF16, 4, 8, 64, on=there), None, q, None, pos, freq, w, dq_out=q)):
        with pytest.raises(ValueError):
            bad()
    assert lib.lib.launches() == []


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 100, -2 ** 31 - 1])
def test_sizes_beyond_32_bits_are_refused(lib, value):
    x = Tensor((4, 8, 64), BF16, "cuda:0")
    cache = types.SimpleNamespace(device=x.device, n_kv_heads=2, head_dim=64, ref=None)
    batch = types.SimpleNamespace(device=x.device, n_seqs=1, max_new=4, ref=None)
    with pytest.raises(ValueError):
        lib.tree_attention(x, cache, batch, Tensor((4, 1), I64, "cuda:0"), window=value, out=x)
    i = lambda *s: Tensor(s, I32, "cuda:0")  # noqa: E731
    with pytest.raises(ValueError):
        binding.PageTable(i(1, 1), i(1), i(1), i(1), value)
    with pytest.raises(ValueError):
        binding.Step(1, value, 0, device="cpu")
    assert lib.lib.launches() == []


def test_a_step_on_the_cpu_is_refused():
    with pytest.raises(ValueError):
        binding.Step(1, 4, 1, device="cpu")
