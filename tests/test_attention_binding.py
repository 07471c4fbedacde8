"""What the binding of the attention side refuses before it calls the library, on the CPU: stand-ins for tensors and
streams of any device, and a library that records its calls."""

import types

import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding

BF16, I32, I64, F64 = torch.bfloat16, torch.int32, torch.int64, torch.float64


class Tensor:
    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device(device), "cuda" in device

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape.numel()

    def record_stream(self, stream):
        pass


class Recorder:
    """Stands for the loaded library: notes which function was called with which arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_bytes") else 0
        return call

    def launches(self):
        return [n for n, _ in self.calls if not n.endswith("_bytes")]


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    x = binding.Library.__new__(binding.Library)
    x.lib, x._attention_bytes, x._attention_ws = Recorder(), {}, {}
    monkeypatch.setattr(x, "_stream_workspace", lambda *a: (None, 1 << 20, 1 << 20), raising=False)
    return x


def stream(device=0):
    return types.SimpleNamespace(cuda_stream=0, device_index=device)


def calls_on(lib, device, s):
    """One call of each operator with everything on `device`."""
    T = lambda dtype, *shape: Tensor(shape, dtype, device)  # noqa: E731
    cache = types.SimpleNamespace(device=torch.device(device), n_kv_heads=2, head_dim=64, ref=None, k=T(BF16, 1), v=T(BF16, 1),
                                  k_scale=None, v_scale=None)
    batch = types.SimpleNamespace(device=torch.device(device), n_seqs=1, max_new=4, ref=None, cu_tokens=T(I32, 2),
                                  kv_len=T(I32, 1), page_table=T(I32, 1, 1))
    q, k, pos, freq, slots = T(BF16, 4, 8, 64), T(BF16, 4, 2, 64), T(I32, 4), T(F64, 32), T(I64, 4)
    out = T(BF16, 4, 8, 64)
    return [lambda: lib.rope_apply(q, pos, freq, out=out, stream=s),
            lambda: lib.kv_append(cache, k, k, slots, pos, freq, q=q, q_out=out, stream=s),
            lambda: lib.paged_attention(q, cache, batch, out=out, stream=s)]


def test_calls_on_the_current_gpu_go_through(fake):
    for call in calls_on(fake, "cuda:0", stream()):
        call()
    assert fake.lib.launches() == ["rope_apply", "kv_append", "paged_attention"]


@pytest.mark.parametrize("device,s", [("cuda:1", stream(1)), ("cuda:1", stream(0)), ("cuda:0", stream(1)), ("cpu", stream())])
def test_calls_elsewhere_are_refused(fake, device, s):
    """The library launches on the current device: pointers and streams of another one must not get there."""
    for call in calls_on(fake, device, s):
        with pytest.raises(ValueError):
            call()
    assert fake.lib.launches() == []


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 100, -2 ** 31 - 1])
def test_sizes_beyond_32_bits_are_refused(fake, value):
    """The library takes them as int32: a window of 2^32 + 100 must not become one of 100, nor a bound on the new
    tokens of 2^32 one of none."""
    q, k = Tensor((4, 8, 64), BF16, "cuda:0"), Tensor((4, 8, 64), BF16, "cuda:0")
    cache = types.SimpleNamespace(device=q.device, n_kv_heads=2, head_dim=64, ref=None, k=k, v=k, k_scale=None, v_scale=None)
    batch = types.SimpleNamespace(device=q.device, n_seqs=1, max_new=4, ref=None, cu_tokens=k, kv_len=k, page_table=k)
    with pytest.raises(ValueError):
        fake.paged_attention(q, cache, batch, window=value, out=k, stream=stream())
    with pytest.raises(ValueError):
        binding.Batch(Tensor((2,), I32, "cuda:0"), Tensor((1,), I32, "cuda:0"), Tensor((1, 1), I32, "cuda:0"), value)
    with pytest.raises(ValueError):
        fake.rope_frequencies(value)
    assert fake.lib.launches() == []
