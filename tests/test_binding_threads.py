"""Calls of several host threads on one stream, whose kernels share that stream's attention workspace (CPU: a library whose
calls take their time, as a real one's launches do, and let other threads run)."""

import threading
import time

import pytest

from tests.test_attention_binding import BF16, F64, I32, Recorder, Tensor, calls_on, fake, stream  # noqa: F401
from tests import test_step_binding as S


class Slow(Recorder):
    """Notes the calls that are inside the library at the same time."""

    def __init__(self):
        super().__init__()
        self.inside, self.most = 0, 0

    def __getattr__(self, name):
        call = super().__getattr__(name)
        if name.endswith("_bytes"):
            return call

        def slow(*args):
            self.inside += 1
            self.most = max(self.most, self.inside)
            time.sleep(0.005)
            self.inside -= 1
            return call(*args)
        return slow


@pytest.fixture
def lib(fake):  # noqa: F811
    fake.lib, fake._tree_bytes, fake._norm_bytes = Slow(), {}, {}
    return fake


def gradient(lib, monkeypatch):
    """A call of qk_norm_rope_backward with everything on the current GPU."""
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    T = lambda dtype, *shape: Tensor(shape, dtype, "cuda:0")  # noqa: E731
    monkeypatch.setattr(binding, "_empty", lambda shape, dtype, *a: T(dtype, *shape))
    q, w = T(BF16, 4, 8, 64), T(BF16, 64)
    return lambda: lib.qk_norm_rope_backward(q, None, q, None, T(I32, 4), T(F64, 32), w, dq_out=q, stream=stream())


def test_workspace_calls_launch_one_at_a_time(lib, monkeypatch):
    calls = [calls_on(lib, "cuda:0", stream())[-1], S.calls_on(lib, "cuda:0", stream())[-1], gradient(lib, monkeypatch)]
    errors = []

    def work():
        try:
            for call in calls:
                call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert sorted(lib.lib.launches()) == sorted(["paged_attention", "tree_attention", "qk_norm_rope_backward"] * 4)
    assert lib.lib.most == 1


def test_a_refused_call_lets_the_next_one_through(lib):
    """The lock is given back when a call fails."""
    class Refuses(Recorder):
        def __getattr__(self, name):
            return (lambda *a: 4096) if name.endswith("_bytes") else (lambda *a: 2)
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    call = S.calls_on(lib, "cuda:0", stream())[-1]
    slow, lib.lib = lib.lib, Refuses()
    with pytest.raises(binding.NVFP4Error):
        call()
    lib.lib = slow
    call()
    assert slow.launches() == ["tree_attention"]
