import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: full-size parity case (minutes of CPU oracle work)")


@pytest.fixture(scope="session")
def lib():
    """The C-ABI library through its Python binding (GPU tests only)."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    return binding.load()


@pytest.fixture(autouse=True)
def attention_counters_are_left_zero(request):
    """After every GPU test: the arrival counters of all attention workspaces are zero, as a completed call leaves them."""
    yield
    if "lib" not in request.fixturenames or request.node.get_closest_marker("gpu") is None:
        return
    import torch
    lib = request.getfixturevalue("lib")
    torch.cuda.synchronize()
    for key, ws in lib._attention_ws.items():
        assert not ws[0][:4096].any(), f"arrival counters of the workspace of {key}"
