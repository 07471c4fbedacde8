"""Attention captured into a graph on a stream that is given to the call while another one is current."""

import pytest
import torch

from tests.gpu_helpers import dev
from tests.test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 300])
def test_a_call_captured_on_a_given_stream_has_its_own_workspace(lib, fp8, new):
    c = Case([(new, 3000), (1, 700), (new, new)], 8, 2, 128, 64, fp8, seed=5)
    cache, batch, s = c.cache(), c.batch(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want, want_lse = lib.paged_attention(c.q, cache, batch, with_lse=True, stream=s)      # the stream's own workspace
    torch.cuda.synchronize()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin(capture_error_mode="thread_local")
    try:
        lib.paged_attention(c.q, cache, batch, out=out, lse=lse, stream=s)
    finally:
        with torch.cuda.stream(s):
            graph.capture_end()
    torch.cuda.synchronize()
    own = lib._attention_ws[(dev().index, s.cuda_stream)][0]
    own[:4096].fill_(255)          # what the stream's workspace holds is nothing to the graph
    torch.cuda.synchronize()
    try:
        for _ in range(2):
            out.zero_(), lse.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert bool((own[:4096] == 255).all())
    finally:
        own[:4096].zero_()
        torch.cuda.synchronize()
    assert lib.device_error() == 0
