"""The tree-decoding example runs: captured steps whose lengths, trees and verdicts change, on both kinds of cache."""

import os
import subprocess
import sys

import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from tests.conftest import ROOT
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

PATH = os.path.join(ROOT, "examples", "tree_decoding.py")


@pytest.mark.parametrize("args", [["--cache", "bf16"], ["--cache", "e4m3", "--seqs", "2"], ["--drafted", "70", "--context", "0"]])
def test_it_runs(args):
    r = subprocess.run([sys.executable, PATH, "--context", "100", "--steps", "4"] + args, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens accepted in 4 steps" in r.stdout


@pytest.mark.parametrize("fp8", [False, True])
def test_empty_calls_go_through_the_binding(lib, fp8):
    """No tokens, no sequences, paths of no entries: nothing is launched on them and nothing written."""
    heads, kv, dim, page = 4, 2, 64, 16
    rows = lambda n, h: torch.zeros(n, h, dim, dtype=torch.bfloat16, device=dev())  # noqa: E731
    none = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device=dev())  # noqa: E731
    pools = torch.ones(2, 3, kv, page, dim, device=dev()).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
    c, w = binding.KVCache(pools[0], pools[1]), torch.ones(dim, dtype=torch.bfloat16, device=dev())
    q, k, pos, freq = rows(0, heads), rows(0, kv), none(0), lib.rope_frequencies(dim, device=dev())
    a, b = lib.qk_norm_rope(q, k, pos, freq, w, w)
    assert a.shape == (0, heads, dim) and b.shape == (0, kv, dim)
    a, b, dq, dk = lib.qk_norm_rope_backward(q, k, q, k, pos, freq, w, w)
    assert a.shape == (0, heads, dim) and b.shape == (0, kv, dim) and not dq.any() and not dk.any()
    assert lib.kv_append(c, k, k, none(0, dtype=torch.int64), pos, freq, q=q, q_norm=w, k_norm=w).shape == (0, heads, dim)
    for batch in (binding.Batch(none(4), none(3), none(3, 2), 1), binding.Batch(none(1), none(0), none(0, 2), 0)):
        out, lse = lib.tree_attention(q, c, batch, none(0, 1, dtype=torch.int64), with_lse=True)
        assert out.shape == (0, heads, dim) and lse.shape == (0, heads)
        assert not lib.kv_accept(c, batch, none(batch.n_seqs, 0)).any()
    torch.cuda.synchronize()
    assert lib.device_error() == 0 and torch.all(pools.float() == 1)
