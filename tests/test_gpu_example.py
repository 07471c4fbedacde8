"""The decode example: its prompt and single-token steps agree with one pass over the whole sequence, and the captured
loop runs."""

import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from tests.conftest import ROOT
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

PATH = os.path.join(ROOT, "examples", "decode_attention.py")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_prefill_in_pieces_equals_one_pass(lib, cache):
    spec = importlib.util.spec_from_file_location("decode_attention", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    heads, kv, dim, total = 8, 4, 128, 150
    qkv = torch.randn(total, heads + 2 * kv, dim, generator=torch.Generator(device=dev()).manual_seed(2), device=dev()).to(torch.bfloat16)
    outs = []
    for cuts in ([0, total], [0, 100, 101, 102, total]):
        block = m.AttentionBlock(lib, 256, heads, kv, dim, 2, 200, page=32, cache=cache)
        outs.append(torch.cat([block.prefill(qkv[a:b], 1, a) for a, b in zip(cuts, cuts[1:])]).double())
    # two roundings of the weights and the results apart: 2 * 2^-8 of the largest value each row can reach
    assert float((outs[0] - outs[1]).abs().max()) <= 4 * 2.0 ** -8 * float(qkv[:, heads + kv:].abs().max())
    assert lib.device_error() == 0 and isinstance(block.cache, binding.KVCache)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_the_loop_runs(cache):
    r = subprocess.run([sys.executable, PATH, "--seqs", "3", "--context", "200", "--steps", "5", "--cache", cache],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "ending at position 207" in r.stdout
