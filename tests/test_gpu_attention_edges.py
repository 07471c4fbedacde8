"""The attention side's calls at their edges: no tokens, signs of the scale, a scale of zero, streams, capture."""

import math

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from tests.gpu_helpers import dev
from tests.test_gpu_attention import Case, run

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


# packed rows of one kv head: tiles of 16, 32 and 64 rows, and the kernel for more
SHAPES = [([(1, 300), (3, 40)], 8, 2), ([(8, 200), (1, 1)], 6, 2), ([(15, 90), (2, 700)], 8, 2), ([(90, 333), (1, 50)], 4, 2)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,heads,kv", SHAPES)
@pytest.mark.parametrize("scale,softcap", [(-0.1, 0.0), (-0.2, 5.0), (0.0, 0.0), (0.0, 5.0)])
def test_negative_and_zero_scales(lib, fp8, dim, lens, heads, kv, scale, softcap):
    c = Case(lens, heads, kv, dim, 32, fp8, seed=dim + heads)
    c.check(*run(lib, c, scale=scale, softcap=softcap), scale=scale, softcap=softcap)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,heads,kv", SHAPES)
def test_a_scale_of_zero_keeps_nan(lib, fp8, dim, lens, heads, kv):
    """0 * NaN is NaN: a query that holds one, and the rows that see a key that holds one."""
    c = Case(lens, heads, kv, dim, 32, fp8, seed=dim)
    c.q[0, 1, 5] = float("nan")
    n, length = c.lens[1]
    raw = c.pools.float()
    raw[0, int(c.table[1, (length - 1) // 32]), 0, (length - 1) % 32, 3] = float("nan")     # the last key of sequence 1
    c.pools = raw.to(c.pools.dtype)
    out, lse = run(lib, c, scale=0.0)
    g, t = heads // kv, c.tokens - 1
    want = torch.zeros(c.tokens, heads, dtype=torch.bool, device=dev())
    want[0, 1] = True
    want[t, :g] = True                     # the last token's rows of kv head 0
    assert torch.equal(torch.isnan(lse), want)
    assert torch.equal(torch.isnan(out), want[..., None].expand_as(out))
