"""E4M3 appends at every bf16 value and at scales of every size: powers of two, scales whose quotients fall on the middle
of two codes, and the ends of fp32, subnormal ones among them.

A code is that of value * (1 / scale) with both in fp32, each rounded once: within 2^-23 of the quotient, so that it lies
between the codes of the quotient times 1 - 2^-22 and 1 + 2^-22.  Where the reciprocal is exact it is the quotient's."""

import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

SCALES = [
    [1.0, 0.5, 2.0 ** -20, 3.0, 5.0, 7.0, 0.75, 1.5], [3.0 / 64, 5.0 / 64, 7.0 / 64, 0.1, 0.3, 0.6, 0.011718750, 0.02],
    [1e-30, 1e-37, 2.0 ** -126, 2.0 ** -127, 2.0 ** -149, 1e-40, 3e-39, 1.1754944e-38],
    [1e30, 1e37, 2.0 ** 126, 2.0 ** 127, 3.4e38, 2.0 ** 60, 2.0 ** 61, 2.0 ** -60], [2.0 ** -61, 3e-19, 1e18, 1e-12, 448.0, 480.0, 1.0 / 448, 1e5],
]


@pytest.mark.parametrize("scales", SCALES)
def test_every_bf16_value(lib, scales):
    kv, dim, page = 8, 128, 64
    tokens = (1 << 16) // dim
    bits = torch.arange(1 << 16, dtype=torch.int32, device=dev()).to(torch.int16).view(torch.bfloat16)
    v = bits.view(tokens, 1, dim).expand(tokens, kv, dim).contiguous()
    s = torch.tensor(scales, dtype=torch.float32, device=dev())
    pool = torch.zeros(2, tokens // page, kv, page, dim, device=dev()).to(torch.float8_e4m3fn)
    lib.kv_append(binding.KVCache(pool[0], pool[1], s, s), v, v, torch.arange(tokens, device=dev()))
    x = v.double() / s.double()[:, None]
    code = lambda t: torch.where(torch.isnan(t), t, t.clamp(-448.0, 448.0)).float().to(torch.float8_e4m3fn)  # noqa: E731
    a, b = code(x * (1 - 2.0 ** -22)).float(), code(x * (1 + 2.0 ** -22)).float()
    nan = torch.isnan(x)
    exact = (torch.frexp(s)[0] == 0.5)[:, None].expand_as(x)       # a power of two
    for p in pool:                                                 # keys that nothing turns, and values
        got = p.permute(0, 2, 1, 3).reshape(tokens, kv, dim)
        g = got.float()
        assert torch.equal(torch.isnan(g), nan)
        assert bool(((g >= torch.minimum(a, b)) & (g <= torch.maximum(a, b)))[~nan].all())
        assert torch.equal(torch.signbit(g)[~nan], torch.signbit(x)[~nan])
        assert torch.equal(got.view(torch.uint8)[exact & ~nan], code(x).view(torch.uint8)[exact & ~nan])
