"""Small angles of the rotation: slow pairs at early positions, whose sines are far below one and stand alone in the
result where the other value of the pair is zero.

Bound.  x_b = 0: y_b = x_a sin t.  The frequency as a 64-bit fraction of a turn is off by less than 2^-63 of a turn a
position, the rest by fp32 roundings: the fraction's 2^-23, its scaling exact, sin 2^-22 (two units), product 2^-24; with the
amplitude's 2^-24 below 2^-21 of the value together.  Then bf16, 2^-8."""

import math

import numpy as np
import pytest
import torch

from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("theta,factor", [(500000.0, 8.0), (1e6, 64.0), (10000.0, 1.0), (1e9, 1.0)])
@pytest.mark.parametrize("positions", [[1, 2, 3, 5, 7], [-1, -3, 100, 1000, -4097]])
def test_slow_pairs_keep_their_sines(lib, interleaved, theta, factor, positions):
    dim, tokens = 128, len(positions)
    w = lib.rope_frequencies(dim, theta, factor)
    x = torch.zeros(tokens, 2, dim, dtype=torch.bfloat16, device=dev())
    first = slice(0, dim, 2) if interleaved else slice(0, dim // 2)
    second = slice(1, dim, 2) if interleaved else slice(dim // 2, dim)
    x[..., first] = torch.randn(tokens, 2, dim // 2, generator=torch.Generator(device=dev()).manual_seed(3), device=dev()).to(torch.bfloat16)
    pos = torch.tensor(positions, dtype=torch.int32, device=dev())
    y = lib.rope_apply(x, pos, w.to(dev()), interleaved).double().cpu().numpy()
    a = x[..., first].double().cpu().numpy()
    angle = np.array(positions, np.float64)[:, None] * w.numpy()          # off by 2^-53 of itself
    for got, want in ((y[..., second], a * np.sin(angle)[:, None]), (y[..., first], a * np.cos(angle)[:, None])):
        turn = 2 * math.pi * 2.0 ** -63 * np.abs(np.array(positions, np.float64))[:, None, None]
        bound = (2.0 ** -8 + 2.0 ** -21) * np.abs(want) + 2.0 ** -21 * np.abs(want) + turn * np.abs(a) + 2.0 ** -50 * np.abs(a) * np.abs(angle)[:, None]
        assert np.all(np.abs(got - want) <= bound), f"{np.max(np.abs(got - want) / np.maximum(bound, 1e-300))} of the bound"
