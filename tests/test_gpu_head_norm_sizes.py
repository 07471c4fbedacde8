"""Norms of heads and weights of opposite sizes: a product of a value and its weight, or of a gradient, its weight and its value,
may leave fp32's range where the normalised result does not.  The tolerances are those of tests/test_gpu_head_norm.py: the
products have the normalised value for a factor, so their sizes are the results', and the roundings are as many."""

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import step as OS
from tests.gpu_helpers import dev
from tests.test_gpu_head_norm import check, sizes_of, want_of, weights
from tests.test_gpu_rope import f64, heads

pytestmark = pytest.mark.gpu

# sizes of x, of the weights and of the gradient: x w and x w dy overflow, or vanish
SIZES = [(1e17, 1e25, 1e-6), (1e-14, 1e-28, 1e6), (1e17, 1e-20, 1e22), (1e-14, 1e10, 1e-36), (1e17, 1e12, 1e12), (1e-14, 1e-12, 1e-15),
         (1e-39, 1.0, 1e-12), (1e37, 1.0, 1e12)]


def sized(tokens, n, dim, seed, size):
    x = heads(tokens, n, dim, seed).double()
    return (x.sign() * x.abs().clamp(0.25, 1.0) * size).to(torch.bfloat16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("x_size,w_size,dy_size", SIZES)
def test_forward_and_backward(lib, x_size, w_size, dy_size, rot, interleaved):
    tokens, n, dim = 5, 3, 64
    x, dy = sized(tokens, n, dim, 1, x_size), sized(tokens, n, dim, 2, dy_size)
    w = (weights(dim, torch.float32, 3)[0].double() * w_size).float()
    pos = torch.arange(tokens, dtype=torch.int32, device=dev()) * 7
    freq = lib.rope_frequencies(rot, device=dev()) if rot else None
    y, _ = lib.qk_norm_rope(x, None, pos, freq, w, eps=0.0, interleaved=interleaved)
    want, slack = want_of(x, w, pos, freq, interleaved, 1.0, 0.0)
    check(y, want, slack, "y")
    dx, _, dw, _ = lib.qk_norm_rope_backward(dy, None, x, None, pos, freq, w, eps=0.0, interleaved=interleaved)
    args = (f64(dy), f64(x), f64(w), pos.cpu().numpy(), freq.cpu().numpy() if rot else np.zeros(0), 0.0, interleaved)
    want, want_w, _, _ = OS.norm_rope_backward(*args)
    r = 1.0 / np.sqrt((args[1] ** 2).mean(-1, keepdims=True))
    u = sizes_of(args[0], rot, interleaved)
    z, unit = u * np.abs(args[2]), np.abs(args[1]) * r
    check(dx, want, 2.0 ** -18 * r * (z + unit * (z * unit).mean(-1, keepdims=True)), "dx")
    assert np.all(np.abs(f64(dw) - want_w) <= (tokens * n * 2.0 ** -24 + 2.0 ** -18) * (u * unit).sum((0, 1)))


@pytest.mark.parametrize("x_size,w_size", [(1e17, 1e25), (1e-14, 1e-28)])
def test_append(lib, x_size, w_size):
    tokens, kv, dim, page = 7, 2, 128, 16
    k = sized(tokens, kv, dim, 4, x_size)
    w = (weights(dim, torch.float32, 5)[0].double() * w_size).float()
    pool = torch.zeros(2, 1, kv, page, dim, dtype=torch.bfloat16, device=dev())
    slots = torch.arange(tokens, device=dev())
    lib.kv_append(binding.KVCache(pool[0], pool[1]), k, k, slots, k_norm=w, eps=0.0)
    pos = torch.zeros(tokens, dtype=torch.int32, device=dev())
    check(pool[0, 0, :, :tokens].transpose(0, 1), *want_of(k, w, pos, None, False, 1.0, 0.0), "k")
