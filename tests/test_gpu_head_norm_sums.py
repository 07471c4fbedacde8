"""The weights' gradients of the norms, share by share: terms of one sign, so that a share that is lost, or counted twice, shows.

Tolerance.  Every addition's result is at most the whole sum, as all terms are positive, and each is rounded by 2^-24 of it.
A term comes through the additions of its thread's run (a block's units: all of them over 608 blocks, rounded up, at least
four), of the block's tokens at once, of every 32nd share, and of the 32 slices; and has 2^-18 of errors of its own."""

import numpy as np
import pytest
import torch

from tests.gpu_helpers import dev
from tests.test_gpu_head_norm import EPS
from tests.test_gpu_rope import heads

pytestmark = pytest.mark.gpu


def additions(tokens, n, kv, dim):
    lanes = 1
    while lanes < dim // 16:
        lanes *= 2
    at_once = 128 // lanes
    units = -(-tokens // at_once) * (n + kv)
    blocks = max(1, min(152 * 4, -(-units // 4)))
    return -(-units // blocks) + at_once + -(-blocks // 32) + 32


CASES = [(1, 1, 1, 64), (37, 5, 2, 128), (600, 3, 1, 256), (4099, 6, 2, 128), (1021, 7, 7, 64), (333, 33, 4, 96), (9001, 1, 0, 16),
         (2500, 16, 16, 512), (8191, 32, 8, 128)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,n,kv,dim", CASES)
def test_terms_of_one_sign(lib, tokens, n, kv, dim, interleaved):
    q, k = heads(tokens, n, dim, 1), heads(tokens, max(kv, 1), dim, 2)
    w = torch.ones(dim, dtype=torch.bfloat16, device=dev())
    if kv:
        _, _, dq_w, dk_w = lib.qk_norm_rope_backward(q, k, q, k, None, None, w, w, eps=EPS, interleaved=interleaved)
    else:
        _, _, dq_w, dk_w = lib.qk_norm_rope_backward(q, None, q, None, None, None, w, eps=EPS, interleaved=interleaved)
        assert dk_w is None
    bound = additions(tokens, n, kv, dim) * 2.0 ** -24 + 2.0 ** -18
    for x, got in ((q, dq_w), (k, dk_w)):
        if got is None:
            continue
        xf = x.double()
        want = (xf * xf * (xf.square().mean(-1, keepdim=True) + EPS).rsqrt()).sum((0, 1))
        worst = ((got.double() - want).abs() / want).max().item()
        assert worst <= bound, f"{worst / bound} of the bound"


@pytest.mark.parametrize("tokens,n,kv,dim", [(5, 2, 1, 128), (700, 3, 2, 128), (4099, 6, 2, 128)])
def test_single_terms_at_the_blocks_borders(lib, tokens, n, kv, dim):
    """One (token, head) has a gradient: its term is the whole sum.  The first and the last unit of blocks, those between the
    queries and the keys among them, and tokens that a block holds at once."""
    at_once = 128 // (dim // 16)
    steps = -(-tokens // at_once)
    units = steps * (n + kv)
    blocks = max(1, min(152 * 4, -(-units // 4)))
    per = -(-units // blocks)
    rng = np.random.default_rng(tokens)
    picked = {0, units - 1, steps * n - 1, steps * n} | {b * per + d for b in rng.integers(0, -(-units // per), 12).tolist() for d in (-1, 0)}
    q, k = heads(tokens, n, dim, 3), heads(tokens, kv, dim, 4)
    w = torch.ones(dim, dtype=torch.float32, device=dev())
    for unit in sorted(u for u in picked if 0 <= u < units):
        kind = 1 if unit >= steps * n else 0
        step, head = divmod(unit - kind * steps * n, (n, kv)[kind])
        for token in {min(step * at_once, tokens - 1), min(step * at_once + at_once - 1, tokens - 1)}:
            dy = [torch.zeros_like(q), torch.zeros_like(k)]
            x = (q, k)[kind][token, head].double()
            dy[kind][token, head] = 1.0
            got = lib.qk_norm_rope_backward(dy[0], dy[1], q, k, None, None, w, w, eps=EPS)
            want = x * (x.square().mean() + EPS).rsqrt()
            assert torch.all((got[2 + kind].double() - want).abs() <= 2.0 ** -18 * want.abs()), (unit, token)
            assert not got[3 - kind].any()
