"""Calls of many rows whose split items are neighbours: an item of 9, 17 or 65 and more shares ends in the range in which
the next split item starts.  Every row of every item against float64 (torch, on the GPU), with the bounds of
test_gpu_attention.py; the counters of the joins are checked after every call."""

import torch
import pytest

from tests.gpu_helpers import dev
from tests.test_attention_plan import NEIGHBOURS
from tests.test_gpu_attention import Case, run

pytestmark = pytest.mark.gpu


def reference(c, b):
    """Sequence b in float64: out, lse, sum_j p_j |v_j| and the largest scale * sum |q| |k| of each row."""
    n, length = c.lens[b]
    g, scale = c.heads // c.kv, c.dim ** -0.5
    q = c.q[int(c.cu[b]):int(c.cu[b + 1])].double()                          # [n, heads, dim]
    pages = torch.tensor(c.table[b, :-(-length // c.page)], device=dev()).long()
    hidden = torch.arange(length, device=dev()) > torch.arange(length - n, length, device=dev())[:, None]
    out, lse = torch.zeros_like(q), torch.zeros(n, c.heads, dtype=torch.float64, device=dev())
    spread, size = torch.zeros_like(q), torch.zeros_like(lse)
    for e in range(c.kv):
        k, v = [(p[pages, e].double() * (s[e].double() if c.fp8 else 1.0)).reshape(-1, c.dim)[:length]
                for p, s in zip(c.pools, c.scales)]
        for h in range(e * g, (e + 1) * g):
            s = (scale * (q[:, h] @ k.T)).masked_fill(hidden, float("-inf"))
            lse[:, h] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[:, h, None])
            out[:, h], spread[:, h] = p @ v, p @ v.abs()
            size[:, h] = (scale * (q[:, h].abs() @ k.abs().T)).masked_fill(hidden, 0.0).amax(-1)
    return out, lse, spread, size


def check(c, out, lse):
    weight = 2.0 ** (-11 if c.fp8 else -8)
    for b, (n, length) in enumerate(c.lens):
        at = slice(int(c.cu[b]), int(c.cu[b + 1]))
        want, wlse, spread, size = reference(c, b)
        delta = c.dim * 2.0 ** -22 * size
        bound = 2.0 ** -8 * want.abs() + spread * (weight + 2.0 * delta[..., None] + 2.0 ** -20 + length * 2.0 ** -22)
        assert bool(((out[at].double() - want).abs() <= bound).all()), f"sequence {b}"
        lbound = delta + 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -22 * wlse.abs()
        assert bool(((lse[at].double() - wlse).abs() <= lbound).all()), f"sequence {b}: lse"


@pytest.mark.parametrize("lens,heads,kv,dim,fp8,shares", NEIGHBOURS)
def test_neighbouring_split_items(lib, lens, heads, kv, dim, fp8, shares):
    c = Case(lens, heads, kv, dim, 64, fp8, seed=shares + dim)
    first = run(lib, c)
    check(c, *first)
    for _ in range(5):
        out, lse = torch.full_like(first[0], float("nan")), torch.full_like(first[1], float("nan"))
        lib.paged_attention(c.q, c.cache(), c.batch(), out=out, lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        for ws in lib._attention_ws.values():
            assert not ws[0][:4096].any()
    assert lib.device_error() == 0
