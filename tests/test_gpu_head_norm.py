"""Norms of queries and keys with the rotation, forward, backward and on the way to a paged cache, against the float64
oracle.

Tolerances.  The sum of squares of a head takes at most 21 roundings (16 in a thread, 5 between lanes), 2^-19.6 of it;
its root halves that, and the reciprocal root adds 2^-22, the three products with r, the weight and cos or sin 2^-24
each, cos and sin themselves 2^-22, the sum of a pair 2^-24: together below 2^-19 of amplitude * (|n_a| + |n_b|), n the
normalised pair.  Then one rounding: 2^-8 of the value for bf16, 2^-4 or half the smallest step, 2^-10, for E4M3.
Backward: dx = r (z - xh m) has the same errors in r, z, xh, and m = mean(z xh) twice that of mean |z xh|: below 2^-18 of
r (|z| + |xh| mean |z xh|), where |z| is taken over the rotated pair.  The weights' gradients are fp32 sums of N =
tokens * heads products (each off by 2^-18 of its size): N * 2^-24 of the sum of their sizes at most."""

import math

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import step as OS
from tests.gpu_helpers import dev
from tests.test_gpu_rope import f64, heads, pair_size

pytestmark = pytest.mark.gpu

EPS = 1e-6


def weights(dim, kind, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return [(1.0 + 0.3 * torch.randn(dim, generator=g, device=dev())).to(kind) for _ in range(2)]


def sizes_of(n, rot, interleaved):
    """|a| + |b| of each value's pair; the value's own size past the rotated ones."""
    out = np.abs(n)
    if rot:
        out[..., :rot] = pair_size(n, rot // 2, rot, interleaved)[..., :rot]
    return out


def want_of(x, w, pos, freq, interleaved, amp, eps=EPS):
    """(normalised and rotated, bound before the last rounding)."""
    args = (f64(x), f64(w), pos.cpu().numpy(), freq.cpu().numpy() if freq is not None else np.zeros(0))
    n = OS.norm_rope(args[0], args[1], args[2], np.zeros(0), eps)
    rot = 2 * len(args[3])
    return OS.norm_rope(*args, eps, interleaved, amp), 2.0 ** -19 * max(amp, 1.0) * sizes_of(n, rot, interleaved)


def check(got, want, slack, what):
    err = np.abs(f64(got) - want)
    bound = 2.0 ** -8 * np.abs(want) + slack
    assert np.all(err <= bound), f"{what}: {np.max(err / np.maximum(bound, 1e-300))} of the bound"


CASES = [(1, 1, 1, 64, 64, 0, torch.bfloat16), (1, 7, 2, 128, 128, 2, torch.float32), (15, 16, 8, 128, 64, 8, torch.bfloat16),
         (33, 5, 5, 96, 48, 1, torch.float32), (7, 4, 1, 256, 256, 0, torch.bfloat16), (3, 3, 1, 80, 0, 1, torch.bfloat16),
         (40, 2, 2, 16, 16, 0, torch.float32), (5, 2, 1, 512, 512, 3, torch.bfloat16), (130, 33, 4, 64, 32, 0, torch.bfloat16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,n,kv,dim,rot,wide,kind", CASES)
def test_forward(lib, tokens, n, kv, dim, rot, wide, kind, interleaved):
    qkv = heads(tokens, n + kv, dim, 3 * tokens + dim, wide)
    q, k = qkv[:, :n], qkv[:, n:]
    qw, kw = weights(dim, kind, dim)
    pos = torch.arange(tokens, dtype=torch.int32, device=dev()) * 31 + 70000
    freq = lib.rope_frequencies(rot, 500000.0, device=dev()) if rot else None
    amp = 1.25 if tokens % 2 else 1.0
    qo, ko = lib.qk_norm_rope(q, k, pos if rot else None, freq, qw, kw, EPS, interleaved, amp)
    torch.cuda.synchronize()
    for got, x, w, what in ((qo, q, qw, "q"), (ko, k, kw, "k")):
        want, slack = want_of(x, w, pos, freq, interleaved, amp)
        check(got, want, slack, what)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,n,kv,dim,rot,wide,kind", CASES)
def test_backward(lib, tokens, n, kv, dim, rot, wide, kind, interleaved):
    qkv = heads(tokens, n + kv, dim, 5 * tokens + dim, wide)
    q, k = qkv[:, :n], qkv[:, n:]
    dq, dk = heads(tokens, n, dim, 6, wide), heads(tokens, kv, dim, 7)
    qw, kw = weights(dim, kind, dim + 1)
    pos = torch.arange(tokens, dtype=torch.int32, device=dev()) * 17 + 3
    freq = lib.rope_frequencies(rot, device=dev()) if rot else None
    amp = 1.25 if tokens % 2 else 1.0
    got = lib.qk_norm_rope_backward(dq, dk, q, k, pos if rot else None, freq, qw, kw, EPS, interleaved, amp)
    again = lib.qk_norm_rope_backward(dq, dk, q, k, pos if rot else None, freq, qw, kw, EPS, interleaved, amp)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for (dx, dw), dy, x, w in (((got[0], got[2]), dq, q, qw), ((got[1], got[3]), dk, k, kw)):
        args = (f64(dy), f64(x), f64(w), pos.cpu().numpy(), freq.cpu().numpy() if rot else np.zeros(0), EPS, interleaved, amp)
        want, want_w, _, size_w = OS.norm_rope_backward(*args)
        z = sizes_of(args[0], rot, interleaved) * max(amp, 1.0) * np.abs(args[2])
        r = 1.0 / np.sqrt((args[1] ** 2).mean(-1, keepdims=True) + EPS)
        unit = np.abs(args[1]) * r
        check(dx, want, 2.0 ** -18 * r * (z + unit * (z * unit).mean(-1, keepdims=True)), "dx")
        u = sizes_of(args[0], rot, interleaved) * max(amp, 1.0)
        bound = (x.shape[0] * x.shape[1] * 2.0 ** -24 + 2.0 ** -18) * (u * unit).sum((0, 1))
        worst = np.max(np.abs(f64(dw) - want_w) / bound)
        assert dw.dtype == torch.float32 and worst <= 1.0, f"weights: {worst} of the bound"
        assert (size_w <= (u * unit).sum((0, 1)) * (1 + 1e-9)).all()


def test_backward_against_differences(lib):
    """Every gradient against central differences of the oracle's forward pass."""
    tokens, n, dim, rot = 2, 2, 32, 16
    x, c = heads(tokens, n, dim, 1), heads(tokens, n, dim, 2)
    (w, _), pos = weights(dim, torch.float32, 4), np.array([3, 901])
    freq = lib.rope_frequencies(rot)
    dx, none, dw, none_w = lib.qk_norm_rope_backward(c, None, x, None, torch.tensor(pos, dtype=torch.int32, device=dev()),
                                                     freq.to(dev()), w, eps=EPS, interleaved=True, amplitude=1.5)
    assert none is None and none_w is None
    xf, cf, wf, h = f64(x), f64(c), f64(w), 1e-5
    f = lambda a, b: (cf * OS.norm_rope(a, b, pos, freq.numpy(), EPS, True, 1.5)).sum()  # noqa: E731
    top = 1.5 * np.abs(cf).max() * np.abs(wf).max() / np.sqrt((xf ** 2).mean(-1).min())
    for idx in np.ndindex(xf.shape):
        up, down = xf.copy(), xf.copy()
        up[idx] += h
        down[idx] -= h
        d = (f(up, wf) - f(down, wf)) / (2 * h)
        # differences are off by h^2 of a third derivative and 2^-52 / h of the sum: below 1e-8 here
        assert abs(f64(dx)[idx] - d) <= 2.0 ** -8 * abs(d) + 2.0 ** -16 * top + 1e-7
    for i in range(dim):
        up, down = wf.copy(), wf.copy()
        up[i] += h
        down[i] -= h
        assert abs(f64(dw)[i] - (f(xf, up) - f(xf, down)) / (2 * h)) <= 2.0 ** -16 * 1.5 * np.abs(cf).max() * 4 * tokens * n + 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_more_tokens_than_one_round_of_blocks(lib, interleaved):
    """Every token of a long call, against torch in fp64 (the oracle walks tokens one by one)."""
    tokens, n, kv, dim, rot = 4099, 6, 2, 128, 64
    q, k, dq, dk = (heads(tokens, m, dim, s, 1) for m, s in ((n, 1), (kv, 2), (n, 3), (kv, 4)))
    qw, kw = weights(dim, torch.bfloat16, 9)
    pos = torch.randint(0, 1 << 17, (tokens,), device=dev()).to(torch.int32)
    freq = lib.rope_frequencies(rot, device=dev())
    qo, ko = lib.qk_norm_rope(q, k, pos, freq, qw, kw, EPS, interleaved)
    got = lib.qk_norm_rope_backward(dq, dk, q, k, pos, freq, qw, kw, EPS, interleaved)

    def turned(x, sign):
        a = (pos.double()[:, None] * freq)[:, None, :] * sign
        lo, hi = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
        y = x.clone()
        u, v = lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()
        if interleaved:
            y[..., 0:rot:2], y[..., 1:rot:2] = u, v
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = u, v
        return y

    for x, w, y, dy, dx, dw in ((q, qw, qo, dq, got[0], got[2]), (k, kw, ko, dk, got[1], got[3])):
        xf, wf = x.double(), w.double()
        r = (xf.square().mean(-1, keepdim=True) + EPS).rsqrt()
        nn = xf * r * wf
        check(y, f64(turned(nn, 1)), 2.0 ** -19 * sizes_of(f64(nn), rot, interleaved), "y")
        u = turned(dy.double(), -1)
        z, unit = u * wf, xf * r
        size = torch.from_numpy(sizes_of(f64(dy), rot, interleaved)).to(dev())
        zs = size * wf.abs()
        slack = 2.0 ** -18 * r * (zs + unit.abs() * (zs * unit.abs()).mean(-1, keepdim=True))
        check(dx, f64(r * (z - unit * (z * unit).mean(-1, keepdim=True))), f64(slack), "dx")
        bound = (tokens * x.shape[1] * 2.0 ** -24 + 2.0 ** -18) * (size * unit.abs()).sum((0, 1))
        assert torch.all((dw.double() - (u * unit).sum((0, 1))).abs() <= bound), "weights"


def test_in_place_strided_outputs_and_queries_alone(lib):
    tokens, n, kv, dim = 19, 6, 2, 128
    q, k = heads(tokens, n, dim, 3, wide=2), heads(tokens, kv, dim, 4)
    dq, dk = heads(tokens, n, dim, 5), heads(tokens, kv, dim, 6, wide=1)
    qw, kw = weights(dim, torch.bfloat16, 1)
    pos = torch.arange(tokens, dtype=torch.int32, device=dev())
    freq = lib.rope_frequencies(dim, device=dev())
    qo, ko = lib.qk_norm_rope(q, k, pos, freq, qw, kw)
    alone, none = lib.qk_norm_rope(q, None, pos, freq, qw)
    assert none is None and torch.equal(alone, qo)
    buf = torch.full((tokens, n + 3, dim), 7.0, dtype=torch.bfloat16, device=dev())
    out, _ = lib.qk_norm_rope(q, k, pos, freq, qw, kw, q_out=buf[:, 1:n + 1])
    assert torch.equal(out, qo) and torch.all(buf[:, 0] == 7.0) and torch.all(buf[:, n + 1:] == 7.0)
    back = lib.qk_norm_rope_backward(dq, dk, q, k, pos, freq, qw, kw)
    dq2, dk2 = dq.clone(), dk.clone()
    got = lib.qk_norm_rope_backward(dq2, dk2, q, k, pos, freq, qw, kw, dq_out=dq2, dk_out=dk2)
    assert got[0] is dq2 and all(torch.equal(a, b) for a, b in zip(got, back))
    q2, k2 = q.clone(), k.clone()
    got = lib.qk_norm_rope_backward(dq, dk, q2, k2, pos, freq, qw, kw, dq_out=q2, dk_out=k2)
    assert got[0] is q2 and all(torch.equal(a, b) for a, b in zip(got, back))
    z, y = q.clone(), k.clone()
    a, b = lib.qk_norm_rope(z, y, pos, freq, qw, kw, q_out=z, k_out=y)
    assert a is z and b is y and torch.equal(z, qo) and torch.equal(y, ko)


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e18, 1e30, 3e38])
def test_heads_of_every_size(lib, size):
    """Squares that overflow or vanish in fp32: without eps the result does not depend on the size."""
    tokens, n, dim = 3, 2, 64
    x, c = heads(tokens, n, dim, 8).clamp(-1.0, 1.0), heads(tokens, n, dim, 9)
    x = (x.double() * size).to(torch.bfloat16)
    w, _ = weights(dim, torch.float32, 2)
    pos = torch.arange(tokens, dtype=torch.int32, device=dev())
    freq = lib.rope_frequencies(dim, device=dev())
    y, _ = lib.qk_norm_rope(x, None, pos, freq, w, eps=0.0)
    want, slack = want_of(x, w, pos, freq, False, 1.0, 0.0)
    check(y, want, slack, "y")
    dx, _, dw, _ = lib.qk_norm_rope_backward(c, None, x, None, pos, freq, w, eps=0.0)
    _, want_w, _, size_w = OS.norm_rope_backward(f64(c), f64(x), f64(w), pos.cpu().numpy(), freq.cpu().numpy(), 0.0)
    assert np.all(np.abs(f64(dw) - want_w) <= 2.0 ** -16 * (size_w + np.abs(f64(c)).sum((0, 1))) * 4)
    if 1e-20 < size < 1e20:  # (elsewhere dx = ... / x leaves bf16's range or its normal numbers)
        want = OS.norm_rope_backward(f64(c), f64(x), f64(w), pos.cpu().numpy(), freq.cpu().numpy(), 0.0)[0]
        r = 1.0 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True))
        z = sizes_of(f64(c), dim, False) * np.abs(f64(w))
        check(dx, want, 2.0 ** -18 * r * (z + np.abs(f64(x)) * r * (z * np.abs(f64(x)) * r).mean(-1, keepdims=True)), "dx")


def test_zeros_infinities_and_nan_stay_in_their_heads(lib):
    tokens, n, dim = 4, 3, 64
    x = heads(tokens, n, dim, 8)
    x[0, 0] = 0.0
    x[1, 1, 5] = float("inf")
    x[2, 2, 7] = float("nan")
    w, _ = weights(dim, torch.bfloat16, 2)
    y, _ = lib.qk_norm_rope(x, None, None, None, w)
    assert torch.all(y[0, 0] == 0.0)
    other = torch.arange(dim, device=dev()) != 5
    assert torch.isnan(y[1, 1, 5]) and torch.all(y[1, 1][other] == 0.0)
    assert torch.isnan(y[2, 2]).all()
    left = torch.ones(tokens, n, dtype=torch.bool, device=dev())
    left[1, 1] = left[2, 2] = False
    assert torch.isfinite(y[left]).all()
    none, _ = lib.qk_norm_rope(x[:0], None, None, None, w)
    assert none.shape == (0, n, dim)
    _, _, dw, _ = lib.qk_norm_rope_backward(x[:0], None, x[:0], None, None, None, w)
    assert torch.all(dw == 0.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,n,kv,dim,rot,page,kind", [
    (1, 4, 1, 64, 64, 16, torch.bfloat16), (16, 16, 8, 128, 128, 64, torch.float32), (37, 6, 2, 256, 128, 32, torch.bfloat16),
    (300, 7, 7, 64, 32, 128, torch.float32), (5, 3, 3, 128, 0, 256, torch.bfloat16), (6, 0, 2, 128, 128, 16, torch.bfloat16)])
def test_append(lib, fp8, tokens, n, kv, dim, rot, page, kind, interleaved):
    g = torch.Generator(device=dev()).manual_seed(77 + tokens)
    pages = -(-tokens // page) + 2
    row = heads(tokens, n + 2 * kv, dim, 21 + tokens)
    q, k, v = row[:, :n] if n else None, row[:, n:n + kv], row[:, n + kv:]
    pool = torch.randn(pages, 2, kv, page, dim, generator=g, device=dev()).to(torch.bfloat16)  # k and v in one pool
    ks = vs = None
    if fp8:
        pool = pool.to(torch.float8_e4m3fn)
        ks = torch.rand(kv, generator=g, device=dev()) * 0.02 + 0.001   # some values saturate
        vs = torch.rand(kv, generator=g, device=dev()) * 0.02 + 0.01
    before = pool.float().cpu().numpy().astype(np.float64)
    cache = binding.KVCache(pool[:, 0], pool[:, 1], ks, vs)
    slots = torch.randperm(pages * page, generator=g, device=dev())[:tokens]
    if tokens > 2:
        slots[tokens // 2] = -1
    pos = torch.randint(0, 100000, (tokens,), generator=g, device=dev()).to(torch.int32)
    freq = lib.rope_frequencies(rot, device=dev()) if rot else None
    qw, kw = weights(dim, kind, dim + 3)
    out = lib.kv_append(cache, k, v, slots, pos if rot else None, freq, interleaved, 1.1, q=q, q_norm=qw if n else None,
                        k_norm=kw, eps=EPS)
    torch.cuda.synchronize()
    assert lib.device_error() == 0
    if n:
        check(out, *want_of(q, qw, pos, freq, interleaved, 1.1), "q")
    else:
        assert out is None
    after = pool.float().cpu().numpy().astype(np.float64)
    want = before.copy()
    s = slots.cpu().numpy()
    wk, slack_k = want_of(k, kw, pos, freq, interleaved, 1.1)
    for which, (rows, slack, scale) in enumerate(((wk, slack_k, ks), (f64(v), np.zeros(v.shape), vs))):
        if fp8:
            sc = scale.cpu().numpy().astype(np.float64)[:, None]
            rows, slack = rows / sc, slack / sc + 2.0 ** -23 * np.abs(rows / sc)
        for t in range(tokens):
            if s[t] < 0:
                continue
            got = after[s[t] // page, which, :, s[t] % page]
            r = np.clip(rows[t], -448.0, 448.0) if fp8 else rows[t]
            half = np.maximum(2.0 ** -4 * np.abs(r), 2.0 ** -10) if fp8 else 2.0 ** -8 * np.abs(r)
            assert np.all(np.abs(got - r) <= half + slack[t] * (1 + 2.0 ** -4)), (which, t)
            want[s[t] // page, which, :, s[t] % page] = got
    assert np.array_equal(after, want), "a slot that no token has was written"


def test_append_reports_slots_outside_the_pool(lib):
    kv, dim, page = 1, 64, 16
    pools = torch.zeros(2, 3, kv, page, dim, dtype=torch.bfloat16, device=dev())
    k, (w, _) = heads(4, kv, dim, 1), weights(dim, torch.bfloat16, 1)
    slots = torch.tensor([0, 3 * page, -5, 1 << 40], device=dev())
    assert lib.device_error() == 0
    lib.kv_append(binding.KVCache(pools[0], pools[1]), k, k, slots, k_norm=w)
    torch.cuda.synchronize()
    assert lib.device_error() == 4
    assert torch.count_nonzero(pools[1]) == torch.count_nonzero(k[0])


def test_binding_refuses(lib):
    kv, dim, page = 2, 64, 16
    pool = torch.zeros(2, 3, kv, page, dim, dtype=torch.bfloat16, device=dev())
    cache = binding.KVCache(pool[0], pool[1])
    x, (w, _) = heads(4, kv, dim, 1), weights(dim, torch.bfloat16, 1)
    pos, f, slots = torch.arange(4, dtype=torch.int32, device=dev()), lib.rope_frequencies(64, device=dev()), torch.arange(4, device=dev())
    for bad in (lambda: lib.qk_norm_rope(x.float(), x, pos, f, w, w), lambda: lib.qk_norm_rope(x, x[:3], pos, f, w, w),
                lambda: lib.qk_norm_rope(x, x, pos.long(), f, w, w), lambda: lib.qk_norm_rope(x, x, None, f, w, w),
                lambda: lib.qk_norm_rope(x, x, pos, f, w[:32], w), lambda: lib.qk_norm_rope(x, x, pos, f, w, w.float()),
                lambda: lib.qk_norm_rope(x, x, pos, f, w.half(), w.half()), lambda: lib.qk_norm_rope(x, x, pos, f, w.cpu(), w),
                lambda: lib.qk_norm_rope(x, None, pos, f, None), lambda: lib.qk_norm_rope(x, None, pos, f, w, k_out=x),
                lambda: lib.qk_norm_rope(x, x, pos, f, w, w, q_out=x[:3]), lambda: lib.qk_norm_rope(x.cpu(), None, pos, f, w),
                lambda: lib.qk_norm_rope(x.transpose(0, 1), None, None, None, w),
                lambda: lib.qk_norm_rope_backward(x[:3], None, x, None, pos, f, w),
                lambda: lib.qk_norm_rope_backward(x, x, x, None, pos, f, w, w),
                lambda: lib.qk_norm_rope_backward(x, x[:, :1], x, x, pos, f, w, w),
                lambda: lib.kv_append(cache, x, x, slots, k_norm=w[:32]), lambda: lib.kv_append(cache, x, x, slots, q_norm=w),
                lambda: lib.kv_append(cache, x, x, slots, q=x, k_norm=w), lambda: lib.kv_append(cache, x, x, slots, q_norm=w, k_norm=w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.qk_norm_rope(x, x, pos, f, w), lambda: lib.qk_norm_rope(x, None, pos, f, w, eps=-1.0),
                lambda: lib.qk_norm_rope(x, None, pos, f, w, eps=math.nan),
                lambda: lib.qk_norm_rope(x, None, pos, lib.rope_frequencies(128, device=dev()), w)):
        with pytest.raises(binding.NVFP4Error):
            bad()
