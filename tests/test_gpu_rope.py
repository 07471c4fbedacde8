"""Rotary positions and the append to a paged cache on the GPU, against the float64 oracle.

Tolerances.  A rotated value is a fp32 combination a c - b s (error of the angle, of cos and sin, two products and a
sum: below 2^-21 of amplitude * (|a| + |b|) together), rounded once: 2^-8 of it for bf16; for E4M3 2^-4, or half the
smallest step, 2^-10, near zero.  Values that nothing turns are bit-exact in bf16."""

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import attention as OA
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -21


def heads(tokens, n, dim, seed, wide=0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randn(tokens, n + wide, dim, generator=g, device=dev()).to(torch.bfloat16)[:, :n]


def f64(t):
    return t.double().cpu().numpy()


def positions_of(kind, tokens, seed):
    rng = np.random.default_rng(seed)
    if kind == "near":
        return np.arange(tokens)
    if kind == "far":
        return rng.integers(1 << 20, (1 << 31) - 1, tokens)
    return rng.integers(-1000, 1000, tokens)


def pair_size(x, half, rot, interleaved):
    """|a| + |b| of each value's pair."""
    a = np.abs(x)
    out = np.zeros_like(a)
    if interleaved:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = s, s
    else:
        s = a[..., :half] + a[..., half:rot]
        out[..., :half], out[..., half:rot] = s, s
    return out


def check_rotated(got, x, want, rot, interleaved, amplitude, what):
    bound = 2.0 ** -8 * np.abs(want) + F32 * amplitude * pair_size(x, rot // 2, rot, interleaved)
    err = np.abs(got - want)
    assert np.all(err <= bound), f"{what}: {np.max(err - bound)} over the bound"
    assert np.array_equal(got[..., rot:], x[..., rot:]), f"{what}: the rest of a head changed"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,n,dim,rot,wide,kind", [
    (1, 1, 16, 16, 0, "near"), (1, 7, 64, 64, 0, "far"), (15, 16, 128, 128, 8, "any"), (33, 5, 128, 64, 3, "near"),
    (7, 2, 256, 96, 0, "far"), (3, 3, 80, 48, 1, "any"), (700, 9, 64, 32, 2, "near"), (2, 1, 512, 512, 0, "near")])
def test_rope_matches_the_oracle(lib, tokens, n, dim, rot, wide, kind, interleaved):
    x = heads(tokens, n, dim, 10 + tokens, wide)
    pos = positions_of(kind, tokens, 5)
    w = lib.rope_frequencies(rot, 500000.0, 8.0, 8192.0)
    amp = 1.25 if tokens % 2 else 1.0
    y = lib.rope_apply(x, torch.tensor(pos, dtype=torch.int32, device=dev()), w.to(dev()), interleaved, amp)
    xf = f64(x)
    step = max(1, tokens // 40)       # the oracle walks tokens one by one
    at = np.unique(np.r_[0:tokens:step, tokens - 1])
    want = OA.rotate(xf[at], pos[at], w.numpy(), interleaved, amp)
    check_rotated(f64(y)[at], xf[at], want, rot, interleaved, amp, "rope")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place_inverse_and_strided_output(lib, interleaved):
    tokens, n, dim, rot = 19, 6, 128, 96
    x = heads(tokens, n, dim, 3, wide=2)
    pos = torch.arange(1000, 1000 + tokens, dtype=torch.int32, device=dev())
    w = lib.rope_frequencies(rot, device=dev())
    y = lib.rope_apply(x, pos, w, interleaved)
    back = lib.rope_apply(y, pos, w, interleaved, inverse=True)
    want = OA.rotate(f64(y), pos.cpu().numpy(), w.cpu().numpy(), interleaved, inverse=True)
    check_rotated(f64(back), f64(y), want, rot, interleaved, 1.0, "inverse")
    buf = torch.full((tokens, n + 3, dim), 7.0, dtype=torch.bfloat16, device=dev())
    out = lib.rope_apply(x, pos, w, interleaved, out=buf[:, 1:n + 1])
    assert torch.equal(out, y) and torch.all(buf[:, 0] == 7.0) and torch.all(buf[:, n + 1:] == 7.0)
    z = x.clone()
    assert lib.rope_apply(z, pos, w, interleaved, out=z) is z and torch.equal(z, y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_inverse_is_the_gradient(lib, interleaved):
    """d <c, rope(x)> / dx = rope^-1(c) * amplitude: against central differences of the oracle."""
    tokens, n, dim, rot = 2, 1, 32, 16
    x, c = heads(tokens, n, dim, 1), heads(tokens, n, dim, 2)
    pos = np.array([3, 901])
    w = lib.rope_frequencies(rot)
    got = f64(lib.rope_apply(c, torch.tensor(pos, dtype=torch.int32, device=dev()), w.to(dev()), interleaved, 1.5,
                             inverse=True))
    xf, cf, h = f64(x), f64(c), 1e-4
    for idx in np.ndindex(xf.shape):
        up, down = xf.copy(), xf.copy()
        up[idx] += h
        down[idx] -= h
        d = (cf * (OA.rotate(up, pos, w.numpy(), interleaved, 1.5) - OA.rotate(down, pos, w.numpy(), interleaved, 1.5))).sum() / (2 * h)
        # the rotation is linear: the difference is exact to its own 1e-16 / h
        assert abs(got[idx] - d) <= 2.0 ** -8 * abs(d) + F32 * 1.5 * 2 * np.abs(cf).max() + 1e-9


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,n,kv,dim,rot,page,interleaved", [
    (1, 4, 1, 64, 64, 16, False), (16, 16, 8, 128, 128, 64, False), (37, 6, 2, 256, 128, 32, True),
    (300, 7, 7, 64, 32, 128, False), (5, 3, 3, 128, 0, 256, False)])
def test_append_matches_the_oracle(lib, fp8, tokens, n, kv, dim, rot, page, interleaved):
    g = torch.Generator(device=dev()).manual_seed(77 + tokens)
    pages = -(-tokens // page) + 2
    row = heads(tokens, n + 2 * kv, dim, 21 + tokens)
    q, k, v = row[:, :n], row[:, n:n + kv], row[:, n + kv:]
    pool = torch.randn(pages, 2, kv, page, dim, generator=g, device=dev()).to(torch.bfloat16)  # k and v in one pool
    ks = vs = None
    if fp8:
        pool = pool.to(torch.float8_e4m3fn)
        ks = torch.rand(kv, generator=g, device=dev()) * 0.02 + 0.001   # some values saturate
        vs = torch.rand(kv, generator=g, device=dev()) * 0.02 + 0.01
    before = pool.float().cpu().numpy().astype(np.float64)
    cache = binding.KVCache(pool[:, 0], pool[:, 1], ks, vs)
    slots = torch.randperm(pages * page, generator=g, device=dev())[:tokens]
    skipped = tokens // 2 if tokens > 2 else -1
    if skipped >= 0:
        slots[skipped] = -1
    pos = torch.randint(0, 100000, (tokens,), generator=g, device=dev()).to(torch.int32)
    w = lib.rope_frequencies(rot) if rot else None
    out = lib.kv_append(cache, k, v, slots, pos if rot else None, w.to(dev()) if rot else None, interleaved, 1.1, q=q)
    torch.cuda.synchronize()
    assert lib.device_error() == 0
    turn = lambda x: OA.rotate(f64(x), pos.cpu().numpy(), w.numpy(), interleaved, 1.1) if rot else f64(x)  # noqa: E731
    check_rotated(f64(out), f64(q), turn(q), rot, interleaved, 1.1, "q")
    after = pool.float().cpu().numpy().astype(np.float64)
    want = before.copy()
    s = slots.cpu().numpy()
    for which, (x, scale) in enumerate(((k, ks), (v, vs))):
        rows = turn(x) if which == 0 else f64(x)
        slack = F32 * 1.1 * pair_size(f64(x), rot // 2, rot, interleaved) if which == 0 else np.zeros_like(rows)
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


def test_append_without_queries_and_in_place(lib):
    tokens, kv, dim, page = 9, 2, 64, 16
    k, v, q = heads(tokens, kv, dim, 1), heads(tokens, kv, dim, 2), heads(tokens, 4, dim, 3)
    pools = torch.zeros(2, 2, kv, page, dim, dtype=torch.bfloat16, device=dev())
    slots = torch.arange(3, 3 + tokens, device=dev())
    pos = torch.arange(tokens, dtype=torch.int32, device=dev())
    w = lib.rope_frequencies(dim, device=dev())
    assert lib.kv_append(binding.KVCache(pools[0], pools[1]), k, v, slots, pos, w) is None
    assert torch.equal(pools[1][0, :, 3:3 + tokens].transpose(0, 1), v)
    assert torch.equal(pools[0][0, :, 3:3 + tokens].transpose(0, 1), lib.rope_apply(k, pos, w))
    want = lib.rope_apply(q, pos, w)
    assert lib.kv_append(binding.KVCache(pools[0], pools[1]), k, v, slots, pos, w, q=q, q_out=q) is q
    assert torch.equal(q, want)


def test_append_reports_slots_outside_the_pool(lib):
    kv, dim, page = 1, 64, 16
    pools = torch.zeros(2, 3, kv, page, dim, dtype=torch.bfloat16, device=dev())
    k = heads(4, kv, dim, 1)
    slots = torch.tensor([0, 3 * page, -5, 1 << 40], device=dev())
    assert lib.device_error() == 0
    lib.kv_append(binding.KVCache(pools[0], pools[1]), k, k, slots)
    torch.cuda.synchronize()
    assert lib.device_error() == 4
    assert lib.device_error() == 0
    assert torch.equal(pools[0][0, 0, 0], k[0, 0]) and torch.count_nonzero(pools[0]) == torch.count_nonzero(k[0])


def test_special_values_reach_the_cache(lib):
    """Infinities and NaN: kept in bf16; in E4M3 an infinity saturates (448) and NaN stays NaN."""
    kv, dim, page = 1, 64, 16
    x = heads(1, kv, dim, 4)
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2] = float("inf"), float("-inf"), float("nan")
    slots = torch.zeros(1, dtype=torch.int64, device=dev())
    pools = torch.zeros(2, 1, kv, page, dim, dtype=torch.bfloat16, device=dev())
    lib.kv_append(binding.KVCache(pools[0], pools[1]), x, x, slots)
    assert torch.equal(pools[0][0, 0, 0].view(torch.int16), x[0, 0].view(torch.int16))
    p8 = torch.zeros(2, 1, kv, page, dim, device=dev()).to(torch.float8_e4m3fn)
    lib.kv_append(binding.KVCache(p8[0], p8[1]), x, x, slots)
    got = p8[0][0, 0, 0].float()
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and torch.isfinite(got[3:]).all()


def test_binding_refuses(lib):
    kv, dim, page = 2, 64, 16
    pool = torch.zeros(2, 3, kv, page, dim, dtype=torch.bfloat16, device=dev())
    cache = binding.KVCache(pool[0], pool[1])
    x = heads(4, kv, dim, 1)
    pos, w, slots = torch.arange(4, dtype=torch.int32, device=dev()), lib.rope_frequencies(64, device=dev()), torch.arange(4, device=dev())
    for bad in (lambda: lib.rope_apply(x.float(), pos, w), lambda: lib.rope_apply(x, pos.long(), w),
                lambda: lib.rope_apply(x, pos[:3], w), lambda: lib.rope_apply(x, pos, w.float()),
                lambda: lib.rope_apply(x.transpose(0, 1), pos, w), lambda: lib.rope_apply(x[..., :32], pos, w),
                lambda: lib.kv_append(cache, x, x[:3], slots), lambda: lib.kv_append(cache, x, x, slots.int()),
                lambda: lib.kv_append(cache, x, x, slots, None, w), lambda: lib.kv_append(cache, x[:, :1], x[:, :1], slots),
                lambda: binding.KVCache(pool[0], pool[1].float()), lambda: binding.KVCache(pool[0].transpose(1, 2), pool[1].transpose(1, 2)),
                lambda: binding.KVCache(pool[0].cpu(), pool[1].cpu()), lambda: binding.KVCache(pool[0], pool[1][:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.NVFP4Error):
        lib.rope_apply(x, pos, lib.rope_frequencies(128, device=dev()))   # rotates more than a head
