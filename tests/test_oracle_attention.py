"""Pins of the attention-side oracle (CPU): closed forms of the rotation and of the stretched frequencies, and
attention against scipy's softmax, one-hot limits and the masks' definitions."""

import numpy as np
import pytest
from scipy.special import log_softmax, logsumexp

from oracle import attention as OA


def test_frequencies_closed_forms():
    w = OA.rope_frequencies(64, 10000.0)
    assert w[0] == 1.0 and w[16] == pytest.approx(0.01, rel=1e-14) and len(w) == 32
    assert np.allclose(OA.rope_frequencies(64, 10000.0, factor=4.0), w / 4.0, rtol=1e-15)
    s = OA.rope_frequencies(64, 10000.0, factor=8.0, trained_context=4096.0)
    turns = 4096.0 * w / (2 * np.pi)
    assert np.allclose(s[turns >= 32], w[turns >= 32], rtol=1e-15)
    assert np.allclose(s[turns <= 1], w[turns <= 1] / 8.0, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(s[mid] < w[mid]) and np.all(s[mid] > w[mid] / 8.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_properties(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 48))
    w = OA.rope_frequencies(32, 10000.0)
    pos = [0, 1, 7, 1000, -3]
    y = OA.rotate(x, pos, w, interleaved, amplitude=1.5)
    assert np.allclose(y[0, :, :32], 1.5 * x[0, :, :32]) and np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose((y[..., :32] ** 2).sum(-1), 2.25 * (x[..., :32] ** 2).sum(-1))
    back = OA.rotate(OA.rotate(x, pos, w, interleaved), pos, w, interleaved, inverse=True)
    assert np.allclose(back, x)
    # only the distance between two positions matters to a product
    a, b = x[:1], x[1:2]
    d1 = (OA.rotate(a, [10], w, interleaved) * OA.rotate(b, [4], w, interleaved)).sum(-1)
    d2 = (OA.rotate(a, [106], w, interleaved) * OA.rotate(b, [100], w, interleaved)).sum(-1)
    assert np.allclose(d1, d2)
    lo, hi = (0, 1) if interleaved else (0, 16)
    assert y[1, 0, lo] == pytest.approx(1.5 * (x[1, 0, lo] * np.cos(1) - x[1, 0, hi] * np.sin(1)))


@pytest.mark.parametrize("window,softcap", [(0, 0.0), (3, 0.0), (0, 5.0), (1, 2.0)])
def test_attention_against_scipy(window, softcap):
    rng = np.random.default_rng(8)
    n, heads, kv, dim, length = 5, 4, 2, 8, 9
    q, k, v = rng.standard_normal((n, heads, dim)), rng.standard_normal((length, kv, dim)), rng.standard_normal((length, kv, dim))
    out, lse, spread, _ = OA.attention(q, k, v, length - n, 0.3, softcap, window)
    for i in range(n):
        for h in range(heads):
            s = 0.3 * k[:, h // 2] @ q[i, h]
            s = softcap * np.tanh(s / softcap) if softcap else s
            j = np.arange(length)
            p = length - n + i
            s = np.where((j <= p) & ((window == 0) | (j > p - window)), s, -np.inf)
            assert lse[i, h] == pytest.approx(logsumexp(s))
            e = np.exp(log_softmax(s))
            assert np.allclose(out[i, h], e @ v[:, h // 2]) and np.allclose(spread[i, h], e @ np.abs(v[:, h // 2]))
    if window == 1:
        assert np.allclose(out, np.repeat(v[length - n:], 2, axis=1))


def test_attention_empty_and_hidden():
    rng = np.random.default_rng(9)
    q, k, v = rng.standard_normal((4, 2, 8)), rng.standard_normal((2, 1, 8)), rng.standard_normal((2, 1, 8))
    out, lse, _, _ = OA.attention(q, k, v, -2, 1.0)      # two tokens before the first key
    assert np.all(out[:2] == 0) and np.all(lse[:2] == -np.inf) and np.allclose(out[2], v[0]) and np.isfinite(lse[2:]).all()
    v[1] = np.nan                                        # a key that token 2 does not see
    again, _, _, _ = OA.attention(q, k, v, -2, 1.0)
    assert np.allclose(again[:3], out[:3]) and np.isnan(again[3]).all()
