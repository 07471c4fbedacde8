"""Pins of the oracle of norms, steps and trees (CPU): closed forms, differences, the causal oracle, brute force."""

import numpy as np
import pytest

from oracle import attention as OA
from oracle import step as OS


def test_a_normalised_head_has_unit_mean_square():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 48)) * 7.0
    n = OS.norm_rope(x, np.ones(48), [0, 5, 9], np.zeros(0), 0.0)
    assert np.allclose((n ** 2).mean(-1), 1.0) and np.allclose(n * np.sqrt((x ** 2).mean(-1, keepdims=True)), x)
    # eps is added to the mean square; weights multiply; the rotation comes after them
    assert np.allclose(OS.norm_rope(np.full((1, 1, 4), 3.0), np.arange(4.0), [0], np.zeros(0), 7.0), 0.75 * np.arange(4.0))
    w = rng.standard_normal(48)
    f = OA.rope_frequencies(32, 10000.0)
    assert np.allclose(OS.norm_rope(x, w, [0, 5, 9], f, 1e-6, True, 1.5), OA.rotate(OS.norm_rope(x, w, [0, 5, 9], np.zeros(0), 1e-6), [0, 5, 9], f, True, 1.5))


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_gradient_is_that_of_differences(interleaved):
    rng = np.random.default_rng(2)
    x, c, w = rng.standard_normal((2, 2, 16)), rng.standard_normal((2, 2, 16)), rng.standard_normal(16)
    f, pos, h = OA.rope_frequencies(16, 100.0), [3, 40], 1e-6
    dx, dw, size, dw_size = OS.norm_rope_backward(c, x, w, pos, f, 1e-3, interleaved, 1.5)
    value = lambda a, b: (c * OS.norm_rope(a, b, pos, f, 1e-3, interleaved, 1.5)).sum()  # noqa: E731
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = h
        assert dx[idx] == pytest.approx((value(x + e, w) - value(x - e, w)) / (2 * h), abs=1e-7)
    for i in range(16):
        e = np.zeros(16)
        e[i] = h
        assert dw[i] == pytest.approx((value(x, w + e) - value(x, w - e)) / (2 * h), abs=1e-7)
    assert np.all(np.abs(dx) <= size * (1 + 1e-12)) and np.all(np.abs(dw) <= dw_size * (1 + 1e-12))


def test_masks_and_ancestors():
    parents = [-1, 0, 1, 0, -1, 4]
    assert [OS.ancestors(parents, i) for i in range(6)] == [[0], [0, 1], [0, 1, 2], [0, 3], [4], [4, 5]]
    assert OS.mask_words([0, 3, 64], 2) == [9, 1] and OS.mask_words([63], 1) == [-(1 << 63)]


def test_assign_by_hand():
    # two requests with pages of 16 keys: one grows over a page border, one finishes, one gets its first page
    table, held, free = [[7, -1], [3, 4], [-1, -1]], [1, 2, 0], [9, 8, 5, 6]
    slots, positions, cu, lengths, _, table, held, free, count, served = OS.assign(table, held, free, 3, [15, 20, 0], [3, -1, 1], 6, 16)
    assert served and slots == [7 * 16 + 15, 5 * 16, 5 * 16 + 1, 8 * 16, -1, -1] and positions == [15, 16, 17, 0, 0, 0]
    assert cu == [0, 3, 3, 4] and lengths == [18, 0, 1]
    assert table == [[7, 5], [3, 4], [8, -1]] and held == [2, 0, 1] and free[:3] == [9, 3, 4] and count == 3


@pytest.mark.parametrize("window,softcap", [(0, 0.0), (5, 0.0), (3, 20.0)])
def test_a_chain_is_causal_attention(window, softcap):
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((7, 4, 8)), rng.standard_normal((19, 2, 8)), rng.standard_normal((19, 2, 8))
    a = OS.tree_attention(q, k, v, np.tril(np.ones((7, 7), bool)), 0.3, softcap, window)
    b = OA.attention(q, k, v, 12, 0.3, softcap, window)
    assert all(np.allclose(x, y) for x, y in zip(a, b))


def test_a_tree_token_sees_its_path():
    """Each token of a tree as the last of the sequence that its path makes."""
    rng = np.random.default_rng(4)
    parents = [-1, 0, 0, 1, 2, 2, 5]
    n, ctx = 7, 6
    q, k, v = rng.standard_normal((n, 2, 8)), rng.standard_normal((ctx + n, 1, 8)), rng.standard_normal((ctx + n, 1, 8))
    mask = np.zeros((n, n), bool)
    for i in range(n):
        mask[i, OS.ancestors(parents, i)] = True
    for window in (0, 4):
        out, lse, _, _ = OS.tree_attention(q, k, v, mask, 0.5, 0.0, window)
        for i in range(n):
            at = list(range(ctx)) + [ctx + t for t in OS.ancestors(parents, i)]
            want, wlse, _, _ = OA.attention(q[i:i + 1], k[at], v[at], len(at) - 1, 0.5, 0.0, window)
            assert np.allclose(out[i], want[0]) and np.allclose(lse[i], wlse[0])
    # nothing seen: zeros; keys before the sequence are not there
    out, lse, _, _ = OS.tree_attention(q, k[:n], v[:n], np.zeros((n, n), bool), 0.5)
    assert not out.any() and np.isneginf(lse).all()
    out, lse, _, _ = OS.tree_attention(q, k[:3], v[:3], mask, 0.5)
    assert np.isneginf(lse[:4]).all() and np.allclose(out[4], v[0]) and np.allclose(out[5], v[1])
