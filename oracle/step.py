"""Norms of queries and keys, a step's bookkeeping, accepted paths and attention of drafted trees in float64 and plain
integers (oracle; test infrastructure only), from their definitions with loops over requests, tokens and heads."""

from __future__ import annotations

import math

import numpy as np

from .attention import rotate


def norm_rope(x, weight, positions, inv_freq, eps, interleaved=False, amplitude=1.0):
    """x [tokens, heads, dim] float64 -> normalised heads, rotated (inv_freq empty: not)."""
    n = np.array(x, np.float64)
    for t in range(n.shape[0]):
        for h in range(n.shape[1]):
            n[t, h] *= weight / math.sqrt(np.mean(x[t, h] ** 2) + eps)
    return rotate(n, positions, inv_freq, interleaved, amplitude)


def norm_rope_backward(dy, x, weight, positions, inv_freq, eps, interleaved=False, amplitude=1.0):
    """(dx, d weight, and the sums of absolute values that their rounding errors are measured by)."""
    u = rotate(dy, positions, inv_freq, interleaved, amplitude, inverse=True)
    dx, size = np.zeros_like(u), np.zeros_like(u)
    dw, dw_size = np.zeros(x.shape[2]), np.zeros(x.shape[2])
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            r = 1.0 / math.sqrt(np.mean(x[t, h] ** 2) + eps)
            z, unit = u[t, h] * weight, x[t, h] * r
            dx[t, h] = r * (z - unit * np.mean(z * unit))
            size[t, h] = r * (np.abs(z) + np.abs(unit) * np.mean(np.abs(z * unit)))
            dw += u[t, h] * unit
            dw_size += np.abs(u[t, h] * unit)
    return dx, dw, size, dw_size


def ancestors(parents, i):
    """Token i of a tree and the tokens before it, the root first."""
    path = []
    while i >= 0:
        path.append(i)
        i = parents[i]
    return path[::-1]


def mask_words(tokens, words):
    """Bit x % 64 of word x / 64 for each of the tokens, as signed 64-bit numbers."""
    out = []
    for w in range(words):
        v = sum(1 << (x - 64 * w) for x in tokens if x // 64 == w)
        out.append(v - (1 << 64) if v >> 63 else v)
    return out


def assign(table, held, free, count, kv_len, new, rows, page, parents=None, words=0):
    """kv_assign, one request after the other: lists of integers in, (slots, positions, cu, kv_len, masks, table, held,
    free, count, served) out; served is False where something was missing."""
    table, held, free = [list(r) for r in table], list(held), list(free)
    slots, positions, masks = [-1] * rows, [0] * rows, [[0] * words for _ in range(rows)]
    cu, lengths, gone, served = [0], [], [], True
    for b, (n, ctx) in enumerate(zip(new, kv_len)):
        if n < 0:
            gone += table[b][:held[b]]
            held[b] = 0
            lengths.append(0)
            cu.append(cu[-1])
            continue
        if n > rows - cu[-1]:
            n, served = rows - cu[-1], False
        cols = len(table[b])
        if ctx + n > cols * page:
            served = False
        while held[b] < min(cols, -(-(ctx + n) // page)):
            if count == 0:
                served = False
                break
            count -= 1
            table[b][held[b]] = free[count]
            held[b] += 1
        for i in range(n):
            t, at = cu[-1] + i, ctx + i
            if at // page < held[b] and table[b][at // page] >= 0:
                slots[t] = table[b][at // page] * page + at % page
            positions[t] = at
            if parents is not None:
                path = ancestors(parents[cu[-1]:cu[-1] + n], i)
                positions[t] = ctx + len(path) - 1
                masks[t] = mask_words(path, words)
            else:
                masks[t] = mask_words(range(min(i + 1, 64 * words)), words)
        cu.append(cu[-1] + n)
        lengths.append(ctx + n)
    for p in gone:
        if count < len(free):
            free[count] = p
            count += 1
        else:
            served = False
    return slots, positions, cu, lengths, masks, table, held, free, count, served


def tree_attention(q, keys, values, mask, scale, softcap=0.0, window=0):
    """One sequence's new tokens q [n, heads, dim]; keys, values [len, kv_heads, dim] float64, the last n of them the new
    tokens' own; mask [n, n] of truth values.  Returns (out, lse, spread, logit_size) as oracle.attention.attention."""
    n, heads, dim = q.shape
    length, kv, _ = keys.shape
    g, ctx = heads // kv, length - n
    out = np.zeros((n, heads, dim))
    spread = np.zeros((n, heads, dim))
    lse = np.full((n, heads), -np.inf)
    size = np.zeros((n, heads))
    for i in range(n):
        at = list(range(max(ctx, 0))) + [ctx + t for t in range(n) if mask[i, t] and ctx + t >= 0]
        if window > 0:
            at = at[-window:]
        if not at:
            continue
        for h in range(heads):
            k, v = keys[at, h // g], values[at, h // g]
            s = scale * (k @ q[i, h])
            size[i, h] = abs(scale) * np.max(np.abs(k) @ np.abs(q[i, h])) if np.all(np.isfinite(k)) else np.inf
            if softcap > 0:
                s = softcap * np.tanh(s / softcap)
            top = np.max(s)
            if np.isnan(top):
                out[i, h], lse[i, h] = np.nan, np.nan
                continue
            if top == -np.inf:
                continue
            e = np.exp(s - top)
            z = e.sum()
            with np.errstate(invalid="ignore"):
                out[i, h] = (e[:, None] * v).sum(0) / z
                spread[i, h] = (e[:, None] * np.abs(v)).sum(0) / z
            lse[i, h] = top + math.log(z)
    return out, lse, spread, size
