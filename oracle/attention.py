"""The attention side in float64 (oracle; test infrastructure only): rotary positions, the append to a paged
cache, and attention over it, from their definitions with loops over tokens and heads.

gemma-cuda-hybrid README, "Everything it has": head-packed GQA attention, an FP8 E4M3 KV cache; TensorSharp
docs/models/gemma4.md: window and global attention, RoPE flavors, paged KV.  The pages give no formulas; these are
the usual ones.
"""

from __future__ import annotations

import math

import numpy as np

from .formats import e4m3_value


def rope_frequencies(rot_dim, theta, factor=1.0, trained_context=0.0, slow=1.0, fast=32.0):
    out = []
    for i in range(rot_dim // 2):
        w = theta ** (-2.0 * i / rot_dim)
        keep = 0.0
        if trained_context > 0:
            turns = trained_context * w / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
        out.append(keep * w + (1.0 - keep) * w / factor)
    return np.array(out, np.float64)


def rotate(x, positions, inv_freq, interleaved=False, amplitude=1.0, inverse=False):
    """x [tokens, heads, dim] float64 -> rotated."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    for t, p in enumerate(positions):
        for i, w in enumerate(inv_freq):
            # off by 2^-53 of p * w: 2^-32 of a radian at two million positions
            a = math.fmod(float(p) * float(w), 2.0 * math.pi)
            c, s = amplitude * math.cos(a), amplitude * math.sin(a)
            if inverse:
                s = -s
            lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            u, v = np.array(x[t, :, lo], np.float64), np.array(x[t, :, hi], np.float64)
            y[t, :, lo], y[t, :, hi] = u * c - v * s, v * c + u * s
    return y


def attention(q, keys, values, position0, scale, softcap=0.0, window=0):
    """One sequence: q [n, heads, dim] at positions position0 + i; keys, values [len, kv_heads, dim] float64.
    Returns (out, lse, spread, logit_size): spread[i, h] = sum_j p_j |v_j| per value, logit_size the largest
    |scale| * sum |q| |k_j| of the row -- what rounding errors are measured by."""
    n, heads, dim = q.shape
    length, kv, _ = keys.shape
    g = heads // kv
    out = np.zeros((n, heads, dim))
    spread = np.zeros((n, heads, dim))
    lse = np.full((n, heads), -np.inf)
    size = np.zeros((n, heads))
    for i in range(n):
        p = position0 + i
        hi = min(p + 1, length)
        lo = max(0, p - window + 1) if window > 0 else 0
        if hi <= lo:
            continue
        for h in range(heads):
            k, v = keys[lo:hi, h // g], values[lo:hi, h // g]
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


def from_e4m3(codes, scales):
    """codes uint8 [..., kv_heads, dim] (heads on axis -2) times the scale of their head."""
    return e4m3_value(codes) * np.asarray(scales, np.float64)[:, None]
