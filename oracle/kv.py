"""Heads, MXFP4 cache rows and attention (oracle; test infrastructure).

"Resumo Técnico: ScaleSweep", 4. Resultados: keys and values of the cache in
FP4 beside weights and activations.  The rotation of a position (rotary
embedding) and softmax attention are the published definitions; the pages
name neither, so their parity is unpinned by the pages.

``map_heads`` follows the definition step by step in float32 (each operation
one rounding; the norm's sum of squares, square root and quotient in
float64).  ``attention`` is float64 throughout.
"""

import numpy as np

from . import hadamard as H


def map_heads(x, positions=None, table=None, interleaved=False, norm_weight=None, eps=0.0, hadamard_n=0):
    """[tokens, heads, head_dim] float32 heads after norm, rotation and block
    Hadamard, in float32."""
    y = np.array(x, dtype=np.float32)
    if norm_weight is not None:
        s = np.sum(y.astype(np.float64) ** 2, axis=-1, keepdims=True) / y.shape[-1]
        r = (1.0 / np.sqrt(s + eps)).astype(np.float32)
        y = (y * r).astype(np.float32) * np.asarray(norm_weight, np.float32)
    if table is not None:
        half = table.shape[1] // 2
        i = np.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c = np.asarray(table, np.float32)[positions][:, None, :half]
        s = np.asarray(table, np.float32)[positions][:, None, half:]
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia] = (a * c) - (b * s)
        y[..., ib] = (b * c) + (a * s)
    return H.block_hadamard(y, hadamard_n) if hadamard_n else y


def rotary_table(positions, rotary_dim, base=10000.0):
    """Cosines then sines of positions 0 .. positions - 1, angles in float64."""
    inv = base ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    a = np.arange(positions, dtype=np.float64)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def attention(q, keys, values, scale, causal=True, window=0):
    """One sequence: q [n, heads, D] float64, its last n tokens; keys, values
    [len, kv_heads, D].  Returns outputs and log-sum-exps, and for error
    bounds the sums of p |v| and the largest sum of |q_d k_d| of a row's
    visible keys."""
    n, heads, dim = q.shape
    length, kv_heads, _ = keys.shape
    g = heads // kv_heads
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, top = np.full((n, heads), -np.inf), np.zeros((n, heads))
    j = np.arange(length)
    for i in range(n):
        p = length - n + i
        see = np.ones(length, dtype=bool)
        if causal:
            see &= j <= p
        if window:
            see &= j > p - window
        if not see.any():
            continue
        for h in range(heads):
            k, v = keys[see, h // g], values[see, h // g]
            s = (k @ q[i, h]) * scale
            m = s.max()
            e = np.exp(s - m)
            w = e / e.sum()
            out[i, h], mag[i, h] = w @ v, w @ np.abs(v)
            lse[i, h] = m + np.log(e.sum())
            top[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mag, top
