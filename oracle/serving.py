"""fp64 NumPy forms of the operators around the attention calls.

TEST INFRASTRUCTURE ONLY, like ``oracle.zebra``: rotary positions, the norm of
queries and keys with the rotation and its gradient, the 8-bit key/value cache
(quantisation, attention over it, the weight its blocks receive) and eviction.
Every function is written from the definition, with plain loops over heads.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["rope_frequencies", "rope", "qk_norm", "qk_norm_rope", "qk_norm_rope_grad", "E4M3_VALUES",
           "quantise_block", "Cache8", "cache_attention", "evict_blocks"]


# --------------------------------------------------------------- positions ----
def rope_frequencies(pairs, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Radians a position of each pair, and the magnitude."""
    i = np.arange(pairs, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (pairs / (pairs - 1))
    f = base ** (-i / pairs)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        keep = np.clip((original_len * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, pos, freq, axes=1, layout="half", magnitude=1.0, inverse=False):
    """x [B, H, N, 64] rotated: pos int [B or 1, axes, N], freq [pairs] in radians a position."""
    y = np.array(x, dtype=np.float64)
    n = len(freq)
    pos = np.broadcast_to(pos, (x.shape[0],) + tuple(pos.shape[1:]))
    for a in range(axes):
        for i in range(n):
            e1, e2 = (2 * n * a + i, 2 * n * a + n + i) if layout == "half" else (2 * n * a + 2 * i, 2 * n * a + 2 * i + 1)
            theta = pos[:, a, :].astype(np.float64) * freq[i]
            c, s = np.cos(theta)[:, None] * magnitude, np.sin(theta)[:, None] * magnitude * (-1 if inverse else 1)
            u, v = np.asarray(x[..., e1], np.float64), np.asarray(x[..., e2], np.float64)
            y[..., e1], y[..., e2] = u * c - v * s, v * c + u * s
    return y


def qk_norm(x, kind, eps):
    """(normalised rows, 1 / sigma) over the last axis."""
    x = np.asarray(x, np.float64)
    if kind == "none":
        return x, np.ones_like(x[..., :1])
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def qk_norm_rope(x, w, b, kind, eps, pos, freq, **how):
    y = qk_norm(x, kind, eps)[0]
    if kind != "none":
        y = y * (1.0 if w is None else w) + (0.0 if b is None else b)
    return y if freq is None else rope(y, pos, freq, **how)


def qk_norm_rope_grad(g, x, w, kind, eps, pos, freq, **how):
    """(dx, dw, db) of qk_norm_rope for the output's gradient g."""
    dy = np.asarray(g, np.float64) if freq is None else rope(g, pos, freq, inverse=True, **how)
    xh, r = qk_norm(x, kind, eps)
    if kind == "none":
        return dy, None, None
    t = dy * (1.0 if w is None else w)
    dx = t - xh * (t * xh).mean(-1, keepdims=True)
    if kind == "layer":
        dx = dx - t.mean(-1, keepdims=True)
    return dx * r, (dy * xh).sum((0, 1, 2)), dy.sum((0, 1, 2))


# ------------------------------------------------------------- 8-bit cache ----
def _e4m3_values():
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3_VALUES = _e4m3_values()   # of the codes 0..126 (+); 448 the last


def quantise_block(x, fmt):
    """(values of the codes, scale) of one block x: scale = fp32(max|x| / M), codes the nearest to x / scale,
    the even one where two are as near; a block with a value that is not finite reads as NaN."""
    x = np.asarray(x, np.float64)
    top = 127.0 if fmt == "int8" else 448.0
    big = np.max(np.abs(x)) if x.size else 0.0
    if not np.isfinite(big):
        return np.zeros_like(x), np.float64(np.nan)
    s = float(np.float32(big / top))
    if s == 0.0:
        return np.zeros_like(x), 0.0
    t = x / s
    if fmt == "int8":
        return np.clip(np.rint(t), -127, 127), s
    hi = np.clip(np.searchsorted(E4M3_VALUES, np.abs(t)), 1, 126)
    lo = hi - 1
    d = (np.abs(t) - E4M3_VALUES[lo]) - (E4M3_VALUES[hi] - np.abs(t))
    up = (d > 0) | ((d == 0) & (hi % 2 == 0))
    return np.copysign(np.where(up, E4M3_VALUES[hi], E4M3_VALUES[lo]), t), s


class Cache8:
    """One head's cache: the original rows, quantised block by block on reading."""

    def __init__(self, block, fmt):
        self.block, self.fmt, self.k, self.v = block, fmt, np.zeros((0, 64)), np.zeros((0, 64))

    def append(self, k, v):
        self.k = np.concatenate([self.k, np.asarray(k, np.float64)])
        self.v = np.concatenate([self.v, np.asarray(v, np.float64)])

    def values(self):
        """Keys and values [len, 64] as the cache holds them, and the scales [blocks]."""
        out = []
        for x in (self.k, self.v):
            parts = [quantise_block(x[i:i + self.block], self.fmt) for i in range(0, len(x), self.block)]
            # what a code stands for: its value times the scale, in fp32
            vals = [np.asarray(c * s, np.float32).astype(np.float64) for c, s in parts]
            out.append((np.concatenate(vals) if vals else np.zeros((0, 64)), np.array([s for _, s in parts])))
        return out[0][0], out[1][0], out[0][1], out[1][1]


def cache_attention(q, k, v, scale, causal, block):
    """q [group, n_q, 64] against one head's k, v [len, 64]: (O, lse, weight of each block).

    Causal: query i of n_q sees keys j <= len - n_q + i.  A row that sees no key gives zeros and -inf."""
    G, n_q, _ = q.shape
    L = len(k)
    O, lse, mass = np.zeros(q.shape), np.full((G, n_q), -np.inf), np.zeros(-(-L // block))
    for g in range(G):
        for i in range(n_q):
            n = max(0, L - n_q + i + 1) if causal else L
            if n == 0:
                continue
            x = scale * (k[:n] @ np.asarray(q[g, i], np.float64))
            top = x.max()
            p = np.exp(x - top)
            lse[g, i] = top + np.log(p.sum())
            p /= p.sum()
            O[g, i] = p @ v[:n]
            mass += np.add.reduceat(np.pad(p, (0, L - n)), np.arange(0, L, block))
    return O, lse, mass


def evict_blocks(table, mass, length, block, budget, sinks, recent):
    """One head: (table, length, kept logical blocks) after keeping at most `budget` blocks."""
    nb = -(-length // block)
    if nb <= budget:
        return list(table), length, list(range(nb))
    middle = sorted(range(sinks, nb - recent), key=lambda b: (-mass[table[b]], b))
    kept = sorted(list(range(sinks)) + middle[:budget - sinks - recent] + list(range(nb - recent, nb)))
    stay = set(kept)
    gone = [b for b in range(nb) if b not in stay]
    return ([table[b] for b in kept] + [table[b] for b in gone] + list(table[nb:]), length - block * len(gone), kept)
