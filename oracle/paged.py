"""Rotary positions, attention over a paged cache, the weights that positions receive, eviction
(oracle).  Test infrastructure only.

Plain 64-bit restatements; the rotary turn is defined with one binary32 rounding per operation and
a last one to fp16, which are made here.
"""
from __future__ import annotations

import numpy as np


def frequencies(rot, base=10000.0, factor=1.0, original=0, low=1.0, high=4.0):
    w = float(base) ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if original == 0:
        return w / factor
    r = original * w / (2 * np.pi)
    g = np.clip((r - low) / (high - low), 0, 1) if high > low else (r >= high).astype(float)
    return w * g + w / factor * (1 - g)


def angles(positions, rot, gain=1.0, **scale):
    """[positions][rot/2][2]: gain * (cos, sin), rounded to binary32."""
    a = np.arange(positions, dtype=np.float64)[:, None] * frequencies(rot, **scale)
    return (gain * np.stack([np.cos(a), np.sin(a)], -1)).astype(np.float32)


def turn(x, heads, table, pos, interleaved, transpose=False):
    """fp16 rows x [n][heads*d] at positions pos [n] -> fp16 [n][heads*d]."""
    rot = 2 * table.shape[1]
    y = x.reshape(len(x), heads, -1).copy()
    h = y[..., :rot].astype(np.float32)
    lo, hi = ((h[..., 0::2], h[..., 1::2]) if interleaved else
              (h[..., :rot // 2], h[..., rot // 2:]))
    c, s = table[pos][:, None, :, 0], table[pos][:, None, :, 1] * np.float32(-1 if transpose else 1)
    a, b = lo * c - hi * s, lo * s + hi * c
    if interleaved:
        h[..., 0::2], h[..., 1::2] = a, b
    else:
        h = np.concatenate([a, b], -1)
    y[..., :rot] = h.astype(np.float16)
    return y.reshape(x.shape)


def seen(first, nq, n, window, sinks):
    """[nq][n]: what query rows at positions first, first + 1, .. see of n keys."""
    i, t = np.arange(first, first + nq)[:, None], np.arange(n)[None]
    ok = t <= i
    if window:
        ok &= (t > i - window) | (t < sinks)
    return ok


def scores(q, k, ok, scale):
    """q [nq][G][d], k [n][d] -> 64-bit scores [nq][G][n], -inf where not seen."""
    with np.errstate(invalid="ignore"):
        s = np.einsum("rgd,td->rgt", q.astype(np.float64), k.astype(np.float64)) * scale
    return np.where(ok[:, None], s, -np.inf)


def attend(q, k, v, ok, scale):
    """Outputs [nq][G][d], log-sum-exp [nq][G], weights [nq][G][n]; what is not seen takes no part."""
    s = scores(q, k, ok, scale)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    l = e.sum(-1, keepdims=True)
    p = e / np.where(l == 0, 1.0, l)
    o = np.zeros(q.shape)
    v = v.astype(np.float64)
    for r in range(q.shape[0]):
        o[r] = p[r][:, ok[r]] @ v[ok[r]]
    with np.errstate(divide="ignore"):
        lse = np.where(l == 0, -np.inf, m + np.log(l))[..., 0]
    return o, lse, p


def evict(acc, n, keep, recent):
    """Positions that stay of the first n, given their weights acc [n]."""
    if n <= keep:
        return np.arange(n)
    old = n - recent
    best = np.argsort(-acc[:old].astype(np.float64), kind="stable")[:keep - recent]
    return np.sort(np.concatenate([best, np.arange(old, n)]))
