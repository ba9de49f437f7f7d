"""Ragged, windowed attention and the ragged cache (oracle).  Test infrastructure only.

Plain 64-bit restatement, one query row and one head at a time.  Position i of a sequence sees
position t when t <= i and (window == 0 or t > i - window or t < sinks); a row that sees nothing
gives 0.  Query head hq reads K/V head hq // (Hq // Hkv).
"""
from __future__ import annotations

import numpy as np


def visible(i: int, n: int, window: int, sinks: int) -> np.ndarray:
    """Indexes of the keys 0 .. n-1 that position i sees."""
    t = np.arange(n)
    ok = t <= i
    if window:
        ok &= (t > i - window) | (t < sinks)
    return t[ok]


def attend(q, k, v, i, window, sinks, scale, kmag=None, vmag=None):
    """One query row q [d] at position i over k, v [n][d] (any float type, read as 64-bit).

    Returns (o [d], info): info holds what error bounds need over the n seen keys -- A [d] =
    sum_t p_t |v_t|, V [d] = sum_t p_t vmag_t, qk and qkmag = the largest scale * sum_j |q_j| |k_tj|
    and scale * sum_j |q_j| kmag_tj, q1 = scale * sum_j |q_j|, l = sum_t exp(s_t - max s), vmax [d].
    kmag, vmag [n][d] (default |k|, |v|): the size of the terms a value is computed from.
    """
    d = q.shape[0]
    t = visible(i, k.shape[0], window, sinks) if i >= 0 else np.zeros(0, int)
    if t.size == 0:
        z = np.zeros(d)
        return z, dict(A=z, V=z, qk=0.0, qkmag=0.0, q1=0.0, l=1.0, n=0, vmax=z)
    kmag = np.abs(np.asarray(k, np.float64)) if kmag is None else kmag
    vmag = np.abs(np.asarray(v, np.float64)) if vmag is None else vmag
    q, k, v, kmag, vmag = (np.asarray(x, np.float64) for x in (q, k[t], v[t], kmag[t], vmag[t]))
    s = (k @ q) * scale
    e = np.exp(s - s.max())
    p = e / e.sum()
    aq = np.abs(q)
    return p @ v, dict(A=p @ np.abs(v), V=p @ vmag, qk=float((np.abs(k) @ aq).max() * scale),
                       qkmag=float((kmag @ aq).max() * scale), q1=float(aq.sum() * scale),
                       l=float(e.sum()), n=int(t.size), vmax=np.abs(v).max(axis=0))


def prefill(q, k, v, q_off, kv_off, Hq, Hkv, window, sinks, scale):
    """q [q_rows][Hq*d], k, v [kv_rows][Hkv*d] -> {row: (o [Hq][d], [info per head])}."""
    d = q.shape[1] // Hq
    out = {}
    for b in range(len(q_off) - 1):
        nq, nk = q_off[b + 1] - q_off[b], kv_off[b + 1] - kv_off[b]
        ks, vs = k[kv_off[b]:kv_off[b + 1]], v[kv_off[b]:kv_off[b + 1]]
        for r in range(nq):
            row = q_off[b] + r
            res = []
            for hq in range(Hq):
                c = (hq // (Hq // Hkv)) * d
                res.append(attend(q[row, hq * d:(hq + 1) * d], ks[:, c:c + d], vs[:, c:c + d],
                                  nk - nq + r, window, sinks, scale))
            out[row] = (np.stack([o for o, _ in res]), [f for _, f in res])
    return out


def decode(q, k, v, lens, Hq, window, sinks, scale, kmag=None, vmag=None):
    """q [B][Hq*d], k, v [B][H][cap][d] restored -> [(o [Hq][d], [info per head])] per sequence.
    kmag, vmag [B][H][cap][d]: as for attend()."""
    H, d = k.shape[1], k.shape[3]
    out = []
    for b, n in enumerate(lens):
        res = []
        for hq in range(Hq):
            at = (b, hq // (Hq // H), slice(0, n))
            res.append(attend(q[b, hq * d:(hq + 1) * d], k[at], v[at], n - 1, window, sinks, scale,
                              None if kmag is None else kmag[at],
                              None if vmag is None else vmag[at]))
        out.append((np.stack([o for o, _ in res]), [f for _, f in res]))
    return out
