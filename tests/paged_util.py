"""Shared helpers of the paged cache's GPU tests: pools of pages, their contents and sequences."""
import numpy as np
import torch

import fg_synth
from oracle import quant as OQ

H16 = 2.0 ** -11          # half a step of fp16, relative
F32 = 2.0 ** -23          # one binary32 operation, rounded or truncated, relative


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def offsets(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(int).tolist()


def tables(need, seed, spare=2, first=0):
    """Page tables (numpy) of sequences that need so many pages, in a shuffled order, unused entries
    bad (-7); and the pages of the pool."""
    pages = sum(need) + spare + first
    order = iter(np.random.default_rng(seed).permutation(pages - first) + first)
    t = np.full((len(need), max(1, max(need, default=1))), -7, np.int32)
    for b, n in enumerate(need):
        t[b, :n] = [next(order) for _ in range(n)]
    return t, pages


class Values:
    """Restored values and their groups' largest magnitudes, by page."""

    def __init__(self, x, big):
        self.x, self.big, self.shape = x, big, x.shape


def restore_error(big):
    """How far a value of the attention may be from its definition fp16(a + q s), s = (b - a)/15.

    It computes fp16((q - z) s1 + fp16((q - z) s2 + c)) with z the code whose value a + z s is nearest
    to 0, c = fp16(a + z s), s1 = fp16(s) and s2 = fp16(s - s1).  With M the larger of |a| and |b| and
    h = 2^-11 half a step: s <= 2 M / 15, so |(q - z) s| <= 2 M, of which s1 + s2 misses h^2 and the
    quotient 2^-21: 2 (h^2 + 2^-21) M < h M / 300; c: h M; the inner sum, M (1 + 2 h) at most: h M (1 +
    2 h); the result: h M (1 + 4 h); the definition's own: h M.  Together less than 4.1 h M.

    Below 2^-14 half a step is 2^-25.  Where s2 is that small, s1 + s2 misses s by 2^-25: 15 times that
    at most.  Where M is, the sums are of multiples of 2^-24, exact, and with them only the definition's
    rounding and c's count; c is a or b, exact, where |q - z| = 15: 15 + 1 or 14 + 2 times 2^-25, which
    is 2^-21."""
    return H16 * 4.1 * big + 2.0 ** -21


def fill(fg, pages, P, H, d, seed, scale=1.0):
    """A pool of pages of quantised normal values, and their restored values [pages][H][P][d] of K
    and of V, each with the largest of its group's magnitudes M beside it (rows_of takes either)."""
    pool = fg.KVPagesQ4(pages, P, H * d, H)
    vals = []
    for codes_t, ab_t, sd in zip(pool.parts()[0::2], pool.parts()[1::2], (0, 1)):
        x = fg_synth.random_fp16((pages * H * P, d), seed=seed * 2 + sd, scale=scale,
                                 offset=0.2 * scale)
        q, a, b = OQ.quantize_g64(x)
        codes_t.copy_(torch.from_numpy(OQ.pack_nibbles(q)).cuda().view(codes_t.shape))
        ab = np.stack([a, b], -1).reshape(pages, H, P, d // 64, 2)
        ab_t.copy_(torch.from_numpy(ab).cuda())
        big = np.maximum(np.abs(a.astype(np.float64)), np.abs(b.astype(np.float64)))
        vals.append(Values(OQ.dequant_g64(q, a, b).reshape(pages, H, P, d),
                           np.repeat(big, 64, axis=1).reshape(pages, H, P, d)))
    return pool, vals[0], vals[1]


def rows_of(vals, table, b, n):
    """Values [H][n][d] of sequence b's first n positions, from values by page."""
    vals = getattr(vals, "x", vals)
    P = vals.shape[2]
    if n == 0:
        return np.zeros((vals.shape[1], 0, vals.shape[3]), vals.dtype)
    x = vals[table[b, :(n + P - 1) // P]]                    # [pages][H][P][d]
    return np.moveaxis(x, 0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def need(lens, P):
    return [(n + P - 1) // P for n in lens]
