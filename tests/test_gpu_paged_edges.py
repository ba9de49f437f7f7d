"""Calls of the paged operators at the edges of what their warps hand to one another, of what values can
be, and of what the callers' arrays hold."""
import math

import numpy as np
import pytest
import torch

from paged_util import H16
from parity_util import dev, host, lib
from test_gpu_paged import check_attend, paged_case, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    return lib()


@pytest.mark.parametrize("G", [1, 4])
def test_blocks_of_two_row_tiles_before_blocks_of_one(fg, G):
    """Prompts of two row tiles, of which the first sees one key tile and the second both, and prompts
    of one, several to a multiprocessor; an infinity in the last V, which only a last row sees, keeps
    the second tile's rows busy far longer than the first's."""
    d, H, P, tpt = 64, 8, 64, 128 // G
    lens = [2 * tpt, 2 * tpt, 17] * 50
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, lens, 71 + G, G)
    t, scale, width = dev(q)[:, :H * G * d], 1.0 / math.sqrt(d), H * G * d
    clean, z = run_attend(fg, t, q_off, H * G, pool, table, lens, scale, max_q=max(lens))
    fg.fg_check_device_error()
    check_attend(clean, z, q, q_off, H * G, k, v, table, lens, scale)
    ab = pool.parts()[3]
    last = [n - 1 for n in lens]
    for b, p in enumerate(last):
        ab[table[b, p // P], :, p % P, 0, 1] = float("inf")
    out, zi = run_attend(fg, t, q_off, H * G, pool, table, lens, scale, max_q=max(lens))
    fg.fg_check_device_error()
    # (the log-sum-exp of rows computed on their own is of other sums: within the oracle's bound, too)
    check_attend(clean, zi, q, q_off, H * G, k, v, table, lens, scale)
    sees = np.zeros(len(q), bool)
    sees[[q_off[b] + p for b, p in enumerate(last)]] = True
    out, clean = host(out), host(clean)
    a, c = out[~sees].astype(np.float64), clean[~sees].astype(np.float64)
    # (rows computed on their own take their sums in another order)
    assert np.all(np.abs(a - c) <= 4 * H16 * np.abs(c) + 2.0 ** -10 * np.abs(c).max())
    assert not np.isfinite(out[sees]).all(axis=1).any()
