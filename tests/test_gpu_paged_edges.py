"""Calls of the paged operators at the edges of what their warps hand to one another, of what values can
be, and of what the callers' arrays hold."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as OP
from paged_util import F32, H16, fill, i32, need, rows_of, tables
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


@pytest.mark.parametrize("n,nq,bad", [(897, 3, 896), (900, 3, 898), (897, 1, 896), (900, 1, 898)])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("G", [1, 9])
def test_pieces_of_cut_blocks_keep_their_nan(fg, n, nq, bad, which, G):
    """A long row's key tiles go to many multiprocessors.  A NaN in K that is all that a row sees of the
    last tile, or that stands among keys whose weights are 0 beside the others', makes the row and its
    log-sum-exp NaN; one in V makes the row NaN.  Rows before it do not show it."""
    d, P = 64, 16
    table, pool, k, v, q_off, q = paged_case(fg, d, 1, P, [n], [nq], 5, G)
    t = torch.ones((len(q), G * d), dtype=torch.float16, device="cuda")
    for p in range(896, n):                                  # scores 800 below 0
        pool.parts()[1][table[0, p // P], 0, p % P] = -100.0
    args = (t, q_off, G, pool, table, [n], 0.125)
    clean, zc = run_attend(fg, *args, max_q=nq)
    pool.parts()[1 + 2 * which][table[0, bad // P], 0, bad % P] = float("nan")
    out, z = run_attend(fg, *args, max_q=nq)
    fg.fg_check_device_error()
    first = q_off[1] - (n - bad)                             # the first row that sees it
    out, z, clean, zc = (host(x)[q_off[0]:q_off[1]] for x in (out, z, clean, zc))
    first = max(0, first - q_off[0])
    assert np.isfinite(clean).all() and np.isfinite(zc).all()
    assert np.isnan(out[first:]).all()
    assert np.isnan(z[first:]).all() if which == 0 else np.array_equal(z[first:], zc[first:])
    # (rows computed on their own take their sums in another order)
    a, c = out[:first].astype(np.float64), clean[:first].astype(np.float64)
    assert np.all(np.abs(a - c) <= 4 * H16 * np.abs(c) + 2.0 ** -10 * np.abs(c).max(initial=0))
    assert np.isfinite(z[:first]).all()


@pytest.mark.parametrize("H,lens,keep,recent", [(2, [2, 40, 200], 20, 4), (2, [2], 1, 0),
                                                (1, [6000], 900, 33), (3, [64, 5000, 17], 30, 0)])
@pytest.mark.parametrize("kind", ["zeros", "nan"])
def test_eviction_order_of_zeros_and_nan(fg, H, lens, keep, recent, kind):
    """Zeros of both signs are equal, NaN of either sign and any payload lie above +inf and are equal:
    among equal ones the lower positions stay.  The weights are handed on as they are."""
    d, P = 64, 16
    both = need(lens, P) + [(keep + P - 1) // P] * len(lens)
    all_tables, pages = tables(both, seed=keep)
    src = np.ascontiguousarray(all_tables[:len(lens)])
    dst = np.ascontiguousarray(all_tables[len(lens):, :both[-1]])
    pool, _, _ = fill(fg, pages, P, H, d, 4)
    rng = np.random.default_rng(keep + H)
    pick = {"zeros": [0x80000000, 0, 0x80000001, 0x00000001, 0xBF800000],
            "nan": [0x7FC00000, 0xFFC00000, 0xFFFFFFFF, 0x7F800001, 0x7F800000, 0xFF800000, 0x3F800000,
                    0x7F7FFFFF]}[kind]
    bits = rng.choice(np.array(pick, np.uint32), (len(lens), H, max(lens) + 3))
    if kind == "nan":                                        # few NaN, so that the last to stay varies
        bits[rng.random(bits.shape) < 0.9] = 0x3F000000
    bits[0, :, :2] = [0x80000000, 0] if kind == "zeros" else [0x7F800000, 0xFFC00000]
    acc = bits.view(np.float32)
    kept = torch.full((len(lens), H, keep), 99, dtype=torch.int32, device="cuda")
    acc_out = torch.full((len(lens), H, keep), 7.0, device="cuda")
    dst_lens = torch.full((len(lens),), 99, dtype=torch.int32, device="cuda")
    fg.fg_kv_evict_q4_paged(pool, dev(src), i32(lens), dev(bits.view(np.int32)).view(torch.float32),
                            recent, dev(dst), kept, acc_out, dst_lens)
    fg.fg_check_device_error()
    with np.errstate(invalid="ignore"):
        wide = acc.astype(np.float64)
    order = np.where(np.isnan(acc), np.inf, np.where(np.isposinf(acc), 1e300, wide))
    got = host(acc_out.view(torch.int32)).view(np.uint32)
    for b, n in enumerate(lens):
        for h in range(H):
            at = OP.evict(order[b, h], n, keep, recent)
            assert np.array_equal(host(kept)[b, h, :len(at)], at), (b, h)
            assert np.array_equal(got[b, h, :len(at)], bits[b, h, at]), (b, h)


@pytest.mark.parametrize("d,H,G,lens,nq", [
    (64, 2, 1, [700, 300], [128, 200]),                      # whole row tiles that all see the first keys
    (128, 1, 4, [600, 257], [64, 33]),
    (64, 1, 7, [500], [40]),                                 # 126 rows a tile
    (128, 2, 2, [700, 40], [8, 1]),                          # few rows: streamed
    (64, 1, 32, [513], [1]),
])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 60000.0])
def test_rows_without_a_log_sum_exp_add_nothing(fg, d, H, G, lens, nq, bad):
    """A row whose log-sum-exp is -inf hands out no weight, whatever its query is; one whose is +inf hands
    out 0 to every finite score."""
    P, Hq, scale = 32, H * G, 1.0 / math.sqrt(d)
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 31 + d, G)
    t = dev(q)[:, :Hq * d].contiguous()
    _, z = run_attend(fg, t, q_off, Hq, pool, table, lens, scale, max_q=max(nq))
    rng = np.random.default_rng(3)
    silent = torch.from_numpy(rng.random(tuple(z.shape)) < 0.2).cuda()
    silent[q_off[0]] = True
    silent[q_off[0], 0] = False

    def weights(rows, lse):
        acc = torch.zeros((len(lens), H, max(lens)), device="cuda")
        fg.fg_attn_weights_q4_paged(rows.reshape(t.shape), i32(q_off), Hq, pool, dev(table), i32(lens),
                                    scale, lse, None, acc, max_q=max(nq))
        fg.fg_check_device_error()
        return host(acc)

    heads = t.view(len(q), Hq, d)
    none = z.masked_fill(silent, -float("inf"))
    want = weights(heads.masked_fill(silent[..., None], 0.0), none)
    assert np.isfinite(want).all() and want.any()
    assert np.array_equal(weights(heads.masked_fill(silent[..., None], bad), none), want)
    assert np.array_equal(weights(heads, z.masked_fill(silent, float("inf"))), want)


@pytest.mark.parametrize("d,H,G,lens,nq,window,sinks", [
    (64, 1, 2, [700, 300, 5], [128, 40, 5], 0, 0),           # pieces, and many rows
    (128, 2, 4, [600, 257], [3, 8], 0, 0),                   # pieces, and few rows
    (128, 1, 7, [500, 90], [40, 20], 64, 3),
    (64, 2, 1, [900, 1, 77, 0], [1, 1, 1, 0], 0, 0),         # single tokens
    (128, 1, 8, [2000, 300], [1, 1], 500, 4),
    (64, 1, 12, [300, 40], [1, 1], 0, 0),                    # single tokens of many heads
])
def test_every_row_hands_out_a_weight_of_one(fg, d, H, G, lens, nq, window, sinks):
    """The received weights with the log-sum-exp that the attention gave: each row and head hands out 1.
    Either call's scores miss theirs by d + 40 binary32 operations on sum |q_j k_j| at most; the
    log-sum-exp and the exponential as in check_attend and test_weights."""
    P, Hq, scale = 32, H * G, 1.0 / math.sqrt(d)
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 83 + d, G)
    t, kw = dev(q)[:, :Hq * d], dict(window=window, sinks=sinks, max_q=max(nq))
    _, z = run_attend(fg, t, q_off, Hq, pool, table, lens, scale, **kw)
    acc = torch.full((len(lens), H, max(lens)), 9.0, device="cuda")
    fg.fg_attn_weights_q4_paged(t, i32(q_off), Hq, pool, dev(table), i32(lens), scale, z, None, acc, **kw)
    fg.fg_check_device_error()
    for b, n in enumerate(lens):
        if nq[b] == 0:
            continue
        ok = OP.seen(n - nq[b], nq[b], n, window, sinks)
        for hk in range(H):
            kk = rows_of(k, table, b, n)[hk].astype(np.float64)
            qq = q[q_off[b]:q_off[b + 1], hk * G * d:(hk + 1) * G * d].reshape(nq[b], G, d)
            mag = np.einsum("rgd,td->rgt", np.abs(qq.astype(np.float64)), np.abs(kk)) * scale
            mag = np.where(ok[:, None], mag, 0).max(-1)
            _, lse, _ = OP.attend(qq, kk, kk, ok, scale)
            off = 2 * mag * (d + 40) * F32 + np.abs(lse) * 8 * F32 + (n + 64) * F32 + 2.0 ** -20 \
                + 2.0 ** -21
            got = host(acc)[b, hk, :n].astype(np.float64).sum()
            want = ok.any(1).sum() * G
            tol = np.expm1(off).sum() + want * (nq[b] * G + 8) * F32
            assert abs(got - want) <= tol, (b, hk, got, want, tol)
