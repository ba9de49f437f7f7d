"""Rotary positions, the paged cache, attention over it, received weights and eviction against the
64-bit oracle, on the GPU.

Turned values, codes, statistics, restored values and evicted caches are compared bit for bit; attention
and weights element by element with bounds that follow the arithmetic."""
import math

import numpy as np
import pytest
import torch

import fg_synth
from oracle import paged as OP
from oracle import quant as OQ
from paged_util import F32, H16, fill, i32, need, offsets, restore_error, rows_of, tables
from parity_util import dev, host, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    return lib()


def table_of(positions, rot, **kw):
    t = OP.angles(positions, rot, **kw)
    return t, dev(t)


# ------------------------------------------------------------------------------- rotary positions


@pytest.mark.parametrize("d,rot,heads", [(64, 64, 1), (64, 16, 5), (128, 128, 3), (128, 32, 2),
                                         (128, 112, 9), (64, 48, 12)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,pos,first", [([1], [5], 0), ([3, 0, 70, 1], [0, 3, 9, 79], 2),
                                            ([1] * 37, list(range(37)), 0)])
def test_rope_is_the_definition(fg, d, rot, heads, interleaved, lens, pos, first):
    table, angles = table_of(80, rot)
    rows = first + sum(lens) + 3
    x = fg_synth.random_fp16((rows, heads * d + 8), seed=rot + heads, scale=3.0)
    t = dev(x)
    y = torch.full((rows, heads * d + 16), 7.0, dtype=torch.float16, device="cuda")
    off = offsets(lens, first)
    fg.fg_rope(t[:, :heads * d], d, i32(off), i32(pos), angles, y[:, :heads * d],
               interleaved=interleaved)
    fg.fg_check_device_error()
    at = np.concatenate([np.arange(p, p + n) for p, n in zip(pos, lens)]).astype(int)
    want = np.full((rows, heads * d + 16), 7.0, np.float16)
    live = slice(first, first + sum(lens))
    want[live, :heads * d] = OP.turn(x[live, :heads * d], heads, table, at, interleaved)
    assert np.array_equal(host(y).view(np.uint16), want.view(np.uint16))
    # in place, and the transposed turn
    back = t[:, :heads * d]
    fg.fg_rope(back, d, i32(off), i32(pos), angles, back, interleaved=interleaved, transpose=True)
    want = x.copy()
    want[live, :heads * d] = OP.turn(x[live, :heads * d], heads, table, at, interleaved, True)
    assert np.array_equal(host(t).view(np.uint16), want.view(np.uint16))


def test_rope_transpose_is_the_gradient(fg):
    """With gain 1.5: sum(g * dy/dx dx) by the formula, and by differences of the call itself (it is
    linear, so a difference is exact but for roundings)."""
    d, rot, heads, n = 64, 32, 2, 9
    table, angles = table_of(30, rot, gain=1.5)
    rng = np.random.default_rng(3)
    x, g, e = (rng.standard_normal((n, heads * d)).astype(np.float16) for _ in range(3))
    off, pos = i32([0, n]), i32([11])

    def turn(v, **kw):
        y = torch.empty((n, heads * d), dtype=torch.float16, device="cuda")
        fg.fg_rope(dev(v), d, off, pos, angles, y, **kw)
        return host(y).astype(np.float64)

    grad = turn(g, transpose=True)
    step = (x.astype(np.float64) + e).astype(np.float16)
    change = turn(step) - turn(x)                            # roundings: half a step of each
    moved = step.astype(np.float64) - x
    # |x0 c - x1 s| <= 2 * 1.5 * 8 and g likewise: half an fp16 step of both sides, summed
    tol = H16 * (np.abs(g.astype(np.float64)) * (np.abs(turn(step)) + np.abs(turn(x)))).sum() \
        + H16 * (np.abs(grad) * np.abs(moved)).sum() + 1e-6
    assert abs((g.astype(np.float64) * change).sum() - (grad * moved).sum()) <= tol
    assert np.array_equal(turn(g, transpose=True).astype(np.float16),
                          OP.turn(g, heads, table, np.arange(11, 11 + n), False, True))


@pytest.mark.parametrize("kw", [{}, dict(factor=4.0), dict(factor=8.0, original=4096),
                                dict(factor=2.0, original=512, low=2.0, high=2.0),
                                dict(gain=1.25, base=500000.0)])
def test_rope_table(fg, kw):
    """Angles of far positions: one binary32 rounding (and the 64-bit functions' last bits)."""
    for rot, positions in ((128, 40000), (16, 1), (48, 257)):
        t = torch.empty((positions, rot // 2, 2), dtype=torch.float32, device="cuda")
        fg.fg_rope_table(t, **kw)
        gain = kw.get("gain", 1.0)
        a = np.arange(positions, dtype=np.float64)[:, None] * OP.frequencies(
            rot, **{k: v for k, v in kw.items() if k != "gain"})
        want = gain * np.stack([np.cos(a), np.sin(a)], -1)
        # one rounding to binary32, half a step: 2^-24 of the value (1.25 lies in [1, 2), whose half
        # step is 2^-24 itself); the frequency's 64-bit roundings, 40000 radians at most, show as
        # 40000 * 2^-50
        tol = 2.0 ** -24 * np.abs(want) + gain * 40000 * 2.0 ** -50
        assert np.all(np.abs(host(t) - want) <= tol)


def test_rope_positions_that_do_not_fit(fg):
    d, rot = 64, 64
    table, angles = table_of(20, rot)
    x = fg_synth.random_fp16((12, d), seed=5)
    y = torch.full((12, d), 7.0, dtype=torch.float16, device="cuda")
    fg.fg_rope(dev(x), d, i32([0, 4, 8, 12]), i32([18, -1, 3]), angles, y)
    with pytest.raises(fg.FgError) as e:
        fg.fg_check_device_error()
    assert e.value.status == fg.FG_ERR_CAPACITY
    want = np.full((12, d), 7.0, np.float16)
    want[:2] = OP.turn(x[:2], 1, table, np.array([18, 19]), False)
    want[8:] = OP.turn(x[8:], 1, table, np.arange(3, 7), False)
    assert np.array_equal(host(y).view(np.uint16), want.view(np.uint16))
    fg.fg_check_device_error()


# ------------------------------------------------------------------------------- append, read


@pytest.mark.parametrize("d,H", [(64, 3), (128, 2)])
@pytest.mark.parametrize("P", [16, 64, 1024])
@pytest.mark.parametrize("rope", [None, "halves", "pairs", "part"])
def test_append_and_read(fg, d, H, P, rope):
    """Codes and statistics of the (turned) rows in the right cells, every other byte as it was, and
    the values back."""
    lens, pos, first = [5, 0, 77, 1, 33], [0, 4, 30, 15, 64], 2
    h, rows = H * d, first + sum(lens) + 3
    buf = fg_synth.random_fp16((rows, 2 * h + 8), seed=d + P, scale=2.0)
    t = dev(buf)
    table, pages = tables(need([p + n for p, n in zip(pos, lens)], P), seed=P)
    pool = fg.KVPagesQ4(pages, P, h, H)
    pool.blocks.fill_(0xA5)
    before = host(pool.blocks).copy()
    off = offsets(lens, first)
    kw, k = {}, buf[:, :h].copy()
    at = np.concatenate([np.arange(p, p + n) for p, n in zip(pos, lens)]).astype(int)
    live = slice(first, first + sum(lens))
    if rope:
        rot = 16 if rope == "part" else d
        tab, angles = table_of(120, rot)
        kw = dict(angles=angles, interleaved=rope == "pairs")
        if rope == "part":                                   # positions of their own
            shift = [3, 0, 9, 100, 1]
            kw["rope_pos"] = i32(shift)
            turn_at = np.concatenate([np.arange(p, p + n) for p, n in zip(shift, lens)]).astype(int)
        else:
            turn_at = at
        k[live] = OP.turn(k[live], H, tab, turn_at, rope == "pairs")
    fg.fg_kv_append_q4_paged(t[:, :h], t[:, h:2 * h], i32(off), i32(pos), pool, dev(table), **kw)
    fg.fg_check_device_error()
    want = fg.KVPagesQ4.of(torch.from_numpy(before.copy()), d)
    seq = np.repeat(np.arange(len(lens)), lens)
    page, cell = table[seq, at // P], at % P
    restored = []
    for x, codes, ab in ((k, *want.parts()[:2]), (buf[:, h:2 * h], *want.parts()[2:])):
        q, a, b = OQ.quantize_g64(np.ascontiguousarray(x[live]).reshape(-1, d))
        codes.numpy()[page, :, cell] = OQ.pack_nibbles(q).reshape(-1, H, d // 2)
        ab.numpy()[page, :, cell] = np.stack([a, b], -1).reshape(-1, H, d // 64, 2)
        restored.append(OQ.dequant_g64(q, a, b).reshape(-1, h))
    assert np.array_equal(host(pool.blocks), want.blocks.numpy())

    out = torch.full((rows, 2 * h), 7.0, dtype=torch.float16, device="cuda")
    fg.fg_kv_read_q4_paged(pool, dev(table), i32(off), i32(pos), out[:, :h], out[:, h:])
    fg.fg_check_device_error()
    back = np.full((rows, 2 * h), 7.0, np.float16)
    back[live, :h], back[live, h:] = restored
    assert np.array_equal(host(out).view(np.uint16), back.view(np.uint16))
    only = torch.full((rows, h), 7.0, dtype=torch.float16, device="cuda")
    fg.fg_kv_read_q4_paged(pool, dev(table), i32(off), i32(pos), None, only)
    assert np.array_equal(host(only).view(np.uint16), back[:, h:].copy().view(np.uint16))


def test_append_extents_that_do_not_fit(fg):
    """Bad pages, positions past the table and turns past the angles: those rows are left out, the
    others written."""
    d, H, P = 64, 2, 16
    lens, pos = [4, 3, 2, 3], [14, 30, -1, 2]
    table = np.array([[3, 99], [1, 2], [0, 0], [4, 5]], np.int32)
    pool = fg.KVPagesQ4(6, P, H * d, H)
    x = fg_synth.random_fp16((12, 2 * H * d), seed=1)
    t = dev(x)
    tab, angles = table_of(32, d)
    fg.fg_kv_append_q4_paged(t[:, :H * d], t[:, H * d:], i32(offsets(lens)), i32(pos), pool,
                             dev(table), angles=angles, rope_pos=i32([0, 0, 0, 30]))
    with pytest.raises(fg.FgError) as e:
        fg.fg_check_device_error()
    assert e.value.status == fg.FG_ERR_CAPACITY
    written = {(3, 14): 0, (3, 15): 1, (2, 14): 4, (2, 15): 5, (4, 2): 9, (4, 3): 10}
    codes = host(pool.parts()[2])
    for page in range(6):
        for cell in range(P):
            row = written.get((page, cell))
            want = 0 if row is None else OQ.pack_nibbles(
                OQ.quantize_g64(x[row:row + 1, H * d:].reshape(-1, d))[0]).reshape(H, -1)
            assert np.array_equal(codes[page, :, cell], np.broadcast_to(want, (H, d // 2))), \
                (page, cell)


# ------------------------------------------------------------------------------- attention


def paged_case(fg, d, H, P, lens, nq, seed, G, first=1, scale=1.0):
    table, pages = tables(need(lens, P), seed=seed)
    pool, k, v = fill(fg, pages, P, H, d, seed, scale)
    q_off = offsets(nq, first)
    rows = first + sum(nq) + 2
    q = fg_synth.random_fp16((rows, H * G * d + 8), seed=seed + 50)
    return table, pool, k, v, q_off, q


def run_attend(fg, q, q_off, Hq, pool, table, lens, scale, out=None, lse=True, max_q=None, **kw):
    width = Hq * pool.d
    if out is None:
        out = torch.full((q.shape[0], width), 7.0, dtype=torch.float16, device="cuda")
    z = torch.full((q.shape[0], Hq), 7.0, device="cuda") if lse else None
    most = max(max_q or q.shape[0], 1)
    ws = torch.full((max(16, fg.fg_attn_paged_workspace_bytes(pool, Hq, most)),), 255,
                    dtype=torch.uint8, device="cuda")
    fg.fg_attn_q4kv_paged(q, i32(q_off), Hq, pool, dev(table), i32(lens), scale, out, ws, lse=z,
                          max_q=max_q, **kw)
    return out, z


def check_attend(got, z, q, q_off, Hq, k, v, table, lens, scale, window=0, sinks=0):
    """Every row within what the arithmetic allows of the oracle's.

    Scores: d + 40 binary32 operations on terms of size |q_j k_j|, and each k within restore_error; an
    error ds moves a weight by a factor within e^(+-2 ds).  Values: within restore_error.  Weights are
    rounded to fp16 (half a step; half of 2^-24 where they are subnormal, at most 2^-31 of the row's largest after their scaling), the exponential adds 2^-21,
    the sums n + 64 binary32 operations; last, the output's own half step."""
    got, z = host(got).astype(np.float64), None if z is None else host(z)
    H, d = k.shape[1], k.shape[3]
    G = Hq // H
    for b, n in enumerate(lens):
        rows = slice(q_off[b], q_off[b + 1])
        nq = q_off[b + 1] - q_off[b]
        if nq == 0:
            continue
        ok = OP.seen(n - nq, nq, n, window, sinks)
        for hk in range(H):
            kk, vv = rows_of(k, table, b, n)[hk], rows_of(v, table, b, n)[hk]
            qq = q[rows, hk * G * d:(hk + 1) * G * d].reshape(nq, G, d)
            o, lse, p = OP.attend(qq, kk, vv, ok, scale)
            mag = np.einsum("rgd,td->rgt", np.abs(qq.astype(np.float64)),
                            np.abs(kk.astype(np.float64))) * scale
            dk, dv = (restore_error(rows_of(x.big, table, b, n)[hk]) for x in (k, v))
            moved = np.einsum("rgd,td->rgt", np.abs(qq.astype(np.float64)), dk) * scale
            ds = np.where(ok[:, None], mag * (d + 40) * F32 + moved, 0).max(-1, initial=0.0)
            V = p @ np.abs(vv.astype(np.float64))
            vmax = np.abs(vv.astype(np.float64)).max(0, initial=0.0)
            tol = ((np.expm1(2 * ds)[..., None] + H16 + 2.0 ** -21 + (n + 64) * F32) * V
                   + p @ dv + n * 2.0 ** -31 * vmax + H16 * np.abs(o) + 2.0 ** -24)
            g = got[rows, hk * G * d:(hk + 1) * G * d].reshape(nq, G, d)
            err = np.abs(g - o)
            assert np.all(err <= tol), (b, hk, float((err - tol).max()), float(err.max()))
            if z is not None:
                zz = z[rows, hk * G:(hk + 1) * G]
                none = ~ok.any(1)
                assert np.all(zz[none] == -np.inf)
                zt = 2 * ds + 2.0 ** -20 + (n + 64) * F32 + np.abs(np.where(none[:, None], 0, lse)) \
                    * 4 * F32
                assert np.all(np.abs(zz[~none] - lse[~none]) <= zt[~none]), (b, hk)


SHAPES = [
    # d, H, G, page, lens, nq, window, sinks
    (128, 2, 1, 16, [1], [1], 0, 0),
    (64, 1, 1, 16, [1, 16, 17, 0, 33], [1, 1, 1, 0, 1], 0, 0),
    (128, 2, 4, 16, [130, 257, 3], [1, 1, 1], 0, 0),
    (128, 1, 7, 32, [300, 40, 129], [5, 40, 1], 0, 0),
    (64, 2, 8, 64, [700, 128, 65], [20, 128, 2], 0, 0),
    (128, 2, 1, 256, [600, 511], [300, 200], 0, 0),
    (128, 3, 2, 16, [257, 1, 400], [257, 1, 33], 0, 0),
    (64, 1, 5, 128, [1000, 77], [60, 77], 100, 4),
    (128, 2, 4, 64, [900, 500, 129], [1, 130, 129], 64, 0),
    (128, 1, 8, 16, [400, 90], [17, 90], 1, 1),
    (64, 4, 1, 32, [2100], [3], 0, 0),
    (64, 1, 128, 1024, [1500, 10], [2, 10], 300, 17),
    (128, 1, 40, 16, [333], [9], 0, 0),
]


@pytest.mark.parametrize("d,H,G,P,lens,nq,window,sinks", SHAPES)
def test_attention(fg, d, H, G, P, lens, nq, window, sinks):
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, sum(lens) + d, G)
    t, width, scale = dev(q), H * G * d, 1.0 / math.sqrt(d)
    kw = dict(window=window, sinks=sinks)
    for max_q in (None, max(nq)):
        out, z = run_attend(fg, t[:, :width], q_off, H * G, pool, table, lens, scale, max_q=max_q,
                            **kw)
        fg.fg_check_device_error()
        check_attend(out, z, q, q_off, H * G, k, v, table, lens, scale, window, sinks)
        outside = np.r_[0:q_off[0], q_off[-1]:len(q)]        # rows of no sequence
        assert np.all(host(out)[outside] == 7.0) and np.all(host(z)[outside] == 7.0)
    # in place, into rows of another width, and without the log-sum-exp
    same, _ = run_attend(fg, t[:, :width], q_off, H * G, pool, table, lens, scale, out=t[:, :width],
                         lse=False, max_q=max(nq), **kw)
    live = slice(q_off[0], q_off[-1])
    assert torch.equal(same[live], out[live])
    assert np.array_equal(host(t)[:, width:], q[:, width:])


def test_attention_rows_before_the_first_position(fg):
    """More query rows than cached positions: the first rows see nothing and get 0."""
    d, H, G, P, lens, nq = 64, 2, 2, 16, [5, 0, 130], [9, 3, 140]
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 3, G)
    out, z = run_attend(fg, dev(q)[:, :H * G * d], q_off, H * G, pool, table, lens, 0.125)
    fg.fg_check_device_error()
    check_attend(out, z, q, q_off, H * G, k, v, table, lens, 0.125)
    assert not host(out)[1:5].any() and not host(out)[10:13].any()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("which", [0, 1])
def test_values_of_masked_positions_do_not_show(fg, bad, which):
    """K or V of a position with an infinity or NaN: only rows that see it show it, whatever else
    shares their tile; stale bytes behind a sequence never do."""
    d, H, G, P, lens, nq = 64, 1, 2, 16, [150, 40], [120, 1]
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 11, G)
    t, scale = dev(q), 0.125
    clean, _ = run_attend(fg, t[:, :G * d], q_off, G, pool, table, lens, scale)
    clean = host(clean).copy()
    ab = pool.parts()[1 + 2 * which]
    at = 100                                                 # seen by rows at positions 100 ..
    ab[table[0, at // P], 0, at % P, 0, 1] = bad
    for p in range(lens[0], need(lens, P)[0] * P):           # behind the sequences
        ab[table[0, p // P], 0, p % P] = bad
    for p in range(lens[1], need(lens, P)[1] * P):
        ab[table[1, p // P], 0, p % P] = bad
    out, _ = run_attend(fg, t[:, :G * d], q_off, G, pool, table, lens, scale)
    fg.fg_check_device_error()
    out = host(out)
    sees = 1 + at - (lens[0] - nq[0])                        # its first query row, packed
    # (rows computed on their own may take their sums in another order)
    a, c = out[1:sees].astype(np.float64), clean[1:sees].astype(np.float64)
    assert np.all(np.abs(a - c) <= 4 * H16 * np.abs(c) + 2.0 ** -10 * np.abs(c).max())
    assert np.array_equal(out[121], clean[121])
    assert not np.isfinite(out[sees:121]).all(axis=1).any()


def test_attention_extents_that_do_not_fit(fg):
    """Bad offsets, lengths, row counts and pages are reported; the other sequences are right."""
    d, H, G, P, lens, nq = 64, 2, 1, 16, [40, 50, 20, 33], [2, 1, 3, 1]
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 21, G)
    t, scale, width = dev(q), 0.125, H * G * d

    def broken(what):
        out, _ = run_attend(fg, t[:, :width], q_off, H * G, pool, what.get("table", table),
                            what.get("lens", lens), scale, max_q=what.get("max_q"))
        with pytest.raises(fg.FgError) as e:
            fg.fg_check_device_error()
        assert e.value.status == fg.FG_ERR_CAPACITY
        return host(out)

    good = host(run_attend(fg, t[:, :width], q_off, H * G, pool, table, lens, scale)[0])
    fg.fg_check_device_error()
    for what, rows in ((dict(lens=[40, 50, 65, 33]), slice(4, 7)),
                       (dict(lens=[40, -1, 20, 33]), slice(3, 4)),
                       (dict(max_q=2), slice(4, 7))):
        out = broken(what)
        others = np.r_[1:rows.start, rows.stop:8]
        assert np.all(out[rows] == 7.0), what
        assert np.array_equal(out[others], good[others]), what
    wrong = table.copy()
    wrong[1, 2] = pool.pages
    out = broken(dict(table=wrong))
    assert np.array_equal(out[np.r_[1:3, 4:8]], good[np.r_[1:3, 4:8]])


# ------------------------------------------------------------------------------- weights, eviction


@pytest.mark.parametrize("d,H,G,P,lens,nq,window,sinks", SHAPES)
def test_weights(fg, d, H, G, P, lens, nq, window, sinks):
    """Scores as in the attention's bound, a term's exponential 2^-21 more and the given log-sum-exp's
    own rounding; one binary32 sum per term.  What lies behind a sequence stays."""
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, sum(lens) + d, G)
    scale, Hq = 1.0 / math.sqrt(d), H * G
    lse = np.full((len(q), Hq), np.nan, np.float32)
    n_acc = max(lens) + 5
    acc = np.random.default_rng(1).random((len(lens), H, n_acc)).astype(np.float32)
    want, tol = acc.astype(np.float64), np.zeros(acc.shape)
    for b, n in enumerate(lens):
        nb = nq[b]
        if nb == 0 or n == 0:
            continue
        ok = OP.seen(n - nb, nb, n, window, sinks)
        for hk in range(H):
            qq = q[q_off[b]:q_off[b + 1], hk * G * d:(hk + 1) * G * d].reshape(nb, G, d)
            kk = rows_of(k, table, b, n)[hk]
            _, z, _ = OP.attend(qq, kk, kk, ok, scale)
            z = z.astype(np.float32)
            lse[q_off[b]:q_off[b + 1], hk * G:(hk + 1) * G] = z
            with np.errstate(invalid="ignore"):
                w = np.exp(OP.scores(qq, kk, ok, scale) - z[..., None].astype(np.float64))
            w = np.where(ok[:, None], w, 0.0)
            mag = np.einsum("rgd,td->rgt", np.abs(qq.astype(np.float64)),
                            np.abs(kk.astype(np.float64))) * scale
            rel = mag * (d + 40) * F32 + np.abs(np.where(np.isfinite(z), z, 0))[..., None] * 4 * F32 \
                + 2.0 ** -21
            want[b, hk, :n] += w.sum((0, 1))
            tol[b, hk, :n] = (w * np.expm1(rel)).sum((0, 1)) \
                + want[b, hk, :n] * (nb * G + 8) * F32
    args = (dev(q)[:, :Hq * d], i32(q_off), Hq, pool, dev(table), i32(lens), scale, dev(lse))
    kw = dict(window=window, sinks=sinks, max_q=max(nq))
    out = torch.full(acc.shape, 7.0, device="cuda")
    fg.fg_attn_weights_q4_paged(*args, dev(acc), out, **kw)
    fg.fg_check_device_error()
    got = host(out)
    for b, n in enumerate(lens):
        err = np.abs(got[b, :, :n] - want[b, :, :n])
        assert np.all(err <= tol[b, :, :n] + 2.0 ** -24 * want[b, :, :n]), (b, err.max())
        assert np.all(got[b, :, n:] == 7.0)
    # in place; from nothing; and the same bits again
    same = dev(acc)
    fg.fg_attn_weights_q4_paged(*args, same, same, **kw)
    for b, n in enumerate(lens):
        assert torch.equal(same[b, :, :n], out[b, :, :n])
        assert np.array_equal(host(same)[b, :, n:], acc[b, :, n:])
    zero, none = torch.zeros(acc.shape, device="cuda"), torch.zeros(acc.shape, device="cuda")
    fg.fg_attn_weights_q4_paged(*args, zero.clone(), zero, **kw)
    fg.fg_attn_weights_q4_paged(*args, None, none, **kw)
    assert torch.equal(zero, none)


@pytest.mark.parametrize("d,H,P", [(64, 2, 16), (128, 3, 64)])
@pytest.mark.parametrize("lens,keep,recent", [([1, 0, 40, 41, 200], 40, 8), ([1500, 2500], 1000, 0),
                                              ([300, 37], 33, 33), ([64, 5000], 1, 0),
                                              ([3000], 2049, 1)])
@pytest.mark.parametrize("kind", ["random", "ties", "extremes"])
def test_evict(fg, d, H, P, lens, keep, recent, kind):
    both = need(lens, P) + [(keep + P - 1) // P] * len(lens)
    all_tables, pages = tables(both, seed=keep)
    src = np.ascontiguousarray(all_tables[:len(lens)])
    dst = np.ascontiguousarray(all_tables[len(lens):, :both[-1]])
    pool, _, _ = fill(fg, pages, P, H, d, 4)
    n_acc = max(lens) + 3
    rng = np.random.default_rng(keep + recent)
    acc = rng.random((len(lens), H, n_acc)).astype(np.float32)
    if kind == "ties":
        acc = np.floor(acc * 3).astype(np.float32)
    if kind == "extremes":
        acc[rng.random(acc.shape) < 0.2] = np.inf
        acc[rng.random(acc.shape) < 0.2] = 0.0
        acc[rng.random(acc.shape) < 0.2] = -1.5
        acc[rng.random(acc.shape) < 0.1] = 1e-42
    before = host(pool.blocks).copy()
    kept = torch.full((len(lens), H, keep), 99, dtype=torch.int32, device="cuda")
    acc_out = torch.full((len(lens), H, keep), 7.0, device="cuda")
    dst_lens = torch.full((len(lens),), 99, dtype=torch.int32, device="cuda")
    fg.fg_kv_evict_q4_paged(pool, dev(src), i32(lens), dev(acc), recent, dev(dst), kept, acc_out,
                            dst_lens)
    fg.fg_check_device_error()
    want = fg.KVPagesQ4.of(torch.from_numpy(before.copy()), d)
    old = fg.KVPagesQ4.of(torch.from_numpy(before), d)
    assert host(dst_lens).tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        for h in range(H):
            at = OP.evict(acc[b, h], n, keep, recent)
            m = len(at)
            assert np.array_equal(host(kept)[b, h, :m], at), (b, h)
            assert np.all(host(kept)[b, h, m:] == -1) and np.all(host(acc_out)[b, h, m:] == 0)
            assert np.array_equal(host(acc_out)[b, h, :m], acc[b, h, at])
            to = np.arange(m)
            for x, y in zip(old.parts(), want.parts()):
                y.numpy()[dst[b, to // P], h, to % P] = x.numpy()[src[b, at // P], h, at % P]
    # the pages of dst behind a sequence's last kept position are nobody's: only they may differ
    got = fg.KVPagesQ4.of(pool.blocks.cpu(), d)
    for g, w in zip(got.parts(), want.parts()):
        assert torch.equal(g, w)


def test_evict_extents_that_do_not_fit(fg):
    d, H, P, lens, keep = 64, 1, 16, [40, 30, 50], 20
    all_tables, pages = tables(need(lens, P) + [2, 2, 2], seed=9)
    src, dst = all_tables[:3].copy(), np.ascontiguousarray(all_tables[3:, :2])
    pool, _, _ = fill(fg, pages, P, H, d, 4)
    before = host(pool.blocks).copy()
    src[0, 0] = -1                                           # a bad page; position 0 stays of it
    acc = np.zeros((3, H, 45), np.float32)
    acc[:, :, 0] = 1.0
    kept = torch.zeros((3, H, keep), dtype=torch.int32, device="cuda")
    acc_out = torch.zeros((3, H, keep), device="cuda")
    dst_lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    # 50 positions do not fit 45 weights: nothing stays of that sequence
    fg.fg_kv_evict_q4_paged(pool, dev(src), i32(lens), dev(acc), 5, dev(dst), kept, acc_out,
                            dst_lens)
    with pytest.raises(fg.FgError) as e:
        fg.fg_check_device_error()
    assert e.value.status == fg.FG_ERR_CAPACITY
    assert host(dst_lens).tolist() == [20, 20, 0]
    got, old = fg.KVPagesQ4.of(pool.blocks.cpu(), d), fg.KVPagesQ4.of(torch.from_numpy(before), d)
    assert np.array_equal(got.parts()[0][dst[2]], old.parts()[0][dst[2]])
    at = OP.evict(acc[1, 0], 30, keep, 5)
    for g, o in zip(got.parts(), old.parts()):
        to = np.arange(keep)
        assert np.array_equal(g[dst[1, to // P], 0, to % P], o[src[1, at // P], 0, at % P])


# ------------------------------------------------------------------------------- together


def test_generation_over_pages(fg):
    """Two prompts in pieces with rotary positions, weights received, caches made smaller, and steps
    behind them, the whole against the oracle's own cache."""
    d, H, G, P = 64, 2, 2, 16
    Hq, scale = H * G, 0.125
    h, rng = H * d, np.random.default_rng(0)
    tab, angles = table_of(400, d)
    pool = fg.KVPagesQ4(80, P, h, H)
    order = rng.permutation(80)
    table, after = order[:40].reshape(2, 20).astype(np.int32), order[40:].reshape(2, 20)
    after = after.astype(np.int32)
    K, V = ([[np.zeros((0, d), np.float16) for _ in range(H)] for _ in range(2)] for _ in range(2))
    acc = torch.zeros((2, H, 320), device="cuda")
    acc_ref, acc_tol = np.zeros((2, H, 320)), np.zeros((2, H, 320))
    pos, rope_pos = [0, 0], [0, 0]

    def step(nq, table):
        rows = sum(nq)
        qkv = rng.standard_normal((rows, (Hq + 2 * H) * d)).astype(np.float16)
        t, off = dev(qkv), offsets(nq)
        q = t[:, :Hq * d]
        fg.fg_rope(q, d, i32(off), i32(rope_pos), angles, q)
        fg.fg_kv_append_q4_paged(t[:, Hq * d:Hq * d + h], t[:, Hq * d + h:], i32(off), i32(pos), pool,
                                 dev(table), angles=angles, rope_pos=i32(rope_pos))
        at = np.concatenate([np.arange(p, p + n) for p, n in zip(rope_pos, nq)]).astype(int)
        qr = OP.turn(qkv[:, :Hq * d], Hq, tab, at, False)
        kr = OP.turn(np.ascontiguousarray(qkv[:, Hq * d:Hq * d + h]), H, tab, at, False)
        for b in range(2):
            r = slice(off[b], off[b + 1])
            for hk in range(H):
                c = slice(hk * d, hk * d + d)
                for store, x in ((K, kr[r, c]), (V, qkv[r, Hq * d + h:][:, c])):
                    new = OQ.dequant_g64(*OQ.quantize_g64(np.ascontiguousarray(x)))
                    store[b][hk] = np.concatenate([store[b][hk], new])
            pos[b] += nq[b]
            rope_pos[b] += nq[b]
        out, lse = run_attend(fg, q, off, Hq, pool, table, pos, scale, max_q=max(nq))
        fg.fg_attn_weights_q4_paged(q, i32(off), Hq, pool, dev(table), i32(pos), scale, lse, acc, acc,
                                    max_q=max(nq))
        fg.fg_check_device_error()
        got = host(out).astype(np.float64)
        for b in range(2):
            r, n = slice(off[b], off[b + 1]), pos[b]
            ok = OP.seen(n - nq[b], nq[b], n, 0, 0)
            for hk in range(H):
                qq = qr[r, hk * G * d:(hk + 1) * G * d].reshape(nq[b], G, d)
                o, _, p = OP.attend(qq, K[b][hk], V[b][hk], ok, scale)
                g = got[r, hk * G * d:(hk + 1) * G * d].reshape(nq[b], G, d)
                # (as in check_attend, with 8 > 4.1 times a row's largest value for its groups' M)
                dk, dv = (restore_error(2 * np.abs(x[b][hk].astype(np.float64)).max(1, keepdims=True))
                          for x in (K, V))
                ds = (np.abs(qq.astype(np.float64)).sum(-1) * dk.max(initial=0) * scale
                      + 2.0 ** -12)[..., None]
                tol = ((np.expm1(2 * ds) + 2 * H16) * (p @ np.abs(V[b][hk].astype(np.float64)))
                       + p @ np.broadcast_to(dv, V[b][hk].shape) + H16 * np.abs(o) + 2.0 ** -20)
                assert np.all(np.abs(g - o) <= tol)
                acc_ref[b, hk, :n] += p.sum((0, 1))
                # the log-sum-exp that the attention gives is within ds too
                acc_tol[b, hk, :n] += (p * np.expm1(2 * ds)).sum((0, 1))
        for b in range(2):
            n = pos[b]
            err = np.abs(host(acc)[b, :, :n] - acc_ref[b, :, :n])
            assert np.all(err <= acc_tol[b, :, :n] + 2.0 ** -16 * acc_ref[b, :, :n])

    for nq in ([130, 1], [77, 90], [1, 1]):
        step(nq, table)
    keep, recent = 96, 32
    kept = torch.empty((2, H, keep), dtype=torch.int32, device="cuda")
    acc_out = torch.empty((2, H, keep), device="cuda")
    dst_lens = torch.empty(2, dtype=torch.int32, device="cuda")
    old = host(acc)
    fg.fg_kv_evict_q4_paged(pool, dev(table), i32(pos), acc, recent, dev(after), kept, acc_out,
                            dst_lens)
    fg.fg_check_device_error()
    acc.zero_()
    acc[:, :, :keep] = acc_out
    acc_ref[:] = acc_tol[:] = 0.0
    for b in range(2):
        for hk in range(H):
            at = OP.evict(old[b, hk], pos[b], keep, recent)
            assert np.array_equal(host(kept)[b, hk, :len(at)], at)
            K[b][hk], V[b][hk] = K[b][hk][at], V[b][hk][at]
            acc_ref[b, hk, :len(at)] = old[b, hk, at]
        pos[b] = min(pos[b], keep)
    assert host(dst_lens).tolist() == pos
    for nq in ([1, 1], [1, 1], [20, 1]):
        step(nq, after)
