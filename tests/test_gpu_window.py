"""The ragged cache calls and the windowed attention against the 64-bit oracle, on the GPU.

Codes, statistics and restored values are compared bit for bit.  Attention outputs are compared
element by element with a bound that follows the arithmetic (see `bound`)."""
import numpy as np
import pytest
import torch

import fg_synth
from oracle import quant as OQ
from oracle import window as OW
from parity_util import dev, host, lib

pytestmark = pytest.mark.gpu

H16 = 2.0 ** -11          # half a step of fp16, relative
F32 = 2.0 ** -23          # one binary32 operation, rounded or truncated, relative


@pytest.fixture(scope="module")
def fg():
    return lib()


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def offsets(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(int).tolist()


def bound(o, info, d, restore):
    """Largest error of one output row that the arithmetic allows.

    Scores: d + 40 binary32 operations on terms of size kmag, and (restore: the cache's values
    enter unrounded where their definition rounds them to fp16) half an fp16 step of each k.
    A score error ds moves every weight by a factor within e^(+-2 ds).  Values: the same half step;
    weights rounded to fp16 (half a step of the terms they multiply; below fp16's normal range half
    of 2^-24, of up to 16 times a value's step, or of a value); n + 64 binary32 sums; the
    exponential's 2^-21.  Last, the output's own half step."""
    n = info["n"]
    ds = info["qkmag"] * (d + 40) * F32
    rel = 0.0
    if restore:
        ds += info["qk"] * H16 + info["q1"] * 2.0 ** -25
        rel = H16
    tiny = n * 2.0 ** -25 / info["l"] * (16.0 if restore else info["vmax"])
    return ((np.expm1(2 * ds) + rel) * info["A"]
            + (H16 + 2.0 ** -21 + (n + 64) * F32) * info["V"]
            + tiny + H16 * np.abs(o) + 2.0 ** -24)


def check_rows(got, want, d, restore, what):
    """got [rows][Hq*d] fp16; want: {row: (o, infos)}."""
    got = host(got).astype(np.float64)
    for row, (o, infos) in want.items():
        g = got[row].reshape(len(infos), d)
        for hq, info in enumerate(infos):
            tol = bound(o[hq], info, d, restore)
            err = np.abs(g[hq] - o[hq])
            assert np.all(err <= tol), (what, row, hq, float((err - tol).max()), float(err.max()))
            if info["n"] == 0:
                assert not g[hq].any(), (what, row, hq)


def fill_cache(fg, B, H, d, cap, seed, scale=1.0):
    """A cache filled with quantised normal values; its restored values (numpy) and the size
    |a| + (b - a) of the terms they are made from, [B][H][cap][d]."""
    cache = fg.KVCacheQ4(B, cap, H * d, H)
    vals, mags = [], []
    for codes_t, ab_t, sd in ((cache.k_codes, cache.k_ab, 0), (cache.v_codes, cache.v_ab, 1)):
        x = fg_synth.random_fp16((B * H * cache.cap, d), seed=seed * 2 + sd, scale=scale,
                                 offset=0.2 * scale)
        q, a, b = OQ.quantize_g64(x)
        codes_t.copy_(dev(OQ.pack_nibbles(q)).view(codes_t.shape))
        ab_t.copy_(dev(OQ.ab_pack_u32(a, b).view(np.int32)).view(ab_t.shape))
        vals.append(OQ.dequant_g64(q, a, b).reshape(B, H, cache.cap, d))
        mag = np.abs(a.astype(np.float64)) + (b.astype(np.float64) - a.astype(np.float64))
        mags.append(np.repeat(mag, 64, axis=1).reshape(B, H, cache.cap, d))
    return cache, vals[0], vals[1], mags[0], mags[1]


def run_decode(fg, q, Hq, cache, lens, scale, window, sinks, out=None):
    if out is None:
        out = torch.full((cache.B, Hq * cache.d), 7.0, dtype=torch.float16, device="cuda")
    n = fg.fg_decode_attn_window_workspace_bytes(cache, Hq)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")   # not initialised to 0
    fg.fg_decode_attn_q4kv_window(q, Hq, cache, lens, scale, out, ws, window=window, sinks=sinks)
    return out


# ------------------------------------------------------------------------------- append, read


def ragged_case(fg, B, H, d, lens, pos, cap, first, spare, seed, x=None):
    """K/V column blocks of one buffer, rows before the first and behind the last sequence."""
    h = H * d
    rows = first + sum(lens) + spare
    buf = fg_synth.random_fp16((rows, 2 * h + 8), seed=seed, scale=2.0)
    if x is not None:
        buf[:, :2 * h] = x
    t = dev(buf)
    cache = fg.KVCacheQ4(B, cap, h, H)
    for c in (cache.k_codes, cache.v_codes):
        c.fill_(0xA5)
    for a in (cache.k_ab, cache.v_ab):
        a.fill_(0x5A5A5A5A)
    return buf, t, cache, i32(offsets(lens, first)), i32(pos)


RAGGED = [
    # B, H, d, lens, pos, cap, rows before, rows behind
    (1, 1, 64, [1], [0], 16, 0, 0),
    (3, 4, 64, [5, 0, 7], [2, 9, 0], 16, 0, 0),
    (4, 2, 128, [1, 1, 1, 1], [15, 0, 7, 31], 32, 0, 0),
    (5, 3, 128, [33, 1, 0, 64, 200], [0, 99, 3, 36, 17], 224, 2, 3),
    (3, 8, 128, [0, 0, 0], [0, 5, 16], 16, 4, 1),
    (2, 12, 64, [129, 300], [3, 0], 304, 1, 0),
    (70, 1, 128, [i % 4 for i in range(70)], [i % 13 for i in range(70)], 16, 0, 5),
]


@pytest.mark.parametrize("B,H,d,lens,pos,cap,first,spare", RAGGED)
def test_append_and_read_bit_exact(fg, B, H, d, lens, pos, cap, first, spare):
    h = H * d
    buf, t, cache, off, ps = ragged_case(fg, B, H, d, lens, pos, cap, first, spare, seed=B + cap)
    fg.fg_kv_append_q4_ragged(t[:, :h], t[:, h:2 * h], off, ps, cache)
    fg.fg_check_device_error()
    o = offsets(lens, first)
    want_vals = []
    for j, (codes_t, ab_t) in enumerate(((cache.k_codes, cache.k_ab),
                                         (cache.v_codes, cache.v_ab))):
        q, a, b = OQ.quantize_g64(np.ascontiguousarray(buf[:, j * h:(j + 1) * h]))
        codes, ab = OQ.pack_nibbles(q), OQ.ab_pack_u32(a, b)
        want_vals.append(OQ.dequant_g64(q, a, b))
        wc = np.full((B, H, cap, d // 2), 0xA5, np.uint8)
        wa = np.full((B, H, cap, d // 64), 0x5A5A5A5A, np.uint32)
        for s in range(B):
            n, p = lens[s], pos[s]
            wc[s, :, p:p + n] = codes[o[s]:o[s] + n].reshape(n, H, d // 2).transpose(1, 0, 2)
            wa[s, :, p:p + n] = ab[o[s]:o[s] + n].reshape(n, H, d // 64).transpose(1, 0, 2)
        assert np.array_equal(host(codes_t), wc)          # and everything else untouched
        assert np.array_equal(host(ab_t).view(np.uint32), wa)
    # read it back beside untouched rows and columns; then each half alone
    rows = t.shape[0]
    for which in ("kv", "k", "v"):
        out = torch.full((rows, 2 * h + 16), 7.0, dtype=torch.float16, device="cuda")
        fg.fg_kv_read_q4_ragged(cache, off, ps, out[:, :h] if "k" in which else None,
                                out[:, h:2 * h] if "v" in which else None)
        fg.fg_check_device_error()
        want = np.full((rows, 2 * h + 16), 7.0, np.float16)
        r = slice(first, first + sum(lens))
        for j, name in enumerate("kv"):
            if name in which:
                want[r, j * h:(j + 1) * h] = want_vals[j][r]
        assert np.array_equal(host(out).view(np.uint16), want.view(np.uint16)), which


def test_append_unusual_values_as_quantize(fg):
    """Ties, constant groups, signed zeros, extremes, infinities and NaN: the bits of
    fg_quantize_g64 on the same rows."""
    rows = fg_synth.adversarial_groups_fp16()
    odd = fg_synth.random_fp16((8, 64), 5)
    odd[0, 3], odd[1, 9], odd[2, 0], odd[2, 1] = np.inf, -np.inf, np.inf, -np.inf
    odd[3, 7], odd[4, :], odd[5, 60] = np.nan, np.nan, -np.nan
    odd[6, 5], odd[6, 6] = np.nan, np.inf
    odd[7].view(np.uint16)[11] = 0xFFFF                      # a NaN with its sign bit set
    g = np.concatenate([rows, odd])
    g = np.concatenate([g, g[::-1]])[:2 * (len(g) // 2) * 2]
    x = g.reshape(-1, 2, 64).reshape(-1, 128)                # rows of one head, d = 128
    n = x.shape[0]
    t = dev(np.concatenate([x, x[::-1]], axis=1))            # K and V
    cache = fg.KVCacheQ4(1, n, 128, 1)
    fg.fg_kv_append_q4_ragged(t[:, :128], t[:, 128:], i32([0, n]), i32([0]), cache)
    for src, codes_t, ab_t in ((t[:, :128], cache.k_codes, cache.k_ab),
                               (t[:, 128:], cache.v_codes, cache.v_ab)):
        codes = torch.empty((n, 64), dtype=torch.uint8, device="cuda")
        ab = torch.empty((n, 2), dtype=torch.int32, device="cuda")
        fg.fg_quantize_g64(src.contiguous(), codes, ab)
        assert torch.equal(codes_t[0, 0, :n], codes)
        assert torch.equal(ab_t[0, 0, :n], ab)
    out = torch.empty((n, 128), dtype=torch.float16, device="cuda")
    fg.fg_kv_read_q4_ragged(cache, i32([0, n]), i32([0]), None, out)
    y = torch.empty_like(out)
    fg.fg_dequant_g64(cache.v_codes[0, 0, :n].contiguous(), cache.v_ab[0, 0, :n].contiguous(), n,
                      128, y)
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(out[~nan].view(torch.int16), y[~nan].view(torch.int16))


@pytest.mark.parametrize("off,pos", [
    ([0, 4, 2, 8], [0, 0, 0]),            # offsets that fall
    ([0, 2, 4, 9], [0, 0, 0]),            # past the rows
    ([-3, 2, 4, 8], [0, 0, 0]),           # before them
    ([0, 2, 4, 8], [0, 15, 0]),           # positions past the capacity
    ([0, 2, 4, 8], [0, -1, 0]),
    ([0, 2, 4, 8], [2 ** 31 - 1, -2 ** 31, 0]),
])
def test_extents_that_do_not_fit(fg, off, pos):
    """Nothing outside the buffers is touched, what fits is written, and the error is told once."""
    h, rows = 128, 8
    x = fg_synth.random_fp16((rows, h), 3)
    guard = torch.full((3, 1, 16, 64), 0xA5, dtype=torch.uint8, device="cuda")
    cache = fg.KVCacheQ4(3, 16, h, 1)
    t = dev(x)
    fg.fg_check_device_error()
    fg.fg_kv_append_q4_ragged(t, t, i32(off), i32(pos), cache)
    with pytest.raises(fg.FgError) as e:
        fg.fg_check_device_error()
    assert e.value.status == fg.FG_ERR_CAPACITY
    out = torch.full((rows, h), 7.0, dtype=torch.float16, device="cuda")
    fg.fg_kv_read_q4_ragged(cache, i32(off), i32(pos), out, None)
    with pytest.raises(fg.FgError):
        fg.fg_check_device_error()
    fg.fg_check_device_error()                               # told once
    assert bool((guard == 0xA5).all())
    if off == [0, 2, 4, 8] and pos[2] == 0:                  # the sequences that fit are there
        q, a, b = OQ.quantize_g64(x)
        assert np.array_equal(host(out)[4:8], OQ.dequant_g64(q, a, b)[4:8])
        if pos[1] < 0:
            assert bool((out[2:4] == 7.0).all())


# ------------------------------------------------------------------------------- decode


DECODE = [
    # B, Hq, H, d, lens, window, sinks
    (1, 1, 1, 64, [1], 0, 0),
    (3, 4, 4, 64, [0, 16, 17], 0, 0),
    (2, 4, 4, 128, [15, 300], 0, 0),
    (4, 2, 2, 128, [48, 49, 47, 96], 1, 0),
    (4, 3, 3, 64, [5, 64, 200, 333], 16, 4),
    (5, 2, 2, 128, [1, 20, 21, 150, 512], 17, 1),
    (3, 4, 2, 128, [100, 0, 511], 100, 16),
    (3, 6, 2, 64, [100, 33, 480], 33, 20),
    (2, 8, 2, 128, [511, 77], 250, 64),
    (2, 7, 1, 128, [400, 31], 64, 3),
    (2, 16, 2, 64, [257, 512], 128, 5),
    (2, 9, 1, 128, [400, 129], 0, 0),
    (2, 16, 1, 128, [500, 16], 90, 40),
    (3, 4, 1, 64, [512, 300, 1], 5, 1000),       # sinks past every length: all visible
    (3, 2, 1, 128, [512, 300, 1], 10000, 2),     # a window past every length
    (37, 2, 2, 64, [(i * 7) % 41 for i in range(37)], 9, 2),
    (1, 32, 32, 128, [5000], 0, 0),
    (1, 8, 1, 128, [9000], 4097, 33),
]


@pytest.mark.parametrize("B,Hq,H,d,lens,window,sinks", DECODE)
def test_decode_window(fg, B, Hq, H, d, lens, window, sinks):
    cap = max(16, max(lens) + 5)
    cache, k, v, km, vm = fill_cache(fg, B, H, d, cap, seed=B * 31 + Hq)
    q16 = fg_synth.random_fp16((B, Hq * d + 24), seed=Hq + d)
    q = dev(q16)[:, :Hq * d]
    buf = torch.full((B, Hq * d + 8), 7.0, dtype=torch.float16, device="cuda")
    scale = 1.0 / np.sqrt(d)
    run_decode(fg, q, Hq, cache, i32(lens), scale, window, sinks, out=buf[:, :Hq * d])
    fg.fg_check_device_error()
    want = OW.decode(q16, k, v, lens, Hq, window, sinks, np.float32(scale), km, vm)
    check_rows(buf[:, :Hq * d], dict(enumerate(want)), d, True, "decode")
    assert bool((buf[:, Hq * d:] == 7.0).all())


@pytest.mark.parametrize("scale_x", [1e-3, 30.0, 3000.0])
def test_decode_window_magnitudes(fg, scale_x):
    """Small and large cached values (the largest near fp16's range)."""
    B, Hq, H, d, lens = 2, 4, 2, 128, [130, 61]
    cache, k, v, km, vm = fill_cache(fg, B, H, d, 144, seed=9, scale=scale_x)
    q16 = fg_synth.random_fp16((B, Hq * d), seed=2, scale=1.0 / scale_x)
    out = run_decode(fg, dev(q16), Hq, cache, i32(lens), 0.1, 50, 7)
    want = OW.decode(q16, k, v, lens, Hq, 50, 7, np.float32(0.1), km, vm)
    check_rows(out, dict(enumerate(want)), d, True, f"decode x {scale_x}")


def test_decode_window_widest_groups(fg):
    """Groups that span fp16's whole range (b - a = 131008): no weight overflows."""
    d, n = 128, 40
    x = np.zeros((n, d), np.float16)
    x[:, ::2], x[:, 1::2] = 65504.0, -65504.0
    x[:, 5] = 100.0
    t = dev(x)
    z = torch.zeros_like(t)
    cache = fg.KVCacheQ4(1, n, d, 1)
    fg.fg_kv_append_q4_ragged(z, t, i32([0, n]), i32([0]), cache)
    out = run_decode(fg, torch.ones((1, d), dtype=torch.float16, device="cuda"), 1, cache,
                     i32([n]), 0.1, 0, 0)
    q, a, b = OQ.quantize_g64(x)
    want = OQ.dequant_g64(q, a, b).astype(np.float64).mean(axis=0)
    got = host(out).astype(np.float64)[0]
    assert np.all(np.isfinite(got)) and np.abs(got - want).max() <= 131008 * 2.0 ** -9


@pytest.mark.parametrize("d,H,G", [(128, 2, 1), (64, 1, 4)])
def test_decode_window_masked_positions_may_hold_anything(fg, d, H, G):
    """Positions behind a sequence and between the first ones and the window hold infinities and
    NaN: the outputs are those of a clean cache, bit for bit."""
    B, cap, lens, window, sinks = 3, 160, [70, 145, 33], 37, 5
    cache, *_ = fill_cache(fg, B, H, d, cap, seed=4)
    q = dev(fg_synth.random_fp16((B, H * G * d), seed=8))
    clean = run_decode(fg, q, H * G, cache, i32(lens), 0.09, window, sinks).clone()
    for b, n in enumerate(lens):
        hide = [t for t in range(cap) if t >= n or (sinks <= t <= n - 1 - window)]
        for ab in (cache.k_ab, cache.v_ab):
            ab[b, :, hide[::2]] = 0x7C00FC00          # (-inf, inf)
            ab[b, :, hide[1::2]] = 0x7E007E00         # (NaN, NaN)
        for c in (cache.k_codes, cache.v_codes):
            c[b, :, hide] = 0xFF
    dirty = run_decode(fg, q, H * G, cache, i32(lens), 0.09, window, sinks)
    assert torch.equal(clean, dirty) and bool(torch.isfinite(dirty).all())


def test_decode_window_matches_dense_call(fg):
    """Equal lengths, no window, one query head per K/V head: what fg_decode_attn_q4kv gives."""
    B, H, d, n = 4, 4, 128, 333
    cache, *_ = fill_cache(fg, B, H, d, n, seed=12)
    q = dev(fg_synth.random_fp16((B, H * d), seed=1))
    a = run_decode(fg, q, H, cache, i32([n] * B), 0.08, 0, 0)
    b = torch.empty_like(a)
    ws = torch.empty(max(16, fg.fg_decode_attn_workspace_bytes(cache, n)), dtype=torch.uint8,
                     device="cuda")
    fg.fg_decode_attn_q4kv(q, H * d, cache, n, 0.08, b, ws)
    assert (a.float() - b.float()).abs().max() <= 4 * H16 * a.float().abs().max()


@pytest.mark.parametrize("lens", [[5, 33, 40], [5, -1, 40], [2 ** 31 - 1, 20, 1]])
def test_decode_window_bad_lengths(fg, lens):
    cache, k, v, km, vm = fill_cache(fg, 3, 1, 64, 32, seed=3)
    q16 = fg_synth.random_fp16((3, 64), 6)
    out = run_decode(fg, dev(q16), 1, cache, i32(lens), 0.1, 0, 0)
    with pytest.raises(fg.FgError) as e:
        fg.fg_check_device_error()
    assert e.value.status == fg.FG_ERR_CAPACITY
    fits = [n if 0 <= n <= 32 else 0 for n in lens]
    want = OW.decode(q16, k, v, fits, 1, 0, 0, np.float32(0.1), km, vm)
    check_rows(out, dict(enumerate(want)), 64, True, "bad lengths")


def test_decode_window_repeats_bit_identical(fg):
    B, Hq, H, d = 6, 8, 2, 128
    cache, *_ = fill_cache(fg, B, H, d, 700, seed=5)
    q = dev(fg_synth.random_fp16((B, Hq * d), seed=3))
    lens = i32([700, 3, 650, 0, 77, 512])
    a = run_decode(fg, q, Hq, cache, lens, 0.09, 300, 4)
    for _ in range(5):
        assert torch.equal(a, run_decode(fg, q, Hq, cache, lens, 0.09, 300, 4))


@pytest.mark.parametrize("B", [384, 385, 1700])
def test_decode_window_many_sequences(fg, B):
    """More sequences than the threads of a CTA (which plans the work in rounds of them), most of
    them short or empty, one long."""
    d, cap = 128, 208
    lens = [(i * 11) % 23 for i in range(B)]
    lens[B - 2] = 207
    cache, k, v, km, vm = fill_cache(fg, B, 1, d, cap, seed=17)
    q16 = fg_synth.random_fp16((B, d), 4)
    out = run_decode(fg, dev(q16), 1, cache, i32(lens), 0.1, 100, 3)
    want = OW.decode(q16, k, v, lens, 1, 100, 3, np.float32(0.1), km, vm)
    check_rows(out, dict(enumerate(want)), d, True, "many sequences")


@pytest.mark.parametrize("G", [1, 4])
def test_decode_window_long_shares(fg, G):
    """65536 positions a warp: what the sums lose does not grow with the length.

    Against the values a + q (b - a)/15 that the kernel sums, the relative error of a row has the
    output's rounding (uniform within half a step of 2^-11 .. 2^-10 relative: 2.1e-4), with G = 4
    that of the fp16 weights (they stand at random before values that sum to the output as the
    rounded ones do: 2^-11/sqrt(3) = 2.8e-4), and the truncation of the 16 additions between two
    corrections, half of 2^-24 a step on average, times the ratio of the uncorrected sums (7.5/15
    of the width, 2.3) to the output's size (0.009): 16 * 2^-25 * 255 / 2 = 6e-5.  Together 3.6e-4;
    the bound is three times that.  Sums that truncate all the way lose 1.5e-2 and more."""
    B, H, d, n = 58, 32, 128, 65536
    g = torch.Generator(device="cuda")
    g.manual_seed(19)
    cache = fg.KVCacheQ4(B, n, H * d, H)
    some = torch.randn(1 << 20, 2, generator=g, device="cuda").abs() * 0.3 + 2.0
    some = (some * torch.tensor([-1.0, 1.0], device="cuda")).half().view(torch.int32).view(-1)
    for c in (cache.k_codes, cache.v_codes):
        c.random_(0, 256, generator=g)
    for t in (cache.k_ab, cache.v_ab):
        t.copy_(some[torch.randint(0, 1 << 20, t.shape, generator=g, device="cuda")])
    q = torch.randn(B, H * G * d, generator=g, device="cuda").half()
    out = run_decode(fg, q, H * G, cache, i32([n] * B), d ** -0.5, 0, 0)
    fg.fg_check_device_error()

    def restored(codes, ab):
        x = torch.stack([codes & 15, codes >> 4], -1).view(n, d // 64, 64).double()
        lo, hi = ab.contiguous().view(torch.float16).view(n, d // 64, 2).double().split(1, -1)
        return (lo + x * ((hi - lo) / 15)).view(n, d)

    for b, h in ((0, 0), (17, 5), (B - 1, H - 1)):
        k = restored(cache.k_codes[b, h], cache.k_ab[b, h])
        v = restored(cache.v_codes[b, h], cache.v_ab[b, h])
        for hq in range(h * G, h * G + G):
            at = slice(hq * d, hq * d + d)
            want = torch.softmax(k @ q[b, at].double() * d ** -0.5, 0) @ v
            rel = ((out[b, at].double() - want).norm() / want.norm()).item()
            assert rel <= 1.1e-3, (b, hq, rel)


@pytest.mark.parametrize("B,G", [(40, 1), (700, 4)])
def test_decode_window_mostly_empty_batch(fg, B, G):
    """A few sequences among many empty places, with runs of more than 32 of those."""
    H, d, cap = 2, 64, 96
    lens = [0] * B
    for i, n in zip((1, 2, 35, B - 1), (96, 17, 50, 33)):
        lens[i] = n
    cache, k, v, km, vm = fill_cache(fg, B, H, d, cap, seed=27)
    q16 = fg_synth.random_fp16((B, H * G * d), 5)
    out = run_decode(fg, dev(q16), H * G, cache, i32(lens), 0.1, 40, 3)
    want = OW.decode(q16, k, v, lens, H * G, 40, 3, np.float32(0.1), km, vm)
    check_rows(out, dict(enumerate(want)), d, True, "mostly empty")


@pytest.mark.parametrize("Hq,H", [(4, 4), (8, 2)])
def test_decode_window_in_place(fg, Hq, H):
    """The output over the queries: the bits of an output of its own."""
    B, d = 9, 128
    lens = i32([0, 600, 1, 33, 250, 599, 16, 17, 420])
    cache, *_ = fill_cache(fg, B, H, d, 600, seed=14)
    q = dev(fg_synth.random_fp16((B, Hq * d), seed=2))
    want = run_decode(fg, q, Hq, cache, lens, 0.09, 0, 0)
    assert torch.equal(want, run_decode(fg, q, Hq, cache, lens, 0.09, 0, 0, out=q))


def test_append_many_sequences(fg):
    """Sequences of none to two rows each: every lookup path of a row's sequence."""
    B, H, d = 3000, 1, 64
    rng = np.random.default_rng(8)
    for lens in ([1] * B, rng.integers(0, 3, B).tolist(), [0] * (B - 1) + [70]):
        pos = rng.integers(0, 10, B).tolist()
        buf, t, cache, off, ps = ragged_case(fg, B, H, d, lens, pos, 80, 1, 2, seed=B)
        fg.fg_kv_append_q4_ragged(t[:, :d], t[:, d:2 * d], off, ps, cache)
        fg.fg_check_device_error()
        q, a, b = OQ.quantize_g64(np.ascontiguousarray(buf[:, d:2 * d]))
        codes, o = OQ.pack_nibbles(q), offsets(lens, 1)
        want = np.full((B, 1, 80, d // 2), 0xA5, np.uint8)
        for s in range(B):
            want[s, 0, pos[s]:pos[s] + lens[s]] = codes[o[s]:o[s + 1]]
        assert np.array_equal(host(cache.v_codes), want)
        out = torch.full((t.shape[0], d), 7.0, dtype=torch.float16, device="cuda")
        fg.fg_kv_read_q4_ragged(cache, off, ps, None, out)
        want = np.full((t.shape[0], d), 7.0, np.float16)
        want[1:o[-1]] = OQ.dequant_g64(q, a, b)[1:o[-1]]
        assert np.array_equal(host(out), want)


# ------------------------------------------------------------------------------- prefill


PREFILL = [
    # Hq, Hkv, d, query rows, K/V rows, window, sinks
    (1, 1, 64, [1], [1], 0, 0),
    (2, 2, 128, [1, 0, 5], [1, 0, 5], 0, 0),
    (2, 2, 64, [37, 128, 129], [37, 128, 129], 0, 0),
    (1, 1, 128, [256, 257], [256, 257], 0, 0),
    (2, 1, 128, [300, 17], [300, 17], 64, 4),
    (1, 1, 64, [400], [400], 1, 0),
    (4, 2, 64, [130, 3], [130, 3], 20, 1),
    (2, 2, 128, [200], [200], 130, 0),
    (2, 1, 128, [515], [515], 128, 128),
    (1, 1, 128, [515], [515], 129, 200),           # sinks past a tile
    (3, 1, 64, [60, 7], [300, 260], 0, 0),         # a piece against what was before it
    (2, 1, 128, [64, 1, 130], [700, 500, 131], 150, 10),
    (1, 1, 64, [20, 300], [7, 180], 0, 0),         # more queries than keys: rows that see nothing
    (1, 1, 128, [20, 300], [0, 40], 8, 2),
    (2, 2, 64, [100, 90], [100, 90], 10000, 7),
    (2, 2, 64, [100, 90], [100, 90], 3, 10000),
    (1, 1, 64, [(i * 5) % 23 for i in range(60)], [(i * 5) % 23 for i in range(60)], 6, 2),
    (1, 1, 128, [900], [2500], 700, 300),
]


def prefill_inputs(Hq, Hkv, d, nq, nk, seed, first=0, spare=0):
    q = fg_synth.random_fp16((first + sum(nq) + spare, Hq * d), seed=seed)
    kv = fg_synth.random_fp16((first + sum(nk) + spare, 2 * Hkv * d + 8), seed=seed + 1)
    return q, kv


def run_prefill(fg, q, q_off, k, v, kv_off, Hq, Hkv, scale, window, sinks, pad=8):
    out = torch.full((q.shape[0], q.shape[1] + pad), 7.0, dtype=torch.float16, device="cuda")
    fg.fg_prefill_attn_window(q, q_off, k, v, kv_off, Hq, Hkv, scale, out[:, :q.shape[1]],
                              window=window, sinks=sinks)
    return out


@pytest.mark.parametrize("Hq,Hkv,d,nq,nk,window,sinks", PREFILL)
def test_prefill_window(fg, Hq, Hkv, d, nq, nk, window, sinks):
    w = Hkv * d
    q16, kv16 = prefill_inputs(Hq, Hkv, d, nq, nk, seed=sum(nq) + d, first=3, spare=2)
    qo, ko = offsets(nq, 3), offsets(nk, 3)
    kv = dev(kv16)
    scale = 1.0 / np.sqrt(d)
    out = run_prefill(fg, dev(q16), i32(qo), kv[:, :w], kv[:, w:2 * w], i32(ko), Hq, Hkv, scale,
                      window, sinks)
    fg.fg_check_device_error()
    want = OW.prefill(q16, kv16[:, :w], kv16[:, w:2 * w], qo, ko, Hq, Hkv, window, sinks,
                      np.float32(scale))
    check_rows(out[:, :Hq * d], want, d, False, "prefill")
    rest = host(out)
    assert (rest[:, Hq * d:] == 7.0).all() and (rest[:3] == 7.0).all()
    assert (rest[qo[-1]:] == 7.0).all()                    # rows behind the last sequence


def test_prefill_window_without_keys(fg):
    """Sequences that hold no K/V row at all, and no K/V buffer: zeros."""
    d, nq = 64, [3, 0, 140]
    q16, _ = prefill_inputs(1, 1, d, nq, [0], seed=2)
    none = torch.empty((0, d), dtype=torch.float16, device="cuda")
    out = run_prefill(fg, dev(q16), i32(offsets(nq)), none, none, i32([0, 0, 0, 0]), 1, 1, 0.1, 8, 2)
    fg.fg_check_device_error()
    assert not host(out)[:, :d].any() and (host(out)[:, d:] == 7.0).all()


def test_prefill_window_extreme_values(fg):
    """Values at the end of fp16's range: the mean does not pass it by rounding."""
    d, n = 128, 200
    q16 = np.zeros((n, d), np.float16)
    kv = dev(np.full((n, 2 * d), 65504.0, np.float16))
    out = run_prefill(fg, dev(q16), i32([0, n]), kv[:, :d], kv[:, d:], i32([0, n]), 1, 1, 0.1, 0, 0)
    assert np.abs(host(out)[:, :d].astype(np.float64) - 65504.0).max() <= 65504.0 * 2 * H16


def test_prefill_window_repeats_bit_identical(fg):
    Hq, Hkv, d, nq, past = 4, 2, 128, [300, 17, 260], 90
    q16, kv16 = prefill_inputs(Hq, Hkv, d, nq, [n + past for n in nq], seed=40)
    kv, w = dev(kv16), Hkv * d
    args = (dev(q16), i32(offsets(nq)), kv[:, :w], kv[:, w:2 * w],
            i32(offsets([n + past for n in nq])), Hq, Hkv, 0.09, 70, 5)
    a = run_prefill(fg, *args)
    for _ in range(5):
        assert torch.equal(a, run_prefill(fg, *args))


def test_prefill_window_large_scores(fg):
    """Scores of a few hundred: the running maximum moves by far more than one step."""
    Hq, d, n = 2, 64, 300
    q16, kv16 = prefill_inputs(Hq, Hq, d, [n], [n], seed=77)
    q16 = (q16 * np.float16(8)).astype(np.float16)
    kv = dev(kv16)
    w = Hq * d
    out = run_prefill(fg, dev(q16), i32([0, n]), kv[:, :w], kv[:, w:2 * w], i32([0, n]), Hq, Hq,
                      0.5, 100, 3)
    want = OW.prefill(q16, kv16[:, :w], kv16[:, w:2 * w], [0, n], [0, n], Hq, Hq, 100, 3, 0.5)
    check_rows(out[:, :w], want, d, False, "large scores")


@pytest.mark.parametrize("d,window,sinks,past", [(64, 0, 0, 0), (128, 70, 5, 0), (128, 40, 9, 150)])
def test_prefill_window_masked_positions_may_hold_anything(fg, d, window, sinks, past):
    """A key's infinities and NaN reach exactly the rows that see it; rows behind the last
    sequence and other sequences' rows reach none."""
    nq = [200, 90]
    nk = [n + past for n in nq]
    q16, kv16 = prefill_inputs(1, 1, d, nq, nk, seed=d + window, spare=40)
    qo, ko = offsets(nq), offsets(nk)
    q = dev(q16)
    clean = run_prefill(fg, q, i32(qo), dev(kv16)[:, :d], dev(kv16)[:, d:2 * d], i32(ko), 1, 1,
                        0.1, window, sinks)
    bad = kv16.copy()
    at = {0: [57 + past, 130 + past], 1: [60 + past]}      # positions of each sequence
    for b, ts in at.items():
        for j, t in enumerate(ts):
            bad[ko[b] + t, :d] = np.nan if j else np.inf
            bad[ko[b] + t, d:2 * d] = np.inf if j else np.nan
    bad[ko[-1]:] = np.nan
    kv = dev(bad)
    out = run_prefill(fg, q, i32(qo), kv[:, :d], kv[:, d:2 * d], i32(ko), 1, 1, 0.1, window, sinks)
    fg.fg_check_device_error()
    c, o = host(clean).astype(np.float64), host(out).astype(np.float64)
    for b in range(2):
        for r in range(nq[b]):
            row, i = qo[b] + r, nk[b] - nq[b] + r
            if any(t in OW.visible(i, nk[b], window, sinks) for t in at[b]):
                assert np.isnan(o[row, :d]).all(), (b, r)
            else:
                err = np.abs(o[row, :d] - c[row, :d]).max()
                assert err <= 2 * H16 * np.abs(c[row, :d]).max(), (b, r, err)
    assert (o[qo[-1]:] == 7.0).all()


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 40), (1, 0), (129, 400)])
def test_prefill_window_few_queries(fg, Hq, Hkv, d, window, sinks):
    """Up to 128 query rows behind many keys, whose tiles two halves of the kernel share; beside
    them a longer sequence, an empty one and one of a single tile."""
    nq, nk = [1, 128, 127, 33, 0, 300, 100, 60], [1000, 257, 129, 700, 50, 500, 1157, 90]
    w = Hkv * d
    q16, kv16 = prefill_inputs(Hq, Hkv, d, nq, nk, seed=d + window, spare=9)
    qo, ko = offsets(nq), offsets(nk)
    kv = dev(kv16)
    scale = 1.0 / np.sqrt(d)
    out = run_prefill(fg, dev(q16), i32(qo), kv[:, :w], kv[:, w:2 * w], i32(ko), Hq, Hkv, scale,
                      window, sinks)
    fg.fg_check_device_error()
    want = OW.prefill(q16, kv16[:, :w], kv16[:, w:2 * w], qo, ko, Hq, Hkv, window, sinks,
                      np.float32(scale))
    check_rows(out[:, :Hq * d], want, d, False, "few queries")
    assert (host(out)[qo[-1]:] == 7.0).all() and (host(out)[:, Hq * d:] == 7.0).all()


@pytest.mark.parametrize("d,window,sinks,past", [(64, 0, 0, 300), (128, 200, 30, 800)])
def test_prefill_window_few_queries_masked_positions(fg, d, window, sinks, past):
    test_prefill_window_masked_positions_may_hold_anything(fg, d, window, sinks, past)


@pytest.mark.parametrize("d,window", [(64, 0), (128, 90)])
@pytest.mark.parametrize("nk", [[1, 130, 127, 300], [17, 255, 33, 129]])
def test_prefill_window_rows_behind_hold_anything(fg, d, window, nk):
    """What stands in the rows behind the last sequence changes no bit of the outputs."""
    q16, kv16 = prefill_inputs(2, 1, d, nk, nk, seed=d + window, spare=70)
    off = offsets(nk)
    outs = []
    for tail in (0.0, np.nan, np.inf, -65504.0):
        q, kv = q16.copy(), kv16.copy()
        q[off[-1]:], kv[off[-1]:] = tail, tail
        t = dev(kv)
        outs.append(run_prefill(fg, dev(q), i32(off), t[:, :d], t[:, d:2 * d], i32(off), 2, 1, 0.1,
                                window, 3))
        assert torch.equal(outs[0], outs[-1]), tail
    fg.fg_check_device_error()
    assert bool(torch.isfinite(outs[0]).all())


@pytest.mark.parametrize("q_off,kv_off", [
    ([0, 30, 20, 64], [0, 30, 40, 64]), ([0, 30, 40, 65], [0, 30, 40, 64]),
    ([-1, 30, 40, 64], [0, 30, 40, 64]), ([0, 30, 40, 64], [0, 50, 40, 64]),
    ([0, 30, 40, 64], [0, 30, 40, 100]), ([0, 30, 40, 64], [-9, 30, 40, 64]),
])
def test_prefill_window_bad_offsets(fg, q_off, kv_off):
    """A sequence whose rows do not fit is left out; the others are computed."""
    d = 64
    q16, kv16 = prefill_inputs(1, 1, d, [64], [64], seed=5)
    kv = dev(kv16)
    out = run_prefill(fg, dev(q16), i32(q_off), kv[:, :d], kv[:, d:2 * d], i32(kv_off), 1, 1, 0.1,
                      12, 2)
    with pytest.raises(fg.FgError) as e:
        fg.fg_check_device_error()
    assert e.value.status == fg.FG_ERR_CAPACITY
    if q_off == [0, 30, 40, 64]:
        o = host(out)
        for b in range(3):
            lo, hi = kv_off[b], kv_off[b + 1]
            rows = slice(q_off[b], q_off[b + 1])
            if not (0 <= lo <= hi <= 64):
                assert (o[rows] == 7.0).all(), b
            else:
                n = q_off[b + 1] - q_off[b]
                want = OW.prefill(q16[rows], kv16[lo:hi, :d], kv16[lo:hi, d:2 * d], [0, n],
                                  [0, hi - lo], 1, 1, 12, 2, np.float32(0.1))
                check_rows(out[rows, :d], want, d, False, "bad offsets")


def test_prefill_window_many_sequences(fg):
    """More sequences than one pass over a plan of them holds, most of them empty or one row."""
    d, n = 64, 2300
    nq = [(i * 7) % 3 for i in range(n)]
    nq[1030] = 150
    q16, kv16 = prefill_inputs(1, 1, d, nq, nq, seed=6)
    kv = dev(kv16)
    off = offsets(nq)
    out = run_prefill(fg, dev(q16), i32(off), kv[:, :d], kv[:, d:2 * d], i32(off), 1, 1, 0.1, 50, 1)
    fg.fg_check_device_error()
    want = OW.prefill(q16, kv16[:, :d], kv16[:, d:2 * d], off, off, 1, 1, 50, 1, np.float32(0.1))
    check_rows(out[:, :d], want, d, False, "many sequences")


def test_prefill_window_matches_equal_prompts_call(fg):
    """Equal prompts, no window: what fg_prefill_attn gives."""
    nseq, s, H, d = 3, 200, 4, 128
    qkv = dev(fg_synth.random_fp16((nseq * s, 3 * H * d), seed=21))
    h = H * d
    off = i32([0, s, 2 * s, 3 * s])
    a = run_prefill(fg, qkv[:, :h], off, qkv[:, h:2 * h], qkv[:, 2 * h:], off, H, H, 0.09, 0, 0)
    b = torch.empty((nseq * s, h), dtype=torch.float16, device="cuda")
    fg.fg_prefill_attn(qkv, nseq, s, H, d, 0.09, b)
    assert (a[:, :h].float() - b.float()).abs().max() <= 4 * H16 * b.float().abs().max()


# ------------------------------------------------------------------------------- together


def serve(fg, B, Hq, H, d, prompts, piece, steps, window, sinks, x, ws, cache, out, stream=None):
    """Prompts written and attended to, a piece of each more against what is read back, then
    single tokens: the calls of a serving loop.  x: fp16 [rows][(Hq + 2H) d], step after step."""
    wq, wk = Hq * d, H * d
    lens = list(prompts)
    scale, row = 0.11, 0

    def qkv(n):
        nonlocal row
        r = slice(row, row + n)
        row += n
        return x[r, :wq], x[r, wq:wq + wk], x[r, wq + wk:], out[r]

    def at(v):
        return torch.tensor(v, dtype=torch.int32).to("cuda")

    q, k, v, o = qkv(sum(prompts))
    off = at(offsets(prompts))
    fg.fg_kv_append_q4_ragged(k, v, off, at([0] * B), cache, stream)
    fg.fg_prefill_attn_window(q, off, k, v, off, Hq, H, scale, o, window, sinks, stream)
    q, k, v, o = qkv(sum(piece))
    off = at(offsets(piece))
    fg.fg_kv_append_q4_ragged(k, v, off, at(lens), cache, stream)
    lens = [a + b for a, b in zip(lens, piece)]
    kv_off = at(offsets(lens))
    kr = torch.empty((sum(lens), wk), dtype=torch.float16, device="cuda")
    vr = torch.empty_like(kr)
    fg.fg_kv_read_q4_ragged(cache, kv_off, at([0] * B), kr, vr, stream)
    fg.fg_prefill_attn_window(q, off, kr, vr, kv_off, Hq, H, scale, o, window, sinks, stream)
    for _ in range(steps):
        q, k, v, o = qkv(B)
        fg.fg_kv_append_q4_ragged(k, v, at(list(range(B + 1))), at(lens), cache, stream)
        lens = [n + 1 for n in lens]
        fg.fg_decode_attn_q4kv_window(q, Hq, cache, at(lens), scale, o, ws, window, sinks, stream)
    return lens


def test_serving_loop(fg):
    """Prompts, a further piece and single tokens of sequences of different lengths."""
    B, Hq, H, d, window, sinks = 3, 4, 2, 64, 40, 4
    prompts, piece, steps = [33, 5, 70], [9, 20, 1], 4
    rows = sum(prompts) + sum(piece) + steps * B
    wq, wk = Hq * d, H * d
    x16 = fg_synth.random_fp16((rows, wq + 2 * wk), seed=31)
    x = dev(x16)
    cache = fg.KVCacheQ4(B, 112, wk, H)
    ws = torch.empty(max(16, fg.fg_decode_attn_window_workspace_bytes(cache, Hq)),
                     dtype=torch.uint8, device="cuda")
    out = torch.zeros((rows, wq), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        serve(fg, B, Hq, H, d, prompts, piece, steps, window, sinks, x, ws, cache, out)
    fg.fg_check_device_error(st)
    # the oracle's run: fp16 K/V for the prompts, the restored ones afterwards
    k16, v16 = x16[:, wq:wq + wk], x16[:, wq + wk:]
    quant = []
    for a16 in (k16, v16):
        q, a, b = OQ.quantize_g64(np.ascontiguousarray(a16))
        mag = np.abs(a.astype(np.float64)) + (b.astype(np.float64) - a.astype(np.float64))
        quant.append((OQ.dequant_g64(q, a, b), np.repeat(mag, 64, axis=1)))
    off = offsets(prompts)
    want = OW.prefill(x16[:, :wq], k16, v16, off, off, Hq, H, window, sinks, np.float32(0.11))
    check_rows(out, want, d, False, "prompts")
    held = [list(range(off[b], off[b + 1])) for b in range(B)]
    row = sum(prompts)
    poff = offsets(piece, row)
    for b in range(B):
        held[b] += range(poff[b], poff[b + 1])
    kv_off = offsets([len(r) for r in held])
    flat = [r for rows_ in held for r in rows_]
    q_rows = x16[row:row + sum(piece), :wq]
    want = OW.prefill(q_rows, quant[0][0][flat], quant[1][0][flat], offsets(piece), kv_off, Hq, H,
                      window, sinks, np.float32(0.11))
    check_rows(out[row:row + sum(piece)], want, d, False, "piece")
    row += sum(piece)
    for s in range(steps):
        for b in range(B):
            held[b].append(row + b)
            n = len(held[b])
            kk, vv, km, vm = (z[held[b]].reshape(n, H, d).transpose(1, 0, 2)[None]
                              for z in (quant[0][0], quant[1][0], quant[0][1], quant[1][1]))
            want = OW.decode(x16[row + b:row + b + 1, :wq], kk, vv, [n], Hq, window, sinks,
                             np.float32(0.11), km, vm)
            check_rows(out[row + b:row + b + 1], dict(enumerate(want)), d, True, f"step {s}")
        row += B


def test_captured_steps_replay(fg):
    """A captured generation step (append, then attention) replayed with lengths that advance on
    the device, and two captured graphs with workspaces of their own."""
    B, Hq, H, d, n0 = 4, 4, 2, 128, 50
    wq, wk = Hq * d, H * d
    cache, *_ = fill_cache(fg, B, H, d, 64, seed=14)
    twin, *_ = fill_cache(fg, B, H, d, 64, seed=14)
    x16 = fg_synth.random_fp16((3 * B, wq + 2 * wk), seed=15)
    steps = dev(x16)
    x = steps[:B].clone()
    pos, lens, off = i32([n0, 3, 0, 20]), i32([n0 + 1, 4, 1, 21]), i32(range(B + 1))
    nws = max(16, fg.fg_decode_attn_window_workspace_bytes(cache, Hq))
    ws = [torch.empty(nws, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.zeros((B, wq), dtype=torch.float16, device="cuda") for _ in range(2)]

    def step(c, w, o):
        fg.fg_kv_append_q4_ragged(x[:, wq:wq + wk], x[:, wq + wk:], off, pos, c)
        fg.fg_decode_attn_q4kv_window(x[:, :wq], Hq, c, lens, 0.1, o, w, window=30, sinks=2)

    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):                        # loads the kernels before the capture
        step(twin, ws[0], out[0])
    torch.cuda.synchronize()
    graphs = []
    for j, c in enumerate((cache, twin)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c, ws[j], out[j])
        graphs.append(g)
    eager_cache, *_ = fill_cache(fg, B, H, d, 64, seed=14)
    eager = torch.zeros((B, wq), dtype=torch.float16, device="cuda")
    ews = torch.empty(nws, dtype=torch.uint8, device="cuda")
    for s in range(3):
        x.copy_(steps[s * B:(s + 1) * B])
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(st):
            graphs[1].replay()
        torch.cuda.synchronize()
        step(eager_cache, ews, eager)
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager) and torch.equal(out[1], eager), s
        pos += 1
        lens += 1
    fg.fg_check_device_error()
    assert torch.equal(cache.k_codes, eager_cache.k_codes)


def test_offsets_past_32_bits(fg):
    """A cache of more than 2^32 bytes of codes, written, read and attended at its far end; and fp16
    rows more than 2^31 elements apart, which give the bits of packed ones."""
    B, H, d, cap, n, window = 2, 2, 64, 1 << 25, 40, 33
    h = H * d
    x16 = fg_synth.random_fp16((n + 3, 3 * h), seed=41)
    x = dev(x16)
    cache = fg.KVCacheQ4(B, cap, h, H)
    off, pos = i32([0, 3, n + 3]), i32([0, cap - n])
    fg.fg_kv_append_q4_ragged(x[:, h:2 * h], x[:, 2 * h:], off, pos, cache)
    back = torch.zeros((n + 3, 2 * h), dtype=torch.float16, device="cuda")
    fg.fg_kv_read_q4_ragged(cache, off, pos, back[:, :h], back[:, h:])
    q = x[[2, n + 2], :h].contiguous()
    out = run_decode(fg, q, H, cache, i32([3, cap]), 0.1, window, 0)
    fg.fg_check_device_error()
    del cache
    vals, mags = [], []
    for j in (1, 2):
        qc, a, b = OQ.quantize_g64(np.ascontiguousarray(x16[:, j * h:(j + 1) * h]))
        vals.append(OQ.dequant_g64(qc, a, b))
        mags.append(np.repeat(np.abs(a.astype(np.float64)) +
                              (b.astype(np.float64) - a.astype(np.float64)), 64, axis=1))
    assert np.array_equal(host(back), np.concatenate(vals, axis=1))
    for row, rows in ((0, slice(0, 3)), (1, slice(3, n + 3))):
        kk, vv, km, vm = (z[rows].reshape(-1, H, d).transpose(1, 0, 2)[None] for z in vals + mags)
        want = OW.decode(host(q)[row:row + 1], kk, vv, [kk.shape[2]], H, window, 0,
                         np.float32(0.1), km, vm)
        check_rows(out[row:row + 1], dict(enumerate(want)), d, True, f"far end {row}")
    # 20 rows 2^27 elements apart
    wide = torch.empty((20, 1 << 27), dtype=torch.float16, device="cuda")
    far = wide[:, :4 * h]
    far[:, :3 * h] = x[:20]
    o20 = i32([0, 7, 20])
    near = torch.empty((20, h), dtype=torch.float16, device="cuda")
    for a, o in ((x[:20], near), (far, far[:, 3 * h:])):
        fg.fg_prefill_attn_window(a[:, :h], o20, a[:, h:2 * h], a[:, 2 * h:3 * h], o20, H, H, 0.1,
                                  o, window=5, sinks=1)
    assert torch.equal(near, far[:, 3 * h:])
    caches = [fg.KVCacheQ4(2, 16, h, H) for _ in range(2)]
    for a, c in zip((x, far), caches):
        fg.fg_kv_append_q4_ragged(a[:20, h:2 * h], a[:20, 2 * h:3 * h], o20, i32([0, 2]), c)
    for name in ("k_codes", "v_codes", "k_ab", "v_ab"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
    fg.fg_check_device_error()


def test_two_streams_at_once(fg):
    """The calls on two streams with nothing between them, each with a cache and a workspace of its
    own, give what they give one after another."""
    sets = []
    for seed, (B, Hq, H, d, lens) in enumerate(((6, 4, 4, 128, [900, 30, 1, 512, 700, 64]),
                                                (3, 8, 2, 64, [1500, 0, 333]))):
        cache, *_ = fill_cache(fg, B, H, d, max(lens), seed=60 + seed)
        q16, kv16 = prefill_inputs(Hq, H, d, lens, lens, seed=70 + seed)
        sets.append(dict(B=B, Hq=Hq, H=H, d=d, cache=cache, lens=i32(lens), off=i32(offsets(lens)),
                         zero=i32([0] * B), q=dev(q16), kv=dev(kv16), st=torch.cuda.Stream(),
                         ws=torch.empty(fg.fg_decode_attn_window_workspace_bytes(cache, Hq),
                                        dtype=torch.uint8, device="cuda")))

    def run(c, stream):
        w, dv = c["H"] * c["d"], c["kv"].device
        k, v = c["kv"][:, :w], c["kv"][:, w:2 * w]
        res = [torch.zeros((c["B"], c["Hq"] * c["d"]), dtype=torch.float16, device=dv),
               torch.zeros_like(c["q"]), torch.zeros_like(c["kv"])]
        torch.cuda.synchronize()
        yield res
        for _ in range(4):
            fg.fg_kv_append_q4_ragged(k, v, c["off"], c["zero"], c["cache"], stream)
            fg.fg_decode_attn_q4kv_window(c["q"][:c["B"]], c["Hq"], c["cache"], c["lens"], 0.1,
                                          res[0], c["ws"], 200, 3, stream)
            fg.fg_prefill_attn_window(c["q"], c["off"], k, v, c["off"], c["Hq"], c["H"], 0.1,
                                      res[1], 200, 3, stream)
            fg.fg_kv_read_q4_ragged(c["cache"], c["off"], c["zero"], res[2][:, :w],
                                    res[2][:, w:2 * w], stream)
            yield res

    alone = []
    for c in sets:
        for res in run(c, None):
            torch.cuda.synchronize()
        alone.append(res)
    both = [run(c, c["st"]) for c in sets]
    together = [next(r) for r in both]
    for _ in range(4):
        for r in both:
            next(r)
    torch.cuda.synchronize()
    fg.fg_check_device_error()
    for a, b in zip(alone, together):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_binding_refuses(fg):
    """What the binding refuses before a pointer is taken."""
    cache = fg.KVCacheQ4(2, 16, 128, 1)
    x = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    off, pos = i32([0, 2, 4]), i32([0, 0])
    bad = [
        lambda: fg.fg_kv_append_q4_ragged(x.float(), x, off, pos, cache),
        lambda: fg.fg_kv_append_q4_ragged(x[:, :64], x, off, pos, cache),
        lambda: fg.fg_kv_append_q4_ragged(x[:3], x, off, pos, cache),
        lambda: fg.fg_kv_append_q4_ragged(x, x, off.long(), pos, cache),
        lambda: fg.fg_kv_append_q4_ragged(x, x, off[:2], pos, cache),
        lambda: fg.fg_kv_append_q4_ragged(x, x, off, pos.cpu(), cache),
        lambda: fg.fg_kv_read_q4_ragged(cache, off, pos, None, None),
        lambda: fg.fg_decode_attn_q4kv_window(x, 1, cache, pos, 0.1, x[:2]),
        lambda: fg.fg_decode_attn_q4kv_window(x[:2], 1, cache, off, 0.1, x[2:]),
        lambda: fg.fg_decode_attn_q4kv_window(x[:2], 1, cache, pos, 0.1, x[2:],
                                              x[:1].expand(64, 128)),
        lambda: fg.fg_prefill_attn_window(x, off, x, x[:3], off, 1, 1, 0.1, x.clone()),
        lambda: fg.fg_prefill_attn_window(x, off, x, x, off[:2], 1, 1, 0.1, x.clone()),
        lambda: fg.fg_prefill_attn_window(x, off, x.t(), x, off, 1, 1, 0.1, x.clone()),
    ]
    for j, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {j} was taken")
    with pytest.raises(fg.FgError):
        fg.fg_prefill_attn_window(x, off, x, x, off, 1, 1, 0.1, x)         # out aliases q
    with pytest.raises(fg.FgError):
        fg.fg_kv_append_q4_ragged(x.view(-1)[4:132].view(1, 128), x.view(-1)[4:132].view(1, 128),
                                  off, pos, cache)                        # misaligned
