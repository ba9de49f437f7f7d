"""Paths of the ragged and windowed kernels that only large calls take: several items per CTA,
several heads per CTA, shares of many positions; and what stands around the buffers."""
import numpy as np
import pytest
import torch

from parity_util import lib
from test_gpu_window import F32, H16, i32, offsets
from test_gpu_window_range import restored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    return lib()


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------------------- prefill


def prefill_rows(q, k, v, first, window, sinks, scale):
    """64-bit outputs [h][n][d] of queries at positions first .. over k, v [h][nk][d], and what the
    arithmetic may be off: scores by d + 40 binary32 operations on terms of their size, which moves
    a weight by a factor within e^(+-2 ds); weights rounded to fp16, half a step of 2^-11 or, times
    2^7 as they are, half of 2^-24; n + 64 binary32 sums; the exponential's 2^-21; the output's half
    step."""
    d = q.shape[-1]
    i = torch.arange(first, first + q.shape[-2], device="cuda")[:, None]
    t = torch.arange(k.shape[-2], device="cuda")
    ok = t <= i
    if window:
        ok &= (t > i - window) | (t < sinks)
    s = (q @ k.mT * scale).masked_fill(~ok, -torch.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m.masked_fill(m == -torch.inf, 0.0))
    l = e.sum(-1, keepdim=True)
    some = l > 0
    p = e / l.masked_fill(~some, 1.0)
    o, A = p @ v, p @ v.abs()
    terms = (q.abs() @ k.abs().mT * scale).masked_fill(~ok, 0.0).amax(-1, keepdim=True)
    n = ok.sum(-1)[..., None]
    tol = (torch.expm1(2 * terms * (d + 40) * F32) + H16 + 2.0 ** -21 + (n + 64) * F32) * A \
        + n * 2.0 ** -32 / l.masked_fill(~some, 1.0) * v.abs().amax(-2, keepdim=True) \
        + H16 * o.abs() + 2.0 ** -24
    return o, torch.where(some, tol, torch.zeros_like(tol))


MIXED = [(700, 0), (1, 2000), (100, 900), (300, 33), (128, 128), (40, 1500), (257, 0), (512, 64),
         (90, 300), (5, 5), (130, -40), (60, -60), (127, 1), (256, 256), (33, 3000), (0, 70)]


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 30), (1, 0), (129, 400)])
def test_prefill_window_many_items_per_cta(fg, Hq, Hkv, d, window, sinks):
    """At least four blocks of query rows per CTA, of sequences whose tiles both halves of the kernel
    share between others whose are not, of many key tiles, one or none."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(window + d)
    seqs = []
    while sum((nq + 255) // 256 for nq, _ in seqs) * Hq < 4 * sms:
        seqs += [MIXED[j] for j in rng.permutation(len(MIXED))]
    nq, nk = [a for a, _ in seqs], [a + b for a, b in seqs]
    qo, ko = offsets(nq), offsets(nk)
    g = generator(d + sinks)
    q = torch.randn(qo[-1], Hq * d, generator=g, device="cuda").half()
    kv = torch.randn(ko[-1], 2 * Hkv * d, generator=g, device="cuda").half()
    k, v = kv[:, :Hkv * d], kv[:, Hkv * d:]
    scale = d ** -0.5
    out = torch.full((qo[-1] + 3, Hq * d), 7.0, dtype=torch.float16, device="cuda")
    for _ in range(2):
        fg.fg_prefill_attn_window(q, i32(qo), k, v, i32(ko), Hq, Hkv, scale, out[:qo[-1]],
                                  window=window, sinks=sinks)
    fg.fg_check_device_error()
    assert bool((out[qo[-1]:] == 7.0).all())
    f32scale = float(np.float32(scale))
    for b in range(len(seqs)):
        if nq[b] == 0:
            continue
        rows = slice(qo[b], qo[b + 1])
        qq = q[rows].double().view(-1, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3)
        kk, vv = (x[ko[b]:ko[b + 1]].double().view(-1, Hkv, 1, d).permute(1, 2, 0, 3)
                  for x in (k, v))
        got = out[rows].double().view(-1, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3)
        if nk[b] == 0:
            assert not got.any(), b
            continue
        o, tol = prefill_rows(qq, kk, vv, nk[b] - nq[b], window, sinks, f32scale)
        over = ((got - o).abs() - tol).max().item()
        assert over <= 0, (b, nq[b], nk[b], over)


# ------------------------------------------------------------------------------- append, read


@pytest.mark.parametrize("H,d,rows,heads", [(96, 128, 1800, 2), (13, 128, 49000, 8),
                                            (40, 64, 34000, 8), (25, 64, 21000, 3)])
def test_append_and_read_several_heads_per_cta(fg, H, d, rows, heads):
    """Calls with so many rows that a CTA walks more than one head (the last CTA of a tile fewer):
    the codes, statistics and values of fg_quantize_g64 and fg_dequant_g64, and nothing else."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per_cta = min(8, (rows + 4096 // d - 1) // (4096 // d) * H // (16 * sms))
    assert per_cta >= heads or sms != 152
    B, h, g = 37, H * d, generator(rows)
    rng = np.random.default_rng(rows)
    lens = rng.multinomial(rows - 12, rng.dirichlet(np.ones(B))).tolist()
    lens[3] = 0
    pos = rng.integers(0, 50, B).tolist()
    cap = (max(n + p for n, p in zip(lens, pos)) + 15) // 16 * 16
    off = offsets(lens, 5)
    x = torch.randn(rows, 2 * h + 8, generator=g, device="cuda").half()
    cache = fg.KVCacheQ4(B, cap, h, H)
    want = {}
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(lens, device="cuda"))
    at = slice(off[0], off[-1])
    t = torch.arange(off[0], off[-1], device="cuda") - i32(off)[seq] + i32(pos)[seq]
    values = []
    for j, name in enumerate("kv"):
        codes_t, ab_t = getattr(cache, name + "_codes"), getattr(cache, name + "_ab")
        codes_t.fill_(0xA5)
        ab_t.fill_(0x5A5A5A5A)
        codes = torch.empty((rows, h // 2), dtype=torch.uint8, device="cuda")
        ab = torch.empty((rows, h // 64), dtype=torch.int32, device="cuda")
        src = x[:, j * h:(j + 1) * h].contiguous()
        fg.fg_quantize_g64(src, codes, ab)
        y = torch.empty_like(src)
        fg.fg_dequant_g64(codes, ab, rows, h, y)
        values.append(y)
        wc, wa = codes_t.clone(), ab_t.clone()
        wc[seq, :, t] = codes[at].view(-1, H, d // 2)
        wa[seq, :, t] = ab[at].view(-1, H, d // 64)
        want[name + "_codes"], want[name + "_ab"] = wc, wa
    fg.fg_kv_append_q4_ragged(x[:, :h], x[:, h:2 * h], i32(off), i32(pos), cache)
    fg.fg_check_device_error()
    for name, w in want.items():
        assert torch.equal(getattr(cache, name), w), name
    for which in ("kv", "k", "v"):
        out = torch.full((rows, 2 * h + 8), 7.0, dtype=torch.float16, device="cuda")
        fg.fg_kv_read_q4_ragged(cache, i32(off), i32(pos), out[:, :h] if "k" in which else None,
                                out[:, h:2 * h] if "v" in which else None)
        w = torch.full_like(out, 7.0)
        for j, name in enumerate("kv"):
            if name in which:
                w[at, j * h:(j + 1) * h] = values[j][at]
        assert torch.equal(out.view(torch.int16), w.view(torch.int16)), which
    fg.fg_check_device_error()


# ------------------------------------------------------------------------------- decode


@pytest.mark.parametrize("d,G", [(64, 1), (64, 2), (64, 4), (128, 2), (128, 8)])
def test_decode_window_long_shares_of_every_kind(fg, d, G):
    """65536 positions a warp for the channel counts and query heads whose second terms sit in other
    columns when sums are corrected; the bound is that of test_decode_window_long_shares: three
    times 3.6e-4, of which 2.1e-4 are the output's rounding, 2.8e-4 the weights' where one fp16
    term is kept, and 6e-5 the truncated sums between two corrections."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H, n = 32, 65536
    sets = (G + 3) // 4                                # row sets per K/V head
    B = (12 if d == 128 else 16) * sms // (H * sets) + 1
    g = generator(23)
    cache = fg.KVCacheQ4(B, n, H * d, H)
    some = torch.randn(1 << 20, 2, generator=g, device="cuda").abs() * 0.3 + 2.0
    some = (some * torch.tensor([-1.0, 1.0], device="cuda")).half().view(torch.int32).view(-1)
    for c in (cache.k_codes, cache.v_codes):
        c.random_(0, 256, generator=g)
    for t in (cache.k_ab, cache.v_ab):
        t.copy_(some[torch.randint(0, 1 << 20, t.shape, generator=g, device="cuda")])
    q = torch.randn(B, H * G * d, generator=g, device="cuda").half()
    out = torch.empty_like(q)
    ws = torch.empty(fg.fg_decode_attn_window_workspace_bytes(cache, H * G), dtype=torch.uint8,
                     device="cuda")
    fg.fg_decode_attn_q4kv_window(q, H * G, cache, i32([n] * B), d ** -0.5, out, ws)
    fg.fg_check_device_error()
    for b, h in ((0, 0), (B // 3, 5), (B - 1, H - 1)):
        k, v = (restored(getattr(cache, c + "_codes")[b, h], getattr(cache, c + "_ab")[b, h], d)
                for c in "kv")
        qq = q[b].double().view(H, G, d)[h]
        want = torch.softmax(qq @ k.T * d ** -0.5, -1) @ v
        got = out[b].double().view(H, G, d)[h]
        rel = ((got - want).norm(dim=-1) / want.norm(dim=-1)).max().item()
        assert rel <= 1.1e-3, (b, h, rel)


# ------------------------------------------------------------------------------- around the buffers


class Guarded:
    """Tensors that are views into the middle of larger buffers filled with one byte."""

    PAD = 1 << 16

    def __init__(self):
        self.bufs = []

    def make(self, shape, dtype):
        size = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((2 * self.PAD + size,), 0xA5, dtype=torch.uint8, device="cuda")
        self.bufs.append((buf, size))
        return buf[self.PAD:self.PAD + size].view(dtype).view(shape)

    def intact(self):
        return all(bool((b[:self.PAD] == 0xA5).all()) and bool((b[self.PAD + n:] == 0xA5).all())
                   for b, n in self.bufs)


def guarded_cache(fg, guard, B, cap, h, H):
    cache, d = fg.KVCacheQ4(B, cap, h, H), h // H
    for name, dtype, w in (("k_codes", torch.uint8, d // 2), ("v_codes", torch.uint8, d // 2),
                           ("k_ab", torch.int32, d // 64), ("v_ab", torch.int32, d // 64)):
        setattr(cache, name, guard.make((B, H, cache.cap, w), dtype))
    return cache


@pytest.mark.parametrize("off,pos", [
    ([0, 4, 2, 8], [0, 0, 0]), ([0, 2, 4, 9], [0, 0, 0]), ([-3, 2, 4, 8], [0, 0, 0]),
    ([0, 2, 4, 200], [0, 0, 0]), ([-100, 2, 4, 8], [0, 0, 0]),
    ([0, 2, 4, 8], [0, 15, 0]), ([0, 2, 4, 8], [0, 0, 14]), ([0, 2, 4, 8], [-1, 0, 0]),
    ([0, 2, 4, 8], [-300, 0, 300]), ([0, 2, 4, 8], [2 ** 31 - 1, -2 ** 31, 0]),
    ([0, 2 ** 31 - 1, -2 ** 31, 8], [0, 0, 0]),
])
def test_extents_that_do_not_fit_stay_inside(fg, off, pos):
    """Rows, offsets and positions that do not fit, right before and behind the buffers and far away:
    not a byte around the cache or the outputs changes."""
    guard, h, rows = Guarded(), 256, 8
    cache = guarded_cache(fg, guard, 3, 16, h, 2)
    kv = guard.make((rows, 2 * h), torch.float16)
    kv.copy_(torch.randn(rows, 2 * h, generator=generator(1), device="cuda"))
    out = guard.make((rows, 2 * h), torch.float16)
    for call in (lambda: fg.fg_kv_append_q4_ragged(kv[:, :h], kv[:, h:], i32(off), i32(pos), cache),
                 lambda: fg.fg_kv_read_q4_ragged(cache, i32(off), i32(pos), out[:, :h], out[:, h:])):
        call()
        with pytest.raises(fg.FgError) as e:
            fg.fg_check_device_error()
        assert e.value.status == fg.FG_ERR_CAPACITY and "ragged cache" in str(e.value)
    assert guard.intact()


def test_attention_stays_inside(fg):
    """Ragged calls with strides, a full cache and lengths or offsets that do not fit: not a byte
    around the cache, the outputs or the workspace changes."""
    g = generator(2)
    for B, Hq, H, d, cap, lens, fits in (
            (4, 4, 4, 128, 48, [48, 0, 47, 1], True), (4, 14, 2, 64, 80, [80, 33, 17, 80], True),
            (3, 4, 2, 128, 32, [33, -1, 32], False)):
        guard = Guarded()
        cache = guarded_cache(fg, guard, B, cap, H * d, H)
        n = B * cap
        kv = torch.randn(n, 2 * H * d, generator=g, device="cuda").half()
        k, v = kv[:, :H * d], kv[:, H * d:]
        fg.fg_kv_append_q4_ragged(k, v, i32(range(0, n + 1, cap)), i32([0] * B), cache)
        q = torch.randn(n, Hq * d, generator=g, device="cuda").half()
        out = guard.make((B, Hq * d), torch.float16)
        ws = guard.make((fg.fg_decode_attn_window_workspace_bytes(cache, Hq),), torch.uint8)
        for window, sinks in ((0, 0), (20, 3)):
            fg.fg_decode_attn_q4kv_window(q[:B], Hq, cache, i32(lens), 0.1, out, ws, window=window,
                                          sinks=sinks)
        wide = guard.make((n, Hq * d + 8), torch.float16)
        ko = offsets([max(0, x) for x in lens])
        ko[-1] += 0 if fits else 10 ** 6
        qo = i32(offsets([cap] * B))
        fg.fg_prefill_attn_window(q, qo, k, v, i32(ko), Hq, H, 0.1, wide[:, :Hq * d], window=20,
                                  sinks=3)
        if fits:
            fg.fg_check_device_error()
        else:
            with pytest.raises(fg.FgError) as e:
                fg.fg_check_device_error()
            assert e.value.status == fg.FG_ERR_CAPACITY
            assert "windowed decode attention, windowed prefill attention" in str(e.value)
        assert guard.intact()
        assert bool((wide[:, Hq * d:].contiguous().view(torch.uint8) == 0xA5).all())


def test_launch_stream_is_the_current_one(fg):
    """The handle that calls without a stream launch on is that of torch.cuda.current_stream()."""
    st = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), st):
        with torch.cuda.stream(s):
            assert fg._stream() == torch.cuda.current_stream().cuda_stream
            assert fg._stream_for(None, torch.empty(1, device="cuda")) == s.cuda_stream
    assert fg._stream(st) == st.cuda_stream


@pytest.mark.parametrize("window,sinks,seen", [(0, 0, 64), (0, 9, 64), (10, 3, 13), (60, 40, 64),
                                               (2 ** 31 - 1, 2 ** 31 - 1, 64)])
def test_profiled_work_of_windowed_decode(fg, window, sinks, seen):
    """The profiler counts what full sequences see, not the whole cache."""
    B, Hq, H, d = 3, 4, 2, 64
    cache = fg.KVCacheQ4(B, 64, H * d, H)
    q = torch.zeros((B, Hq * d), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(fg.fg_decode_attn_window_workspace_bytes(cache, Hq), dtype=torch.uint8,
                     device="cuda")
    fg.fg_prof_reset()
    fg.fg_prof_enable()
    try:
        fg.fg_decode_attn_q4kv_window(q, Hq, cache, i32([64, 5, 0]), 0.1, out, ws, window=window,
                                      sinks=sinks)
        torch.cuda.synchronize()
        r = fg.fg_prof_query(fg.K_DECODE_ATTN_WINDOW)
    finally:
        fg.fg_prof_enable(False)
        fg.fg_prof_reset()
    assert r["launches"] == 1
    assert r["work"] == 2 * B * seen * H * d * 0.5625 + 4 * B * Hq * d
