"""The windowed attention over the whole range of softmax weights and of values: what a few large
weights must not take away from many small ones."""
import pytest
import torch

from parity_util import lib
from test_gpu_window import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    return lib()


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def restored(codes, ab, d):
    """64-bit a + q (b - a)/15 of cached positions [..][n][d]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (d // 64, 64)).double()
    lo, hi = ab.contiguous().view(torch.float16).unflatten(-1, (-1, 2)).double().split(1, -1)
    return (lo + q * ((hi - lo) / 15)).flatten(-2)


def relative(got, want):
    return ((got.double() - want).norm(dim=-1) / want.norm(dim=-1)).max().item()


@pytest.mark.parametrize("G", [1, 2, 4, 7])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sigma,gap,n", [(0.01, 12, 2048), (0.05, 14, 8192), (0.01, 12, 8192),
                                         (1.0, 13, 2048), (0.0005, 0, 2048)])
def test_decode_window_one_large_weight(fg, G, d, sigma, gap, n):
    """A first position `gap` nats above thousands of others, as attention sinks are, and small
    values; 4000 row sets or more, so that most lie within one warp's share.

    Relative error of a row: the output's rounding, at most 2^-11, and for the smallest values (near
    0.0005 / sqrt(2048) = 1e-5 without a gap) half of fp16's smallest step, 2^-25 = 3e-8 an element
    of 1e-5: 3e-3; the weights' rounding where one fp16 term is kept (G > 2), at most 2^-11 of each
    (c - 7.5) (b - a)/15, which are 1.2 times the values at most (their middle is not their mean);
    the truncated sums between corrections (6e-5, as for long shares); scores of up to 14 from d +
    40 operations: 14 (d + 40) 2^-23 = 2.8e-4 of the small weights together, which are a twentieth
    of the sum: 1.4e-5.  Together 4.9e-4 + 5.9e-4 + 8e-5 = 1.2e-3."""
    H, B = 8, 500
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    x = torch.randn(n, 2, H * d, generator=g, device="cuda")
    k, v = (0.3 * x[:, 0]).half(), (sigma * x[:, 1]).half()
    q = (1.0 + 0.3 * torch.randn(H * G * d, generator=g, device="cuda")).half()
    if gap:
        k[0] = gap / d ** 0.5
    one = fg.KVCacheQ4(1, n, H * d, H)
    fg.fg_kv_append_q4_ragged(k, v, i32([0, n]), i32([0]), one)
    cache = fg.KVCacheQ4(B, n, H * d, H)
    for name in ("k_codes", "k_ab", "v_codes", "v_ab"):
        getattr(cache, name).copy_(getattr(one, name).expand_as(getattr(cache, name)))
    qs = q.expand(B, -1).contiguous()
    out = torch.empty_like(qs)
    ws = torch.empty(fg.fg_decode_attn_window_workspace_bytes(cache, H * G), dtype=torch.uint8,
                     device="cuda")
    fg.fg_decode_attn_q4kv_window(qs, H * G, cache, i32([n] * B), d ** -0.5, out, ws)
    fg.fg_check_device_error()
    kk, vv = (restored(getattr(one, c + "_codes")[0], getattr(one, c + "_ab")[0], d) for c in "kv")
    p = torch.softmax(torch.einsum("hgd,hnd->hgn", q.view(H, G, d).double(), kk) * d ** -0.5, -1)
    want = torch.einsum("hgn,hnd->hgd", p, vv)
    if gap:
        assert p[:, :, 0].min() > 0.5 and p[:, :, 1:].max() < 1e-2     # one large, the rest small
    got = out.view(B, H, G, d)
    assert relative(got, want) <= 1.2e-3 + (3e-3 if sigma < 0.001 else 0.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [300, 64])          # an item per Q tile, and one that both share
def test_prefill_window_one_large_weight(fg, d, nq):
    """A first key 14.2 nats above 16384 equal ones, with a value of 0: the output is the small
    weights' (2^-20.5 of the first).

    Relative error of a row: the output's rounding and the weights', at most 2^-11 each (the
    weights are all alike, so their errors have one sign); scores of 14.2 from d + 40 operations:
    14.2 (d + 40) 2^-23 = 2.9e-4; the exponential's 2^-21.  Together 1.3e-3."""
    n = 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    k = torch.zeros(n, d, dtype=torch.float16, device="cuda")
    k[0] = 14.2 / d ** 0.5
    v = (1.0 + 0.3 * torch.randn(n, d, generator=g, device="cuda")).half()
    v[0] = 0
    q = torch.ones(nq, d, dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    fg.fg_prefill_attn_window(q, i32([0, nq]), k, v, i32([0, n]), 1, 1, d ** -0.5, out)
    fg.fg_check_device_error()
    s = (q.double() @ k.double().T) * d ** -0.5
    t = torch.arange(n, device="cuda")
    s = s.masked_fill(t > torch.arange(n - nq, n, device="cuda")[:, None], -torch.inf)
    assert relative(out, torch.softmax(s, -1) @ v.double()) <= 1.3e-3


@pytest.mark.parametrize("nq", [256, 100])
def test_prefill_window_visible_nan_costs_little(fg, nq):
    """Rows that see a NaN in a key or in a whole value row have their answer without their keys
    being gone over again (which takes 500 times as long); a NaN in one channel stays in it."""
    d, n, H = 128, 16384, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    q, k, v = (torch.randn(r, H * d, generator=g, device="cuda").half() for r in (nq, n, n))
    qo, ko = i32([0, nq]), i32([0, n])

    def timed(k, v):
        best = 1e9
        for _ in range(4):
            out = torch.empty_like(q)
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            fg.fg_prefill_attn_window(q, qo, k, v, ko, H, H, d ** -0.5, out)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        fg.fg_check_device_error()
        return out, best

    clean, t0 = timed(k, v)
    assert bool(torch.isfinite(clean).all())
    for t, bad_k, bad_v in ((5, True, True), (5, False, True), (n - nq, True, False)):
        kk, vv = k.clone(), v.clone()
        if bad_k:
            kk[t] = torch.nan
        if bad_v:
            vv[t] = torch.nan
        out, dt = timed(kk, vv)
        assert bool(torch.isnan(out).all()), (t, bad_k, bad_v)
        assert dt <= 10 * t0, (dt, t0)
    vv = v.clone()
    vv[7, 3], vv[9, d + 5] = torch.nan, torch.inf
    out, _ = timed(k, vv)
    assert bool(torch.isnan(out[:, 3]).all()) and bool((out[:, d + 5] == torch.inf).all())
    rest = [c for c in range(H * d) if c not in (3, d + 5)]
    assert (out[:, rest].float() - clean[:, rest].float()).abs().max() <= 2e-3 * clean.abs().max()


@pytest.mark.parametrize("G", [1, 2, 4, 7])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("decades", [5, -5, 8, -8])
def test_decode_window_values_of_growing_size(fg, G, d, decades):
    """Values that grow (or shrink) by many orders along a sequence while the scores fall (or rise)
    alike, so that every part of it contributes as much: widths and scores move all along.

    Relative error of a row: the output's rounding, at most 2^-11 = 4.9e-4, and for outputs near
    4.5e-5 (8 decades) half of fp16's smallest step, 2^-25: 6.6e-4; the weights' rounding where one
    fp16 term is kept (G > 2), at most 2^-11 of each (c - 7.5) (b - a)/15, at random before values
    that sum up at random, 1.2 times these: 5.9e-4; the truncated sums, 6e-5; scores of up to 18.4
    from d + 40 operations: 18.4 (d + 40) 2^-23 = 3.7e-4 of the weights.  Together 1.6e-3, and 7e-4
    more for 8 decades."""
    H, B, n = 8, 500, 2048
    g = generator(37)
    up = torch.arange(n, device="cuda") / n * abs(decades)
    size = up + 4 - abs(decades)                            # powers of ten, at most 10^4
    if decades < 0:
        size, up = size.flip(0), up.flip(0)
    v = (torch.randn(n, H * d, generator=g, device="cuda") * 10 ** size[:, None]).half()
    k = (-up * 2.302585 / d ** 0.5).half()[:, None].expand(n, H * d).contiguous()
    q = torch.ones(H * G * d, dtype=torch.float16, device="cuda")
    one = fg.KVCacheQ4(1, n, H * d, H)
    fg.fg_kv_append_q4_ragged(k, v, i32([0, n]), i32([0]), one)
    cache = fg.KVCacheQ4(B, n, H * d, H)
    for name in ("k_codes", "k_ab", "v_codes", "v_ab"):
        getattr(cache, name).copy_(getattr(one, name).expand_as(getattr(cache, name)))
    qs = q.expand(B, -1).contiguous()
    out = torch.empty_like(qs)
    ws = torch.empty(fg.fg_decode_attn_window_workspace_bytes(cache, H * G), dtype=torch.uint8,
                     device="cuda")
    fg.fg_decode_attn_q4kv_window(qs, H * G, cache, i32([n] * B), d ** -0.5, out, ws)
    fg.fg_check_device_error()
    kk, vv = (restored(getattr(one, c + "_codes")[0], getattr(one, c + "_ab")[0], d) for c in "kv")
    p = torch.softmax(torch.einsum("hgd,hnd->hgn", q.view(H, G, d).double(), kk) * d ** -0.5, -1)
    want = torch.einsum("hgn,hnd->hgd", p, vv)
    parts = (p[0, 0, :, None] * vv[0]).norm(dim=-1).view(4, -1).norm(dim=-1)
    assert parts.max() < 8 * parts.min()                   # every quarter of the sequence counts
    assert relative(out.view(B, H, G, d), want) <= (1.6e-3 if abs(decades) == 5 else 2.3e-3)
