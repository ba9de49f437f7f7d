"""Attention over pages over the range of what the 4-bit format holds: K^ and V^ are the format's values
bit for bit, and small and large groups lose nothing that the arithmetic does not say."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as OP
from oracle import quant as OQ
from paged_util import F32, H16, i32, offsets, rows_of
from parity_util import dev, host, lib
from test_gpu_paged import paged_case, run_attend

pytestmark = pytest.mark.gpu

SCALES = [1e-6, 1e-5, 1e-4, 1e-2, 1.0, 4000.0]


@pytest.fixture(scope="module")
def fg():
    return lib()


def batch(n, single):
    """Every position of one page table row as a query: a prompt of n, or n single tokens that share its
    pages."""
    return (list(range(1, n + 1)), [1] * n) if single else ([n], [n])


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("d,G,P", [(64, 1, 16), (128, 4, 64), (64, 9, 256), (128, 7, 32)])
@pytest.mark.parametrize("single", [False, True])
def test_attention_takes_the_formats_values(fg, scale, d, G, P, single):
    """A window of one position: a row's output is that position's V^, its weight 1 (2^7 before the sum,
    2^7, divides it), and with a query of one channel its log-sum-exp is that of K^."""
    n, H = 300, 2
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, [n], [n], 3 + d, G, scale=scale)
    lens, nq = batch(n, single)
    q[:] = 0
    ch = (np.arange(n)[:, None] * 7 + np.arange(H * G)[None]) % d
    rows = np.arange(n)[:, None]
    q[q_off[0] + rows, np.arange(H * G) * d + ch] = 1.0
    a = 1.0 / scale
    out, z = run_attend(fg, dev(q)[:, :H * G * d], offsets(nq, q_off[0]), H * G, pool,
                        np.repeat(table, len(nq), 0), lens, a, window=1, max_q=max(nq))
    fg.fg_check_device_error()
    live = slice(q_off[0], q_off[1])
    got, z = host(out)[live].reshape(n, H, G, d), host(z)[live].astype(np.float64)
    assert np.array_equal(got, np.broadcast_to(
        np.moveaxis(rows_of(v, table, 0, n), 0, 1)[:, :, None], got.shape))
    kk = rows_of(k, table, 0, n).astype(np.float64)                    # [H][n][d]
    want = a * kk[np.arange(H * G) // G, rows, ch]
    # nine binary32 roundings (the scale, twice, the score, its shifts by 7 and by the maximum and back,
    # log2, ln 2) of numbers of |want| / ln 2 + 7 at most, half a step each, the exponential and log2
    # one or two: 16 halves
    assert np.all(np.abs(z - want) <= 16 * 2.0 ** -24 * (np.abs(want) * 1.5 + 7))


@pytest.mark.parametrize("d,G,P", [(64, 1, 16), (128, 4, 64), (64, 9, 256), (128, 8, 32)])
@pytest.mark.parametrize("single", [False, True])
def test_infinite_statistics(fg, d, G, P, single):
    """Infinities and NaN of V^ where the format has them (codes of 0 among them), and in no other row."""
    n, H = 200, 1
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, [n], [n], 9 + d, G)
    lens, nq = batch(n, single)
    codes, ab = (host(x).copy() for x in pool.parts()[2:])
    at = np.arange(0, n, 7)
    for i, p in enumerate(at):
        word = [(1.0, np.inf), (-np.inf, 2.0), (np.nan, 1.0), (0.5, np.nan), (-np.inf, np.inf)][i % 5]
        ab[table[0, p // P], 0, p % P, i % (d // 64)] = word
    pool.parts()[3].copy_(torch.from_numpy(ab))
    with np.errstate(invalid="ignore"):
        c = np.stack([codes & 15, codes >> 4], -1).reshape(-1, d)
        vals = OQ.dequant_g64(c, *(ab.reshape(-1, d // 64, 2)[..., i] for i in (0, 1)))
    want = rows_of(vals.reshape(ab.shape[0], H, P, d), table, 0, n)[0]
    out, _ = run_attend(fg, dev(q)[:, :G * d], offsets(nq, q_off[0]), G, pool,
                        np.repeat(table, len(nq), 0), lens, 0.125, window=1, max_q=max(nq))
    fg.fg_check_device_error()
    got = host(out)[q_off[0]:q_off[1]].reshape(n, G, d)
    assert not np.isfinite(want[at]).all(1).any() and np.isposinf(want).any()
    assert np.array_equal(got, np.broadcast_to(want[:, None], got.shape), equal_nan=True)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("d,H,G,P,lens,nq,window,sinks", [
    (128, 2, 1, 16, [300], [200], 0, 0),
    (64, 1, 4, 64, [900], [33], 0, 0),
    (128, 1, 12, 32, [700], [9], 300, 5),
    (128, 2, 1, 16, [300, 5, 1111], [1, 1, 1], 0, 0),
    (64, 1, 2, 32, [2000], [1], 500, 4),
    (128, 2, 4, 64, [130, 900], [1, 1], 0, 0),
    (64, 1, 7, 16, [700, 77], [1, 1], 0, 0),
])
def test_attention_over_the_range_of_values(fg, scale, d, H, G, P, lens, nq, window, sinks):
    """As check_attend's bound, without an error of K^ and V^.  The weights of streamed single tokens are
    two fp16 terms: 2^-22 of a weight."""
    table, pool, k, v, q_off, q = paged_case(fg, d, H, P, lens, nq, 5 + d + G, G, scale=scale)
    a = 1.0 / (math.sqrt(d) * scale)
    out, z = run_attend(fg, dev(q)[:, :H * G * d], q_off, H * G, pool, table, lens, a, max_q=max(nq),
                        window=window, sinks=sinks)
    fg.fg_check_device_error()
    got, z = host(out).astype(np.float64), host(z)
    for b, n in enumerate(lens):
        r = slice(q_off[b], q_off[b + 1])
        ok = OP.seen(n - nq[b], nq[b], n, window, sinks)
        for hk in range(H):
            kk, vv = (rows_of(x, table, b, n)[hk].astype(np.float64) for x in (k, v))
            qq = q[r, hk * G * d:(hk + 1) * G * d].reshape(nq[b], G, d)
            o, lse, p = OP.attend(qq, kk, vv, ok, a)
            aq = np.abs(qq.astype(np.float64))
            moved = np.einsum("rgd,td->rgt", aq, np.abs(kk) * (d + 40) * F32) * a
            ds = np.where(ok[:, None], moved, 0).max(-1)
            V = p @ np.abs(vv)
            rounded = 2.0 ** -22 if max(nq) == 1 and G <= 8 else H16
            tol = ((np.expm1(2 * ds)[..., None] + rounded + 2.0 ** -21 + (n + 64) * F32) * V
                   + n * 2.0 ** -31 * np.abs(vv).max(0) + H16 * np.abs(o) + 2.0 ** -25)
            err = np.abs(got[r, hk * G * d:(hk + 1) * G * d].reshape(nq[b], G, d) - o)
            assert np.all(err <= tol), (b, hk, float((err / tol).max()))
            zt = 2 * ds + 2.0 ** -20 + (n + 64) * F32 + np.abs(lse) * 4 * F32
            assert np.all(np.abs(z[r, hk * G:(hk + 1) * G] - lse) <= zt), (b, hk)


@pytest.mark.parametrize("d,G", [(64, 1), (128, 4)])
def test_sums_do_not_lose_with_the_length(fg, d, G):
    """65,536 positions of values around 2 that one warp adds up: the outputs' errors have no common
    direction.  A rounding of an output is half a step at most, either way; 1500 of them that agree in
    no direction lie within 0.17 half steps on average (Hoeffding's bound, one in 10^9), and the weights'
    errors, of 65,536 each, within less; 128 truncated additions before a sum is moved lose 2^-23 of it
    each, and 32 rounded ones 2^-24: together less than 0.3 half steps."""
    H, P, n = 8, 64, 65536
    warps = 16 if d == 64 else 12
    B = torch.cuda.get_device_properties(0).multi_processor_count * warps // H
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    pool = fg.KVPagesQ4(n // P, P, H * d, H)
    for codes, ab, mid in zip(pool.parts()[0::2], pool.parts()[1::2], (0.0, 2.0)):
        codes.copy_(torch.randint(0, 256, codes.shape, generator=gen, device="cuda", dtype=torch.uint8))
        half = 1.0 + torch.rand(ab.shape[:-1], generator=gen, device="cuda")
        ab.copy_(torch.stack((mid - half, mid + half), -1))
    order = torch.randperm(n // P, generator=gen, device="cuda").int()
    table = order.expand(B, -1).contiguous()
    q = torch.randn((B, H * G * d), generator=gen, device="cuda").half()
    scale = 1.0 / math.sqrt(d)
    out, z = run_attend(fg, q, list(range(B + 1)), H * G, pool, host(table), [n] * B, scale, max_q=1)
    fg.fg_check_device_error()
    at = i32([0, n]), i32([0])
    kv = torch.empty((n, 2 * H * d), dtype=torch.float16, device="cuda")
    fg.fg_kv_read_q4_paged(pool, table[:1].contiguous(), *at, kv[:, :H * d], kv[:, H * d:])
    k, v = (x.double().view(n, H, d).transpose(0, 1) for x in (kv[:, :H * d], kv[:, H * d:]))
    rel = []
    for b in (0, B // 2, B - 1):
        s = q[b].double().view(H, G, d) @ k.mT * scale
        o = torch.softmax(s, -1) @ v
        rel.append(((out[b].double().view(H, G, d) - o) / o.abs()).flatten())
        assert (torch.logsumexp(s, -1).flatten() - z[b]).abs().max() <= 2.0 ** -16
    rel = torch.cat(rel)
    assert rel.abs().max() <= 4 * H16 and rel.mean().abs() <= 0.3 * H16
