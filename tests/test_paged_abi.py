"""Host-side refusals of the rotary positions and the paged cache's calls (no GPU needed), and the
device's index arithmetic and frequencies compiled for the host."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

from oracle import paged as OP

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, MISALIGNED = 0x10000, 0x10008        # never dereferenced: validation fails before any use
OUT = 0x40000000


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__ as g
    g.build()
    from bit_compressed_throughput_gb300 import fg as mod
    return mod


def pool(fg, blocks=FAKE, pages=8, page=32, h=256, H=2):
    return fg.fg_kvpages(blocks, pages, page, h, H)


def rope(fg, angles=FAKE, pos=FAKE, positions=64, rot=64, interleaved=0):
    return fg.fg_rope_rows(angles, pos, positions, rot, interleaved)


BAD_POOLS = [dict(page=24), dict(page=8), dict(page=2048), dict(page=0), dict(H=8), dict(H=3),
             dict(H=0), dict(pages=-1)]


def test_rope_validation(fg):
    L = fg.lib

    def call(x=FAKE, xs=256, rows=4, heads=2, d=128, off=FAKE, nseq=2, r=None, t=0, y=OUT, ys=256):
        return L.fg_rope(x, xs, rows, heads, d, off, nseq, C.byref(r or rope(fg)), t, y, ys, None)

    assert call(d=96) == fg.FG_ERR_SHAPE and call(heads=0) == fg.FG_ERR_SHAPE
    assert call(rows=-1) == fg.FG_ERR_SHAPE and call(nseq=-1) == fg.FG_ERR_SHAPE
    assert call(xs=248) == fg.FG_ERR_SHAPE and call(ys=260) == fg.FG_ERR_SHAPE
    for rot in (0, 8, 40, 144):
        assert call(r=rope(fg, rot=rot)) == fg.FG_ERR_SHAPE
    assert call(r=rope(fg, positions=0)) == fg.FG_ERR_SHAPE
    assert call(r=rope(fg, angles=None)) == fg.FG_ERR_ARG
    assert call(r=rope(fg, angles=MISALIGNED)) == fg.FG_ERR_ARG
    assert call(r=rope(fg, pos=None)) == fg.FG_ERR_ARG
    assert call(r=rope(fg, pos=FAKE + 1)) == fg.FG_ERR_ARG
    assert call(r=rope(fg, interleaved=2)) == fg.FG_ERR_ARG
    assert call(t=2) == fg.FG_ERR_ARG and call(off=None) == fg.FG_ERR_ARG
    assert call(x=None) == fg.FG_ERR_ARG and call(y=MISALIGNED) == fg.FG_ERR_ARG
    assert call(y=FAKE + 32) == fg.FG_ERR_ARG                # rows that overlap
    assert call(y=FAKE, ys=264) == fg.FG_ERR_ARG             # in place with another stride
    assert call(rows=0, x=None, y=None) == fg.FG_OK
    assert call(nseq=0, x=None, y=None, off=None) == fg.FG_OK
    assert L.fg_rope(FAKE, 256, 4, 2, 128, FAKE, 2, None, 0, OUT, 256, None) == fg.FG_ERR_ARG


def test_rope_table_validation(fg):
    def call(t=FAKE, n=16, rot=64, base=1e4, factor=1.0, original=0, low=1.0, high=4.0, gain=1.0):
        return fg.lib.fg_rope_table(t, n, rot, base, factor, original, low, high, gain, None)

    assert call(n=-1) == fg.FG_ERR_SHAPE and call(rot=0) == fg.FG_ERR_SHAPE
    assert call(rot=7) == fg.FG_ERR_SHAPE and call(original=-1) == fg.FG_ERR_SHAPE
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert call(base=bad) == fg.FG_ERR_ARG and call(factor=bad) == fg.FG_ERR_ARG
    assert call(gain=float("nan")) == fg.FG_ERR_ARG
    assert call(original=4096, low=5.0) == fg.FG_ERR_ARG     # low above high
    assert call(t=None) == fg.FG_ERR_ARG and call(t=MISALIGNED) == fg.FG_ERR_ARG
    assert call(t=None, n=0) == fg.FG_OK


def test_paged_rows_validation(fg):
    L = fg.lib

    def append(k=FAKE, v=FAKE, stride=256, rows=4, off=FAKE, pos=FAKE, r=None, kv=None, table=FAKE,
               ts=4, nseq=2):
        return L.fg_kv_append_q4_paged(k, v, stride, rows, off, pos, r and C.byref(r),
                                       C.byref(kv or pool(fg)), table, ts, nseq, None)

    def read(k=FAKE, v=OUT, stride=256, rows=4, off=FAKE, pos=FAKE, kv=None, table=FAKE, ts=4,
             nseq=2):
        return L.fg_kv_read_q4_paged(C.byref(kv or pool(fg)), table, ts, nseq, off, pos, rows, k, v,
                                     stride, None)

    for call in (append, read):
        for bad in BAD_POOLS:
            assert call(kv=pool(fg, **bad)) == fg.FG_ERR_SHAPE, bad
        assert call(stride=248) == fg.FG_ERR_SHAPE and call(stride=260) == fg.FG_ERR_SHAPE
        assert call(rows=-1) == fg.FG_ERR_SHAPE and call(nseq=-1) == fg.FG_ERR_SHAPE
        assert call(nseq=65536) == fg.FG_ERR_SHAPE
        assert call(ts=-1) == fg.FG_ERR_SHAPE and call(ts=1 << 26) == fg.FG_ERR_SHAPE
        assert call(kv=pool(fg, blocks=None)) == fg.FG_ERR_ARG
        assert call(kv=pool(fg, blocks=MISALIGNED)) == fg.FG_ERR_ARG
        assert call(table=None) == fg.FG_ERR_ARG and call(table=FAKE + 2) == fg.FG_ERR_ARG
        assert call(off=None) == fg.FG_ERR_ARG and call(pos=FAKE + 1) == fg.FG_ERR_ARG
        assert call(k=MISALIGNED) == fg.FG_ERR_ARG
        assert call(rows=0, k=None, v=None, off=None, pos=None, table=None) == fg.FG_OK
        assert call(nseq=0, k=None, v=None, off=None, pos=None, table=None) == fg.FG_OK
    assert append(k=None) == fg.FG_ERR_ARG and append(v=None) == fg.FG_ERR_ARG
    assert append(r=rope(fg, rot=24)) == fg.FG_ERR_SHAPE
    assert append(r=rope(fg, angles=None)) == fg.FG_ERR_ARG
    assert read(k=None, v=None) == fg.FG_ERR_ARG and read(v=FAKE) == fg.FG_ERR_ARG
    assert read(v=FAKE + 64) == fg.FG_ERR_ARG                # one output over the other
    assert L.fg_kv_read_q4_paged(None, FAKE, 4, 2, FAKE, FAKE, 4, FAKE, OUT, 256, None) \
        == fg.FG_ERR_ARG


def test_paged_attention_validation(fg):
    L = fg.lib
    wsb = 1 << 30

    def attend(q=FAKE, qs=512, qr=8, off=FAKE, most=4, Hq=4, kv=None, table=FAKE, ts=4, lens=FAKE,
               nseq=2, window=0, sinks=0, scale=0.1, out=OUT, os_=512, lse=None, ws=FAKE, n=wsb):
        return L.fg_attn_q4kv_paged(q, qs, qr, off, most, Hq, C.byref(kv or pool(fg)), table, ts,
                                    lens, nseq, window, sinks, scale, out, os_, lse, ws, n, None)

    def weights(q=FAKE, qs=512, qr=8, off=FAKE, most=4, Hq=4, kv=None, table=FAKE, ts=4, lens=FAKE,
                nseq=2, window=0, sinks=0, scale=0.1, lse=FAKE, acc=FAKE, out=OUT, stride=64):
        return L.fg_attn_weights_q4_paged(q, qs, qr, off, most, Hq, C.byref(kv or pool(fg)), table,
                                          ts, lens, nseq, window, sinks, scale, lse, acc, out,
                                          stride, None)

    for call in (attend, weights):
        for bad in BAD_POOLS:
            assert call(kv=pool(fg, **bad)) == fg.FG_ERR_SHAPE, bad
        assert call(Hq=3) == fg.FG_ERR_SHAPE and call(Hq=0) == fg.FG_ERR_SHAPE
        assert call(Hq=258, qs=258 * 128) == fg.FG_ERR_SHAPE       # 129 heads per K/V head
        assert call(qs=504) == fg.FG_ERR_SHAPE and call(qs=516) == fg.FG_ERR_SHAPE
        assert call(qr=-1) == fg.FG_ERR_SHAPE and call(most=-1) == fg.FG_ERR_SHAPE
        assert call(window=-1) == fg.FG_ERR_SHAPE and call(sinks=-1) == fg.FG_ERR_SHAPE
        for s in (0.0, -1.0, float("inf"), float("nan")):
            assert call(scale=s) == fg.FG_ERR_ARG
        assert call(q=None) == fg.FG_ERR_ARG and call(off=FAKE + 2) == fg.FG_ERR_ARG
        assert call(lens=None) == fg.FG_ERR_ARG and call(table=None) == fg.FG_ERR_ARG
        assert call(nseq=0, q=None, out=None, off=None, lens=None, table=None) == fg.FG_OK
    assert attend(os_=504) == fg.FG_ERR_SHAPE and attend(out=None) == fg.FG_ERR_ARG
    assert attend(lse=FAKE + 2) == fg.FG_ERR_ARG
    assert attend(out=FAKE + 64) == fg.FG_ERR_ARG            # rows that overlap
    assert attend(qr=0, q=None, out=None) == fg.FG_OK
    need = L.fg_attn_paged_workspace_bytes(C.byref(pool(fg)), 4, 4)
    assert need > 0
    assert attend(n=need - 1) == fg.FG_ERR_WORKSPACE
    assert attend(ws=None) == fg.FG_ERR_WORKSPACE and attend(ws=MISALIGNED) == fg.FG_ERR_WORKSPACE
    for bad in BAD_POOLS:
        assert L.fg_attn_paged_workspace_bytes(C.byref(pool(fg, **bad)), 4, 4) == 0
    assert L.fg_attn_paged_workspace_bytes(C.byref(pool(fg)), 3, 4) == 0
    assert L.fg_attn_paged_workspace_bytes(None, 4, 4) == 0
    assert weights(stride=-1) == fg.FG_ERR_SHAPE
    assert weights(lse=None) == fg.FG_ERR_ARG and weights(out=None) == fg.FG_ERR_ARG
    assert weights(acc=FAKE + 1) == fg.FG_ERR_ARG
    assert weights(acc=OUT + 64) == fg.FG_ERR_ARG            # one sum over another's
    many = dict(nseq=65535, Hq=256, qs=1 << 15)              # 2^40 tiles of 16 positions and heads
    assert attend(os_=1 << 15, ts=65472, n=0, **many) == fg.FG_ERR_SHAPE
    assert attend(os_=1 << 15, ts=16384, n=0, **many) == fg.FG_ERR_WORKSPACE
    assert weights(ts=65472, lse=None, **many) == fg.FG_ERR_SHAPE
    assert weights(ts=16384, lse=None, **many) == fg.FG_ERR_ARG


def test_evict_validation(fg):
    def call(kv=None, table=FAKE, ts=4, nseq=2, lens=FAKE, acc=FAKE, stride=64, keep=32, recent=8,
             dst=0x20000, ds=4, kept=OUT, acc_out=OUT + 0x10000, dl=OUT + 0x20000):
        return fg.lib.fg_kv_evict_q4_paged(C.byref(kv or pool(fg)), table, ts, nseq, lens, acc,
                                           stride, keep, recent, dst, ds, kept, acc_out, dl, None)

    for bad in BAD_POOLS:
        assert call(kv=pool(fg, **bad)) == fg.FG_ERR_SHAPE, bad
    assert call(keep=0) == fg.FG_ERR_SHAPE and call(recent=-1) == fg.FG_ERR_SHAPE
    assert call(recent=33) == fg.FG_ERR_SHAPE and call(stride=-1) == fg.FG_ERR_SHAPE
    assert call(keep=129) == fg.FG_ERR_CAPACITY              # four pages of 32
    for name in ("table", "lens", "acc", "dst", "kept", "acc_out", "dl"):
        assert call(**{name: None}) == fg.FG_ERR_ARG, name
        assert call(**{name: FAKE + 2}) == fg.FG_ERR_ARG, name
    assert call(dst=FAKE) == fg.FG_ERR_ARG                   # the same table
    assert call(dl=FAKE) == fg.FG_ERR_ARG                    # lengths in place
    assert call(acc_out=FAKE + 128) == fg.FG_ERR_ARG         # weights that overlap
    assert call(nseq=0, table=None, lens=None, acc=None) == fg.FG_OK


def test_binding_refuses_what_the_library_cannot_see(fg):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        fg.KVPagesQ4(4, 24, 128, 2, device="cpu")
    with pytest.raises(ValueError):
        fg.KVPagesQ4(4, 16, 192, 2, device="cpu")            # d = 96
    with pytest.raises(ValueError):
        fg.KVPagesQ4.of(torch.zeros((2, 2, 100), dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        fg.KVPagesQ4.of(torch.zeros((2, 2, 1152), dtype=torch.int8), 64)
    pool_t = fg.KVPagesQ4(4, 16, 128, 2, device="cpu")
    shapes = [tuple(p.shape) for p in pool_t.parts()]
    assert shapes == [(4, 2, 16, 32), (4, 2, 16, 1, 2)] * 2
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    h16 = lambda *s: torch.zeros(s, dtype=torch.float16)
    f32 = lambda *s: torch.zeros(s)
    ok = dict(k=h16(3, 128), v=h16(3, 128), off=i32(3), pos=i32(2), table=i32(2, 2), ang=None,
              rp=None)

    def append(**kw):
        a = {**ok, **kw}
        fg.fg_kv_append_q4_paged(a["k"], a["v"], a["off"], a["pos"], pool_t, a["table"],
                                 angles=a["ang"], rope_pos=a["rp"])

    for kw in (dict(k=h16(3, 64)), dict(v=h16(2, 128)), dict(k=f32(3, 128)), dict(off=i32(2)),
               dict(pos=i32(3)), dict(table=i32(2)), dict(table=torch.zeros((2, 2))),
               dict(ang=f32(8, 32)), dict(ang=f32(8, 32, 2), rp=i32(3)), dict(rp=i32(2))):
        with pytest.raises(ValueError):
            append(**kw)
    with pytest.raises(ValueError):
        fg.fg_rope(h16(3, 100), 64, i32(3), i32(2), f32(8, 32, 2), h16(3, 100))
    with pytest.raises(ValueError):
        fg.fg_rope(h16(3, 128), 64, i32(3), i32(2), f32(8, 32, 2), h16(2, 128))
    with pytest.raises(ValueError):
        fg.fg_rope(h16(3, 128), 64, i32(4), i32(2), f32(8, 32, 2), h16(3, 128))

    def attend(q=h16(3, 256), off=i32(3), table=i32(2, 2), lens=i32(2), out=h16(3, 256), lse=None,
               **kw):
        fg.fg_attn_q4kv_paged(q, off, 4, pool_t, table, lens, 0.1, out, None, lse=lse, **kw)

    for kw in (dict(q=h16(3, 128)), dict(out=h16(2, 256)), dict(lens=i32(3)), dict(off=i32(4)),
               dict(lse=f32(3, 2)), dict(window=1 << 31), dict(table=i32(2, 2).long())):
        with pytest.raises(ValueError):
            attend(**kw)
    with pytest.raises(ValueError):
        fg.fg_attn_weights_q4_paged(h16(3, 256), i32(3), 4, pool_t, i32(2, 2), i32(2), 0.1,
                                    f32(3, 4), f32(2, 2, 8), f32(2, 2, 9))
    with pytest.raises(ValueError):
        fg.fg_kv_evict_q4_paged(pool_t, i32(2, 2), i32(2), f32(2, 2, 8), 1, i32(2, 2), i32(2, 2, 4),
                                f32(2, 2, 5), i32(2))


HOST_SRC = r"""
#include "paged.cuh"
#include "rope.h"
using namespace fg;
extern "C" {
long long h_slot(const int32_t* table, long long stride, int pages, int lg, int b, long long p) {
  return PagedCache{nullptr, table, stride, pages, lg, 2, 3}.slot(b, p);
}
long long h_block(int lg, int H, long long slot, int head, int d) {
  PagedCache c{nullptr, nullptr, 0, 0, lg, H, 0};
  return c.block(slot, head, d) - (uint8_t*)nullptr;
}
double h_frequency(double base, double factor, int original, double low, double high, int j,
                   int half) {
  return rope_frequency(RopeScale{base, factor, low, high, 1.0, original}, j, half);
}
}
"""


@pytest.fixture(scope="module")
def dll(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src, so = d / "p.cpp", d / "p.so"
    src.write_text(HOST_SRC)
    inc = os.path.join(ROOT, "bit_compressed_throughput_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o",
                    str(so)], check=True)
    dll = C.CDLL(str(so))
    dll.h_slot.restype = dll.h_block.restype = C.c_longlong
    dll.h_slot.argtypes = [C.c_void_p, C.c_longlong, C.c_int, C.c_int, C.c_int, C.c_longlong]
    dll.h_block.argtypes = [C.c_int, C.c_int, C.c_longlong, C.c_int, C.c_int]
    dll.h_frequency.restype = C.c_double
    dll.h_frequency.argtypes = [C.c_double, C.c_double, C.c_int, C.c_double, C.c_double, C.c_int,
                                C.c_int]
    return dll


def test_slots_and_blocks(dll):
    table = np.array([[3, 0], [7, -1], [1 << 30, 2]], np.int32)
    at = lambda b, p, lg=5, pages=8: dll.h_slot(table.ctypes.data, 2, pages, lg, b, p)
    assert at(0, 0) == 96 and at(0, 31) == 127 and at(0, 32) == 0 and at(1, 5) == 229
    assert at(1, 40) == -1 and at(2, 0) == -1 and at(2, 33) == 65
    assert at(2, 0, lg=10, pages=(1 << 30) + 1) == 1 << 40   # past 32 bits
    for d, per in ((64, 72), (128, 144)):
        assert dll.h_block(4, 3, 16 * 5, 2, d) == (5 * 3 + 2) * 16 * per
        assert dll.h_block(10, 96, 1 << 33, 95, d) == ((1 << 23) * 96 + 95) * 1024 * per


def test_frequencies(dll):
    for kw in (dict(), dict(factor=4.0), dict(factor=8.0, original=8192, low=1.0, high=4.0),
               dict(base=5e5, factor=2.0, original=512, low=2.0, high=2.0)):
        w = OP.frequencies(128, **kw)
        for j in range(64):
            got = dll.h_frequency(kw.get("base", 1e4), kw.get("factor", 1.0), kw.get("original", 0),
                                  kw.get("low", 1.0), kw.get("high", 4.0), j, 64)
            assert abs(got - w[j]) <= 1e-14 * w[j], (kw, j)
