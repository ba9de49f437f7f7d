"""Host-side refusals of the ragged cache calls and the windowed attention (no GPU needed), and
the device's index arithmetic compiled for the host."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, MISALIGNED = 0x10000, 0x10008        # never dereferenced: validation fails before any use


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__ as g
    g.build()
    from bit_compressed_throughput_gb300 import fg as mod
    return mod


def kvs(fg, B=2, cap=32, h=256, H=2, k=FAKE):
    return fg.fg_kvcache(k, FAKE, FAKE, FAKE, B, cap, h, H)


def test_ragged_cache_validation(fg):
    L = fg.lib

    def append(k=FAKE, v=FAKE, stride=256, rows=4, off=FAKE, pos=FAKE, kv=None):
        return L.fg_kv_append_q4_ragged(k, v, stride, rows, off, pos,
                                        C.byref(kv or kvs(fg)), None)

    def read(k=FAKE, v=FAKE, stride=256, rows=4, off=FAKE, pos=FAKE, kv=None):
        return L.fg_kv_read_q4_ragged(C.byref(kv or kvs(fg)), off, pos, rows, k, v, stride, None)

    for call in (append, read):
        assert call(stride=248) == fg.FG_ERR_SHAPE
        assert call(stride=260) == fg.FG_ERR_SHAPE
        assert call(rows=-1) == fg.FG_ERR_SHAPE
        assert call(kv=kvs(fg, cap=20)) == fg.FG_ERR_SHAPE
        assert call(kv=kvs(fg, H=8)) == fg.FG_ERR_SHAPE               # d = 32
        assert call(kv=kvs(fg, k=None)) == fg.FG_ERR_ARG
        assert call(k=MISALIGNED) == fg.FG_ERR_ARG
        assert call(off=None) == fg.FG_ERR_ARG
        assert call(pos=None) == fg.FG_ERR_ARG
        assert call(off=FAKE + 2) == fg.FG_ERR_ARG
        assert call(rows=0, k=None, v=None, off=None, pos=None) == fg.FG_OK
        assert call(kv=kvs(fg, B=0), k=None, v=None, off=None, pos=None) == fg.FG_OK
    assert append(k=None) == fg.FG_ERR_ARG and append(v=None) == fg.FG_ERR_ARG
    assert read(k=None, v=None) == fg.FG_ERR_ARG
    assert read(k=FAKE, v=FAKE) == fg.FG_ERR_ARG                      # one output over the other


def test_decode_window_validation(fg):
    L = fg.lib
    wsb = 1 << 30

    def call(q=FAKE, qs=512, Hq=4, kv=None, lens=FAKE, window=8, sinks=2, scale=0.1, out=FAKE,
             os_=512, ws=FAKE, n=wsb):
        return L.fg_decode_attn_q4kv_window(q, qs, Hq, C.byref(kv or kvs(fg)), lens, window, sinks,
                                            scale, out, os_, ws, n, None)

    assert call(Hq=3) == fg.FG_ERR_SHAPE and call(Hq=0) == fg.FG_ERR_SHAPE
    assert call(qs=504) == fg.FG_ERR_SHAPE and call(qs=516) == fg.FG_ERR_SHAPE
    assert call(os_=504) == fg.FG_ERR_SHAPE
    assert call(window=-1) == fg.FG_ERR_SHAPE and call(sinks=-1) == fg.FG_ERR_SHAPE
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=s) == fg.FG_ERR_ARG
    assert call(q=None) == fg.FG_ERR_ARG and call(out=MISALIGNED) == fg.FG_ERR_ARG
    assert call(lens=None) == fg.FG_ERR_ARG and call(lens=FAKE + 1) == fg.FG_ERR_ARG
    assert call(kv=kvs(fg, B=0), q=None, out=None, lens=None) == fg.FG_OK
    need = L.fg_decode_attn_window_workspace_bytes(C.byref(kvs(fg)), 4)
    if need:
        assert call(n=need - 1) == fg.FG_ERR_WORKSPACE
        assert call(ws=None) == fg.FG_ERR_WORKSPACE and call(ws=MISALIGNED) == fg.FG_ERR_WORKSPACE
    assert L.fg_decode_attn_window_workspace_bytes(C.byref(kvs(fg, cap=20)), 4) == 0
    assert L.fg_decode_attn_window_workspace_bytes(C.byref(kvs(fg)), 3) == 0
    assert L.fg_decode_attn_window_workspace_bytes(None, 4) == 0
    # more heads, or more tiles of row sets, than the kernel can number
    many = kvs(fg, h=64, H=1)
    assert call(kv=many, Hq=65537, qs=65537 * 64, os_=65537 * 64) == fg.FG_ERR_SHAPE
    assert L.fg_decode_attn_window_workspace_bytes(C.byref(many), 65536) > 0
    assert L.fg_decode_attn_window_workspace_bytes(C.byref(many), 65537) == 0
    long = kvs(fg, B=64, cap=1 << 26, h=64, H=1)
    assert call(kv=long, Hq=8192, qs=8192 * 64, os_=8192 * 64) == fg.FG_ERR_SHAPE
    assert L.fg_decode_attn_window_workspace_bytes(C.byref(long), 8192) == 0


def test_prefill_window_validation(fg):
    L = fg.lib

    def call(q=FAKE, qs=256, qr=8, qo=FAKE, k=FAKE, v=FAKE, ks=128, kr=8, ko=FAKE, nseq=2, Hq=4,
             Hkv=2, d=64, window=0, sinks=0, scale=0.1, out=0x90000, os_=256):
        return L.fg_prefill_attn_window(q, qs, qr, qo, k, v, ks, kr, ko, nseq, Hq, Hkv, d, window,
                                        sinks, scale, out, os_, None)

    assert call(Hkv=3) == fg.FG_ERR_SHAPE and call(d=32) == fg.FG_ERR_SHAPE
    assert call(Hq=0) == fg.FG_ERR_SHAPE and call(Hkv=0) == fg.FG_ERR_SHAPE
    assert call(Hq=1 << 17, Hkv=1 << 17, qs=1 << 23, os_=1 << 23, ks=1 << 23) == fg.FG_ERR_SHAPE
    assert call(nseq=-1) == fg.FG_ERR_SHAPE and call(qr=-1) == fg.FG_ERR_SHAPE
    assert call(kr=-1) == fg.FG_ERR_SHAPE
    assert call(qs=248) == fg.FG_ERR_SHAPE and call(ks=132) == fg.FG_ERR_SHAPE
    assert call(os_=260) == fg.FG_ERR_SHAPE and call(ks=120) == fg.FG_ERR_SHAPE
    assert call(window=-1) == fg.FG_ERR_SHAPE and call(sinks=-5) == fg.FG_ERR_SHAPE
    assert call(scale=0.0) == fg.FG_ERR_ARG
    assert call(q=None) == fg.FG_ERR_ARG and call(k=None) == fg.FG_ERR_ARG
    assert call(v=MISALIGNED) == fg.FG_ERR_ARG and call(qo=None) == fg.FG_ERR_ARG
    assert call(ko=FAKE + 2) == fg.FG_ERR_ARG
    for alias in ("q", "k", "v"):
        assert call(**{alias: 0x90000}) == fg.FG_ERR_ARG
    assert call(nseq=0, q=None, out=None, qo=None, ko=None) == fg.FG_OK
    assert call(qr=0, q=None, out=None, k=None, v=None) == fg.FG_OK


HOST_SRC = r"""
#include "ragged.cuh"
using namespace fg;
extern "C" {
int h_sequence_of_row(const int32_t* off, int n, int r) { return sequence_of_row(off, n, r); }
int h_offsets_ok(const int32_t* off, int n, int rows) { return offsets_ok(off, n, rows, 0, 1); }
void h_seq_tiles(int len, int window, int sinks, int32_t* o) {
  const SeqTiles s = seq_tiles(len, window, sinks);
  o[0] = s.len; o[1] = s.wstart; o[2] = s.nt; o[3] = s.ns; o[4] = s.tw;
}
int h_tile_pos(int len, int window, int sinks, int u) {
  return tile_pos(seq_tiles(len, window, sinks), u);
}
int h_run_tiles(int len, int window, int sinks, int u, int u1) {
  return run_tiles(seq_tiles(len, window, sinks), u, u1);
}
int64_t h_first_tile(int64_t total, int nw, int w) { return Shares(total, nw).first(w); }
int h_share_of(int64_t total, int nw, int64_t x) { return Shares(total, nw).share_of(x); }
void h_key_tiles(int r0, int nq, int nk, int window, int sinks, int32_t* o) {
  const KeyTiles k = key_tiles(r0, nq, nk, window, sinks);
  o[0] = k.ns; o[1] = k.tw; o[2] = k.te;
}
void h_either(const int32_t* a, const int32_t* b, int32_t* o) {
  const KeyTiles k = either(KeyTiles{a[0], a[1], a[2]}, KeyTiles{b[0], b[1], b[2]});
  o[0] = k.ns; o[1] = k.tw; o[2] = k.te;
}
void h_key_steps(int tile, int lo, int hi, int window, int sinks, int32_t* o) {
  const KeySteps k = key_steps(tile, lo, hi, window, sinks);
  o[0] = k.s0; o[1] = k.s1;
}
unsigned h_visible_bits(int c0, int i, int window, int sinks) {
  return visible_bits(c0, i, window, sinks);
}
int h_visible(int t, int i, int window, int sinks) { return visible(t, i, window, sinks); }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("ragged")
    src, lib = d / "h.cpp", d / "h.so"
    src.write_text(HOST_SRC)
    inc = os.path.join(ROOT, "bit_compressed_throughput_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o",
                    str(lib)], check=True)
    dll = C.CDLL(str(lib))
    dll.h_first_tile.argtypes = [C.c_int64, C.c_int, C.c_int]
    dll.h_first_tile.restype = C.c_int64
    dll.h_visible_bits.restype = C.c_uint32
    dll.h_share_of.argtypes = [C.c_int64, C.c_int, C.c_int64]
    return dll


def arr(x):
    a = np.asarray(x, np.int32)
    return a, a.ctypes.data_as(C.POINTER(C.c_int32))


def test_sequence_of_row(host):
    rng = np.random.default_rng(1)
    for _ in range(200):
        n = int(rng.integers(1, 20))
        lens = rng.integers(0, 4, n)
        off = np.concatenate([[0], np.cumsum(lens)]) + int(rng.integers(0, 3))
        keep, p = arr(off)
        for r in range(-1, int(off[-1]) + 3):
            want = [b for b in range(n) if off[b] <= r < off[b + 1]]
            assert host.h_sequence_of_row(p, n, r) == (want[0] if want else -1)


def test_sequence_of_row_stays_inside_for_any_offsets(host):
    """Offsets that fall, repeat or overflow: the answer is a sequence or -1."""
    rng = np.random.default_rng(2)
    for _ in range(500):
        n = int(rng.integers(1, 9))
        keep, p = arr(rng.choice([-2 ** 31, -5, 0, 1, 3, 7, 2 ** 31 - 1], n + 1))
        for r in (0, 1, 3, 6, 2 ** 31 - 1):
            assert -1 <= host.h_sequence_of_row(p, n, r) < n


def test_offsets_ok(host):
    for off, rows, ok in (([0, 2, 2, 5], 5, 1), ([1, 2, 2, 5], 9, 1), ([0, 3, 2, 5], 5, 0),
                          ([0, 2, 2, 6], 5, 0), ([-1, 2, 2, 5], 5, 0), ([0, 0], 0, 1)):
        keep, p = arr(off)
        assert host.h_offsets_ok(p, len(off) - 1, rows) == ok, off


def test_visible(host):
    from oracle import window as OW
    for n in (1, 7, 20):
        for window in (0, 1, 5, 2 ** 31 - 1):
            for sinks in (0, 2, 2 ** 31 - 1):
                for i in range(n):
                    got = [t for t in range(n) if host.h_visible(t, i, window, sinks)]
                    assert got == OW.visible(i, n, window, sinks).tolist()


def test_decode_tiles_are_the_visible_ones(host):
    """The tiles of a sequence are those that hold a visible position, each once and in order, in
    at most two runs of positions."""
    from oracle import window as OW
    for n in (1, 15, 16, 17, 47, 48, 100, 161):
        for window in (0, 1, 2, 15, 16, 17, 40, 160, 2 ** 31 - 1):
            for sinks in (0, 1, 15, 16, 17, 33, 64, 200, 2 ** 31 - 1):
                o = np.zeros(5, np.int32)
                host.h_seq_tiles(n, window, sinks, o.ctypes.data_as(C.POINTER(C.c_int32)))
                want = sorted(set((OW.visible(n - 1, n, window, sinks) // 16).tolist()))
                pos = [host.h_tile_pos(n, window, sinks, u) for u in range(o[2])]
                assert pos == [16 * t for t in want], (n, window, sinks)
                assert o[1] == (max(0, n - window) if window else 0)
                for u1 in range(1, len(pos) + 1):
                    u = runs = 0
                    while u < u1:
                        c = host.h_run_tiles(n, window, sinks, u, u1)
                        assert 1 <= c and u + c <= u1
                        assert pos[u + c - 1] == pos[u] + 16 * (c - 1)
                        u += c
                        runs += 1
                    assert runs <= 2
    o = np.zeros(5, np.int32)
    for n in (0, 2 ** 31 - 16):                            # nothing, and the longest
        host.h_seq_tiles(n, 0, 0, o.ctypes.data_as(C.POINTER(C.c_int32)))
        assert o[2] == n // 16


def test_worker_ranges(host):
    """The ranges cover the order without gaps, differ by one tile at most, and share_of is
    their inverse, for small and for very large totals."""
    for total, nw in ((1, 1), (7, 3), (576, 192), (5000, 2432), (2 ** 40 + 12345, 2432),
                      (2 ** 55 + 1, 24576)):
        first = [host.h_first_tile(total, nw, w) for w in range(nw + 1)]
        assert first[0] == 0 and first[-1] == total
        size = np.diff(np.array(first, dtype=object))
        assert min(size) >= total // nw and max(size) <= total // nw + 1
        for w in list(range(0, nw, max(1, nw // 50))) + [nw - 1]:
            for x in {first[w], first[w + 1] - 1}:
                assert host.h_share_of(total, nw, x) == w, (total, nw, w)


def tiles(host, *args):
    o = np.zeros(3, np.int32)
    host.h_key_tiles(*args, o.ctypes.data_as(C.POINTER(C.c_int32)))
    ns, tw, te = (int(x) for x in o)
    return o, set(range(ns)) | set(range(tw, te)), ns + te - tw


def test_prefill_key_tiles(host):
    """The key tiles of a query tile hold every key that one of its rows sees, each once, and no
    tile without one except between two rows' windows; the tiles of a pair are the union."""
    from oracle import window as OW
    rng = np.random.default_rng(5)
    cases = [(nq, nk, w, s) for nq in (1, 100, 128, 129, 300) for nk in (0, 1, 99, 128, 257, 700)
             for w, s in ((0, 0), (1, 0), (2, 130), (64, 4), (128, 128), (129, 300), (500, 1),
                          (2 ** 31 - 1, 2 ** 31 - 1))]
    cases += [tuple(int(x) for x in rng.integers(1, 900, 4)) for _ in range(60)]
    for nq, nk, w, s in cases:
        for r0 in range(0, nq + 128, 128):
            o, got, n = tiles(host, r0, nq, nk, w, s)
            assert n == len(got)
            want = set()
            for r in range(r0, min(nq, r0 + 128)):
                if nk - nq + r >= 0:
                    want |= set((OW.visible(nk - nq + r, nk, w, s) // 128).tolist())
            assert want == got, (nq, nk, w, s, r0, want, got)
            for tile in got:
                seen = set()
                for r in range(r0, min(nq, r0 + 128)):
                    v = OW.visible(nk - nq + r, nk, w, s) if nk - nq + r >= 0 else np.zeros(0, int)
                    seen |= set(((v[v // 128 == tile] - 128 * tile) // 16).tolist())
                host.h_key_steps(tile, nk - nq + r0, nk - nq + min(r0 + 128, nq) - 1, w, s, o.ctypes.data_as(C.POINTER(C.c_int32)))
                assert 0 <= o[0] < o[1] <= 8
                assert min(seen) == o[0] and max(seen) == o[1] - 1, (nq, nk, w, s, r0, tile)
            assert not got or max(got) * 128 < nk
            o, _, _ = tiles(host, r0, nq, nk, w, s)
            o2, got2, _ = tiles(host, r0 + 128, nq, nk, w, s)
            u = np.zeros(3, np.int32)
            ptr = [x.ctypes.data_as(C.POINTER(C.c_int32)) for x in (o, o2, u)]
            host.h_either(*ptr)
            union = set(range(u[0])) | set(range(u[1], u[2]))
            assert got | got2 <= union and len(union) == u[0] + u[2] - u[1]
            assert union == got | got2, (nq, nk, w, s, r0)


def test_visible_bits(host):
    for c0 in (0, 32, 64, 96, 1024):
        for i in (0, 1, 31, 32, 40, 95, 96, 1023, 1030, 1055, 5000):
            for w in (0, 1, 3, 31, 32, 33, 1000, 2 ** 31 - 1):
                for s in (0, 1, 31, 33, 70, 1040, 2 ** 31 - 1):
                    got = host.h_visible_bits(c0, i, w, s)
                    want = sum(1 << e for e in range(32)
                               if c0 + e <= i and (w == 0 or c0 + e > i - w or c0 + e < s))
                    assert got == want, (c0, i, w, s)
