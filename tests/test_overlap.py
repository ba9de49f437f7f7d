"""Overlapping rows: the rule against every byte, and the calls that refuse them (no GPU needed)."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x100000                             # never dereferenced: validation fails before any use

SRC = r"""
#include "overlap.h"
extern "C" int overlap(uint64_t a, int64_t ra, int64_t sa, int64_t wa, uint64_t b, int64_t rb,
                       int64_t sb, int64_t wb) {
  return fg::rows_overlap(fg::RowSet{a, ra, sa, wa}, fg::RowSet{b, rb, sb, wb});
}
"""


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    src, lib = d / "o.cpp", d / "o.so"
    src.write_text(SRC)
    inc = os.path.join(ROOT, "bit_compressed_throughput_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o",
                    str(lib)], check=True)
    fn = C.CDLL(str(lib)).overlap
    fn.argtypes = ([C.c_uint64] + [C.c_int64] * 3) * 2
    return fn


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__ as g
    g.build()
    from bit_compressed_throughput_gb300 import fg as mod
    return mod


def cells(at, rows, stride, width):
    return {at + r * stride + c for r in range(rows) for c in range(width)}


def test_rows_overlap_is_every_byte(overlap):
    rng = np.random.default_rng(3)
    seen = [0, 0]
    for i in range(20000):
        sets = []
        for _ in range(2):
            width = int(rng.integers(1, 9))
            sets.append((int(rng.integers(100, 160)), int(rng.integers(0, 7)),
                         int(rng.integers(width, 20)), width))
        if i % 2:                           # equal strides
            s = max(sets[0][3], sets[1][3], sets[0][2])
            sets = [(a, r, s, w) for a, r, _, w in sets]
        want = bool(cells(*sets[0]) & cells(*sets[1]))
        assert bool(overlap(*sets[0], *sets[1])) == want, sets
        assert bool(overlap(*sets[1], *sets[0])) == want, sets
        seen[want] += 1
    assert min(seen) > 2000


def test_rows_overlap_of_large_sets(overlap):
    big = 1 << 40
    assert not overlap(0x1000, 1 << 31, big, 256, 0x1100, 1 << 31, big, 256)
    assert overlap(0x1000, 1 << 31, big, 256, 0x10FF, 1 << 31, big, 256)
    assert overlap(0x1000, 1 << 31, big, 256, 0x1000 + 5 * big - 100, 1, 1 << 62, 256)
    assert not overlap(0x1000, 4, big, 256, 0x1000 + 4 * big, 4, big, 256)


def test_calls_refuse_overlapping_rows(fg):
    L, ARG = fg.lib, fg.FG_ERR_ARG
    kv = fg.fg_kvcache(0x10000, 0x10000, 0x10000, 0x10000, 4, 32, 256, 2)

    def read(k, v, stride):
        return L.fg_kv_read_q4_ragged(C.byref(kv), 0x10000, 0x10000, 8, k, v, stride, None)

    assert read(BASE, BASE + 16, 256) == ARG
    assert read(BASE, BASE + 496, 512) == ARG
    assert read(BASE + 7 * 512, BASE, 256) == ARG

    def decode(q, out, qs=256, os_=256):
        return L.fg_decode_attn_q4kv_window(q, qs, 2, C.byref(kv), 0x10000, 0, 0, 0.1, out, os_,
                                            0x10000, 1 << 30, None)

    assert decode(BASE, BASE, os_=512) == ARG            # in place, but not row over row
    assert decode(BASE, BASE + 512) == ARG               # shifted by a row
    assert decode(BASE + 16, BASE) == ARG

    def prefill(q, k, v, out, qs=256, ks=256, os_=256):
        return L.fg_prefill_attn_window(q, qs, 8, 0x10000, k, v, ks, 8, 0x10000, 2, 4, 4, 64, 0, 0,
                                        0.1, out, os_, None)

    far = [0x900000, 0xA00000, 0xB00000]
    for i in range(3):
        for shift in (16, 512, 7 * 512, -16):
            p = list(far)
            p[i] = BASE + shift
            assert prefill(*p, BASE) == ARG, (i, shift)
    # a column block of the queries' buffer that begins inside their rows
    assert prefill(BASE, *far[1:], BASE + 2 * 248, qs=512, os_=512) == ARG
