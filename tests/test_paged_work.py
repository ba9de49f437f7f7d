"""The order and the division of the work over the paged cache (CPU, from the kernels' own header):
every key tile that a row sees is worked on exactly once, and cut blocks find their pieces."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HOST_SRC = r"""
#include "paged_work.cuh"
using namespace fg;
// Shares 0 .. n-1 of the order over nseq sequences (q_off, lens), walked as the kernel walks them:
// a record per segment, {share, b, hk, q0, ntok, pos, j0, j1, slot, single, tiles, cut pieces, cut
// q0} and its key tiles behind it.  Returns the records; -1: `room` is too small.
extern "C" int h_walk(const int32_t* q_off, const int32_t* lens, int nseq, int H, int tpt, int window,
                      int sinks, int lead, int n_shares, int32_t* out,
                      int room) {
  const PagedShape sh{tpt, window, sinks, lead};
  auto seq = [&](int b) { return PagedSeq{q_off[b], q_off[b + 1] - q_off[b], lens[b]}; };
  int64_t total = 0;
  for (int b = 0; b < nseq; ++b) total += H * head_units(seq(b), sh);
  if (total == 0) return 0;
  // (so few shares that each holds the start of a key tile)
  if (n_shares > total / (2 + lead)) n_shares = total < 2 + lead ? 1 : (int)(total / (2 + lead));
  const Shares shares(total, n_shares);
  int used = 0, recs = 0;
  for (int w = 0; w < n_shares; ++w) {
    PagedWalk k;
    k.sh = sh; k.share = w; k.H = H; k.x0 = shares.first(w); k.x1 = shares.first(w + 1);
    if (k.x0 >= k.x1) continue;
    int64_t before = 0;
    int b = 0;
    for (;; ++b) {
      const int64_t u = H * head_units(seq(b), sh);
      if (before + u > k.x0) break;
      before += u;
    }
    k.start(seq(b), b, before);
    bool first = true;
    while (k.at < k.x1 && k.b < nseq) {
      const PagedBlock blk = paged_block(k.s, k.blk, sh);
      PagedSeg g;
      if (k.segment(g, blk)) {
        int32_t cut[2] = {0, 0};
        if (first && g.j0 > 0 && shares.share_of(k.at) == w - 1) {
          const int64_t last = k.at + blk.begin(blk.kt.count() - 1);
          cut[0] = shares.share_of(last) - w + 2;
          cut[1] = g.q0;
        }
        first = false;
        const int n = g.j1 - g.j0;
        if (used + 13 + n > room) return -1;
        const int32_t r[13] = {w, g.b, g.hk, g.q0, g.ntok, g.pos, g.j0, g.j1, g.slot, g.single,
                               blk.kt.count(), cut[0], cut[1]};
        for (int i = 0; i < 13; ++i) out[used++] = r[i];
        for (int j = g.j0; j < g.j1; ++j) out[used++] = g.kt.tile(j);
        ++recs;
      }
      k.at += blk.units();
      if (++k.blk >= paged_blocks(k.s, tpt)) {
        k.blk = 0;
        if (++k.hk == H) {
          k.hk = 0;
          do {
            if (++k.b >= nseq) break;
            k.s = seq(k.b);
            k.per_head = head_units(k.s, sh);
          } while (k.per_head == 0);
        }
      }
    }
  }
  return recs;
}
extern "C" int h_cut_slot(int w, int pieces, int i) { return cut_slot(w, pieces, i); }
extern "C" int h_span_sees(int tile, int lo, int hi, int window, int sinks) {
  return span_sees(tile, lo, hi, window, sinks);
}
extern "C" int h_weight_item(int q0, int nq, int n, int i, int tpt, int window, int sinks,
                             int32_t* out) {
  const WeightItem w = weight_item(PagedSeq{q0, nq, n}, i, PagedShape{tpt, window, sinks, 0});
  out[0] = w.k0;
  out[1] = w.t0;
  out[2] = w.t1;
  return weight_items(PagedSeq{q0, nq, n});
}
"""


@pytest.fixture(scope="module")
def dll(tmp_path_factory):
    d = tmp_path_factory.mktemp("work")
    src, so = d / "w.cpp", d / "w.so"
    src.write_text(HOST_SRC)
    inc = os.path.join(ROOT, "bit_compressed_throughput_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o",
                    str(so)], check=True)
    dll = C.CDLL(str(so))
    dll.h_walk.argtypes = [C.c_void_p, C.c_void_p] + [C.c_int] * 7 + [C.c_void_p, C.c_int]
    dll.h_weight_item.argtypes = [C.c_int] * 7 + [C.c_void_p]
    return dll


def seen(i, n, window, sinks):
    """The positions t < n that position i sees."""
    t = np.arange(n)
    return (t <= i) & ((window == 0) | (t > i - window) | (t < sinks))


CASES = [
    # lens, nq, H, tokens per tile, window, sinks
    ([1], [1], 1, 128, 0, 0),
    ([1000, 1, 0, 129, 4000], [1, 1, 0, 129, 300], 2, 32, 0, 0),
    ([5, 0, 130], [9, 3, 140], 3, 64, 0, 0),                 # more rows than positions
    ([3000, 700], [600, 700], 2, 16, 500, 4),
    ([3000, 700], [37, 1], 1, 1, 1, 0),
    ([260, 900, 2000], [260, 1, 55], 2, 18, 128, 300),
    ([0, 0], [0, 0], 2, 8, 0, 0),
]


@pytest.mark.parametrize("lens,nq,H,tpt,window,sinks", CASES)
@pytest.mark.parametrize("n_shares", [1, 2, 7, 152])
@pytest.mark.parametrize("lead", [0, 4, 7])
def test_every_key_tile_once(dll, lens, nq, H, tpt, window, sinks, n_shares, lead):
    off = np.concatenate([[3], 3 + np.cumsum(nq)]).astype(np.int32)
    ln = np.asarray(lens, np.int32)
    out = np.zeros(1 << 20, np.int32)
    recs = dll.h_walk(off.ctypes.data, ln.ctypes.data, len(lens), H, tpt, window, sinks, lead,
                      n_shares, out.ctypes.data, len(out))
    assert recs >= 0
    at, work, pieces, slots, cuts = 0, {}, {}, set(), {}
    for _ in range(recs):
        w, b, hk, q0, ntok, pos, j0, j1, slot, single, count, cut, cut_q0 = out[at:at + 13].tolist()
        tiles = out[at + 13:at + 13 + j1 - j0].tolist()
        at += 13 + j1 - j0
        assert 0 < ntok <= 2 * tpt and single == (ntok <= tpt)
        assert off[b] <= q0 and q0 + ntok <= off[b + 1] and pos == lens[b] - nq[b] + q0 - off[b]
        work.setdefault((b, hk, q0, ntok), []).extend(tiles)
        if slot >= 0:
            assert slot not in slots and slot // 2 == w
            slots.add(slot)
            pieces.setdefault((b, hk, q0), []).append((w, slot))
        else:
            assert (j0, j1) == (0, count)
        if cut:
            assert cut_q0 == q0 and (b, hk, q0) not in cuts
            cuts[b, hk, q0] = (w, cut)
    # every row of a sequence lies in one block, whose tiles are those that one of its rows sees
    rows = {}
    for (b, hk, q0, ntok), tiles in work.items():
        first = lens[b] - nq[b] + q0 - off[b]
        any_row = np.zeros(lens[b], bool)
        for i in range(max(first, 0), first + ntok):
            any_row |= seen(i, lens[b], window, sinks)
        assert sorted(tiles) == sorted(set(np.flatnonzero(any_row) // 128)), (b, hk, q0)
        for r in range(q0, q0 + ntok):
            rows[b, hk, r] = rows.get((b, hk, r), 0) + 1
    for b in range(len(lens)):
        for hk in range(H):
            for r in range(nq[b]):
                sees = lens[b] - nq[b] + r >= 0
                assert rows.get((b, hk, off[b] + r), 0) in ((1,) if sees else (0, 1))
    # the pieces of a cut block lie where the merge looks for them
    assert set(cuts) == set(pieces)
    for key, (w, n) in cuts.items():
        assert [s for _, s in pieces[key]] == [dll.h_cut_slot(w, n, i) for i in range(n)], key


def test_what_a_span_sees(dll):
    rng = np.random.default_rng(5)
    for _ in range(2000):
        window, sinks = int(rng.choice([0, 1, 5, 127, 128, 129, 600])), int(rng.integers(0, 400))
        lo = int(rng.integers(-20, 900))
        hi = lo + int(rng.integers(0, 200))
        got = [dll.h_span_sees(t, lo, hi, window, sinks) for t in range(9)]
        want = np.zeros(9 * 128, bool)
        for i in range(max(lo, 0), hi + 1):
            want |= seen(i, 9 * 128, window, sinks)
        assert all(g for g, w in zip(got, want.reshape(9, 128).any(1)) if w), (lo, hi, window, sinks)


def test_tokens_of_a_weight_item(dll):
    rng = np.random.default_rng(6)
    out = np.zeros(3, np.int32)
    for _ in range(500):
        window, sinks = int(rng.choice([0, 1, 5, 255, 256, 700])), int(rng.integers(0, 600))
        n = int(rng.integers(1, 1500))
        nq = int(rng.integers(1, n + 40))
        items = dll.h_weight_item(0, nq, n, 0, 8, window, sinks, out.ctypes.data)
        assert items == (n + 255) // 256
        sees = np.zeros((nq, n), bool)
        for r in range(nq):
            if n - nq + r >= 0:
                sees[r] = seen(n - nq + r, n, window, sinks)
        for i in range(items):
            dll.h_weight_item(0, nq, n, i, 8, window, sinks, out.ctypes.data)
            k0, t0, t1 = out.tolist()
            tok = np.flatnonzero(sees[:, k0:k0 + 256].any(1))
            assert k0 == 256 * i
            # the range holds every token that sees one of the positions
            assert len(tok) == 0 or (t0 <= tok[0] and tok[-1] < t1), (n, nq, window, sinks, i)
