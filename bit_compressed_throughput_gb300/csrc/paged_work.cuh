// The work order of the attention over the paged cache (sm_103a; host and device, the host's use
// is its tests).
//
// The query rows of a K/V head are its tokens' G query heads, token by token; a row tile holds tpt =
// 128 / G whole tokens, a block two row tiles (a sequence's last one, or its only one, may hold one:
// a single block).  A block works on the 128-position key tiles that one of its tokens sees.  All
// blocks stand in one order: sequences, K/V heads, blocks, key tiles.  A key tile of a block counts
// one unit, of a block of two row tiles two, and the first one `lead` more, for what a block costs
// beside its tiles; the units are cut evenly into shares, and a share owns the key tiles that begin
// in it.  So every CTA has the same work whatever the lengths, and a block
// that a cut divides is put together afterwards from its pieces, one per share.
#pragma once
#include <stdint.h>

#include "ragged.cuh"

namespace fg {

struct PagedSeq {
  int q0, nq, n;       // first query row, query rows, cached positions
};
struct PagedShape {
  int tpt, window, sinks, lead;
};

// The key tiles that tokens at positions pos .. pos + ntok - 1 see (pos may be negative).
FG_HD KeyTiles span_tiles(int pos, int ntok, int window, int sinks) {
  KeyTiles k{0, 0, 0};
  const int hi = pos + ntok - 1, lo = pos > 0 ? pos : 0;
  if (ntok <= 0 || hi < 0) return k;
  k.te = hi / kKeyTile + 1;
  k.tw = (window == 0 || lo < window) ? 0 : (lo - window + 1) / kKeyTile;
  const int seen = sinks <= hi ? sinks : hi + 1;
  k.ns = seen > 0 ? (seen - 1) / kKeyTile + 1 : 0;
  if (k.ns >= k.tw) k.ns = k.tw = 0;
  return k;
}
// Whether tokens at positions lo .. hi see a position of key tile `tile`.
FG_HD bool span_sees(int tile, int lo, int hi, int window, int sinks) {
  const int k0 = tile * kKeyTile;
  return hi >= lo && k0 <= hi &&
         (window == 0 || (int64_t)k0 + kKeyTile - 1 > (int64_t)lo - window || k0 < sinks);
}

struct PagedBlock {
  int t0, ntok, pos;   // first token of the sequence, tokens, the first one's position
  int cost, lead;      // units per key tile, and the first one's more
  KeyTiles kt;
  FG_HD int64_t begin(int64_t j) const { return j > 0 ? lead + cost * j : 0; }  // of tile number j
  FG_HD int64_t units() const { return kt.count() > 0 ? begin(kt.count()) : 0; }
};
FG_HD int paged_blocks(const PagedSeq& s, int tpt) {
  return (int)(((int64_t)s.nq + 2 * tpt - 1) / (2 * tpt));
}
FG_HD PagedBlock paged_block(const PagedSeq& s, int blk, const PagedShape& sh) {
  PagedBlock b;
  b.t0 = blk * 2 * sh.tpt;
  b.ntok = s.nq - b.t0 < 2 * sh.tpt ? s.nq - b.t0 : 2 * sh.tpt;
  b.pos = s.n - s.nq + b.t0;
  b.cost = b.ntok > sh.tpt ? 2 : 1;
  b.lead = sh.lead;
  b.kt = span_tiles(b.pos, b.ntok, sh.window, sh.sinks);
  return b;
}
// Units of one K/V head of a sequence.
FG_HD int64_t head_units(const PagedSeq& s, const PagedShape& sh) {
  int64_t u = 0;
  for (int i = paged_blocks(s, sh.tpt) - 1; i >= 0; --i) u += paged_block(s, i, sh).units();
  return u;
}

// A share's part of a block: key tiles number j0 .. j1 - 1 of its list.
struct PagedSeg {
  int b, hk;           // sequence (-1: no more segments) and K/V head
  int q0, ntok, pos;   // the block's first row in q, tokens, the first one's position
  int n;               // cached positions
  int single;          // one row tile
  KeyTiles kt;
  int j0, j1;
  int slot;            // partial slot; -1: the whole block is here
};
// What is to be put together at a share: the block that its first segment ends, when the share
// before holds (at its end) the block's first key tile.
struct PagedCut {
  int pieces;          // 0: nothing
  int q0, ntok, hk;
};
// Partial slots: 2 share + 1 for a segment whose block goes on in the next share, 2 share for one
// that ends a block.  Piece i of a cut at share w:
FG_HD int cut_slot(int w, int pieces, int i) {
  return 2 * (w - 1 + i) + (i + 1 < pieces ? 1 : 0);
}

// ---- Q buffers.  Chain 0 multiplies buffer 0, chain 1 buffer 1, or 0 too where a block has one row
// tile; both wait for buffer 0 in every segment.  A buffer's use ends with two arrivals at its
// barrier.  Where a block has two row tiles one of buffer 0's is chain 1's, behind its wait: else the
// next segment's rows could come while chain 1 has not passed that wait, which a parity cannot tell
// from the phase before.  Arrivals at buffer 0's barrier behind the wait; at the barrier of the buffer
// that the chain multiplies, after its last product:
FG_HD int q_given_at_once(int chain, bool single) { return chain == 1 && !single ? 1 : 0; }
FG_HD int q_given_after_use(int chain, bool single) { return chain == 1 && !single ? 2 : 1; }

// Walks the segments of share [x0, x1) of the order.
struct PagedWalk {
  PagedShape sh;
  int share, H;
  int64_t x0, x1;
  int64_t at;          // unit at which the current block begins
  int64_t per_head;    // units of one head of the current sequence
  PagedSeq s;
  int b, hk, blk;

  // At the first block of sequence b, which begins at unit `before` and holds unit x0.
  FG_HD void start(const PagedSeq& seq, int b_, int64_t before) {
    s = seq;
    b = b_;
    per_head = head_units(s, sh);
    hk = (int)((x0 - before) / per_head);
    at = before + hk * per_head;
    blk = 0;
  }
  FG_HD static int64_t tiles_before(int64_t x, const PagedBlock& k) {    // that begin before unit x
    if (x <= 0) return 0;                                                // of the block
    return x <= k.lead + k.cost ? 1 : (x - k.lead + k.cost - 1) / k.cost;
  }
  // The current block's segment (false: none in this share), without moving on.
  FG_HD bool segment(PagedSeg& g, const PagedBlock& k) const {
    const int64_t nt = k.kt.count(), j0 = tiles_before(x0 - at, k), j1 = tiles_before(x1 - at, k);
    g.j0 = (int)(j0 < nt ? j0 : nt);
    g.j1 = (int)(j1 < nt ? j1 : nt);
    if (g.j0 >= g.j1) return false;
    g.b = b;
    g.hk = hk;
    g.q0 = s.q0 + k.t0;
    g.ntok = k.ntok;
    g.pos = k.pos;
    g.n = s.n;
    g.single = k.cost == 1;
    g.kt = k.kt;
    g.slot = g.j1 < nt ? 2 * share + 1 : (g.j0 > 0 ? 2 * share : -1);
    return true;
  }
};

// ---- the weights that positions receive: items of 256 positions of one K/V head (two key tiles), for
// each the row tiles that see one of them.  An item costs as many units as tokens see it, and its
// restoring as many as two row tiles hold; a share owns the items that begin in it, so its sums have
// one owner each.
constexpr int kItemKeys = 2 * kKeyTile;
struct WeightItem {
  int k0;              // first position
  int t0, t1;          // the tokens that see one of its positions
};
FG_HD int weight_items(const PagedSeq& s) {
  return (int)(((int64_t)s.n + kItemKeys - 1) / kItemKeys);
}
FG_HD WeightItem weight_item(const PagedSeq& s, int i, const PagedShape& sh) {
  WeightItem w;
  w.k0 = i * kItemKeys;
  const int first = s.n - s.nq;                        // position of the first token
  const int last = (s.n - w.k0 < kItemKeys ? s.n : w.k0 + kItemKeys) - 1;
  w.t0 = w.k0 > first ? w.k0 - first : 0;              // the first token that sees position k0
  w.t1 = s.nq;                                         // behind the last that sees one
  if (sh.window != 0 && w.k0 >= sh.sinks && (int64_t)last + sh.window - first < w.t1)
    w.t1 = last + sh.window - first;
  if (w.t1 < w.t0) w.t1 = w.t0;
  return w;
}
FG_HD int64_t weight_cost(const WeightItem& w, const PagedShape& sh) {
  return 2 * sh.tpt + w.t1 - w.t0;
}
FG_HD int64_t weight_units(const PagedSeq& s, const PagedShape& sh) {   // of one K/V head
  int64_t u = 0;
  for (int i = weight_items(s) - 1; i >= 0; --i) u += weight_cost(weight_item(s, i, sh), sh);
  return u;
}

}  // namespace fg
