// Sequences of different lengths and what a query sees of them (sm_103a): shared by the ragged
// K/V-cache operators and the windowed attention.
//
// Extents come from device arrays that the host never reads, so the kernels check them: a
// sequence whose extent does not fit its buffers takes no part, and a bit of the translation
// unit's error word tells (read by fg_check_device_error).
#pragma once
#include <stdint.h>

// The index arithmetic also compiles for the host, where its tests run.
#ifdef __CUDACC__
#define FG_HD __host__ __device__ __forceinline__
#else
#define FG_HD inline
#endif

namespace fg {

constexpr unsigned int kErrExtent = 1u << 16;    // bit of a device error word: an extent does not
                                                 // fit (the low bits: a bounded wait ran out)

// The sequence holding row r: the last b of 0 .. n-1 with off[b] <= r, or -1 when r lies before
// the first or behind the last sequence.  For offsets that do not grow the answer may not hold
// r; callers test off[b] <= r < off[b + 1].
FG_HD int sequence_of_row(const int32_t* off, int n, int r) {
  if (r < off[0] || r >= off[n]) return -1;
  int lo = 0, hi = n;                      // off[lo] <= r, and r < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// Offsets 0 <= off[b] <= off[b + 1] <= rows for b = i, i + step, ...
FG_HD bool offsets_ok(const int32_t* off, int n, int rows, int i, int step) {
  bool ok = true;
  for (int b = i; b < n; b += step) {
    const int lo = off[b], hi = off[b + 1];
    ok = ok && lo >= 0 && lo <= hi && hi <= rows;
  }
  return ok;
}

// The keys that query position i sees: t <= i inside the window (0: no window) or among the
// first `sinks` positions.
FG_HD bool visible(int t, int i, int window, int sinks) {
  return t <= i && (window == 0 || t > i - window || t < sinks);
}

// ---- decode: the 16-position tiles of a sequence that its newest position sees
//
// Tiles 0 .. ns-1 hold the first positions, tiles tw .. te-1 the window; where they touch or
// overlap ns is 0 and tw is 0 (one run of tiles).  Each of the nt tiles holds a visible position.
constexpr int kTilePos = 16;
struct SeqTiles {
  int len, wstart;     // length; first position of the window
  int nt, ns, tw;      // tiles; of them first-position tiles; first tile of the window
};
FG_HD SeqTiles seq_tiles(int len, int window, int sinks) {
  SeqTiles s;
  s.len = len;
  s.wstart = (window == 0 || window >= len) ? 0 : len - window;
  const int te = (int)(((int64_t)len + kTilePos - 1) / kTilePos);
  const int seen = sinks < len ? sinks : len;
  s.ns = (int)(((int64_t)seen + kTilePos - 1) / kTilePos);
  s.tw = s.wstart / kTilePos;
  if (s.ns >= s.tw) s.ns = s.tw = 0;
  s.nt = s.ns + te - s.tw;
  return s;
}
// Position of the first row of tile u (0 <= u < nt), and the tiles from there to u1 that are one
// run of positions (either the first positions' or the window's).
FG_HD int tile_pos(const SeqTiles& s, int u) {
  return (u < s.ns ? u : u - s.ns + s.tw) * kTilePos;
}
FG_HD int run_tiles(const SeqTiles& s, int u, int u1) {
  return ((u < s.ns && s.ns < u1) ? s.ns : u1) - u;
}

// ---- prefill: the 128-key tiles that a tile of 128 query rows sees
//
// Key tiles 0 .. ns-1 hold first positions, tw .. te-1 the rows' windows (ns and tw 0 where the two
// touch).  Row r of a sequence with nq query rows and nk keys is position nk - nq + r.
constexpr int kKeyTile = 128, kQueryTile = 128;
struct KeyTiles {
  int ns, tw, te;
  FG_HD int count() const { return ns + te - tw; }
  FG_HD bool has(int tile) const { return tile < ns || (tile >= tw && tile < te); }
  FG_HD int tile(int j) const { return j < ns ? j : j - ns + tw; }
};
FG_HD KeyTiles key_tiles(int r0, int nq, int nk, int window, int sinks) {
  KeyTiles k{0, 0, 0};
  const int last = r0 < nq - kQueryTile ? r0 + kQueryTile - 1 : nq - 1;
  const int hi = nk - nq + last;           // the last row's position
  if (r0 >= nq || hi < 0) return k;
  const int lo = nk - nq + r0 > 0 ? nk - nq + r0 : 0;     // the first row's that has one
  k.te = hi / kKeyTile + 1;
  k.tw = (window == 0 || lo < window) ? 0 : (lo - window + 1) / kKeyTile;
  const int seen = sinks <= hi ? sinks : hi + 1;
  k.ns = seen > 0 ? (seen - 1) / kKeyTile + 1 : 0;
  if (k.ns >= k.tw) k.ns = k.tw = 0;
  return k;
}
// The tiles that either of two neighbouring query tiles sees.
FG_HD KeyTiles either(const KeyTiles& a, const KeyTiles& b) {
  if (a.count() == 0) return b;
  if (b.count() == 0) return a;
  KeyTiles k;
  k.te = a.te > b.te ? a.te : b.te;
  k.tw = a.tw < b.tw ? a.tw : b.tw;
  k.ns = a.ns > b.ns ? a.ns : b.ns;
  if (k.ns >= k.tw) k.ns = k.tw = 0;
  return k;
}
// The 16-key steps s0 .. s1-1 of key tile `tile` that hold what rows at positions lo .. hi (lo may
// be negative) see of it; not empty for a tile that the query tile has.
struct KeySteps {
  int s0, s1;
};
FG_HD KeySteps key_steps(int tile, int lo, int hi, int window, int sinks) {
  const int k0 = tile * kKeyTile;
  const int w0 = (window == 0 || lo < window) ? 0 : lo - window + 1;     // the windows' first key
  const int first = k0 < sinks || w0 <= k0 ? 0 : w0 - k0;
  int end = hi - k0 < kKeyTile ? hi - k0 + 1 : kKeyTile;
  if (w0 >= k0 + kKeyTile && sinks - k0 < end) end = sinks - k0;         // first positions only
  return KeySteps{first / 16, (end + 15) / 16};
}
// Bits e of 32 columns (keys c0 + e of the sequence) that position i sees, i < nk.
FG_HD uint32_t bits_below(int n) { return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u); }
FG_HD uint32_t visible_bits(int c0, int i, int window, int sinks) {
  const uint32_t past = bits_below(i - c0 < 32 ? i - c0 + 1 : 32);
  const int w0 = (window == 0 || i < window) ? 0 : i - window + 1;    // the window's first key
  return past & (~bits_below(w0 - c0) | bits_below(sinks > c0 ? sinks - c0 : 0));
}

// `total` tiles in one order, cut evenly into n shares (n < 2^16): share i is tiles first(i) ..
// first(i + 1) - 1; share_of is the inverse.
struct Shares {
  int64_t each;        // tiles per share, rounded down
  uint32_t more;       // the tiles left over, per share, times 2^32, rounded up
  int n;               // shares
  FG_HD Shares(int64_t total, int shares) : n(shares) {
    uint32_t rest;
    if (total < (1ll << 32)) {             // a 32-bit division takes a fraction of the time
      each = (uint32_t)total / (uint32_t)n;
      rest = (uint32_t)total - (uint32_t)each * (uint32_t)n;
    } else {
      each = total / n;
      rest = (uint32_t)(total - each * n);
    }
    // (rest 2^32 + n - 1) / n in two digits of 16 bits, as n < 2^16
    const uint32_t hi = (rest << 16) / (uint32_t)n, left = (rest << 16) - hi * (uint32_t)n;
    more = (hi << 16) + ((left << 16) + (uint32_t)n - 1) / (uint32_t)n;
  }
  // (first(n) = total: n more lies within n of rest 2^32)
  FG_HD int64_t first(int i) const {
    return each * i + (int64_t)(((uint64_t)more * (uint32_t)i) >> 32);
  }
  FG_HD int share_of(int64_t x) const {
    // a guess in binary32, then the definition
    int i = (int)((float)x / ((float)each + (float)more * 0x1p-32f));
    i = i < 0 ? 0 : (i >= n ? n - 1 : i);
    while (i > 0 && first(i) > x) --i;
    while (i + 1 < n && first(i + 1) <= x) ++i;
    return i;
  }
};

}  // namespace fg
