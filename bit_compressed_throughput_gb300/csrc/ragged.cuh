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

constexpr unsigned int kErrExtent = 4u;    // bit of a device error word: an extent does not fit

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

}  // namespace fg
