// Whether two sets of equally spaced rows share a byte (host code without CUDA, so that its tests
// run anywhere).
#pragma once
#include <stdint.h>

namespace fg {

struct RowSet {
  uint64_t at;         // address of the first row
  int64_t rows;
  int64_t stride;      // bytes between rows, >= width
  int64_t width;       // bytes of a row
};
inline RowSet fp16_rows(const void* p, int64_t rows, int64_t stride, int64_t width) {
  return RowSet{reinterpret_cast<uint64_t>(p), rows, 2 * stride, 2 * width};
}

// Column blocks of one buffer, whose ranges overlap while their rows do not, are apart.  Row i of
// a, at offset x = at_a - at_b + i stride_a, shares a byte with row j of b when
// x - width_b < j stride_b < x + width_a.  For equal strides (or a single row) only j - i matters;
// else the rows of the smaller set inside the other's range are gone through.
inline bool rows_overlap(RowSet a, RowSet b) {
  using Wide = __int128;
  if (a.rows <= 0 || b.rows <= 0) return false;
  if (a.rows > b.rows) {
    const RowSet t = a;
    a = b;
    b = t;
  }
  if (a.rows == 1) a.stride = b.stride;    // arbitrary for one row
  const Wide d = (Wide)a.at - (Wide)b.at;  // of the first rows
  const Wide end_a = d + (Wide)(a.rows - 1) * a.stride + a.width;
  const Wide end_b = (Wide)(b.rows - 1) * b.stride + b.width;
  if (d >= end_b || end_a <= 0) return false;
  auto floor_div = [](Wide x, Wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };
  // the rows j of b, unbounded, that a row at offset x meets
  auto first = [&](Wide x) { return floor_div(x - b.width, b.stride) + 1; };
  auto last = [&](Wide x) { return floor_div(x + a.width - 1, b.stride); };
  if (a.stride == b.stride) {
    // j - i from first(d) to last(d); pairs of rows have differences 1 - rows_a .. rows_b - 1
    const Wide lo = first(d), hi = last(d);
    return lo <= hi && lo <= b.rows - 1 && hi >= 1 - a.rows;
  }
  Wide i0 = d < 0 ? floor_div(-d - a.width, a.stride) : 0, i1 = floor_div(end_b - d, a.stride);
  i0 = i0 < 0 ? 0 : i0;
  i1 = i1 > a.rows - 1 ? a.rows - 1 : i1;
  for (Wide i = i0; i <= i1; ++i) {
    const Wide x = d + i * a.stride;
    Wide lo = first(x), hi = last(x);
    lo = lo < 0 ? 0 : lo;
    hi = hi > b.rows - 1 ? b.rows - 1 : hi;
    if (lo <= hi) return true;
  }
  return false;
}

}  // namespace fg
