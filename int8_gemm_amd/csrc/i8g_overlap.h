// i8g_overlap.h -- whether two matrices in memory share a byte (host code of
// the C ABI and of the binding; no HIP).
#pragma once
#include <stdint.h>

namespace i8g {

// rows x width bytes, `ld` >= width bytes from row to row (of one row: unused).
struct ByteRows {
  uintptr_t at;
  int64_t rows, width, ld;
  bool operator==(const ByteRows& o) const {
    return at == o.at && rows == o.rows && width == o.width && (ld == o.ld || rows <= 1);
  }
};

// Exact: the columns of one buffer's two halves lie between each other's rows
// and share nothing.  One division for equal leading dimensions, else one for
// each row of the matrix with fewer.
inline bool share_bytes(ByteRows a, ByteRows b) {
  if (a.rows <= 0 || a.width <= 0 || b.rows <= 0 || b.width <= 0) return false;
  if (a.rows > b.rows) {
    const ByteRows t = a;                                 // a has the fewer
    a = b;
    b = t;
  }
  const auto end = [](const ByteRows& m) { return m.at + (uintptr_t)(m.rows - 1) * (uintptr_t)m.ld + (uintptr_t)m.width; };
  if (end(a) <= b.at || end(b) <= a.at) return false;
  if (a.rows > 1 && a.ld == b.ld) {
    // row i of a and row i + k of b start d + k ld bytes from each other, k from 1 - a.rows to b.rows - 1
    const int64_t d = (int64_t)(b.at - a.at);
    const int64_t k = -(d / a.ld);                        // (rounded towards 0: it or a neighbour is nearest)
    for (int64_t j = k - 1; j <= k + 1; ++j)
      if (j >= 1 - a.rows && j <= b.rows - 1 && d + j * a.ld < a.width && d + j * a.ld > -b.width) return true;
    return false;
  }
  for (int64_t i = 0; i < a.rows; ++i) {
    const uintptr_t lo = a.at + (uintptr_t)(i * a.ld), hi = lo + (uintptr_t)a.width;
    if (hi <= b.at) continue;
    int64_t j = 0;                                        // the last row of b that starts before hi
    if (b.rows > 1) j = (int64_t)((hi - 1 - b.at) / (uintptr_t)b.ld);
    if (j > b.rows - 1) j = b.rows - 1;
    if (b.at + (uintptr_t)(j * b.ld + b.width) > lo) return true;
  }
  return false;
}

// An output that may be the input itself, or lie apart from it.
inline bool itself_or_apart(const ByteRows& out, const ByteRows& in) { return out == in || !share_bytes(out, in); }

}  // namespace i8g
