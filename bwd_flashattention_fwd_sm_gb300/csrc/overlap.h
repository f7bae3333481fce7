// Whether tensors of rows share memory: host code, for the refusals of the row operators' entries.
#pragma once

#include <stdint.h>

namespace gbattn {

// Rows of `width` bytes, `step` >= width bytes apart.
struct RowSpan {
  const void* at;
  int64_t rows, step, width;

  bool empty() const { return !at || rows <= 0 || width <= 0; }
  __int128 begin() const { return (__int128)reinterpret_cast<uintptr_t>(at); }
  __int128 end() const { return begin() + (__int128)(rows - 1) * step + width; }
  // Whether any row has a byte in [lo, hi).
  bool meets(__int128 lo, __int128 hi) const {
    if (lo >= end() || hi <= begin()) return false;
    if (lo < begin()) return true;
    const __int128 i = (lo - begin()) / step;  // the row that lo lies in, or in whose gap it lies
    return lo < begin() + i * step + width || (i + 1 < rows && hi > begin() + (i + 1) * step);
  }
};

inline bool same_rows(const RowSpan& a, const RowSpan& b) {
  return a.at == b.at && a.rows == b.rows && a.width == b.width && (a.rows == 1 || a.step == b.step);
}

// Whether two tensors share a byte.  Rows that lie between the other's rows do not.
inline bool rows_meet(RowSpan a, RowSpan b) {
  if (a.empty() || b.empty() || a.end() <= b.begin() || b.end() <= a.begin()) return false;
  if (a.begin() > b.begin()) {
    const RowSpan t = a;
    a = b;
    b = t;
  }
  // b's first row begins among a's; with one step for both every later row repeats it
  if (a.step == b.step || b.rows == 1) return a.meets(b.begin(), b.begin() + b.width);
  if (a.rows == 1) return b.meets(a.begin(), a.end());
  // only where spans meet that a program keeps apart: row by row of the shorter one, while it is within the other's span
  const RowSpan& few = a.rows < b.rows ? a : b;
  const RowSpan& many = a.rows < b.rows ? b : a;
  for (int64_t i = 0; i < few.rows; ++i) {
    const __int128 lo = few.begin() + (__int128)i * few.step;
    if (lo >= many.end()) break;
    if (many.meets(lo, lo + few.width)) return true;
  }
  return false;
}

}  // namespace gbattn
