// rows_meet and same_rows against a count of every byte.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "overlap.h"

using namespace gbattn;

static bool by_bytes(const RowSpan& a, const RowSpan& b) {
  if (!a.at || !b.at) return false;
  std::set<uintptr_t> of_a;
  for (int64_t r = 0; r < a.rows; ++r)
    for (int64_t c = 0; c < a.width; ++c) of_a.insert(reinterpret_cast<uintptr_t>(a.at) + r * a.step + c);
  for (int64_t r = 0; r < b.rows; ++r)
    for (int64_t c = 0; c < b.width; ++c)
      if (of_a.count(reinterpret_cast<uintptr_t>(b.at) + r * b.step + c)) return true;
  return false;
}

int main() {
  std::srand(1);
  int meeting = 0, apart = 0;
  for (int n = 0; n < 300000; ++n) {
    RowSpan s[2];
    const int64_t step = 1 + std::rand() % 12;
    for (RowSpan& x : s) {
      x.step = std::rand() % 3 ? step : 1 + std::rand() % 12;
      x.width = std::rand() % 20 ? 1 + std::rand() % x.step : 0;
      x.rows = std::rand() % 20 ? 1 + std::rand() % 6 : 0;
      x.at = std::rand() % 50 ? reinterpret_cast<const void*>((uintptr_t)(100 + std::rand() % 60)) : nullptr;
    }
    const bool want = by_bytes(s[0], s[1]);
    (want ? meeting : apart)++;
    if (rows_meet(s[0], s[1]) != want || rows_meet(s[1], s[0]) != want) {
      std::printf("%p %ld %ld %ld, %p %ld %ld %ld: %d\n", s[0].at, (long)s[0].rows, (long)s[0].step, (long)s[0].width,
                  s[1].at, (long)s[1].rows, (long)s[1].step, (long)s[1].width, want);
      return 1;
    }
  }
  if (meeting < 50000 || apart < 50000) return std::printf("%d meet, %d do not\n", meeting, apart), 1;
  // the largest tensors: no product passes its type, and what does not meet is found at once
  const RowSpan all{reinterpret_cast<const void*>((uintptr_t)4096), INT64_MAX, INT64_MAX, 1 << 20};
  const RowSpan last{reinterpret_cast<const void*>(~(uintptr_t)0), 1, 1, 1};
  if (!rows_meet(all, all) || !same_rows(all, all) || rows_meet(all, last)) return std::printf("large\n"), 1;
  const RowSpan one{all.at, 1, 7, 64}, other{all.at, 1, 9, 64}, two{all.at, 2, 64, 64};
  if (!same_rows(one, other) || same_rows(one, two)) return std::printf("same\n"), 1;
  std::printf("ok\n");
  return 0;
}
