// The index arithmetic of the 4-bit cache's kernels, run on the host.
#include <cstdio>
#include <vector>

#include "kv4.h"

using namespace gbattn;

static int failures = 0;
#define EXPECT(c)                                             \
  do {                                                        \
    if (!(c)) {                                               \
      std::printf("failed at line %d: %s\n", __LINE__, #c);   \
      ++failures;                                             \
    }                                                         \
  } while (0)

int main() {
  Kv4Args a = {};
  std::vector<int> table = {3, 0, -1, 5, 4, 2}, lens = {40, -2, 1000}, cu = {0, 2, 7, 6};
  a.table = table.data();
  a.table_stride = 2;
  a.lens = lens.data();
  a.batch = 3;
  a.heads_kv = 2;
  a.seqlen = 5;
  a.page = 16;
  a.n_pages = 5;
  a.max_pages = 2;
  bool bad = false;
  // rows of pages that exist
  EXPECT(kv4_row_index(a, 0, 1, 17, &bad) == (0 * 2 + 1) * 16 + 1 && !bad);
  EXPECT(kv4_row_index(a, 0, 0, 15, &bad) == (3 * 2 + 0) * 16 + 15 && !bad);
  // a negative page, and one past the cache's last
  EXPECT(kv4_row_index(a, 1, 0, 3, &bad) == -1 && bad);
  bad = false;
  EXPECT(kv4_row_index(a, 1, 0, 16, &bad) == -1 && bad);
  bad = false;
  // lengths: above what the page list can hold (32), below 0
  EXPECT(kv4_seq_of(a, 0, &bad).len == 32 && bad);
  bad = false;
  EXPECT(kv4_seq_of(a, 1, &bad).len == 0 && bad);
  bad = false;
  lens[2] = 32;
  EXPECT(kv4_seq_of(a, 2, &bad).len == 32 && !bad);
  // packed rows: a sequence of 2, one of 5, one whose end lies before its start
  a.cu = cu.data();
  a.total = 7;
  lens[0] = lens[1] = 3;
  EXPECT(kv4_seq_of(a, 0, &bad).n == 2 && !bad);
  EXPECT(kv4_seq_of(a, 1, &bad).n == 5 && kv4_seq_of(a, 1, &bad).row0 == 2 && !bad);
  EXPECT(kv4_seq_of(a, 2, &bad).n == 0 && bad);
  bad = false;
  a.total = 6;  // the second sequence ends behind the tensor
  EXPECT(kv4_seq_of(a, 1, &bad).n == 0 && bad);
  bad = false;
  a.total = 7;
  a.seqlen = 4;  // or has more rows than the call says
  EXPECT(kv4_seq_of(a, 1, &bad).n == 0 && bad);
  bad = false;
  // a large cache: 64-bit rows
  a.n_pages = 1 << 20;
  a.heads_kv = 64;
  a.page = 1 << 10;
  table[0] = (1 << 20) - 1;
  EXPECT(kv4_row_index(a, 0, 63, 1023, &bad) == (1ll << 36) - 1 && !bad);
  // a page list that holds more than 2^31 - 1 positions
  a.max_pages = 1 << 30;
  lens[0] = 0x7FFFFFFF;
  a.cu = nullptr;
  EXPECT(kv4_seq_of(a, 0, &bad).len == 0x7FFFFFFF && !bad);
  if (!failures) std::printf("ok\n");
  return failures != 0;
}
