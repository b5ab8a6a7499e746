// Host-side check of the row operators' rules (plain C++, no CUDA): where strided row tensors lie, against every
// byte's owner, and how many blocks share a row.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <set>

#include "da_rows.h"

static int fails = 0;
#define CHECK(c) do { if (!(c)) { std::printf("FAIL line %d: %s\n", __LINE__, #c); ++fails; } } while (0)

using da::RowRuns;

static std::multiset<int64_t> bytes_of(const RowRuns& t) {
  std::multiset<int64_t> s;
  for (int64_t r = 0; r < t.rows; ++r)
    for (int64_t h = 0; h < t.heads; ++h)
      for (int64_t i = 0; i < t.run; ++i) s.insert((int64_t)t.address + r * t.row + h * t.head + i);
  return s;
}

int main() {
  unsigned seed = 1;
  auto pick = [&](int n) { seed = seed * 1664525u + 1013904223u; return (int)((seed >> 8) % (unsigned)n); };
  int shared = 0, apart = 0, unsure = 0;
  for (int n = 0; n < 60000; ++n) {
    RowRuns a, b;
    for (RowRuns* t : {&a, &b}) {
      t->address = 10000 + pick(40);
      t->rows = 1 + pick(4);
      t->heads = 1 + pick(3);
      t->run = 4;
      t->head = pick(3) ? 4 * (1 + pick(4)) : pick(19) - 6;
      t->row = pick(3) ? 4 * (1 + pick(12)) : pick(60) - 20;
    }
    b.run = a.run;
    if (pick(2)) b.row = a.row, b.head = a.head;
    const auto x = bytes_of(a), y = bytes_of(b);
    bool meet = false;
    for (int64_t i : x) meet |= y.count(i) > 0;
    const bool says = da::may_share(a, b);
    CHECK(says == da::may_share(b, a));
    if (meet) CHECK(says);                 // never taken for apart
    shared += meet;
    apart += !says;
    unsure += says && !meet;
    // rows on one another
    bool once = true;
    for (int64_t i : x) once &= x.count(i) == 1;
    if (da::lie_apart(a)) CHECK(once);
  }
  CHECK(shared > 10000 && apart > 10000);
  // parts of one tensor's rows (q, k and v of a projection), of its heads, and every other head
  auto part = [](uint64_t at, int64_t rows, int64_t row, int64_t heads, int64_t head) {
    return RowRuns{1u << 20, rows, row, heads, head, 256};
  };
  RowRuns q = part(0, 1000, 48 * 256, 32, 256), k = q, even = part(0, 50, 8 * 256, 4, 512), odd = even;
  k.address += 32 * 256;
  k.heads = 8;
  odd.address += 256;
  CHECK(!da::may_share(q, k) && !da::may_share(even, odd));
  k.address -= 1;
  CHECK(da::may_share(q, k));
  RowRuns first = part(0, 50, 256, 4, 100 * 256), second = first;   // [heads, rows, d]
  second.address += 50 * 256;
  CHECK(!da::may_share(first, second) && da::lie_apart(first));
  second.address -= 256;
  CHECK(da::may_share(first, second));
  // an input one row on: out = x[1:]
  RowRuns x = part(0, 64, 8 * 256, 8, 256), shifted = x;
  shifted.address += 8 * 256;
  CHECK(da::may_share(x, shifted) && !da::result_ok(x, shifted) && da::result_ok(x, x));
  RowRuns other = x;
  other.row *= 2;
  CHECK(!da::result_ok(x, other));
  // one row read for all
  RowRuns all = part(0, 64, 0, 8, 256);
  CHECK(da::may_share(all, x) && !da::lie_apart(all));
  // strides whose products pass 64 bits
  RowRuns huge = part(0, 2147483647, 1ll << 62, 1 << 20, 1ll << 45);
  CHECK(!da::lie_apart(huge));
  huge.head = 256;
  CHECK(da::lie_apart(huge));
  huge.row = -(1ll << 62);
  CHECK(!da::lie_apart(huge));
  RowRuns low = part(0, 2, 256, 1, 256);
  low.address = 4096;
  CHECK(!da::may_share(low, part(0, 2, INT64_MAX, 1 << 20, INT64_MAX)));
  // blocks a row: enough for two an SM, by the SMs at hand, and a pass of heads each
  for (int sms : {1, 2, 40, 132, 152, 160})
    for (int64_t rows : {1, 2, 3, 5, 64, 79, 80, 263, 264, 303, 304, 305, 5000, 2147483647})
      for (int passes : {1, 2, 5, 64, 1000}) {
        const int n = da::row_slices(rows, passes, sms);
        int want = 1;
        while (want < passes && rows * want < 2 * sms) ++want;
        CHECK(n == want);
      }
  if (fails == 0) std::printf("ok\n");
  return fails ? 1 : 0;
}
