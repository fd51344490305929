// norm_rows_main.hip -- walks on the host over the rows that the norm's backward kernels share
// out among slots (test only): every row belongs to one slot, and where slots have whole
// groups each gate row's gradient is written by exactly one of them.
#include <stdio.h>

#include <vector>

#include "norm_rows.hpp"

using namespace nvfp4;

static bool check(int64_t rows, int64_t groups, int streams, int64_t workgroups) {
  const Split s = split_rows(rows, groups, streams, workgroups);
  const int64_t per = rows / groups;
  std::vector<int> rows_seen(rows, 0), gates_written(groups, 0);
  bool good = s.sums * streams >= s.slots;
  for (int64_t slot = 0; slot < s.sums * streams; ++slot) {   // (the last ones may have no rows)
    int64_t row, end;
    slot_rows(s, slot, row, end);
    const int64_t last = (end < rows ? end : rows) - 1 > 0 ? (end < rows ? end : rows) - 1 : 0;
    const int64_t group = (row < last ? row : last) / per;
    for (int64_t r = row; r < end; ++r) ++rows_seen[r];
    if (s.parts) good &= row >= end || row / per == (end - 1) / per;   // (a slot stays in one group)
    if (one_group(s)) {   // closes its group after its rows, also if it has none
      ++gates_written[group];
    } else {   // a group is closed at its last row
      for (int64_t r = row; r < end; ++r) gates_written[r / per] += (r + 1) % per == 0 || r + 1 == end;
    }
  }
  for (int n : rows_seen) good &= n == 1;
  if (s.parts == 0)
    for (int n : gates_written) good &= n == 1;
  if (!good) printf("rows %lld groups %lld streams %d workgroups %lld\n", (long long)rows, (long long)groups, streams, (long long)workgroups);
  return good;
}

int main() {
  int64_t wrong = 0, cases = 0;
  for (int64_t rows = 1; rows <= 2100; rows += rows < 80 ? 1 : 101)
    for (int64_t groups = 1; groups <= rows; ++groups) {
      if (rows % groups) continue;
      for (int streams : {1, 2, 4, 8})
        for (int64_t workgroups : {1, 3, 128, 256}) {
          ++cases;
          wrong += !check(rows, groups, streams, workgroups);
        }
    }
  printf("%lld of %lld splits wrong\n", (long long)wrong, (long long)cases);
  return wrong != 0;
}
