// The ends of moved ranges (csrc/pace_move_range.h) over random and extreme starts, counts and tables: what is read of a
// row of nodes lies in it, and every entry is moved once.  Built for the CPU with AddressSanitizer and
// UndefinedBehaviorSanitizer and run by tests/test_move_range.py; prints "OK <checks>" on success.
#include <climits>
#include <cstdio>
#include <random>
#include <vector>

#include "../../bit_recurrent_state_amd/csrc/pace_move_range.h"

using namespace pace;

static int fails = 0;
static long checks = 0;
#define EXPECT(c)                                        \
  do {                                                   \
    ++checks;                                            \
    if (!(c) && fails++ < 30) printf("FAIL line %d: %s\n", __LINE__, #c); \
  } while (0)

int main() {
  std::mt19937 rng(11);
  const std::vector<int> starts = {INT_MIN, INT_MIN + 1, -40, -17, -16, -1, 0, 1, 5, 15, 16, 37, 63, 64, 100, 1000, INT_MAX - 1, INT_MAX};
  const std::vector<int> counts = {INT_MIN, -3, -1, 0, 1, 2, 15, 16, 17, 40, 64, 65, 100, INT_MAX};
  const std::vector<int64_t> limits = {16, 32, 64, 112, 1008, (INT64_C(1) << 31) - 16};
  for (int T : {1, 2, 16, 17, 64, 65, 90})
    for (int start : starts)
      for (int count : counts)
        for (int64_t limit : limits)
          for (int step : {64, 512}) {
            std::vector<int> row(T), seen(T, 0);
            for (int& x : row) x = (int)(rng() % 1000);
            MoveRange r;
            const bool any = move_range(start, count, T, limit, r);
            const int n = count < 0 ? 0 : count < T ? count : T;
            int there = 0;
            for (int i = 0; i < n; ++i) there += (int64_t)start + i >= 0 && (int64_t)start + i < limit;
            EXPECT(any == (there > 0));
            if (!any) continue;
            // every step, and those behind the last whose nodes are asked for ahead
            const int64_t steps = (r.end - r.base + step - 1) / step;
            EXPECT(steps >= 1 && r.base >= 0 && r.base % 16 == 0 && r.first - r.base < 16);
            long sum = 0;
            for (int64_t pos = r.base; pos < r.base + (steps + 4) * step; ++pos) {
              const int64_t at = node_place(r, pos);
              EXPECT(at >= 0 && at < n);
              sum += row[(size_t)at];
              if (pos >= r.first && pos < r.end) {
                EXPECT(pos - start == at);
                ++seen[(size_t)at];
              }
            }
            for (int i = 0; i < T; ++i) EXPECT(seen[i] == (i < n && (int64_t)start + i >= 0 && (int64_t)start + i < limit ? 1 : 0));
            EXPECT(sum >= 0);
          }
  if (fails) {
    printf("%d of %ld failed\n", fails, checks);
    return 1;
  }
  printf("OK %ld\n", checks);
  return 0;
}
