// The index arithmetic of ragged sequences (igc_ragged.h) on the host, under AddressSanitizer and
// UndefinedBehaviorSanitizer (built and run by tests/test_host_sanitizers.py), walked as the attention kernels walk it:
// every slot of a launch finds its sequence and tile, and every row of that tile its query row. Whatever the
// offsets hold, all of them lie inside the sequence and the array. Ascending offsets, from any first row to any last,
// are covered row by row exactly once, and rows outside of them never.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "igc_ragged.h"

using namespace igc;

static int fail(const std::vector<int32_t>& off, int64_t n, int group, int bm, int64_t slot, const char* what) {
  std::fprintf(stderr, "ragged driver: %s (n %lld, group %d, tiles of %d, slot %lld, offsets", what, (long long)n, group,
               bm, (long long)slot);
  for (int32_t x : off) std::fprintf(stderr, " %d", x);
  std::fprintf(stderr, ")\n");
  return 1;
}

// One launch; the offsets may be empty (no offsets, one sequence).
static int walk(const std::vector<int32_t>& off, int64_t n, int group, int bm) {
  const int32_t* o = off.empty() ? nullptr : off.data();
  const int batch = off.empty() ? 1 : (int)off.size() - 1;
  bool ascending = true;
  for (size_t i = 1; i < off.size(); ++i) ascending = ascending && off[i - 1] <= off[i];
  std::vector<int> seen((size_t)(n * group), 0);
  const int64_t slots = n * group / bm + batch;
  for (int64_t slot = 0; slot < slots; ++slot) {
    int b = -1;
    const int64_t tile = find_tile(o, batch, n, group, bm, slot, b);
    if (b < 0 || b >= batch) return fail(off, n, group, bm, slot, "sequence out of range");
    int64_t begin, end;
    seq_rows(o, b, n, begin, end);
    if (begin < 0 || end < begin || end > n) return fail(off, n, group, bm, slot, "rows of the sequence out of range");
    const int64_t rows = (end - begin) * group;
    if (tile * bm >= rows) continue;
    if (tile < 0) return fail(off, n, group, bm, slot, "negative tile");
    for (int64_t r = tile * bm; r < rows && r < (tile + 1) * bm; ++r) {
      int64_t q;
      int g;
      split_row(r, group, q, g);
      if (q < 0 || begin + q >= end || g < 0 || g >= group) return fail(off, n, group, bm, slot, "row out of range");
      ++seen[(size_t)((begin + q) * group + g)];
    }
  }
  if (!ascending) return 0;
  const int64_t first = o ? clamp64(off.front(), 0, n) : 0, last = o ? clamp64(off.back(), 0, n) : n;
  for (int64_t r = 0; r < n * group; ++r)
    if (seen[(size_t)r] != (r >= first * group && r < last * group))
      return fail(off, n, group, bm, -1, "a row is missed, met twice or not of any sequence");
  return 0;
}

int main() {
  int bad = 0;
  const std::vector<std::vector<int32_t>> some = {
      {}, {0, 10}, {1, 2, 3}, {300, 400, 700}, {0, 0, 0, 700}, {700, 700}, {350, 350, 351, 351}, {0, 300},
      {5, 3, 1}, {700, 0}, {0, 500, 200, 700}, {-5, 100, 1 << 30}, {1 << 30, 1 << 30}, {-9, -3, -1}, {600, 100, 650, 20},
      {INT32_MIN, INT32_MAX}, {INT32_MAX, INT32_MIN, 3}};
  for (const auto& off : some)
    for (int64_t n : {0, 1, 3, 700})
      for (int group : {1, 2, 3, 5})
        for (int bm : {1, 2, 4, 128, 256}) bad += walk(off, n, group, bm);
  uint32_t seed = 12345;
  auto next = [&](uint32_t m) {
    seed = seed * 1664525u + 1013904223u;
    return (seed >> 8) % m;
  };
  for (int i = 0; i < 3000 && !bad; ++i) {
    const int64_t n = next(900);
    const int batch = 1 + (int)next(12);
    std::vector<int32_t> off((size_t)batch + 1);
    const bool up = next(4) != 0;
    int32_t at = (int32_t)next(200) - 20;
    for (auto& x : off) {
      x = up ? at : (int32_t)next(1200) - 100;
      at += (int32_t)(next(3) ? next(150) : 0);
    }
    const int bm[] = {1, 2, 4, 128, 256};
    bad += walk(off, n, 1 + (int)next(6), bm[next(5)]);
  }
  if (bad) return 1;
  std::puts("ragged driver: ok");
  return 0;
}
