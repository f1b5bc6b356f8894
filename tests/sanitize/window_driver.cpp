// The index arithmetic of sliding windows (igc_ragged.h) on the host, under AddressSanitizer and UndefinedBehaviorSanitizer (built
// and run by tests/test_window_rows.py), walked as the attention kernels walk it: each tile's axis of keys holds every key
// that one of its queries sees exactly once and leads nowhere else, each row's places are the keys that the formula
// gives, and the queries of a key tile, near and far, are those that see it.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "igc_ragged.h"

using namespace igc;

static bool sees(const Window& w, int64_t i, int64_t j, int64_t lq, int64_t lk) {
  const int64_t p = i + lk - lq;
  if (w.right >= 0 && j > p + w.right) return false;
  return w.left < 0 || j >= p - w.left || j < w.sinks;
}

static int fail(const Window& w, int64_t lq, int64_t lk, int64_t at, const char* what) {
  std::fprintf(stderr, "window driver: %s (left %lld, right %lld, sinks %d, %lld queries, %lld keys, at %lld)\n", what,
               (long long)w.left, (long long)w.right, w.sinks, (long long)lq, (long long)lk, (long long)at);
  return 1;
}

// Tiles of bm queries over bn keys at a time, as many parts; key tiles of bm keys.
static int walk(const Window& w, int64_t lq, int64_t lk, int bm, int bn, int parts) {
  for (int64_t i0 = 0; i0 < lq; i0 += bm) {
    const int64_t i1 = (i0 + bm < lq ? i0 + bm : lq) - 1;
    const WindowAxis a = window_axis(w, i0, i1, lq, lk);
    if (a.keys < 0 || a.keys > lk || a.sinks < 0 || a.jump < 0) return fail(w, lq, lk, i0, "axis out of range");
    std::vector<int> met((size_t)lk, 0);
    for (int part = 0; part < parts; ++part) {
      int64_t x0, x1;
      split_axis(a.keys, parts, part, bn, x0, x1);
      if (x0 < 0 || x1 < x0 || x1 > a.keys) return fail(w, lq, lk, part, "part out of range");
      for (int64_t x = x0; x < x1; ++x) {
        const int64_t j = a.key(x);
        if (j < 0 || j >= lk || met[(size_t)j]++) return fail(w, lq, lk, x, "a place leads nowhere or to a key met before");
        for (int64_t i = i0; i <= i1; ++i) {
          const WindowRow r = window_tile(w, a, x0, i0, lq, lk).row((int32_t)(i - i0));
          const int32_t at = (int32_t)(x - x0);
          if ((at < r.first || (at >= r.low && at < r.high)) != sees(w, i, j, lq, lk))
            return fail(w, lq, lk, i, "a row's places are not its keys");
        }
      }
    }
    for (int64_t i = i0; i <= i1; ++i)
      for (int64_t j = 0; j < lk; ++j)
        if (sees(w, i, j, lq, lk) && !met[(size_t)j]) return fail(w, lq, lk, i, "a key is missed");
  }
  for (int64_t j0 = 0; j0 < lk; j0 += bm) {
    const int64_t j1 = (j0 + bm < lk ? j0 + bm : lk) - 1;
    int64_t from, to, none;
    window_queries(w, j0, lq, lk, true, from, none);
    window_queries(w, j1, lq, lk, true, none, to);
    if (to < from) to = from;
    const bool far = j0 < w.sinks;
    for (int64_t j = j0; j <= j1; ++j) {
      int64_t a, b;
      window_queries(w, j, lq, lk, false, a, b);
      if (a < 0 || b < a || b > lq) return fail(w, lq, lk, j, "queries of a key out of range");
      for (int64_t i = 0; i < lq; ++i) {
        const bool near_it = i >= from && i < to && i >= a && i < b, far_it = far && j < w.sinks && i >= to && i >= a && i < b;
        if ((near_it || far_it) != sees(w, i, j, lq, lk)) return fail(w, lq, lk, j, "a key's queries are not those that see it");
      }
    }
  }
  return 0;
}

int main() {
  int bad = 0;
  for (int64_t left : {-1, 0, 3, 40, 500, INT32_MAX})
    for (int64_t right : {-1, 0, 1, 50, INT32_MAX})
      for (int sinks : {0, 1, 5, 64, 90, INT32_MAX})
        for (int64_t lq : {0, 1, 2, 65, 90})
          for (int64_t lk : {0, 1, 64, 90, 150})
            if (!bad) bad += walk({left, right, left < 0 ? 0 : sinks}, lq, lk, 32, 16, 1 + (int)(lk % 3));
  uint32_t seed = 999;
  auto next = [&](uint32_t m) {
    seed = seed * 1664525u + 1013904223u;
    return (int64_t)((seed >> 8) % m);
  };
  for (int i = 0; i < 3000 && !bad; ++i) {
    Window w = {next(8) ? next(60) : -1, next(3) ? next(60) : next(2) - 1, (int32_t)next(40)};
    if (w.left < 0) w.sinks = 0;
    const int64_t lk = next(160), lq = next(3) ? lk : next(160);
    const int bm[] = {1, 2, 4, 32, 64}, bn[] = {8, 32, 64};
    bad += walk(w, lq, lk, bm[next(5)], bn[next(3)], 1 + (int)next(4));
  }
  // Rows and windows near 2^31: nothing overflows (the undefined behaviour sanitizer watches).
  const int64_t big = INT32_MAX - 1023;
  for (int64_t i : {(int64_t)0, big / 2, big - 1})
    for (int64_t left : {(int64_t)-1, (int64_t)0, (int64_t)INT32_MAX})
      for (int64_t right : {(int64_t)-1, (int64_t)0, (int64_t)INT32_MAX}) {
        const Window w = {left, right, left < 0 ? 0 : 7};
        const WindowAxis a = window_axis(w, i, i, big, big);
        const WindowRow r = window_tile(w, a, 0, i, big, big).row(0);
        int64_t from, to;
        window_queries(w, i, big, big, false, from, to);
        if (a.keys < 0 || a.keys > big || r.high < 0 || r.high <= r.low || from > i || to <= i) bad += fail(w, big, big, i, "far rows");
        // The row's own key is on the axis where the formula puts it.
        const int64_t x = i - a.jump;
        if (a.key(x) != i || !(x < r.first || (x >= r.low && x < r.high))) bad += fail(w, big, big, i, "the key of a far row");
      }
  if (bad) return 1;
  std::puts("window driver: ok");
  return 0;
}
