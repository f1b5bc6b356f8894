// Rows and tiles of ragged sequences, from their row offsets: index arithmetic alone, so that host code runs it too.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace igc {

__host__ __device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) {
  return x < lo ? lo : x > hi ? hi : x;
}

// Rows [begin, end) of sequence b; whatever the offsets hold, within [0, n].
__host__ __device__ __forceinline__ void seq_rows(const int32_t* off, int b, int64_t n, int64_t& begin, int64_t& end) {
  if (!off) {
    begin = 0, end = n;
    return;
  }
  begin = clamp64(off[b], 0, n);
  end = clamp64(off[b + 1], begin, n);
}

// Rows [begin, end) that the sequences cover together (ascending offsets); the rest is left unwritten.
__host__ __device__ __forceinline__ void covered_rows(const int32_t* off, int batch, int64_t n, int64_t& begin,
                                                      int64_t& end) {
  begin = off ? clamp64(off[0], 0, n) : 0;
  end = off ? clamp64(off[batch], begin, n) : n;
}

// Tiles of `bm` rows over ragged sequences without a plan: sequence b of rows [begin, end) (times mul)
// owns the slots from (begin - first) * mul / bm + b on, with `first` the first sequence's first row, which are at
// least as many as its tiles, so that n * mul / bm + batch slots cover everything and a slot finds its sequence by a
// binary search. Returns the tile in sequence b. It may lie past the sequence's end, but is never negative, whatever the
// offsets hold: sequence 0 starts at slot 0, and a later one is taken only if it starts at or before `slot`.
__host__ __device__ __forceinline__ int64_t find_tile(const int32_t* off, int batch, int64_t n, int mul, int bm,
                                                      int64_t slot, int& b) {
  b = 0;
  if (!off) return slot;
  const int64_t first = clamp64(off[0], 0, n);
  int hi = batch;  // slots of hi and beyond start after `slot`
  while (hi - b > 1) {
    const int mid = (b + hi) >> 1;
    if ((clamp64(off[mid], 0, n) - first) * mul / bm + mid <= slot) b = mid;
    else hi = mid;
  }
  return slot - ((clamp64(off[b], 0, n) - first) * mul / bm + b);
}

// Query and head of the group of row r of a sequence (rows of all sequences together stay below 2^31).
__host__ __device__ __forceinline__ void split_row(int64_t r, int group, int64_t& query, int& g) {
  const uint32_t x = (uint32_t)r, q = group == 1 ? x : x / (uint32_t)group;
  query = q;
  g = (int)(x - q * (uint32_t)group);
}

// Query of row r of a sequence.
__host__ __device__ __forceinline__ int64_t row_query(int64_t r, int group) {
  return group == 1 ? r : (uint32_t)r / (uint32_t)group;
}

// Part `part` of `parts` of an axis of n places (below 2^31 - 1024), [begin, end): all but the last a multiple of `step` long.
__host__ __device__ __forceinline__ void split_axis(int64_t n, int parts, int part, int step, int64_t& begin, int64_t& end) {
  begin = 0, end = n;
  if (parts == 1) return;
  const int64_t each = ((uint32_t)(n + parts - 1) / (uint32_t)parts + step - 1) / step * step;
  begin = part * each < n ? part * each : n;
  end = begin + each < n ? begin + each : n;
}

// A sliding window: query i of a sequence of lq queries and lk keys stands at p = i + lk - lq and sees the keys j <= p + right
// that are no more than `left` behind it or among the first `sinks`. left or right -1: no limit.
struct Window {
  int64_t left, right;
  int32_t sinks;
};

// The keys that the queries i0 .. i1 of a sequence see, as one axis of `keys` places: place x is key x before `sinks`, key x +
// jump from there on.
struct WindowAxis {
  int64_t keys, sinks, jump;
  __host__ __device__ __forceinline__ int64_t key(int64_t x) const { return x < sinks ? x : x + jump; }
};
__host__ __device__ __forceinline__ WindowAxis window_axis(const Window& w, int64_t i0, int64_t i1, int64_t lq, int64_t lk) {
  const int64_t high = w.right < 0 ? lk : clamp64(i1 + lk - lq + w.right + 1, 0, lk);
  const int64_t low = w.left < 0 ? 0 : clamp64(i0 + lk - lq - w.left, 0, high);
  WindowAxis a;
  a.sinks = w.sinks < low ? w.sinks : low;
  a.jump = low - a.sinks;
  a.keys = high - a.jump;
  return a;
}

// The places that a query sees on that axis, counted from place x0: those before `first` and those of [low, high).
struct WindowRow {
  int32_t first, low, high;
};
// The same for query i0 + i of a tile (i < 1024) in 32 bits: what leads far outside of the axis saturates.
struct WindowTile {
  int32_t sinks, low, high, end;
  __host__ __device__ __forceinline__ WindowRow row(int32_t i) const {
    WindowRow r;
    r.low = low + i;
    r.high = high + i < end ? high + i : end;
    r.first = sinks < r.high ? sinks : r.high;  // places before the jump: the row's window never ends there
    return r;
  }
};
__host__ __device__ __forceinline__ WindowTile window_tile(const Window& w, const WindowAxis& a, int64_t x0, int64_t i0, int64_t lq,
                                                           int64_t lk) {
  const int64_t p = i0 + lk - lq - a.jump - x0, far = INT32_MAX - 1023;
  WindowTile t;
  t.sinks = (int32_t)clamp64(w.sinks - x0, -far, far);
  t.low = (int32_t)(w.left < 0 ? -far : clamp64(p - w.left, -far, far));
  t.high = (int32_t)(w.right < 0 ? far : clamp64(p + w.right + 1, -far, far));
  t.end = (int32_t)(a.keys - x0);
  return t;
}

// The queries [begin, end) that see key j; `window`: of a sink, only those whose window holds it too.
__host__ __device__ __forceinline__ void window_queries(const Window& w, int64_t j, int64_t lq, int64_t lk, bool window,
                                                        int64_t& begin, int64_t& end) {
  begin = w.right < 0 ? 0 : clamp64(j - w.right - (lk - lq), 0, lq);
  end = w.left < 0 || (!window && j < w.sinks) ? lq : clamp64(j + w.left + 1 - (lk - lq), begin, lq);
}

}  // namespace igc
