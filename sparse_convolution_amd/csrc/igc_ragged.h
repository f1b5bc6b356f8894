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

}  // namespace igc
