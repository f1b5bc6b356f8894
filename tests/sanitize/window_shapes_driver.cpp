// The choice of window attention's shapes (window_few) on the host, under AddressSanitizer and UndefinedBehaviorSanitizer (built
// and run by tests/test_window_shapes.py): the forms that share a row's axis between two waves are taken only where all
// workgroups of the launch run at a time, and wherever they do.
#include <cstdio>

#include "igc_host.h"

using namespace igc;

// Workgroups that a launch over `batch` sequences of `rows` rows has in tiles of `bm`: the slots that find_tile searches.
static int64_t launched(int64_t rows, int batch, int kv_heads, int bm) { return (rows * batch / bm + batch) * kv_heads; }

static int check(int dtype, int dim, int64_t rows, int batch, int kv_heads) {
  const bool wide = dim > (dtype == IGC_F32 ? 32 : 64), eight = dtype == IGC_F32 && dim > 32 && dim <= 64;
  const int got = window_few(dtype, dim, rows, batch, kv_heads);
  const bool one = launched(rows, batch, kv_heads, 64) <= (wide ? 256 : 512), two = eight && launched(rows, batch, kv_heads, 128) <= 256;
  const int want = one ? 1 : two ? 2 : 0;
  if (got == want) return 0;
  std::fprintf(stderr, "window shapes: %d, not %d (type %d, dim %d, %d sequences of %lld rows, %d key heads)\n", got, want, dtype, dim, batch,
               (long long)rows, kv_heads);
  return 1;
}

int main() {
  int bad = 0;
  for (int dtype : {IGC_F32, IGC_BF16})
    for (int dim : {8, 32, 33, 40, 64, 65, 96, 128})
      for (int64_t rows : {1, 20, 40, 63, 64, 65, 100, 128, 192, 256, 400, 2000, 4501, 8300, 16000, 33000, 2147482624})
        for (int batch : {1, 2, 3, 9, 34, 68, 100, 135, 200, 300, 1000})
          for (int kv_heads : {1, 2, 4, 8})
            if (rows * batch < 2147483648) bad += check(dtype, dim, rows, batch, kv_heads);
  // 200 sequences of 64 rows and 2 key heads: 400 tiles, but as many workgroups of eight waves, for 256 CUs.
  if (window_few(IGC_F32, 64, 64, 200, 2) != 0) ++bad, std::fprintf(stderr, "window shapes: 200 sequences of 64 rows\n");
  if (bad) return 1;
  std::puts("window shapes driver: ok");
  return 0;
}
