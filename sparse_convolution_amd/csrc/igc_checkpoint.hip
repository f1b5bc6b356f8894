// 8-bit activation checkpoints: packing features after the forward pass and restoring them in
// the backward pass.
//
// Groups of 64 consecutive channels of a row share one fp32 scale (the last group of a row may
// be shorter); see q8_scale for the formula. Memory bound: each value is read and written once. 4,100,003 fp32 rows of
// 16: pack 75 us, 4.6 TB/s, restore 54 us, 6.4 TB/s; 2,000,003 bf16 rows of 128: restore 129 us, 6.1 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "igc_host.h"
#include "igc_row.h"
#include "igc_wave.h"

namespace igc {
namespace {

constexpr int kNT = 256;

// Two tiles a workgroup once there are more than fill the GPU. Pack and restore of 128 M values, bf16 / fp32, us: 143 / 240; one
// tile 148 / 254, four 147 / 243, at most 8192 and 16384 workgroups 152 / 270.
unsigned wgs_for(int64_t tiles) {
  return (unsigned)std::min(std::max<int64_t>(std::min<int64_t>(tiles, 2048), (tiles + 1) / 2), kMaxWgs);
}

// GL lanes hold a group of up to 64 channels, V each; unit u = (row, group).
template <typename T, int V, int GL, bool TAIL>
__global__ __launch_bounds__(kNT) void k_pack(const T* __restrict__ x, uint32_t units, int c, int groups,
                                              int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int SL = kNT / GL;
  const int l = threadIdx.x % GL, slot = threadIdx.x / GL;
  for (uint64_t u0 = (uint64_t)blockIdx.x * SL; u0 < units; u0 += (uint64_t)gridDim.x * SL) {
    const uint32_t u = (uint32_t)u0 + slot;
    const bool live = u0 + slot < units;
    const uint32_t r = groups == 1 ? u : u / (uint32_t)groups;
    const RowPos<V, TAIL> e((int)(u - r * groups) * kQ8Group + l * V, c);
    float v[V];
    float a = 0.f;
    if (live && e.in) load_vec<T, V>(x + (int64_t)r * c + e.at, v);
#pragma unroll
    for (int i = 0; i < V; ++i) a = live && e.in && e.own(i) ? absmax2(a, v[i]) : a;
    a = lanes_absmax<GL>(a);
    float inv, scale;
    q8_scale(a, inv, scale);
    if (live && e.in) {
      store_codes<V>(codes + (int64_t)r * c + e.at, v, inv, e.skip);
      if (l == 0) scales[u] = scale;
    }
  }
}

// V channels of one row per thread.
template <typename T, int V, bool TAIL>
__global__ __launch_bounds__(kNT) void k_unpack(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                int64_t items, int per_row, int c, int groups, T* __restrict__ x) {
  const bool small = items <= UINT32_MAX;
  for (int64_t at = (int64_t)blockIdx.x * kNT + threadIdx.x; at < items; at += (int64_t)gridDim.x * kNT) {
    const int64_t r = small ? (int64_t)((uint32_t)at / (uint32_t)per_row) : at / per_row;
    const int first = (int)(at - r * per_row) * V;
    const RowPos<V, TAIL> e(first, c);
    float v[V];
    load_codes<V>(codes + r * c + e.at, v);
    const float sc = scales[r * groups + first / kQ8Group];
    const float before = TAIL ? scales[r * groups + e.at / kQ8Group] : sc;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= e.own(i) ? sc : before;
    store_vec<T, V>(x + r * c + e.at, v);
  }
}

template <typename T, int V, int GL>
void pack_go(const T* x, int64_t n, int c, int8_t* codes, float* scales, hipStream_t s) {
  const int groups = (c + kQ8Group - 1) / kQ8Group;
  // 32-bit units: rows of more groups are packed 2^25 rows at a time.
  for (int64_t r = 0; r < n; r += (int64_t)1 << 25) {
    const int64_t rows = std::min<int64_t>(n - r, (int64_t)1 << 25);
    const uint32_t units = (uint32_t)(rows * groups);
    const unsigned blocks = wgs_for(((int64_t)units + kNT / GL - 1) / (kNT / GL));
    const T* xr = x + r * c;
    if (c % V == 0) k_pack<T, V, GL, false><<<blocks, kNT, 0, s>>>(xr, units, c, groups, codes + r * c, scales + r * groups);
    else k_pack<T, V, GL, true><<<blocks, kNT, 0, s>>>(xr, units, c, groups, codes + r * c, scales + r * groups);
  }
}

template <typename T, int V>
void pack_v(const T* x, int64_t n, int c, int8_t* codes, float* scales, hipStream_t s) {
  const int lanes = (std::min(c, kQ8Group) + V - 1) / V;
  if (lanes <= 1) return pack_go<T, V, 1>(x, n, c, codes, scales, s);
  if (lanes <= 2) return pack_go<T, V, 2>(x, n, c, codes, scales, s);
  if constexpr (V >= 4) {
    if (lanes <= 4) return pack_go<T, V, 4>(x, n, c, codes, scales, s);
    if (lanes <= 8) return pack_go<T, V, 8>(x, n, c, codes, scales, s);
    if constexpr (V == 4) pack_go<T, V, 16>(x, n, c, codes, scales, s);
  }
}

template <typename T, int V>
void unpack_v(const int8_t* codes, const float* scales, int64_t n, int c, T* x, hipStream_t s) {
  const int per_row = (c + V - 1) / V, groups = (c + kQ8Group - 1) / kQ8Group;
  const int64_t items = n * per_row;
  const unsigned blocks = wgs_for((items + kNT - 1) / kNT);
  if (c % V == 0) k_unpack<T, V, false><<<blocks, kNT, 0, s>>>(codes, scales, items, per_row, c, groups, x);
  else k_unpack<T, V, true><<<blocks, kNT, 0, s>>>(codes, scales, items, per_row, c, groups, x);
}

// 16 bytes a load, less only for rows of fewer channels than that.
template <typename T>
void pack_t(const T* x, int64_t n, int c, int8_t* codes, float* scales, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (c >= 8) return pack_v<T, 8>(x, n, c, codes, scales, s);
  }
  if (c >= 4) return pack_v<T, 4>(x, n, c, codes, scales, s);
  if (c >= 2) return pack_v<T, 2>(x, n, c, codes, scales, s);
  pack_v<T, 1>(x, n, c, codes, scales, s);
}

template <typename T>
void unpack_t(const int8_t* codes, const float* scales, int64_t n, int c, T* x, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (c >= 8) return unpack_v<T, 8>(codes, scales, n, c, x, s);
  }
  if (c >= 4) return unpack_v<T, 4>(codes, scales, n, c, x, s);
  if (c >= 2) return unpack_v<T, 2>(codes, scales, n, c, x, s);
  unpack_v<T, 1>(codes, scales, n, c, x, s);
}

}  // namespace

int launch_pack(const void* x, int32_t dtype, int64_t n, int32_t c, int8_t* codes, float* scales, hipStream_t s) {
  if (dtype == IGC_BF16) pack_t<bf16_t>((const bf16_t*)x, n, c, codes, scales, s);
  else pack_t<float>((const float*)x, n, c, codes, scales, s);
  IGC_HIP(hipGetLastError(), "igc_checkpoint_pack: launch");
  return IGC_OK;
}

int launch_unpack(const int8_t* codes, const float* scales, int64_t n, int32_t c, int32_t dtype, void* x,
                  hipStream_t s) {
  if (dtype == IGC_BF16) unpack_t<bf16_t>(codes, scales, n, c, (bf16_t*)x, s);
  else unpack_t<float>(codes, scales, n, c, (float*)x, s);
  IGC_HIP(hipGetLastError(), "igc_checkpoint_unpack: launch");
  return IGC_OK;
}

}  // namespace igc
