// 8-bit activation checkpoints: packing features after the forward pass and restoring them in
// the backward pass.
//
// Groups of 64 consecutive channels of a row share one fp32 scale (the last group of a row may
// be shorter); see q8_scale for the formula. Memory bound: each value is read and written once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "igc_host.h"
#include "igc_row.h"
#include "igc_wave.h"

namespace igc {
namespace {

constexpr int kNT = 256;

// GL lanes hold a group of up to 64 channels, V each; unit u = (row, group).
template <typename T, int V, int GL>
__global__ __launch_bounds__(kNT) void k_pack(const T* __restrict__ x, int64_t units, int c, int groups,
                                              int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int SL = kNT / GL;
  const int l = threadIdx.x % GL, slot = threadIdx.x / GL;
  for (int64_t u0 = (int64_t)blockIdx.x * SL; u0 < units; u0 += (int64_t)gridDim.x * SL) {
    const int64_t u = u0 + slot;
    const int64_t r = u / groups;
    const int ch = (int)(u - r * groups) * kQ8Group + l * V;
    const bool in = u < units && ch < c;
    float v[V];
    float a = 0.f;
    if (in) load_vec<T, V>(x + r * c + ch, v);
#pragma unroll
    for (int i = 0; i < V; ++i) a = in ? absmax2(a, v[i]) : 0.f;
    a = lanes_absmax<GL>(a);
    float inv, scale;
    q8_scale(a, inv, scale);
    if (in) {
      store_codes<V>(codes + r * c + ch, v, inv);
      if (l == 0) scales[u] = scale;
    }
  }
}

// V channels of one group per thread.
template <typename T, int V>
__global__ __launch_bounds__(kNT) void k_unpack(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                int64_t items, int per_row, int c, int groups, T* __restrict__ x) {
  for (int64_t e = (int64_t)blockIdx.x * kNT + threadIdx.x; e < items; e += (int64_t)gridDim.x * kNT) {
    const int64_t r = e / per_row;
    const int ch = (int)(e - r * per_row) * V;
    float v[V];
    load_codes<V>(codes + r * c + ch, v);
    const float sc = scales[r * groups + ch / kQ8Group];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= sc;
    store_vec<T, V>(x + r * c + ch, v);
  }
}

template <typename T>
int vec_of(int c, const void* x, const void* codes) {
  for (int v = 16 / (int)sizeof(T); v >= 4; v /= 2)
    if (c % v == 0 && (uintptr_t)x % (v * sizeof(T)) == 0 && (uintptr_t)codes % v == 0) return v;
  return 1;
}

template <typename T, int V, int GL>
void pack_go(const T* x, int64_t n, int c, int8_t* codes, float* scales, hipStream_t s) {
  const int groups = (c + kQ8Group - 1) / kQ8Group;
  const int64_t blocks = (n * groups + kNT / GL - 1) / (kNT / GL);
  k_pack<T, V, GL><<<(unsigned)std::min<int64_t>(blocks, 8192), kNT, 0, s>>>(x, n * groups, c, groups, codes, scales);
}

template <typename T, int V>
void pack_v(const T* x, int64_t n, int c, int8_t* codes, float* scales, hipStream_t s) {
  const int lanes = (std::min(c, kQ8Group) + V - 1) / V;
  if (lanes <= 1) return pack_go<T, V, 1>(x, n, c, codes, scales, s);
  if (lanes <= 2) return pack_go<T, V, 2>(x, n, c, codes, scales, s);
  if (lanes <= 4) return pack_go<T, V, 4>(x, n, c, codes, scales, s);
  if (lanes <= 8) return pack_go<T, V, 8>(x, n, c, codes, scales, s);
  if constexpr (V < 8) {
    if (lanes <= 16) return pack_go<T, V, 16>(x, n, c, codes, scales, s);
    if constexpr (V < 4) {
      if (lanes <= 32) return pack_go<T, V, 32>(x, n, c, codes, scales, s);
      pack_go<T, V, 64>(x, n, c, codes, scales, s);
    }
  }
}

template <typename T, int V>
void unpack_v(const int8_t* codes, const float* scales, int64_t n, int c, T* x, hipStream_t s) {
  const int64_t items = n * (c / V);
  const int64_t blocks = (items + kNT - 1) / kNT;
  k_unpack<T, V><<<(unsigned)std::min<int64_t>(blocks, 16384), kNT, 0, s>>>(codes, scales, items, c / V, c,
                                                                           (c + kQ8Group - 1) / kQ8Group, x);
}

template <typename T>
void pack_t(const T* x, int64_t n, int c, int8_t* codes, float* scales, hipStream_t s) {
  const int v = vec_of<T>(c, x, codes);
  if constexpr (sizeof(T) == 2) {
    if (v == 8) return pack_v<T, 8>(x, n, c, codes, scales, s);
  }
  if (v == 4) return pack_v<T, 4>(x, n, c, codes, scales, s);
  pack_v<T, 1>(x, n, c, codes, scales, s);
}

template <typename T>
void unpack_t(const int8_t* codes, const float* scales, int64_t n, int c, T* x, hipStream_t s) {
  const int v = vec_of<T>(c, x, codes);
  if constexpr (sizeof(T) == 2) {
    if (v == 8) return unpack_v<T, 8>(codes, scales, n, c, x, s);
  }
  if (v == 4) return unpack_v<T, 4>(codes, scales, n, c, x, s);
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
