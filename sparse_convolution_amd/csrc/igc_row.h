// Row-wise helpers shared by the layer norm and the 8-bit activation checkpoints: vector loads
// and stores of fp32 / bf16 values as floats, and reductions over the lanes that hold one row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace igc {

typedef __bf16 bf16_t;

// Channels of a row that share one scale of an 8-bit checkpoint.
constexpr int kQ8Group = 64;

// Vectors of V values at any address that T allows: global memory takes 16-byte accesses at every alignment, so
// rows of an odd number of channels are read as wide as others (see RowPos).
template <typename T, int V>
struct VecOf {
  typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};
template <typename T>
struct VecOf<T, 1> {
  typedef T type;
};

// Where a lane's V channels of a row of c >= V channels lie: from `first` on, where its turn comes, or, at the end of a
// row that V does not divide, the row's last V; the first `skip` of them belong to the lane before, which
// computes and stores the same values, and stay out of every sum.
template <int V, bool TAIL>
struct RowPos {
  int at, skip;
  bool in;
  __device__ __forceinline__ RowPos(int first, int c) : at(first), skip(0), in(first < c) {
    if (TAIL && in && first + V > c) at = c - V, skip = first - at;
  }
  __device__ __forceinline__ bool own(int i) const { return !TAIL || i >= skip; }
};

// V consecutive values at p as floats.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
  const typename VecOf<T, V>::type t = *(const typename VecOf<T, V>::type*)p;
  if constexpr (V == 1) {
    v[0] = (float)t;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)t[i];
  }
}

// Stores floats as T (bf16: rounded to nearest even).
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = (T)v[0];
  } else {
    typename VecOf<T, V>::type t;
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = (T)v[i];
    *(typename VecOf<T, V>::type*)p = t;
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Reduction over aligned groups of L lanes (L a power of two up to 64); every lane gets the
// result. Up to 16 lanes the exchange stays in the vector unit: quad permutes, then the mirrors
// of 8 and of 16 lanes (after the quads agree, lane 7 - i or 15 - i holds the other half).
template <int L, typename F>
__device__ __forceinline__ float lanes_reduce(float v, F f) {
  if constexpr (L >= 2) v = f(v, dpp<0xB1>(v));   // lane ^ 1
  if constexpr (L >= 4) v = f(v, dpp<0x4E>(v));   // lane ^ 2
  if constexpr (L >= 8) v = f(v, dpp<0x141>(v));  // 7 - lane of each 8
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v)); // 15 - lane of each 16
  if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16, 64));
  if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32, 64));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_reduce<L>(v, [](float a, float b) { return a + b; });
}
// Maximum that keeps a NaN: the hardware maximum drops it, so the lanes reduce the bit patterns
// of non-negative floats, whose integer order is theirs, with every NaN above infinity.
template <int L>
__device__ __forceinline__ float lanes_absmax(float v) {
  return lanes_reduce<L>(v, [](float a, float b) {
    const uint32_t x = __builtin_bit_cast(uint32_t, a), y = __builtin_bit_cast(uint32_t, b);
    return __builtin_bit_cast(float, x > y ? x : y);
  });
}
__device__ __forceinline__ float absmax2(float m, float x) {
  const uint32_t a = __builtin_bit_cast(uint32_t, m), b = __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
  return __builtin_bit_cast(float, a > b ? a : b);
}

// 8-bit checkpoint of one group with largest magnitude a: inv = 127 (1/a) maps a to 127, code =
// rint(x inv), value = code * scale with scale = a (1/127), each step rounded to fp32. Groups below
// 2^-100 store zeros (1/a of smaller ones would overflow); a group that holds an infinity or a
// NaN gets a NaN scale and zero codes, so that it reads back as NaN instead of as numbers.
__device__ __forceinline__ void q8_scale(float a, float& inv, float& scale) {
  const bool finite = a <= 3.402823466e38f;
  const bool zero = a < 0x1p-100f;
  inv = !finite || zero ? 0.f : __fmul_rn(1.0f / a, 127.f);
  scale = zero ? 0.f : finite ? __fmul_rn(a, 1.0f / 127.f) : __builtin_nanf("");
}
// inv == 0 gives 0 whatever x is (0 * infinity included).
__device__ __forceinline__ int q8_code(float x, float inv) {
  const float q = inv == 0.f ? 0.f : rintf(__fmul_rn(x, inv));
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// V codes to memory, without the first `skip` (their group may be another).
template <int V>
__device__ __forceinline__ void store_codes(int8_t* p, const float (&x)[V], float inv, int skip) {
  typedef int8_t i8x __attribute__((ext_vector_type(V < 2 ? 2 : V), aligned(1)));
  typedef uint32_t u32u __attribute__((aligned(1)));
  typedef uint16_t u16u __attribute__((aligned(1)));
  uint64_t w = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) w |= (uint64_t)((uint32_t)q8_code(x[i], inv) & 0xFFu) << (8 * i);
  if (skip == 0) {
    if constexpr (V == 1) *p = (int8_t)w;
    else *(i8x*)p = __builtin_bit_cast(i8x, typename std::conditional<V == 8, uint64_t, typename std::conditional<V == 4, uint32_t, uint16_t>::type>::type(w));
    return;
  }
  p += skip;
  w >>= 8 * skip;
  const int n = V - skip;
  if (n & 4) *(u32u*)p = (uint32_t)w, p += 4, w >>= 32;
  if (n & 2) *(u16u*)p = (uint16_t)w, p += 2, w >>= 16;
  if (n & 1) *p = (int8_t)w;
}
template <int V>
__device__ __forceinline__ void load_codes(const int8_t* p, float (&v)[V]) {
  typedef int8_t i8x __attribute__((ext_vector_type(V < 2 ? 2 : V), aligned(1)));
  if constexpr (V == 1) {
    v[0] = (float)*p;
  } else {
    const i8x t = *(const i8x*)p;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)t[i];
  }
}

// V channels of a weight or bias vector held in fp32 or in bf16, `none` where there is no vector.
template <int V>
__device__ __forceinline__ void load_params(const void* p, int at, bool f32, float none, float (&v)[V]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = none;
  } else if (f32) {
    load_vec<float, V>((const float*)p + at, v);
  } else {
    load_vec<bf16_t, V>((const bf16_t*)p + at, v);
  }
}

}  // namespace igc
