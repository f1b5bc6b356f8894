// Pieces shared by the cross-attention kernels: ragged tiles, matrix-core fragments and staging.
//
// Fragments. All products run on 32x32 matrix instructions whose result puts one column in each
// lane (lane % 32) and 16 rows in its registers: register r of lane half h = lane / 32 is row
// 8 (r / 4) + 4 h + r % 4. Scores are computed transposed where the next product sums over keys (so
// that a lane owns a query: softmax statistics stay in the lane) and straight where it sums over
// queries; either way, registers 8 m .. 8 m + 7 of a score tile are, without any exchange between lanes,
// the second operand of the next product over the tile's 16 rows m, provided its first operand lists
// the same rows: 16 m + 4 h + 0..3, then 16 m + 8 + 4 h + 0..3. load_tr reads that operand.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "igc_host.h"
#include "igc_ragged.h"
#include "igc_row.h"
#include "igc_wave.h"

namespace igc {

typedef bf16_t bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16_t bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef float f32x8v __attribute__((ext_vector_type(8), aligned(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Operands of the matrix instructions are bf16. An fp32 value is split into three parts of 8 significant
// bits each, x = x0 + x1 + x2 exactly, and a product takes the six part products down to 2^-16 of it, which
// leaves out 2^-24: fp32 results at six bf16 instructions instead of eight fp32 ones that each take twice as
// long (fp32 tiles of 32 x 32 x 16: 192 cycles instead of 512). An infinite operand gives NaN.
template <typename T>
constexpr int kParts = sizeof(T) == 2 ? 1 : 3;

// 8 values of one lane along the summed axis, as operands.
template <typename T>
struct Frag {
  bf16x8v p[kParts<T>];
};
// The same as they are in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  typedef bf16x8v type;
};
template <>
struct Raw8<float> {
  typedef f32x8v type;
};

__device__ __forceinline__ Frag<bf16_t> to_parts(const bf16x8v& x) { return {{x}}; }
__device__ __forceinline__ Frag<float> to_parts(f32x8v x) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  Frag<float> f;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    u32x4 w;  // the upper halves of two values each: truncation to bf16
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_amdgcn_perm(__float_as_uint(x[2 * i + 1]), __float_as_uint(x[2 * i]), 0x07060302u);
    f.p[k] = __builtin_bit_cast(bf16x8v, w);
    if (k < 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] -= __uint_as_float(__float_as_uint(x[i]) & 0xFFFF0000u);
    }
  }
  return f;
}

// c += a b over 16 values of the summed axis.
__device__ __forceinline__ f32x16 mma(const bf16x8v& a, const bf16x8v& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<bf16_t>& a, const Frag<bf16_t>& b, const f32x16& c) {
  return mma(a.p[0], b.p[0], c);
}
__device__ __forceinline__ f32x16 mma(const Frag<float>& a, const Frag<float>& b, f32x16 c) {
  c = mma(a.p[1], b.p[1], c);
  c = mma(a.p[0], b.p[2], c);
  c = mma(a.p[2], b.p[0], c);
  c = mma(a.p[0], b.p[1], c);
  c = mma(a.p[1], b.p[0], c);
  return mma(a.p[0], b.p[0], c);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// 8 values at p; only the first `have` exist. vec: p is 16-byte aligned and 8 or none exist.
template <typename T>
__device__ __forceinline__ typename Raw8<T>::type load8(const T* p, int have, bool vec) {
  typename Raw8<T>::type f;
  if (vec) {
    f = typename Raw8<T>::type{};
    if (have > 0) f = *(const typename Raw8<T>::type*)p;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < have ? p[i] : (T)0.f;
  }
  return f;
}

// An LDS tile holds its parts one after the other, PS values apart, each row-major with row stride LD.
// First operand from rows (the summed axis along the row).
template <typename T, int PS>
__device__ __forceinline__ Frag<T> load_row(const bf16_t* p) {
  Frag<T> f;
#pragma unroll
  for (int k = 0; k < kParts<T>; ++k) f.p[k] = *(const bf16x8v*)(p + k * PS);
  return f;
}

// First operand whose summed axis runs over rows: this lane's column col0 + lane % 32 of rows
// row0 + 4 h + 0..3 and row0 + 8 + 4 h + 0..3, by the transposing LDS read: 16 lanes give the addresses
// of a 4 x 16 block (4 values each) and get a column of 4 each (layout measured).
template <typename T, int LD, int PS>
__device__ __forceinline__ Frag<T> load_tr(const bf16_t* s, int row0, int col0) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* lds;
  const int lane = lane_id();
  const bf16_t* p = s + (row0 + 4 * (lane >> 5) + ((lane & 15) >> 2)) * LD + col0 + (lane & 16) + (lane & 3) * 4;
  Frag<T> f;
#pragma unroll
  for (int k = 0; k < kParts<T>; ++k) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p + k * PS));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p + k * PS + 8 * LD));
    f.p[k] = __builtin_shufflevector(__builtin_bit_cast(bf16x4, a), __builtin_bit_cast(bf16x4, b), 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return f;
}

// x - part[i] in one instruction, a dot product with (-1, 0) or (0, -1); exact where part[i] is x rounded to bf16. An
// infinite neighbour makes it NaN, so the neighbours have to belong to the same sum. The pair comes from a register: as an
// inline constant, which the compiler would take for (-1, 0), the instruction reads -1 into the other half.
__device__ __forceinline__ float minus_part(const bf16x8v& part, int i, float x) {
  typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 pair = {part[i & ~1], part[i | 1]};
  uint32_t pick = i & 1 ? 0xBF800000u : 0x0000BF80u;
  asm("" : "+s"(pick));
  return __builtin_amdgcn_fdot2_f32_bf16(pair, __builtin_bit_cast(bf16x2, pick), x, false);
}

// Registers 8 m .. 8 m + 7 of a score tile as the second operand (bf16 data: rounded to nearest).
template <typename T>
__device__ __forceinline__ Frag<T> to_frag(const f32x16& s, int m) {
  if constexpr (sizeof(T) == 2) {
    Frag<T> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.p[0][i] = (bf16_t)s[8 * m + i];
    return f;
  } else {
    f32x8v x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s[8 * m + i];
    return to_parts(x);
  }
}

// The same as two operands, the rounded values and what the rounding left (fp32 data: all in the first).
template <typename T>
__device__ __forceinline__ void to_frag2(const f32x16& s, int m, Frag<T>& hi, Frag<T>& lo) {
  hi = to_frag<T>(s, m);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) lo.p[0][i] = (bf16_t)minus_part(hi.p[0], i, s[8 * m + i]);
  }
}

// Largest of a tile's 16 registers. Not as inline assembly, which would save passing the operands through a
// maximum with themselves first: the compiler places no wait between a matrix instruction and assembly that
// reads its result.
__device__ __forceinline__ float max16(const f32x16& x) {
  float top = x[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) top = fmaxf(top, x[r]);
  return top;
}

// Maximum over the two lanes that hold one column.
__device__ __forceinline__ float halves_max(float x) {
  const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
}

// Row of register r within a 32-row result tile, for lane half h.
__device__ __forceinline__ int reg_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// Row stride of an LDS tile of DP columns. Padding by 8 leaves row reads without bank conflicts, by 16 the
// column reads. 60,000 x 1,500, 128 channels: forward 136 us with 8, 132 with 16, dk and dv 298 and 280; 64 channels: 174.6
// and 179.5 (dq), 232 and 239. Permuting the granules frees both, but the address arithmetic costs more (dk, dv 264).
template <int DP>
constexpr int lds_ld() {
  return DP + (DP >= 128 ? 16 : 8);
}

// Copies tiles of ROWS rows of an operand (columns from dim on are zero) into an LDS tile of row stride
// LD in two steps, so that the loads of the next tile are in flight while this one is computed on: load()
// into registers, store() to LDS. Rows of keys step by the row stride. Rows of queries (group > 1) step
// through the heads that share a key head before the next query: row r is query r / group, head r % group.
// The tile's address is uniform and each thread keeps the offsets of its 8-value granules from it, which
// cost nothing per tile while ROWS is a multiple of group (the tile starts at a multiple of ROWS).
// VEC: 16-byte loads are allowed, dim is a multiple of 8 and a tile spans less than 2 GiB.
template <typename T, int ROWS, int DP, int NT, bool VEC>
struct Stage {
  static constexpr int CG = DP / 8;                    // granules of a row
  static constexpr int N = (ROWS * CG + NT - 1) / NT;  // granules of a thread
  typedef typename std::conditional<VEC, uint32_t, int64_t>::type Off;
  typename Raw8<T>::type r[N];
  Off off[N];  // bytes
  const char* base;
  int64_t row_stride, head_stride, at;
  int dim, group;
  static __device__ __forceinline__ bool mine(int i) {
    return (ROWS * CG) % NT == 0 || (int)threadIdx.x + i * NT < ROWS * CG;
  }
  static __device__ __forceinline__ int row(int i) { return (threadIdx.x + i * NT) / CG; }
  static __device__ __forceinline__ int col(int i) { return (threadIdx.x + i * NT) % CG * 8; }
  // first: row 0 of the sequence; the first tile starts at row r0 (a multiple of ROWS).
  __device__ __forceinline__ void start(const T* first, int64_t r0, int64_t rs, int64_t hs, int group_, int dim_) {
    row_stride = rs * (int64_t)sizeof(T), head_stride = hs * (int64_t)sizeof(T), group = group_, dim = dim_, at = r0;
    int64_t q;
    int g;
    split_row(r0, group, q, g);
    base = (const char*)first + q * row_stride;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int64_t q2;
      int g2;
      split_row(g + row(i), group, q2, g2);
      off[i] = (Off)(q2 * row_stride + g2 * head_stride + col(i) * (int)sizeof(T));
    }
  }
  // Loads the tile and steps to the next one. Rows from `have` on are zero.
  __device__ __forceinline__ void load(int have) {
    if (VEC && have >= ROWS && dim == DP && (ROWS * CG) % NT == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = *(const typename Raw8<T>::type*)(base + off[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        r[i] = load8<T>((const T*)(base + off[i]), mine(i) && row(i) < have ? dim - col(i) : 0, VEC);
    }
    if (ROWS % group == 0) {
      base += (int64_t)(ROWS / group) * row_stride;
    } else {
      int64_t q, q1;
      int g, g1;
      split_row(at, group, q, g);
      split_row(at + ROWS, group, q1, g1);
      at += ROWS;
      base += (q1 - q) * row_stride;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        int64_t q2;
        int g2;
        split_row(g1 + row(i), group, q2, g2);
        off[i] = (Off)(q2 * row_stride + g2 * head_stride + col(i) * (int)sizeof(T));
      }
    }
  }
  // Rows whose bit in `keep` is off are written as zeros.
  template <int LD, int PS>
  __device__ __forceinline__ void store(bf16_t* s, uint64_t keep) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (mine(i)) {
        typename Raw8<T>::type x = r[i];
        if (!(keep >> row(i) & 1)) x = typename Raw8<T>::type{};
        put<LD, PS>(s, i, x);
      }
  }
  template <int LD, int PS>
  __device__ __forceinline__ void store(bf16_t* s) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (mine(i)) put<LD, PS>(s, i, r[i]);
  }
  template <int LD, int PS>
  static __device__ __forceinline__ void put(bf16_t* s, int i, const typename Raw8<T>::type& x) {
    const Frag<T> f = to_parts(x);
#pragma unroll
    for (int k = 0; k < kParts<T>; ++k) *(bf16x8v*)(s + k * PS + row(i) * LD + col(i)) = f.p[k];
  }
};

// LDS bytes a workgroup of four waves needs for its tiles (values of bf16) and for store_tile.
template <typename T, int DP>
constexpr int lds_bytes(int tile_values) {
  const int out = 4 * 32 * (DP + 4) * 4;  // fp32 results: the larger form
  return tile_values * 2 > out ? tile_values * 2 : out;
}

// Stores a wave's result tile (32 rows in the lanes, DP / 32 register tiles of columns) scaled by f as rows of
// `dim` values: row `row` of this lane, none if negative. Through LDS (32 (DP + 4) fp32 values of the wave's own),
// since a lane's values lie 8 bytes at a time a row apart: 16-byte stores of whole rows instead. vec: dim is a
// multiple of 8 and out 16-byte aligned; otherwise value by value. 200,000 queries x 77 keys, 4 heads of 64: 84 us without
// LDS, 68 with.
template <typename T, int DP>
__device__ __forceinline__ void store_tile(T* out, void* lds, const f32x16 (&c)[DP / 32], float f, int64_t row, int dim,
                                           bool vec) {
  if (!vec) {
    if (row >= 0) {
#pragma unroll
      for (int t = 0; t < DP / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int at = t * 32 + reg_row(r, lane_id() >> 5);
          if (at < dim) out[row * dim + at] = (T)(c[t][r] * f);
        }
    }
    return;
  }
  constexpr int V = 16 / (int)sizeof(T), LD = DP + V, LPR = DP / V;
  const int lane = lane_id();
  T* s = (T*)lds;
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = c[t][4 * g + i] * f;
      store_vec<T, 4>(s + (lane & 31) * LD + t * 32 + 8 * g + 4 * (lane >> 5), v);
    }
  wave_sync();
#pragma unroll
  for (int i = 0; i < LPR / 2; ++i) {
    const int e = i * 64 + lane, r = e / LPR, col = e % LPR * V;
    const int64_t to = (int64_t)shfl64((uint64_t)row, r);
    const uint4 x = *(const uint4*)(s + r * LD + col);
    if (to >= 0 && col < dim) *(uint4*)(out + to * dim + col) = x;
  }
  wave_sync();
}

}  // namespace igc
