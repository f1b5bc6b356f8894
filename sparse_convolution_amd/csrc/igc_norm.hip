// Layer norm over the channels of each voxel, forward and backward, and its forms that keep the
// normalised input as an 8-bit checkpoint.
//
//   forward:  mu = mean(x), var = mean((x - mu)^2), rstd = 1 / sqrt(var + eps),
//             xhat = (x - mu) rstd, y = xhat w + b
//   backward: g = dy w, dx = rstd (g - mean(g) - xhat mean(g xhat)),
//             dw = sum over rows of dy xhat, db = sum over rows of dy
//
// A row is held in registers by LPR lanes (a power of two, or the whole workgroup for rows over
// 1024 channels), V channels a load, so memory is read once and the variance is summed around
// the mean rather than from squares. The mean is corrected by the mean of the differences from it: its
// rounding error would otherwise be scaled by rstd, up to 316 in a constant row (eps 1e-5). All sums are
// fp32; weight and bias gradients are fp32 per lane over the lane's rows, then added in a fixed order: the
// workgroup's row slots, then all workgroups in fp64, so reruns are bit-identical.
//
// Memory bound, each array moved once (a 4 GiB copy reaches 4.8 TB/s). bf16: 2,000,003 rows of 64, 93 us,
// 5.6 TB/s; backward of 4,000,037 rows of 256, 1.17 ms, 5.3 TB/s; with the checkpoint, 2,000,003 rows of
// 128, forward 248 us, 5.3 TB/s, backward 232 us, 5.6 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "igc_host.h"
#include "igc_row.h"
#include "igc_wave.h"

// Fused multiply-adds only where written: the compiler's own choice differs between a kernel's
// forms, and y must not depend on whether the checkpoint is written too.
#pragma clang fp contract(off)

namespace igc {
namespace {

constexpr int kNT = 256;  // threads of a workgroup

// Sums a and b over the LPR lanes of a row (LPR == kNT: over the workgroup, through s).
template <int LPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* s) {
  if constexpr (LPR <= 64) {
    a = lanes_sum<LPR>(a);
    b = lanes_sum<LPR>(b);
  } else {
    a = lanes_sum<64>(a);
    b = lanes_sum<64>(b);
    __syncthreads();  // the previous sums have been read
    if (lane_id() == 0) s[threadIdx.x >> 6] = a, s[4 + (threadIdx.x >> 6)] = b;
    __syncthreads();
    a = (s[0] + s[1]) + (s[2] + s[3]);
    b = (s[4] + s[5]) + (s[6] + s[7]);
  }
}
template <int LPR>
__device__ __forceinline__ float row_sum(float a, float* s) {
  float unused = 0.f;
  if constexpr (LPR <= 64) return lanes_sum<LPR>(a);
  row_sum2<LPR>(a, unused, s);
  return a;
}

template <typename T, int V, int LPR, int NV, bool TAIL, bool Q8>
__global__ __launch_bounds__(kNT) void k_norm(const T* __restrict__ x, int64_t n, int c, const void* __restrict__ w,
                                              const void* __restrict__ b, int wf32, float eps, T* __restrict__ y,
                                              float* __restrict__ mean, float* __restrict__ rstd,
                                              int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int SL = kNT / LPR;                                    // rows of a workgroup at a time
  constexpr int GL = LPR < kQ8Group / V ? LPR : kQ8Group / V;      // lanes of a scale group
  __shared__ float s_red[8];
  const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const float inv_c = 1.0f / (float)c;
  const int groups = (c + kQ8Group - 1) / kQ8Group;
  float pw[NV][V], pb[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const RowPos<V, TAIL> e((j * LPR + l) * V, c);
    if (e.in) {
      load_params<V>(w, e.at, wf32, 1.f, pw[j]);
      load_params<V>(b, e.at, wf32, 0.f, pb[j]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) pw[j][i] = pb[j][i] = 0.f;
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * SL; r0 < n; r0 += (int64_t)gridDim.x * SL) {
    const int64_t r = r0 + slot;
    const bool live = r < n;
    float v[NV][V];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const RowPos<V, TAIL> e((j * LPR + l) * V, c);
      if (live && e.in) {
        load_vec<T, V>(x + r * c + e.at, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum += e.own(i) ? v[j][i] : 0.f;
    }
    const float mu0 = row_sum<LPR>(sum, s_red) * inv_c;
    float sq = 0.f, rest = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const RowPos<V, TAIL> e((j * LPR + l) * V, c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[j][i] = e.in ? v[j][i] - mu0 : 0.f;
        const float d = e.own(i) ? v[j][i] : 0.f;
        rest += d;
        sq = fmaf(d, d, sq);
      }
    }
    row_sum2<LPR>(rest, sq, s_red);
    rest *= inv_c;
    // An infinite mean leaves NaN differences: it stays as it is, and the variance is NaN (a maximum with 0 would drop that).
    const float mu = rest - rest == 0.f ? mu0 + rest : mu0;
    const float var = fmaf(-rest, rest, sq * inv_c);
    const float rs = 1.0f / sqrtf((var < 0.f ? 0.f : var) + eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int first = (j * LPR + l) * V;
      const RowPos<V, TAIL> e(first, c);
      float o[V];
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[j][i] = e.in ? (v[j][i] - rest) * rs : 0.f;
        o[i] = fmaf(v[j][i], pw[j][i], pb[j][i]);
        if (Q8) a = absmax2(a, e.own(i) ? v[j][i] : 0.f);
      }
      if (live && e.in) store_vec<T, V>(y + r * c + e.at, o);
      if constexpr (Q8) {
        a = lanes_absmax<GL>(a);
        float inv, scale;
        q8_scale(a, inv, scale);
        if (live && e.in) {
          store_codes<V>(codes + r * c + e.at, v[j], inv, e.skip);
          if (l % GL == 0) scales[r * groups + first / kQ8Group] = scale;
        }
      }
    }
    if (live && l == 0) {
      if (!Q8) mean[r] = mu;
      rstd[r] = rs;
    }
  }
}

// Q8: xhat comes from codes and scales, otherwise from x, mean and rstd. part (may be null) gets
// the workgroup's partial dw and db, [gridDim.x][2][c].
template <typename T, int V, int LPR, int NV, bool TAIL, bool Q8>
__global__ __launch_bounds__(kNT) void k_norm_bwd(const T* __restrict__ dy, const T* __restrict__ x,
                                                  const float* __restrict__ mean, const int8_t* __restrict__ codes,
                                                  const float* __restrict__ scales, const float* __restrict__ rstd,
                                                  const void* __restrict__ w, int wf32, int64_t n, int c,
                                                  T* __restrict__ dx, float* __restrict__ part) {
  constexpr int SL = kNT / LPR;
  extern __shared__ float s_part[];  // [2][c]
  __shared__ float s_red[8];
  const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const float inv_c = 1.0f / (float)c;
  const int groups = (c + kQ8Group - 1) / kQ8Group;
  float pw[NV][V], aw[NV][V], ab[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const RowPos<V, TAIL> e((j * LPR + l) * V, c);
#pragma unroll
    for (int i = 0; i < V; ++i) pw[j][i] = aw[j][i] = ab[j][i] = 0.f;
    if (e.in) load_params<V>(w, e.at, wf32, 1.f, pw[j]);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * SL; r0 < n; r0 += (int64_t)gridDim.x * SL) {
    const int64_t r = r0 + slot;
    const bool live = r < n;
    const float rs = live ? rstd[r] : 0.f;
    const float mu = !Q8 && live ? mean[r] : 0.f;
    float g[NV][V], h[NV][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int first = (j * LPR + l) * V;
      const RowPos<V, TAIL> e(first, c);
#pragma unroll
      for (int i = 0; i < V; ++i) g[j][i] = h[j][i] = 0.f;
      if (live && e.in) {
        load_vec<T, V>(dy + r * c + e.at, g[j]);
        if constexpr (Q8) {
          load_codes<V>(codes + r * c + e.at, h[j]);
          const float sc = scales[r * groups + first / kQ8Group];
          const float before = TAIL ? scales[r * groups + e.at / kQ8Group] : sc;
#pragma unroll
          for (int i = 0; i < V; ++i) h[j][i] *= e.own(i) ? sc : before;
        } else {
          load_vec<T, V>(x + r * c + e.at, h[j]);
#pragma unroll
          for (int i = 0; i < V; ++i) h[j][i] = (h[j][i] - mu) * rs;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const RowPos<V, TAIL> e((j * LPR + l) * V, c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gi = e.own(i) ? g[j][i] : 0.f;
        aw[j][i] = fmaf(gi, h[j][i], aw[j][i]);
        ab[j][i] += gi;
        g[j][i] *= pw[j][i];
        const float gw = e.own(i) ? g[j][i] : 0.f;
        s1 += gw;
        s2 = fmaf(gw, h[j][i], s2);
      }
    }
    row_sum2<LPR>(s1, s2, s_red);
    s1 *= inv_c;
    s2 *= inv_c;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const RowPos<V, TAIL> e((j * LPR + l) * V, c);
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = rs * fmaf(-h[j][i], s2, g[j][i] - s1);
      if (live && e.in) store_vec<T, V>(dx + r * c + e.at, o);
    }
  }
  if (!part) return;
  // The row slots of a wave by lane exchange, then the waves one after the other.
  constexpr int WL = LPR < 64 ? LPR : 64;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int m = WL; m < 64; m <<= 1) {
        aw[j][i] += __shfl_xor(aw[j][i], m, 64);
        ab[j][i] += __shfl_xor(ab[j][i], m, 64);
      }
    }
  if constexpr (LPR == kNT) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const RowPos<V, TAIL> e((j * LPR + l) * V, c);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e.in && e.own(i)) {
          part[(size_t)blockIdx.x * 2 * c + e.at + i] = aw[j][i];
          part[(size_t)blockIdx.x * 2 * c + c + e.at + i] = ab[j][i];
        }
    }
  } else {
    for (int q = 0; q < kNT / 64; ++q) {
      if ((int)(threadIdx.x >> 6) == q && lane_id() < WL) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const RowPos<V, TAIL> e((j * LPR + l) * V, c);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (e.in && e.own(i)) {
              const int ch = e.at + i;
              s_part[ch] = q ? s_part[ch] + aw[j][i] : aw[j][i];
              s_part[c + ch] = q ? s_part[c + ch] + ab[j][i] : ab[j][i];
            }
        }
      }
      __syncthreads();
    }
    for (int e = threadIdx.x; e < 2 * c; e += kNT) part[(size_t)blockIdx.x * 2 * c + e] = s_part[e];
  }
}

// dw[e] (e < c) and db[e - c] = sum over chunks of part[chunk][e] in fp64, in a fixed order.
__global__ __launch_bounds__(kNT) void k_norm_reduce(const float* __restrict__ part, int chunks, int c,
                                                     float* __restrict__ dw, float* __restrict__ db) {
  constexpr int EL = 16, NG = kNT / EL;
  __shared__ double s_sum[NG][EL];
  const int el = threadIdx.x % EL, q = threadIdx.x / EL;
  const int e = blockIdx.x * EL + el;
  double acc = 0.0;
  if (e < 2 * c) {
#pragma unroll 8
    for (int k = q; k < chunks; k += NG) acc += (double)part[(size_t)k * 2 * c + e];
  }
  s_sum[q][el] = acc;
  __syncthreads();
  if (q == 0 && e < 2 * c) {
    double t = 0.0;
#pragma unroll
    for (int k = 0; k < NG; ++k) t += s_sum[k][el];
    if (e < c) dw[e] = (float)t;
    else db[e - c] = (float)t;
  }
}

template <int V>
using IntC = std::integral_constant<int, V>;

// Calls f(V, LPR, NV) as compile-time integers for rows of c channels loaded V at a time (V < 4: only the rows of
// fewer than 4 channels).
template <int V, typename F>
void with_row_shape(int c, F f) {
  const int lanes = (c + V - 1) / V;  // loads of a row
  if (lanes <= 1) return f(IntC<V>{}, IntC<1>{}, IntC<1>{});
  if (lanes <= 2) return f(IntC<V>{}, IntC<2>{}, IntC<1>{});
  if constexpr (V >= 4) {
    if (lanes <= 4) return f(IntC<V>{}, IntC<4>{}, IntC<1>{});
    if (lanes <= 8) return f(IntC<V>{}, IntC<8>{}, IntC<1>{});
    if (lanes <= 16) return f(IntC<V>{}, IntC<16>{}, IntC<1>{});
    if (lanes <= 32) return f(IntC<V>{}, IntC<32>{}, IntC<1>{});
    if (lanes <= 64) return f(IntC<V>{}, IntC<64>{}, IntC<1>{});
    if (lanes <= 128) return f(IntC<V>{}, IntC<64>{}, IntC<2>{});
    if constexpr (V == 4) {
      if (lanes <= 256) return f(IntC<V>{}, IntC<64>{}, IntC<4>{});
      if (lanes <= 512) return f(IntC<V>{}, IntC<kNT>{}, IntC<2>{});
      return f(IntC<V>{}, IntC<kNT>{}, IntC<4>{});
    } else {
      if (lanes <= 256) return f(IntC<V>{}, IntC<kNT>{}, IntC<1>{});
      return f(IntC<V>{}, IntC<kNT>{}, IntC<2>{});
    }
  }
}

// Calls f(V, LPR, NV, TAIL): 16 bytes a load, less only for rows of fewer channels than that.
template <typename T, typename F>
void with_shape(int c, F f) {
  auto with = [&](auto V) {
    with_row_shape<V>(c, [&](auto v, auto lpr, auto nv) {
      if (c % v == 0) f(v, lpr, nv, std::false_type{});
      else f(v, lpr, nv, std::true_type{});
    });
  };
  if constexpr (sizeof(T) == 2) {
    if (c >= 8) return with(IntC<8>{});
  }
  if (c >= 4) return with(IntC<4>{});
  if (c >= 2) return with(IntC<2>{});
  with(IntC<1>{});
}

template <typename T, bool Q8>
int norm_t(const NormArgs& a, hipStream_t s) {
  with_shape<T>(a.c, [&](auto V, auto L, auto NV, auto TAIL) {
    // A workgroup takes four (bf16) or two (fp32) tiles of rows, the grid apart: enough to spread the reading of the
    // weights over, while the workgroups in flight stay on neighbouring rows. 128 M values in rows of 64, bf16 / fp32, us:
    // one tile 114 / 173, two 99 / 177, four 100 / 188 (rows of 100: 144, 114 and 107 bf16), 4096 workgroups for
    // everything 110 / 223.
    const int64_t blocks = (a.n + kNT / L - 1) / (kNT / L);
    constexpr int kTiles = sizeof(T) == 2 ? 4 : 2;
    const int64_t wgs =
        std::min(std::max<int64_t>(std::min<int64_t>(blocks, 2048), (blocks + kTiles - 1) / kTiles), kMaxWgs);
    k_norm<T, V, L, NV, TAIL, Q8><<<(unsigned)wgs, kNT, 0, s>>>(
        (const T*)a.x, a.n, a.c, a.w, a.b, a.wf32, a.eps, (T*)a.y, a.mean, a.rstd, a.codes, a.scales);
  });
  IGC_HIP(hipGetLastError(), a.fn);
  return IGC_OK;
}

template <typename T, bool Q8>
int norm_bwd_t(const NormArgs& a, void* ws, hipStream_t s) {
  const int parts = norm_bwd_parts(a.n, a.c);
  float* part = a.dw ? (float*)ws : nullptr;
  with_shape<T>(a.c, [&](auto V, auto L, auto NV, auto TAIL) {
    k_norm_bwd<T, V, L, NV, TAIL, Q8><<<(unsigned)parts, kNT, 8 * (size_t)a.c, s>>>(
        (const T*)a.dy, (const T*)a.x, a.mean, a.codes, a.scales, a.rstd, a.w, a.wf32, a.n, a.c, (T*)a.y, part);
  });
  IGC_HIP(hipGetLastError(), a.fn);
  if (part) {
    k_norm_reduce<<<(unsigned)((2 * a.c + 15) / 16), kNT, 0, s>>>(part, parts, a.c, a.dw, a.db);
    IGC_HIP(hipGetLastError(), a.fn);
  }
  return IGC_OK;
}

}  // namespace

int norm_bwd_parts(int64_t n, int32_t c) {
  // One partial of 2 c floats per workgroup; three workgroups per CU walk all rows. 128 M bf16 values in rows of 64: 152 us with
  // 768 workgroups, 154 with 512, 158 with 1024, 179 with 2048; from a checkpoint 126, 143, 133 and 154.
  const int64_t rows = 64;
  return (int)std::max<int64_t>(1, std::min<int64_t>((n + rows - 1) / rows, 768));
}

int launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.dtype == IGC_BF16) return a.codes ? norm_t<bf16_t, true>(a, s) : norm_t<bf16_t, false>(a, s);
  return a.codes ? norm_t<float, true>(a, s) : norm_t<float, false>(a, s);
}

int launch_norm_bwd(const NormArgs& a, void* ws, hipStream_t s) {
  if (a.dtype == IGC_BF16) return a.codes ? norm_bwd_t<bf16_t, true>(a, ws, s) : norm_bwd_t<bf16_t, false>(a, ws, s);
  return a.codes ? norm_bwd_t<float, true>(a, ws, s) : norm_bwd_t<float, false>(a, ws, s);
}

}  // namespace igc
