// Norm of queries and keys for each head and the rotation by their positions, in one pass over both, and its gradients.
//
//   rstd = 1 / sqrt(mean(x^2) + eps), z = x rstd w
//   pair (z1, z2) of axis a and frequency f turns by positions[row, a] * f:
//   y1 = amplitude (z1 cos - z2 sin), y2 = amplitude (z2 cos + z1 sin); channels behind the pairs: y = z
//   backward: g = the transposed rotation of dy, h = g w, dx = rstd (h - xhat mean(h xhat)), dw = sum of g xhat, xhat = x rstd
//
// A row's cosines and sines are computed once for all of its heads: the LPR lanes of a row first make a table in LDS, then
// keep what their channels need of it and walk the heads, V channels a load, with the loads of the next heads in flight.
//
// Memory bound, each array moved once (a copy of 4 GiB reaches 4.8 TB/s); the vector unit is busy for 73% of the time with bf16
// data. 1,000,003 rows of 4 + 4 heads of 64 by voxel coordinates, bf16: 391 us, 5.2 TB/s; gradients 598 us, 5.1 TB/s. Rotation alone of
// 500,003 rows of 4 heads of 48, fp32: 150 us, 5.1 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "igc_host.h"
#include "igc_row.h"
#include "igc_wave.h"

namespace igc {
namespace {

constexpr int kNT = 256;

// Cosine and sine of position * frequency. The product and its share of a turn are formed in 64 bits with the rounding
// errors carried along, whole turns leave before these are added (behind them they could be more than a turn themselves), so that
// positions up to 2^31 keep an angle exact to fp32 for frequencies up to 2^40, and a bounded one beyond; the rest of an eighth of a
// turn to either side goes through the Taylor series, whose first missing terms are below 2^-29.
__device__ __forceinline__ float2 cos_sin(int32_t position, float frequency) {
#pragma clang fp contract(off)  // t - rint(t) is of the rounded t: a fused one would hold what t_low adds
  constexpr double kTurn = 0.15915494309189535, kTurnLow = -9.839338337591534e-18;  // 1 / (2 pi) in two parts
  const double a = position, f = frequency;
  const double p = a * f, p_low = fma(a, f, -p);
  const double t = p * kTurn, t_low = fma(p_low, kTurn, fma(p, kTurnLow, fma(p, kTurn, -t)));
  const double u = (t - rint(t)) + t_low, quarter = rint(4.0 * u);
  const float x = (float)(fma(quarter, -0.25, u) * 6.283185307179586);
  const int q = (int)quarter & 3;
  const float x2 = x * x;
  const float s = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float c = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float co = q & 1 ? s : c, si = q & 1 ? c : s;
  return make_float2(q == 1 || q == 2 ? -co : co, q >= 2 ? -si : si);
}

// What a lane holds of a head: NV times V channels. The LPR lanes of a row, and with them its table, lie in one wave.
template <typename T, int V, int LPR, int NV>
struct Head {
  static constexpr int SL = kNT / LPR;       // rows of a workgroup
  static constexpr int WS = 64 / LPR;        // and of a wave
  static constexpr int DP = LPR * NV * V;    // channels that the lanes could hold
  static constexpr int kPairs = DP / 2 > 0 ? DP / 2 : 1;
  typedef typename VecOf<T, V>::type Raw;

  static __device__ __forceinline__ int lane_in() { return (int)threadIdx.x % LPR; }
  static __device__ __forceinline__ int channel(int j, int i) { return (j * LPR + lane_in()) * V + i; }

  // Cosines and sines of row r's pairs: each lane of the row makes every LPR-th.
  static __device__ __forceinline__ void fill(const QkArgs& a, int64_t r, bool live, float2* s_table) {
    const int pairs = a.axes * a.pairs;
    float2* const mine = s_table + lane_id() / LPR * kPairs;
    if (live)
      for (int p = lane_in(); p < pairs; p += LPR) {
        const int axis = (p >= a.pairs) + (p >= 2 * a.pairs);
        const float2 t = cos_sin(a.positions[r * a.axes + axis], a.frequencies[p]);
        mine[p] = make_float2(t.x * a.amplitude, t.y * a.amplitude);
      }
  }
  // This lane's factors: y[c] = z[c] co[c] + z[partner of c] si[c]. A row behind the last has no table: what lies there instead may
  // be NaN, which would enter the weights' gradients.
  static __device__ __forceinline__ void factors(const QkArgs& a, bool live, const float2* s_table, float (&co)[NV][V],
                                                 float (&si)[NV][V]) {
    const int pairs = a.axes * a.pairs;
    const float2* const mine = s_table + lane_id() / LPR * kPairs;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int ch = channel(j, i);
        co[j][i] = 1.f, si[j][i] = 0.f;
        if (live && ch < 2 * pairs) {
          const bool second = a.interleaved ? ch & 1 : ch >= pairs;
          const float2 t = mine[a.interleaved ? ch >> 1 : second ? ch - pairs : ch];
          co[j][i] = t.x;
          si[j][i] = second ? t.y : -t.y;
        }
      }
  }
  // Where the partners of this lane's channels lie in the wave's exchange (see partners); channels behind the pairs read its last
  // place, which holds 0.
  static constexpr int kExchange = NV * V * 64 + 1;
  static __device__ __forceinline__ void places(const QkArgs& a, float* s_x, int (&at)[NV][V]) {
    s_x[kExchange - 1] = 0.f;
    const int pairs = a.axes * a.pairs, first = lane_id() / LPR * LPR;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int ch = channel(j, i), to = a.interleaved ? ch ^ 1 : ch < pairs ? ch + pairs : ch - pairs, group = to / V;
        at[j][i] = ch < 2 * pairs ? (group / LPR * V + to % V) * 64 + first + group % LPR : kExchange - 1;
      }
  }
  // The partners' values of v; 0 for channels behind the pairs, whose own may be infinite. Channel c of a row lies at (c % V) * 64 +
  // its lane in the wave's part of LDS, so that neither the writes nor the reads, whose channels lie a fixed distance apart, meet
  // in a bank.
  static __device__ __forceinline__ void partners(const QkArgs& a, float* s_x, const int (&at)[NV][V], const float (&v)[NV][V],
                                                  float (&o)[NV][V]) {
    if (V % 2 == 0 && a.interleaved) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) o[j][i] = at[j][i] < kExchange - 1 ? v[j][i ^ 1] : 0.f;
      return;
    }
    wave_sync();  // the last values have been read
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s_x[(j * V + i) * 64 + lane_id()] = v[j][i];
    wave_sync();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) o[j][i] = s_x[at[j][i]];
  }
  // p: the head's values from this lane's first channel on.
  static __device__ __forceinline__ void load(const T* p, int dim, bool live, Raw (&v)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v[j] = Raw{};
      if (live && channel(j, 0) < dim) v[j] = *(const Raw*)(p + j * LPR * V);
    }
  }
  static __device__ __forceinline__ void floats(const Raw (&r)[NV], float (&v)[NV][V]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (V == 1) {
        v[j][0] = (float)r[j];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = (float)r[j][i];
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, int dim, bool live, const float (&v)[NV][V]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (live && channel(j, 0) < dim) store_vec<T, V>(p + j * LPR * V, v[j]);
    }
  }
  // The weights of queries and keys, 0 behind the head, kept in LDS: a head's are read where its turn comes.
  static __device__ __forceinline__ void keep_weights(const QkArgs& a, float (*s_w)[DP]) {
    for (int e = threadIdx.x; e < 2 * DP; e += kNT) {
      const void* w = a.w[e / DP];
      const int ch = e % DP;
      float x = ch < a.dim ? 1.f : 0.f;
      if (w && ch < a.dim) x = a.wf32 ? ((const float*)w)[ch] : (float)((const bf16_t*)w)[ch];
      s_w[e / DP][ch] = x;
    }
    __syncthreads();
  }
};

// How many heads' loads are in flight; the registers that this takes are bounded by the waves per SIMD (k_qk five, k_qk_bwd
// four). 1,000,003 rows of 4 + 4 heads of 64, bf16, us: forward 4 heads 393, 3 399, 2 with six waves 459, 1 435; without a bound 457;
// backward 1 head 602, 2 609, 2 with three waves 663. At five waves bf16 heads of 16 to 128 channels in steps of 8 spill two registers.
constexpr int kAhead = 4, kAheadBwd = 1;

// blockIdx.x: the rows, blockIdx.y: a share of the heads (those of the queries first).
template <typename T, int V, int LPR, int NV>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(5))) void k_qk(QkArgs a) {
  typedef Head<T, V, LPR, NV> H;
  __shared__ float2 s_table[kNT / 64][H::WS * H::kPairs];
  __shared__ float s_x[kNT / 64][H::kExchange];
  __shared__ float s_w[2][H::DP];
  const int wave = threadIdx.x >> 6;
  const float inv_d = 1.0f / (float)a.dim;
  const int h0 = blockIdx.y * a.heads_each, h1 = min(h0 + a.heads_each, a.heads[0] + a.heads[1]);
  int at[NV][V];
  H::places(a, s_x[wave], at);
  if (a.norm) H::keep_weights(a, s_w);
  for (int64_t r0 = (int64_t)blockIdx.x * H::SL; r0 < a.n; r0 += (int64_t)gridDim.x * H::SL) {
    const int64_t r = r0 + threadIdx.x / LPR;
    const bool live = r < a.n;
    typename H::Raw raw[kAhead][NV];
    // This lane's first channel of its row's first head: a head is a uniform step away.
    const T *px[2];
    T* py[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      px[t] = (const T*)a.x[t] + r * a.xs[t][0] + H::channel(0, 0);
      py[t] = (T*)a.y[t] + r * ((int64_t)a.heads[t] * a.dim) + H::channel(0, 0);
    }
    auto fetch = [&](int h, typename H::Raw (&x)[NV]) {
      if (h >= h1) return;
      if (h < a.heads[0]) H::load(px[0] + h * a.xs[0][1], a.dim, live, x);
      else H::load(px[1] + (h - a.heads[0]) * a.xs[1][1], a.dim, live, x);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(h0 + u, raw[u]);
    float co[NV][V], si[NV][V];
    wave_sync();  // the last row's table has been read
    H::fill(a, r, live, s_table[wave]);
    wave_sync();
    H::factors(a, live, s_table[wave], co, si);
    for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (h + u >= h1) break;
        const int t = h + u >= a.heads[0], g = h + u - (t ? a.heads[0] : 0);
        float x[NV][V], o[NV][V];
        H::floats(raw[u], x);
        fetch(h + u + kAhead, raw[u]);
        if (a.norm) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(x[j][i], x[j][i], ss);
          const float rstd = rsqrtf(fmaf(lanes_sum<LPR>(ss), inv_d, a.eps));
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) x[j][i] *= rstd * s_w[t][H::channel(j, i)];
        }
        H::partners(a, s_x[wave], at, x, o);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) x[j][i] = fmaf(x[j][i], co[j][i], o[j][i] * si[j][i]);
        if (t == 0) H::store(py[0] + (int64_t)g * a.dim, a.dim, live, x);
        else H::store(py[1] + (int64_t)g * a.dim, a.dim, live, x);
      }
    }
  }
}

template <typename T, int V, int LPR, int NV>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(4))) void k_qk_bwd(QkArgs a) {
  typedef Head<T, V, LPR, NV> H;
  __shared__ float2 s_table[kNT / 64][H::WS * H::kPairs];
  __shared__ float s_x[kNT / 64][H::kExchange];
  __shared__ float s_w[2][H::DP];
  const int wave = threadIdx.x >> 6;
  const float inv_d = 1.0f / (float)a.dim;
  const int h0 = blockIdx.y * a.heads_each, h1 = min(h0 + a.heads_each, a.heads[0] + a.heads[1]);
  float aw[2][NV][V];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) aw[t][j][i] = 0.f;
  int at[NV][V];
  H::places(a, s_x[wave], at);
  if (a.norm) H::keep_weights(a, s_w);
  for (int64_t r0 = (int64_t)blockIdx.x * H::SL; r0 < a.n; r0 += (int64_t)gridDim.x * H::SL) {
    const int64_t r = r0 + threadIdx.x / LPR;
    const bool live = r < a.n;
    typename H::Raw raw_g[kAheadBwd][NV], raw_x[kAheadBwd][NV];
    const T *px[2];
    int64_t dense[2];  // of dy and dx
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      px[t] = (const T*)a.x[t] + r * a.xs[t][0] + H::channel(0, 0);
      dense[t] = r * ((int64_t)a.heads[t] * a.dim) + H::channel(0, 0);
    }
    auto fetch = [&](int h, typename H::Raw (&g)[NV], typename H::Raw (&x)[NV]) {
      if (h >= h1) return;
      if (h < a.heads[0]) {
        H::load((const T*)a.dy[0] + (int64_t)h * a.dim + dense[0], a.dim, live, g);
        if (a.norm) H::load(px[0] + h * a.xs[0][1], a.dim, live, x);
      } else {
        const int k = h - a.heads[0];
        H::load((const T*)a.dy[1] + (int64_t)k * a.dim + dense[1], a.dim, live, g);
        if (a.norm) H::load(px[1] + k * a.xs[1][1], a.dim, live, x);
      }
    };
#pragma unroll
    for (int u = 0; u < kAheadBwd; ++u) fetch(h0 + u, raw_g[u], raw_x[u]);
    float co[NV][V], si[NV][V];
    wave_sync();
    H::fill(a, r, live, s_table[wave]);
    wave_sync();
    H::factors(a, live, s_table[wave], co, si);
    for (int h = h0; h < h1; h += kAheadBwd) {
#pragma unroll
      for (int u = 0; u < kAheadBwd; ++u) {
        if (h + u >= h1) break;
        const int t = h + u >= a.heads[0], k = h + u - (t ? a.heads[0] : 0);
        float g[NV][V], x[NV][V], o[NV][V];
        H::floats(raw_g[u], g);
        if (a.norm) H::floats(raw_x[u], x);
        fetch(h + u + kAheadBwd, raw_g[u], raw_x[u]);
        H::partners(a, s_x[wave], at, g, o);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) g[j][i] = fmaf(g[j][i], co[j][i], -o[j][i] * si[j][i]);
        if (a.norm) {
          float ss = 0.f, dot = 0.f, w[NV][V];
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              w[j][i] = s_w[t][H::channel(j, i)];
              ss = fmaf(x[j][i], x[j][i], ss);
              dot = fmaf(g[j][i] * w[j][i], x[j][i], dot);
            }
          // A row behind the last adds nothing to dw, not even NaN where eps is 0.
          const float rstd = live ? rsqrtf(fmaf(lanes_sum<LPR>(ss), inv_d, a.eps)) : 0.f;
          const float mean = lanes_sum<LPR>(dot) * inv_d * rstd;
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float xhat = x[j][i] * rstd, add = g[j][i] * xhat;
              if (t) aw[1][j][i] += add;
              else aw[0][j][i] += add;
              g[j][i] = rstd * fmaf(-xhat, mean, g[j][i] * w[j][i]);
            }
        }
        if (t == 0) H::store((T*)a.y[0] + (int64_t)k * a.dim + dense[0], a.dim, live, g);
        else H::store((T*)a.y[1] + (int64_t)k * a.dim + dense[1], a.dim, live, g);
      }
    }
  }
  if (!a.part) return;
  // The row slots of a wave by lane exchange, then the waves in order.
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int m = LPR; m < 64; m <<= 1) aw[t][j][i] += __shfl_xor(aw[t][j][i], m, 64);
  __shared__ float s_sum[kNT / 64][2][H::DP];
  if (lane_id() < LPR)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s_sum[wave][t][H::channel(j, i)] = aw[t][j][i];
  __syncthreads();
  float* const part = a.part + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.dim;
  for (int e = threadIdx.x; e < 2 * a.dim; e += kNT) {
    const int t = e / a.dim, ch = e % a.dim;
    part[e] = (s_sum[0][t][ch] + s_sum[1][t][ch]) + (s_sum[2][t][ch] + s_sum[3][t][ch]);
  }
}

template <int V>
using IntC = std::integral_constant<int, V>;

// Calls f(V, LPR, NV) for heads of `dim` channels: 16 bytes a load where that divides the head, so that pairs of
// neighbouring channels stay in a lane; less for other sizes.
template <typename T, typename F>
void with_head(int dim, F f) {
  auto lanes = [&](auto V) {
    const int l = dim / V;
    if (l <= 1) return f(V, IntC<1>{}, IntC<1>{});
    if (l <= 2) return f(V, IntC<2>{}, IntC<1>{});
    if (l <= 4) return f(V, IntC<4>{}, IntC<1>{});
    if (l <= 8) return f(V, IntC<8>{}, IntC<1>{});
    if (l <= 16) return f(V, IntC<16>{}, IntC<1>{});
    if constexpr (V <= 4) {
      if (l <= 32) return f(V, IntC<32>{}, IntC<1>{});
    }
    if constexpr (V <= 2) {
      if (l <= 64) return f(V, IntC<64>{}, IntC<1>{});
    }
    if constexpr (V == 1) return f(V, IntC<64>{}, IntC<2>{});
  };
  if constexpr (sizeof(T) == 2) {
    if (dim % 8 == 0) return lanes(IntC<8>{});
  }
  if (dim % 4 == 0) return lanes(IntC<4>{});
  if (dim % 2 == 0) return lanes(IntC<2>{});
  lanes(IntC<1>{});
}

// Heads of a workgroup: all of them, so that a row's table is made once, unless that leaves the GPU empty.
int heads_each(int64_t wgs, int heads) {
  const int64_t shares = std::max<int64_t>(1, std::min<int64_t>(heads, 1024 / std::max<int64_t>(1, wgs)));
  return (int)((heads + shares - 1) / shares);
}

template <typename T>
int rows_each(int dim) {
  int rows = 1;
  with_head<T>(dim, [&](auto V, auto L, auto NV) { rows = kNT / L; });
  return rows;
}

struct QkGrid {
  int64_t x;
  int heads_each, y;
};
QkGrid qk_grid(int dtype, int64_t n, int heads, int dim, int64_t most) {
  const int rows = dtype == IGC_BF16 ? rows_each<bf16_t>(dim) : rows_each<float>(dim);
  QkGrid g;
  const int64_t wgs = (n + rows - 1) / rows;
  g.heads_each = heads_each(wgs, heads);
  g.y = (heads + g.heads_each - 1) / g.heads_each;
  g.x = std::max<int64_t>(1, std::min<int64_t>(wgs, most));
  return g;
}

// Workgroups of the backward pass, each with partial weight gradients: as many as run at a time.
constexpr int64_t kBwdWgs = 1024;

template <typename T>
void qk_t(QkArgs a, bool backward, hipStream_t s) {
  const QkGrid g = qk_grid(a.dtype, a.n, a.heads[0] + a.heads[1], a.dim, backward ? kBwdWgs : kMaxWgs);
  a.heads_each = g.heads_each;
  const dim3 grid((unsigned)g.x, (unsigned)g.y);
  with_head<T>(a.dim, [&](auto V, auto L, auto NV) {
    if (backward) k_qk_bwd<T, V, L, NV><<<grid, kNT, 0, s>>>(a);
    else k_qk<T, V, L, NV><<<grid, kNT, 0, s>>>(a);
  });
}

}  // namespace

int qk_parts(int32_t dtype, int64_t n, int32_t heads, int32_t dim) {
  const QkGrid g = qk_grid(dtype, n, heads, dim, kBwdWgs);
  return (int)g.x * g.y;
}

int launch_qk(const QkArgs& a, bool backward, hipStream_t s) {
  if (a.dtype == IGC_BF16) qk_t<bf16_t>(a, backward, s);
  else qk_t<float>(a, backward, s);
  IGC_HIP(hipGetLastError(), a.fn);
  if (backward && a.part)
    return launch_pair_sum(a.fn, a.part, qk_parts(a.dtype, a.n, a.heads[0] + a.heads[1], a.dim), a.dim, a.dw[0], a.dw[1], s);
  return IGC_OK;
}

}  // namespace igc
