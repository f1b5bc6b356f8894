// Cross attention, backward pass.
//
//   p_ij = exp(s_ij - lse_i), delta_i = dout_i . out_i, ds_ij = p_ij (dout_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j
//   dk_j = scale sum_i ds_ij q_i, dv_j = sum_i p_ij dout_i, over the queries of the sequence and the
//          query heads that share the key head
//
// Two kernels, each keeping its output in registers while it walks the other axis: k_attn_dq owns
// query rows and walks keys, k_attn_dkv owns keys and walks query rows, so nothing is added by atomics
// and reruns are bit-identical. Scores are computed again in both (seven products instead of five; nine with bf16 data, where
// those with ds are done in two parts).
//
// With bf16 data p is rounded to bf16 for dv; ds is kept in two bf16 parts for dq and dk, since its terms cancel (see
// k_attn_dkv for both sides). Bound like the forward pass, by the vector unit beside the matrix cores: bf16, 100,003 queries,
// 4 heads on 2 key heads of 64, three sequences of ~800 keys: 443 us in all (400 with ds rounded once for dk, on the same GPU);
// under the profiler, whose clock is lower, dq 227 us, dk and dv 290, sums 7.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "igc_attn.h"
#include "igc_host.h"

namespace igc {
namespace {

constexpr int kNT = 256;

// lse in base 2; +infinity for rows without keys, whose probabilities are then exp2(-infinity) = 0.
__device__ __forceinline__ float lse_base2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// dq and delta: four waves of 32 NQ query rows over tiles of BN keys (see k_attn_fwd for rows).
template <typename T, int DP, int NQ, int BN, int WPE, bool VEC>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_dq(AttnArgs a) {
  typedef Frag<T> frag;
  constexpr int LD = lds_ld<DP>(), PS = BN * LD;
  constexpr int BM = 128 * NQ;
  constexpr int KT = BN / 32, DT = DP / 32;
  constexpr uint64_t kAll = BN == 64 ? ~0ull : (1ull << (BN & 63)) - 1;
  constexpr int TILE = kParts<T> * PS;
  __shared__ __attribute__((aligned(16))) char s_mem[lds_bytes<T, DP>(4 * TILE)];
  auto s_k = [&](int buf) { return (bf16_t*)s_mem + buf * TILE; };
  auto s_v = [&](int buf) { return (bf16_t*)s_mem + (2 + buf) * TILE; };

  const int lane = lane_id(), wave = threadIdx.x >> 6, h = lane >> 5;
  const int kh = blockIdx.x % a.kv_heads;
  const int split = (blockIdx.x / a.kv_heads) % a.splits;
  int b;
  const int64_t tile = find_tile(a.qo, a.batch, a.nq, a.group, BM, blockIdx.x / (a.kv_heads * a.splits), b);
  int64_t q0, q1, k0, k1;
  seq_rows(a.qo, b, a.nq, q0, q1);
  seq_rows(a.ko, b, a.nk, k0, k1);
  const int64_t rows = (q1 - q0) * a.group;
  if (tile * BM >= rows) return;
  if (!a.dq) k1 = k0;  // only delta is wanted
  if (a.splits > 1) {
    const int64_t part = ((k1 - k0 + a.splits - 1) / a.splits + BN - 1) / BN * BN;
    k0 = k0 + split * part < k1 ? k0 + split * part : k1;
    k1 = k0 + part < k1 ? k0 + part : k1;
  }
  const int keys = (int)(k1 - k0);
  Stage<T, BN, DP, kNT, VEC> sk, sv;
  sk.start((const T*)a.k + kh * a.ks[1] + k0 * a.ks[0], 0, a.ks[0], 0, 1, a.dim);
  sv.start((const T*)a.v + kh * a.vs[1] + k0 * a.vs[0], 0, a.vs[0], 0, 1, a.dim);
  // As in k_attn_fwd: the ballot comes a tile later, so that it waits for no loads (100,003 queries, masked: 231 and 213 us).
  auto key_ok = [&](int j) -> int { return lane < BN && j + lane < keys ? (a.mask ? a.mask[k0 + j + lane] : 1) : 0; };
  sk.load(keys);
  sv.load(keys);
  int next_ok = key_ok(0);

  int64_t row[NQ];  // row of out and lse, -1: none
  frag fq[NQ][DP / 16], fo[NQ][DP / 16];
  float delta[NQ], lse[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t r = tile * BM + (wave * NQ + n) * 32 + (lane & 31);
    int64_t qi;
    int head;
    split_row(r < rows ? r : 0, a.group, qi, head);
    qi += q0;
    head += kh * a.group;
    const int64_t at = qi * a.heads + head;
    row[n] = r < rows ? at : -1;
    const T* p = (const T*)a.q + qi * a.qs[0] + head * a.qs[1];
    delta[n] = 0.f;
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      const int d = kk * 16 + h * 8, have = r < rows ? a.dim - d : 0;
      fq[n][kk] = to_parts(load8<T>(p + d, have, VEC));
      const auto g = load8<T>((const T*)a.dout + at * a.dim + d, have, VEC);
      const auto f = load8<T>((const T*)a.out_in + at * a.dim + d, have, VEC);
      fo[n][kk] = to_parts(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) delta[n] = fmaf((float)g[i], (float)f[i], delta[n]);
    }
    delta[n] += __shfl_xor(delta[n], 32, 64);
    if (row[n] >= 0 && h == 0 && split == 0) a.delta[row[n]] = delta[n];
    lse[n] = lse_base2(row[n] >= 0 ? a.lse_in[row[n]] : -INFINITY);
  }
  const float c = a.scale * kLog2e;
  f32x16 dq[NQ][DT];
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[n][t] = zero16();

  int buf = 0;
  for (int j = 0; j < keys; j += BN, buf ^= 1) {
    const uint64_t bits = __ballot(next_ok != 0);
    if (a.mask) {
      sk.template store<LD, PS>(s_k(buf), bits);
      sv.template store<LD, PS>(s_v(buf), bits);
    } else {
      sk.template store<LD, PS>(s_k(buf));
      sv.template store<LD, PS>(s_v(buf));
    }
    if (j + BN < keys) {
      sk.load(keys - j - BN);
      sv.load(keys - j - BN);
      next_ok = key_ok(j + BN);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      f32x16 s[NQ], dp[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n] = zero16(), dp[n] = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const int at = (t * 32 + (lane & 31)) * LD + kk * 16 + h * 8;
        const frag fk = load_row<T, PS>(s_k(buf) + at), fv = load_row<T, PS>(s_v(buf) + at);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          s[n] = mma(fk, fq[n][kk], s[n]);
          dp[n] = mma(fv, fo[n][kk], dp[n]);
        }
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], c, -lse[n])) * (dp[n][i] - delta[n]);
      if (bits != kAll) {
        const uint32_t w = (uint32_t)(bits >> (32 * t)) >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool keep = w & (1u << (8 * (i >> 2) + (i & 3)));
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][i] = keep ? s[n][i] : 0.f;
        }
      }
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        // ds in two parts: rounded once, dq would be off by more than one and a half times what its own rounding to
        // bf16 costs, since the terms of a row cancel (their ds add up to 0). In two parts by 1.00.
        frag hi[NQ], lo[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) to_frag2<T>(s[n], mm, hi[n], lo[n]);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const frag fk = load_tr<T, LD, PS>(s_k(buf), t * 32 + mm * 16, d * 32);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            if constexpr (sizeof(T) == 2) dq[n][d] = mma(fk, lo[n], dq[n][d]);
            dq[n][d] = mma(fk, hi[n], dq[n][d]);
          }
        }
      }
    }
  }
  if (!a.dq) return;
  __syncthreads();  // every wave is past reading the tiles: their space takes the results
  void* const s_out = s_mem + wave * (32 * (DP + 4) * 4);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (a.splits > 1)
      store_tile<float, DP>(a.part_a + (int64_t)split * a.nq * a.heads * a.dim, s_out, dq[n], a.scale, row[n], a.dim,
                            a.dim % 4 == 0);
    else
      store_tile<T, DP>((T*)a.dq, s_out, dq[n], a.scale, row[n], a.dim, a.ovec);
  }
}

// dk and dv: four waves of 32 NK keys each over tiles of BQ query rows of the sequence. bf16 data: ds in two parts for the
// product with q, as for dq, since its terms cancel too: rounded once, dk is off by 1.40 to 1.46 times what its own rounding
// to bf16 costs (30 to 1,500 keys a sequence, 256 queries, heads of 64, rms against 64 bits), in two parts by 1.00. The
// second product costs 4 to 12% of the backward pass over 300 to 1,500 keys (60,000 queries on 1,500 keys, heads of 128 and of
// 32: 433 and 453 us, 466 and 521). It is done at every length, so that a sequence's gradients are as exact whatever its
// neighbours are. A score costs its exponential, two multiplications, three roundings and a remainder: the products with dout
// start from -delta (read into their accumulators from LDS), and what the mask leaves out is cleared in the results
// instead of per score (100,003 queries, three sequences of ~800 keys, 4 heads of 64, ds rounded once: 252 and 223 us).
template <typename T, int DP, int NK, int BQ, int WPE, bool VEC>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_dkv(AttnArgs a) {
  typedef Frag<T> frag;
  constexpr int LD = lds_ld<DP>(), PS = BQ * LD;
  constexpr int BM = 128 * NK;
  constexpr int QT = BQ / 32, DT = DP / 32;
  constexpr int TILE = kParts<T> * PS;
  __shared__ __attribute__((aligned(16))) char s_mem[lds_bytes<T, DP>(4 * TILE)];
  auto s_q = [&](int buf) { return (bf16_t*)s_mem + buf * TILE; };
  auto s_o = [&](int buf) { return (bf16_t*)s_mem + (2 + buf) * TILE; };
  __shared__ __attribute__((aligned(16))) float s_lse[2][BQ], s_delta[2][BQ];  // s_delta: -delta

  const int lane = lane_id(), wave = threadIdx.x >> 6, h = lane >> 5;
  const int kh = blockIdx.x % a.kv_heads;
  const int split = (blockIdx.x / a.kv_heads) % a.splits;
  int b;
  const int64_t tile = find_tile(a.ko, a.batch, a.nk, 1, BM, blockIdx.x / (a.kv_heads * a.splits), b);
  int64_t q0, q1, k0, k1;
  seq_rows(a.qo, b, a.nq, q0, q1);
  seq_rows(a.ko, b, a.nk, k0, k1);
  if (k0 + tile * BM >= k1) return;
  int64_t r0 = 0, r1 = (q1 - q0) * a.group;
  if (a.splits > 1) {
    const int64_t part = ((r1 + a.splits - 1) / a.splits + BQ - 1) / BQ * BQ;
    r0 = split * part < r1 ? split * part : r1;
    r1 = r0 + part < r1 ? r0 + part : r1;
  }
  // Query rows step through the heads of the group before the next query.
  const int n_rows = (int)(r1 - r0);
  Stage<T, BQ, DP, kNT, VEC> sq, so;
  float n_lse = 0.f, n_delta = 0.f;  // as loaded: worked on a tile later (with ds rounded once 223 and 211 us)
  auto fetch = [&](int t0) {
    sq.load(n_rows - t0);
    so.load(n_rows - t0);
    if (threadIdx.x < BQ) {
      n_lse = -INFINITY;
      n_delta = 0.f;
      if (t0 + (int)threadIdx.x < n_rows) {
        int64_t qi;
        int g;
        split_row(r0 + t0 + threadIdx.x, a.group, qi, g);
        const int64_t at = (q0 + qi) * a.heads + kh * a.group + g;
        n_lse = a.lse_in[at];
        n_delta = a.delta[at];
      }
    }
  };
  if (n_rows > 0) {
    sq.start((const T*)a.q + q0 * a.qs[0] + kh * a.group * a.qs[1], r0, a.qs[0], a.qs[1], a.group, a.dim);
    so.start((const T*)a.dout + (q0 * a.heads + kh * a.group) * a.dim, r0, (int64_t)a.heads * a.dim, a.dim, a.group, a.dim);
    fetch(0);
  }

  int64_t key[NK];
  bool keep[NK];
  frag fk[NK][DP / 16], fv[NK][DP / 16];
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    const int64_t j = k0 + tile * BM + (wave * NK + n) * 32 + (lane & 31);
    key[n] = j < k1 ? j : -1;
    keep[n] = j < k1 && (!a.mask || a.mask[j]);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      const int d = kk * 16 + h * 8, have = keep[n] ? a.dim - d : 0;
      const int64_t at = keep[n] ? j : 0;
      fk[n][kk] = to_parts(load8<T>((const T*)a.k + at * a.ks[0] + kh * a.ks[1] + d, have, VEC));
      fv[n][kk] = to_parts(load8<T>((const T*)a.v + at * a.vs[0] + kh * a.vs[1] + d, have, VEC));
    }
  }
  const float c = a.scale * kLog2e;
  f32x16 dk[NK][DT], dv[NK][DT];
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int t = 0; t < DT; ++t) dk[n][t] = zero16(), dv[n][t] = zero16();

  int buf = 0;
  for (int t0 = 0; t0 < n_rows; t0 += BQ, buf ^= 1) {
    sq.template store<LD, PS>(s_q(buf));
    so.template store<LD, PS>(s_o(buf));
    if (threadIdx.x < BQ) s_lse[buf][threadIdx.x] = lse_base2(n_lse), s_delta[buf][threadIdx.x] = -n_delta;
    if (t0 + BQ < n_rows) fetch(t0 + BQ);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      f32x16 s[NK], dp[NK];
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        s[n] = zero16();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4v x = *(const f32x4v*)&s_delta[buf][t * 32 + 8 * g + 4 * h];
#pragma unroll
          for (int i = 0; i < 4; ++i) dp[n][4 * g + i] = x[i];
        }
      }
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const int at = (t * 32 + (lane & 31)) * LD + kk * 16 + h * 8;
        const frag fq = load_row<T, PS>(s_q(buf) + at), fo = load_row<T, PS>(s_o(buf) + at);
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          s[n] = mma(fq, fk[n][kk], s[n]);
          dp[n] = mma(fo, fv[n][kk], dp[n]);
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4v lse = *(const f32x4v*)&s_lse[buf][t * 32 + 8 * g + 4 * h];
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // Of a key that the mask leaves out this may be anything: it stays in the key's own results.
            const float p = __builtin_amdgcn_exp2f(fmaf(s[n][4 * g + i], c, -lse[i]));
            dp[n][4 * g + i] *= p;
            s[n][4 * g + i] = p;
          }
      }
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        frag fp[NK], fs[NK], lo[NK];
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          // bf16 data: rounded once, as in the forward pass. dv is off by 1.38 to 1.45 times its own rounding; in two parts by
          // 1.00, for 5 to 10% of the backward pass (60,000 x 1,500, heads of 32, 64 and 128: 543 and 599 us, 450 and 490, 471
          // and 496). p is positive, so the error is at most 2^-8 of the sum of p |dout| (in out 2^-8 of the sum of p |v|);
          // that of ds can be far more than its sum.
          fp[n] = to_frag<T>(s[n], mm);
          to_frag2<T>(dp[n], mm, fs[n], lo[n]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const frag go = load_tr<T, LD, PS>(s_o(buf), t * 32 + mm * 16, d * 32);
          const frag gq = load_tr<T, LD, PS>(s_q(buf), t * 32 + mm * 16, d * 32);
#pragma unroll
          for (int n = 0; n < NK; ++n) {
            dv[n][d] = mma(go, fp[n], dv[n][d]);
            if constexpr (sizeof(T) == 2) dk[n][d] = mma(gq, lo[n], dk[n][d]);
            dk[n][d] = mma(gq, fs[n], dk[n][d]);
          }
        }
      }
    }
  }
  __syncthreads();
  void* const s_out = s_mem + wave * (32 * (DP + 4) * 4);
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    const int64_t row = key[n] < 0 ? -1 : key[n] * a.kv_heads + kh;
    if (!keep[n]) {
#pragma unroll
      for (int t = 0; t < DT; ++t) dk[n][t] = zero16(), dv[n][t] = zero16();
    }
    if (a.splits > 1) {
      const int64_t first = (int64_t)split * a.nk * a.kv_heads * a.dim;
      store_tile<float, DP>(a.part_a + first, s_out, dk[n], a.scale, row, a.dim, a.dim % 4 == 0);
      store_tile<float, DP>(a.part_b + first, s_out, dv[n], 1.f, row, a.dim, a.dim % 4 == 0);
    } else {
      store_tile<T, DP>((T*)a.dk, s_out, dk[n], a.scale, row, a.dim, a.ovec);
      store_tile<T, DP>((T*)a.dv, s_out, dv[n], 1.f, row, a.dim, a.ovec);
    }
  }
}

// out[e] = sum over splits of part[split][e] in a fixed order, over the rows (of `width` values) that the sequences of
// `off` cover: eight groups of threads take every eighth part, and
// their sums are added in order. Two results of n values each (blockIdx.y). With one thread for all parts of an
// element, 128 parts of 77 keys x 256 channels took 31 us.
template <typename T, int V>
__global__ __launch_bounds__(kNT) void k_attn_sum(const float* __restrict__ part0, const float* __restrict__ part1,
                                                  int splits, const int32_t* __restrict__ off, int batch, int64_t rows,
                                                  int64_t width, T* __restrict__ out0, T* __restrict__ out1) {
  constexpr int G = 8, EL = kNT / G;
  __shared__ float s_sum[G][EL][V];
  const float* part = blockIdx.y ? part1 : part0;
  T* out = blockIdx.y ? out1 : out0;
  const int el = threadIdx.x % EL, g = threadIdx.x / EL;
  const int64_t e = ((int64_t)blockIdx.x * EL + el) * V, n = rows * width;  // V divides width
  int64_t first, last;
  covered_rows(off, batch, rows, first, last);
  const bool mine = e >= first * width && e < last * width;
  float t[V];
#pragma unroll
  for (int i = 0; i < V; ++i) t[i] = 0.f;
  if (mine) {
#pragma unroll 4
    for (int s = g; s < splits; s += G) {
      float v[V];
      load_vec<float, V>(part + (int64_t)s * n + e, v);
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s_sum[g][el][i] = t[i];
  __syncthreads();
  if (g == 0 && mine) {
#pragma unroll
    for (int k = 1; k < G; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] += s_sum[k][el][i];
    store_vec<T, V>(out + e, t);
  }
}

template <typename T>
void sum_go(const float* part0, const float* part1, int splits, const int32_t* off, int batch, int64_t rows, int heads,
            int dim, bool vec, void* out0, void* out1, hipStream_t s) {
  const int64_t width = (int64_t)heads * dim, n = rows * width;
  const int per = vec && dim % 4 == 0 ? 128 : 32;  // values of a workgroup
  const dim3 grid((unsigned)((n + per - 1) / per), out1 ? 2 : 1);
  if (per == 128)
    k_attn_sum<T, 4><<<grid, kNT, 0, s>>>(part0, part1, splits, off, batch, rows, width, (T*)out0, (T*)out1);
  else
    k_attn_sum<T, 1><<<grid, kNT, 0, s>>>(part0, part1, splits, off, batch, rows, width, (T*)out0, (T*)out1);
}

// Tiles of the two kernels: 32 NQ (NK) query rows (keys) of a wave, rows of an LDS tile, waves per SIMD.
// bf16, measured on 60,000 queries x 1,500 keys and 256 channels (dq / dkv, us; with ds rounded once and delta subtracted
// per score. Since then, with heads of 64: ds in two parts took dq from 175 to 220; delta as the products' start took dkv from 231
// to 208, and ds in two parts adds 41): heads of 32: dq 209 with three waves, 228 with NQ 2; dkv 286 with NK 2, 346 with
// NK 1. Heads of 64: dq 175 with NQ 2 on 32-key tiles, 184 on 64, 187 with NQ 1; dkv 231, with NK 2 (one wave) 317, on
// 32-row tiles 254. Heads of 128: dq 184 with two waves, 242 with one; dkv 290 with one wave, 470 with two (spills).
template <typename T, int DP>
struct BwdShape;
template <int DP>
struct BwdShape<bf16_t, DP> {
  static constexpr int NQ = DP == 64 ? 2 : 1, QWPE = DP <= 32 ? 3 : 2, QB = DP == 64 ? 32 : 64;
  static constexpr int NK = DP <= 32 ? 2 : 1, KWPE = DP <= 64 ? 2 : 1, KB = 64;
};
template <int DP>
struct BwdShape<float, DP> {
  static constexpr int NQ = 1, QWPE = DP <= 64 ? 2 : 1, QB = 32, NK = 1, KWPE = DP <= 32 ? 2 : 1, KB = 32;
};
struct BwdRows {
  int q, k;
};
template <typename T>
BwdRows bwd_rows_t(int dim) {
  if (dim <= 32) return {128 * BwdShape<T, 32>::NQ, 128 * BwdShape<T, 32>::NK};
  if (dim <= 64) return {128 * BwdShape<T, 64>::NQ, 128 * BwdShape<T, 64>::NK};
  return {128 * BwdShape<T, 128>::NQ, 128 * BwdShape<T, 128>::NK};
}
BwdRows bwd_rows(int dtype, int dim) { return dtype == IGC_BF16 ? bwd_rows_t<bf16_t>(dim) : bwd_rows_t<float>(dim); }

template <typename T, int DP>
void bwd_go(AttnArgs a, const AttnBwdPlan& p, float* ws, hipStream_t s) {
  typedef BwdShape<T, DP> S;
  const bool vec = a.qvec && a.kvec && a.ovec;
  a.delta = ws;
  ws += (a.nq * a.heads + 63) / 64 * 64;
  if (a.nq > 0) {
    AttnArgs d = a;
    d.splits = a.dq ? p.dq_splits : 1;
    d.part_a = ws;
    const unsigned wgs = (unsigned)((a.nq * a.group / (128 * S::NQ) + a.batch) * a.kv_heads * d.splits);
    if (vec) k_attn_dq<T, DP, S::NQ, S::QB, S::QWPE, true><<<wgs, kNT, 0, s>>>(d);
    else k_attn_dq<T, DP, S::NQ, S::QB, S::QWPE, false><<<wgs, kNT, 0, s>>>(d);
    if (a.dq && d.splits > 1)
      sum_go<T>(ws, nullptr, d.splits, a.qo, a.batch, a.nq, a.heads, a.dim, a.ovec, a.dq, nullptr, s);
  }
  if (a.dk && a.nk > 0) {
    const int64_t n = a.nk * a.kv_heads * a.dim;
    a.splits = p.dkv_splits;
    a.part_a = ws;
    a.part_b = ws + (p.dkv_splits > 1 ? p.dkv_splits * n : 0);
    const unsigned wgs = (unsigned)((a.nk / (128 * S::NK) + a.batch) * a.kv_heads * a.splits);
    if (vec) k_attn_dkv<T, DP, S::NK, S::KB, S::KWPE, true><<<wgs, kNT, 0, s>>>(a);
    else k_attn_dkv<T, DP, S::NK, S::KB, S::KWPE, false><<<wgs, kNT, 0, s>>>(a);
    if (a.splits > 1)
      sum_go<T>(a.part_a, a.part_b, a.splits, a.ko, a.batch, a.nk, a.kv_heads, a.dim, a.ovec, a.dk, a.dv, s);
  }
}

template <typename T>
void bwd_t(const AttnArgs& a, const AttnBwdPlan& p, float* ws, hipStream_t s) {
  if (a.dim <= 32) return bwd_go<T, 32>(a, p, ws, s);
  if (a.dim <= 64) return bwd_go<T, 64>(a, p, ws, s);
  if (a.dim <= 96) return bwd_go<T, 96>(a, p, ws, s);
  bwd_go<T, 128>(a, p, ws, s);
}

// Parts of the axis a kernel walks: enough to fill the GPU, each of at least `least` rows. The query axis goes down to
// 64 rows: its partial results are small next to what a part reads.
int parts(int64_t wgs, int64_t axis, int64_t least) {
  const int64_t want = wgs >= 512 ? 1 : 512 / std::max<int64_t>(1, wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 128), axis / least));
}

}  // namespace

AttnBwdPlan attn_bwd_plan(int dtype, int64_t nq, int64_t nk, int batch, int heads, int kv_heads, int dim) {
  AttnBwdPlan p;
  const BwdRows t = bwd_rows(dtype, dim);
  const int64_t rows = (nq + batch - 1) / batch * (heads / kv_heads), keys = (nk + batch - 1) / batch;
  p.dq_splits = parts(batch * ((rows + t.q - 1) / t.q) * kv_heads, keys, 256);
  p.dkv_splits = parts(batch * ((keys + t.k - 1) / t.k) * kv_heads, rows, 64);
  const size_t dq = p.dq_splits > 1 ? (size_t)p.dq_splits * nq * heads * dim : 0;
  const size_t dkv = p.dkv_splits > 1 ? (size_t)2 * p.dkv_splits * nk * kv_heads * dim : 0;
  // The two kernels run one after the other, so their partial results share the space.
  p.floats = (size_t)(nq * heads + 63) / 64 * 64 + std::max(dq, dkv);
  return p;
}

int launch_attn_bwd(const AttnArgs& a, int dtype, const AttnBwdPlan& p, void* ws, hipStream_t s) {
  if (dtype == IGC_BF16) bwd_t<bf16_t>(a, p, (float*)ws, s);
  else bwd_t<float>(a, p, (float*)ws, s);
  IGC_HIP(hipGetLastError(), a.fn);
  return IGC_OK;
}

}  // namespace igc
