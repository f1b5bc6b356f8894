// Cross attention and window attention (WIN), backward pass.
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
// Windows (ten products, p in two parts for dv): 100,003 rows, 512 to either side and 16 sinks, masked, 4 heads on 2 of 64: 678 to
// 731 us in all by the GPU's clock, 326 to 351 TFLOP/s of the five products of visible pairs; under the profiler, whose clock is lower, dq 318, dk
// and dv 445, sinks 6.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "igc_attn.h"
#include "igc_host.h"

namespace igc {
namespace {

constexpr int kNT = 256;

// lse in base 2; +infinity for rows without keys, whose probabilities are then exp2(-infinity) = 0.
__device__ __forceinline__ float lse_base2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// dq and delta: NW waves of 32 NQ query rows over tiles of BN keys (see k_attn_fwd for rows, WIN, KS and the key mask's bias).
template <typename T, int DP, int NQ, int BN, int WPE, bool VEC, int WIN, int NW, int KS>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_dq(AttnArgs a) {
  typedef Frag<T> frag;
  constexpr int LD = lds_ld<DP>(), PS = BN * LD;
  constexpr int NT = 64 * NW, BM = 32 * NQ * NW / KS;
  constexpr int KT = BN / 32, DT = DP / 32;
  constexpr uint64_t kAll = BN == 64 ? ~0ull : (1ull << (BN & 63)) - 1;
  constexpr int TILE = kParts<T> * PS;
  __shared__ __attribute__((aligned(16))) char s_mem[lds_bytes<T, DP>(4 * TILE, NW)];
  __shared__ __attribute__((aligned(16))) float s_bias[WIN == 2 ? 2 : 1][WIN == 2 ? BN : 1];
  auto s_k = [&](int buf) { return (bf16_t*)s_mem + buf * TILE; };
  auto s_v = [&](int buf) { return (bf16_t*)s_mem + (2 + buf) * TILE; };

  static_assert(KS == 1 || (NQ == 1 && KT == KS && handover_bytes<DP / 32>(0) * NW / KS <= lds_bytes<T, DP>(4 * TILE, NW)), "KS");
  const int lane = lane_id(), wave = threadIdx.x >> 6, h = lane >> 5;
  const int row_wave = wave / KS, share = wave % KS;
  const int kh = blockIdx.x % a.kv_heads;
  const int split = (blockIdx.x / a.kv_heads) % a.splits;
  int b;
  const int64_t tile = tile_of<WIN != 0>(a.qo, a.batch, a.nq, a.group, BM, blockIdx.x / (a.kv_heads * a.splits), b);
  int64_t q0, q1, k0, k1;
  seq_rows(a.qo, b, a.nq, q0, q1);
  seq_rows(a.ko, b, a.nk, k0, k1);
  const int64_t rows = (q1 - q0) * a.group;
  if (tile * BM >= rows) return;
  WindowAxis axis = {};  // as in k_attn_fwd
  const int64_t lq = q1 - q0, lk = k1 - k0;
  int64_t x0 = 0, x1 = 0, i0 = 0;
  WindowTile tile_sees = {};
  if (!a.dq) k1 = k0;  // only delta is wanted
  if constexpr (WIN) {
    i0 = row_query(tile * BM, a.group);
    axis = window_axis(a.win, i0, row_query(((tile + 1) * BM < rows ? (tile + 1) * BM : rows) - 1, a.group), lq, lk);
    split_axis(a.dq ? axis.keys : 0, a.splits, split, BN, x0, x1);
    tile_sees = window_tile(a.win, axis, x0, i0, lq, lk);
  } else if (a.splits > 1) {
    const int64_t part = ((k1 - k0 + a.splits - 1) / a.splits + BN - 1) / BN * BN;
    k0 = k0 + split * part < k1 ? k0 + split * part : k1;
    k1 = k0 + part < k1 ? k0 + part : k1;
  }
  const int keys = WIN ? (int)(x1 - x0) : (int)(k1 - k0);
  Stage<T, BN, DP, NT, VEC> sk, sv;
  sk.start((const T*)a.k + kh * a.ks[1] + k0 * a.ks[0], 0, a.ks[0], 0, 1, a.dim);
  sv.start((const T*)a.v + kh * a.vs[1] + k0 * a.vs[0], 0, a.vs[0], 0, 1, a.dim);
  // As in k_attn_fwd: the ballot comes a tile later, so that it waits for no loads (100,003 queries, masked: 231 and 213 us).
  auto key_ok = [&](int j) -> int {
    if constexpr (WIN == 1) return 1;
    if constexpr (WIN == 2) return lane < BN && j + lane < keys ? a.mask[k0 + axis.key(x0 + j + lane)] : 0;
    return lane < BN && j + lane < keys ? (a.mask ? a.mask[k0 + j + lane] : 1) : 0;
  };
  // Tiles up to the one behind the last sink start where the axis says, others a tile behind the last.
  const int near_sinks = WIN ? (int)clamp64(axis.sinks - x0 + BN, 0, keys) : 0;
  auto fetch = [&](int j) {
    if constexpr (WIN) {
      if (j == 0 || j < near_sinks) {
        const int64_t x = x0 + j, cut = axis.sinks - x;
        const int64_t r = cut > 0 ? x : x + axis.jump;
        const int until = cut > 0 && cut < BN ? (int)cut : BN;
        sk.load_at((const T*)a.k + kh * a.ks[1] + k0 * a.ks[0], r, keys - j, until, axis.jump * sk.row_stride);
        sv.load_at((const T*)a.v + kh * a.vs[1] + k0 * a.vs[0], r, keys - j, until, axis.jump * sv.row_stride);
        return key_ok(j);
      }
    }
    sk.load(keys - j);
    sv.load(keys - j);
    return key_ok(j);
  };
  int next_ok = fetch(0);

  int64_t row[NQ];  // row of out and lse, -1: none
  frag fq[NQ][DP / 16], fo[NQ][DP / 16];
  float delta[NQ], lse[NQ];
  WindowRow see[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t r = tile * BM + (row_wave * NQ + n) * 32 + (lane & 31);
    int64_t qi;
    int head;
    split_row(r < rows ? r : WIN ? rows - 1 : 0, a.group, qi, head);
    if constexpr (WIN) see[n] = tile_sees.row((int)(qi - i0));
    qi += q0;
    head += kh * a.group;
    const int64_t at = qi * a.heads + head;
    row[n] = r < rows ? at : -1;
    const T* p = (const T*)a.q + qi * a.qs[0] + head * a.qs[1];
    const float row_lse = row[n] >= 0 ? a.lse_in[row[n]] : -INFINITY;
    const bool blind = WIN == 2 && row_lse == -INFINITY;  // what a row without keys holds need not be finite
    lse[n] = lse_base2(row_lse);
    delta[n] = 0.f;
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      typedef typename Raw8<T>::type raw;
      const int d = kk * 16 + h * 8, have = r < rows ? a.dim - d : 0;
      const raw x = load8<T>(p + d, have, VEC);
      const raw g = load8<T>((const T*)a.dout + at * a.dim + d, have, VEC);
      const raw f = load8<T>((const T*)a.out_in + at * a.dim + d, have, VEC);
      fq[n][kk] = to_parts(blind ? raw{} : x);
      fo[n][kk] = to_parts(blind ? raw{} : g);
#pragma unroll
      for (int i = 0; i < 8; ++i) delta[n] = fmaf((float)g[i], (float)f[i], delta[n]);
    }
    delta[n] += __shfl_xor(delta[n], 32, 64);
    if (blind) delta[n] = 0.f;
    if (row[n] >= 0 && h == 0 && split == 0 && share == 0) a.delta[row[n]] = delta[n];
  }
  WindowWave wave_sees;
  if constexpr (WIN) wave_sees.start(see[0], see[NQ - 1]);
  const float c = a.scale * kLog2e;
  f32x16 dq[NQ][DT];
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[n][t] = zero16();

  int buf = 0;
  for (int j = 0; j < keys; j += BN, buf ^= 1) {
    const uint64_t bits = WIN == 1 ? kAll : __ballot(next_ok != 0);
    if (WIN != 1 && a.mask) {
      sk.template store<LD, PS>(s_k(buf), bits);
      sv.template store<LD, PS>(s_v(buf), bits);
      if (WIN == 2 && wave == 0 && lane < BN) s_bias[buf][lane] = next_ok ? 0.f : -INFINITY;
    } else {
      sk.template store<LD, PS>(s_k(buf));
      sv.template store<LD, PS>(s_v(buf));
    }
    if (j + BN < keys) next_ok = fetch(j + BN);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      if (KS > 1 && t != share) continue;
      if (WIN && wave_sees.none(j + 32 * t, 32)) continue;
      f32x16 s[NQ], dp[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        s[n] = WIN == 2 ? n ? s[0] : from_bias(s_bias[buf] + 32 * t) : zero16();
        dp[n] = zero16();
      }
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
      if (WIN && !wave_sees.all(j + 32 * t, 32)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) clear_unseen(s[n], see[n], wave_sees, j + 32 * t, 0.f);
      } else if (!WIN && bits != kAll) {
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
  if constexpr (KS > 1) {
    float* const s = (float*)(s_mem + row_wave * handover_bytes<DT>(0));
    if (share == 1) hand_over(s, dq[0]);
    __syncthreads();
    if (share == 0) take_over(s, dq[0], 1.f, 1.f);
    __syncthreads();
    if (share == 1) return;
  }
  void* const s_out = s_mem + row_wave * (32 * (DP + 4) * 4);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (a.splits > 1)
      store_tile<float, DP>(a.part_a + (int64_t)split * a.nq * a.heads * a.dim, s_out, dq[n], a.scale, row[n], a.dim,
                            a.dim % 4 == 0);
    else
      store_tile<T, DP>((T*)a.dq, s_out, dq[n], a.scale, row[n], a.dim, a.ovec);
  }
}

// dk and dv: NW waves of 32 NK keys each over tiles of BQ query rows of the sequence. bf16 data: ds in two parts for the
// product with q, as for dq, since its terms cancel too: rounded once, dk is off by 1.40 to 1.46 times what its own rounding
// to bf16 costs (30 to 1,500 keys a sequence, 256 queries, heads of 64, rms against 64 bits), in two parts by 1.00. The
// second product costs 4 to 12% of the backward pass over 300 to 1,500 keys (60,000 queries on 1,500 keys, heads of 128 and of
// 32: 433 and 453 us, 466 and 521). It is done at every length, so that a sequence's gradients are as exact whatever its
// neighbours are. A score costs its exponential, two multiplications, three roundings and a remainder: the products with dout
// start from -delta (read into their accumulators from LDS), and what the mask leaves out is cleared in the results
// instead of per score (100,003 queries, three sequences of ~800 keys, 4 heads of 64, ds rounded once: 252 and 223 us).
//
// WIN: the workgroup of a key tile walks the rows whose windows hold any of its keys. Sinks among its keys are seen by all later
// rows too: those are walked by far_parts workgroups of their own for each tile with sinks (the launch's first), so that none walks
// a whole sequence alone, and k_attn_sinks adds up.
// KS 2 (WIN): pairs of waves share their keys, each takes every second block of 32 rows.
template <typename T, int DP, int NK, int BQ, int WPE, bool VEC, int WIN, int NW, int KS>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_dkv(AttnArgs a) {
  typedef Frag<T> frag;
  constexpr int LD = lds_ld<DP>(), PS = BQ * LD;
  constexpr int NT = 64 * NW, BM = 32 * NK * NW / KS;
  constexpr int QT = BQ / 32, DT = DP / 32;
  constexpr int TILE = kParts<T> * PS;
  __shared__ __attribute__((aligned(16))) char s_mem[lds_bytes<T, DP>(4 * TILE, NW)];
  auto s_q = [&](int buf) { return (bf16_t*)s_mem + buf * TILE; };
  auto s_o = [&](int buf) { return (bf16_t*)s_mem + (2 + buf) * TILE; };
  __shared__ __attribute__((aligned(16))) float s_lse[2][BQ], s_delta[2][BQ];  // s_delta: -delta

  static_assert(KS == 1 || (NK == 1 && QT == KS && handover_bytes<2 * DP / 32>(0) * NW / KS <= lds_bytes<T, DP>(4 * TILE, NW)), "KS");
  const int lane = lane_id(), wave = threadIdx.x >> 6, h = lane >> 5;
  const int key_wave = wave / KS, share = wave % KS;
  const bool far = WIN && blockIdx.x < a.far_wgs;
  const unsigned wg = WIN && !far ? blockIdx.x - a.far_wgs : blockIdx.x;
  const int kh = wg % a.kv_heads;
  const int parts = far ? a.far_parts : a.splits;
  const int split = (wg / a.kv_heads) % parts;
  int b;
  int64_t tile = wg / (a.kv_heads * parts);
  if (far && !a.far_by_key) {
    const int tiles = (a.win.sinks + BM - 1) / BM;
    b = (int)(tile / tiles);
    tile %= tiles;
  } else {
    tile = tile_of<WIN != 0>(a.ko, a.batch, a.nk, 1, BM, tile, b);
  }
  int64_t q0, q1, k0, k1;
  seq_rows(a.qo, b, a.nq, q0, q1);
  seq_rows(a.ko, b, a.nk, k0, k1);
  if (k0 + tile * BM >= k1) return;
  int64_t r0 = 0, r1 = (q1 - q0) * a.group;
  const int64_t lq = q1 - q0, lk = k1 - k0;
  bool sinks = false;  // some of the tile's keys are
  if constexpr (WIN) {
    sinks = tile * BM < a.win.sinks;
    if (far && !sinks) return;
    int64_t from, to, none;
    window_queries(a.win, tile * BM, lq, lk, true, from, none);
    window_queries(a.win, (tile + 1) * BM < lk ? (tile + 1) * BM - 1 : lk - 1, lq, lk, true, none, to);
    r0 = (far ? to : from) * a.group;
    r1 = far ? r1 : to * a.group;
    if (r1 < r0) r1 = r0;
  }
  if (parts > 1) {
    const int64_t part = ((r1 - r0 + parts - 1) / parts + BQ - 1) / BQ * BQ;
    r0 = r0 + split * part < r1 ? r0 + split * part : r1;
    r1 = r0 + part < r1 ? r0 + part : r1;
  }
  // Query rows step through the heads of the group before the next query.
  const int n_rows = (int)(r1 - r0);
  Stage<T, BQ, DP, NT, VEC> sq, so;
  float n_lse = 0.f, n_delta = 0.f;  // as loaded: worked on a tile later (with ds rounded once 223 and 211 us)
  // A mask may leave rows without keys among those that a tile of keys walks, and what such rows hold need not be finite: each
  // wave then looks at the tile's lse and makes them zeros. (Windows alone leave none there.)
  const bool masked = WIN && a.mask;
  auto fetch = [&](int t0) {
    sq.load(n_rows - t0);
    so.load(n_rows - t0);
    if (lane < BQ && (wave == 0 || masked)) {
      n_lse = -INFINITY;
      n_delta = 0.f;
      if (t0 + lane < n_rows) {
        int64_t qi;
        int g;
        split_row(r0 + t0 + lane, a.group, qi, g);
        const int64_t at = (q0 + qi) * a.heads + kh * a.group + g;
        n_lse = a.lse_in[at];
        if (wave == 0) n_delta = a.delta[at];
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
  int from[NK], to[NK];               // rows that see this lane's key, from this part's first on
  int any_from = 0, any_to = 0, all_from = 0, all_to = 0;  // rows that see any, and all, of the wave's keys
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    const int64_t j = k0 + tile * BM + (key_wave * NK + n) * 32 + (lane & 31);
    key[n] = j < k1 ? j : -1;
    keep[n] = j < k1 && (!a.mask || a.mask[j]);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      const int d = kk * 16 + h * 8, have = keep[n] ? a.dim - d : 0;
      const int64_t at = keep[n] ? j : 0;
      fk[n][kk] = to_parts(load8<T>((const T*)a.k + at * a.ks[0] + kh * a.ks[1] + d, have, VEC));
      fv[n][kk] = to_parts(load8<T>((const T*)a.v + at * a.vs[0] + kh * a.vs[1] + d, have, VEC));
    }
    if constexpr (WIN) {
      int64_t x, y;
      window_queries(a.win, j - k0, lq, lk, false, x, y);
      if (j >= k1 || (far && j - k0 >= a.win.sinks)) x = y = 0;  // nothing to do for it here
      from[n] = (int)(clamp64(x * a.group, r0, r1) - r0);
      to[n] = (int)(clamp64(y * a.group, r0, r1) - r0);
    }
  }
  if constexpr (WIN) {
    any_from = all_to = n_rows;
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      any_from = min(any_from, from[n] < to[n] ? from[n] : n_rows), any_to = max(any_to, from[n] < to[n] ? to[n] : 0);
      all_from = max(all_from, from[n]), all_to = min(all_to, to[n]);
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      any_from = min(any_from, __shfl_xor(any_from, m, 64)), any_to = max(any_to, __shfl_xor(any_to, m, 64));
      all_from = max(all_from, __shfl_xor(all_from, m, 64)), all_to = min(all_to, __shfl_xor(all_to, m, 64));
    }
    any_from = __builtin_amdgcn_readfirstlane(any_from), any_to = __builtin_amdgcn_readfirstlane(any_to);
    all_from = __builtin_amdgcn_readfirstlane(all_from), all_to = __builtin_amdgcn_readfirstlane(all_to);
  }
  const float c = a.scale * kLog2e;
  f32x16 dk[NK][DT], dv[NK][DT];
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int t = 0; t < DT; ++t) dk[n][t] = zero16(), dv[n][t] = zero16();

  int buf = 0;
  for (int t0 = 0; t0 < n_rows; t0 += BQ, buf ^= 1) {
    if (masked) {
      const uint64_t seeing = __ballot(n_lse != -INFINITY);
      if (seeing != ~0ull >> (64 - BQ)) sq.clear(seeing), so.clear(seeing);
    }
    sq.template store<LD, PS>(s_q(buf));
    so.template store<LD, PS>(s_o(buf));
    if (threadIdx.x < BQ) s_lse[buf][threadIdx.x] = lse_base2(n_lse), s_delta[buf][threadIdx.x] = -n_delta;
    if (t0 + BQ < n_rows) fetch(t0 + BQ);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int r32 = t0 + 32 * t;
      if (KS > 1 && t != share) continue;
      if (WIN && (any_to <= r32 || any_from >= r32 + 32)) continue;
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
      // Scores of rows that do not see the key need not be below their lse: minus infinity, so that p is 0.
      if (WIN && all_from > r32) {
#pragma unroll
        for (int n = 0; n < NK; ++n) clear_before(s[n], from[n] - r32, -INFINITY);
      }
      if (WIN && all_to < r32 + 32) {
#pragma unroll
        for (int n = 0; n < NK; ++n) clear_behind(s[n], to[n] - r32, -INFINITY);
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
        constexpr bool kTwo = WIN != 0 && sizeof(T) == 2;
        frag fp[NK], fs[NK], lo[NK], lp[NK];
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          // bf16 data: p as in the forward pass, without windows rounded once. dv is then off by 1.38 to 1.45 times its own
          // rounding; in two parts by 1.00, for 5 to 10% of the backward pass (60,000 x 1,500, heads of 32, 64 and 128: 543 and
          // 599 us, 450 and 490, 471 and 496). p is positive, so the error is at most 2^-8 of the sum of p |dout| (in out 2^-8 of
          // the sum of p |v|); that of ds can be far more than its sum. With windows two parts: dv is off by 1.00 (rounded once
          // 1.38 to 1.44) for 2 to 8% of the backward pass (100,003 rows, 256 to either side, 4 heads of 64 and 128: 429 and 449
          // us, 861 and 894; 512 to either side, masked, 4 heads on 2 of 64: 650 and 703).
          if constexpr (kTwo) to_frag2<T>(s[n], mm, fp[n], lp[n]);
          else fp[n] = to_frag<T>(s[n], mm);
          to_frag2<T>(dp[n], mm, fs[n], lo[n]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const frag go = load_tr<T, LD, PS>(s_o(buf), t * 32 + mm * 16, d * 32);
          const frag gq = load_tr<T, LD, PS>(s_q(buf), t * 32 + mm * 16, d * 32);
#pragma unroll
          for (int n = 0; n < NK; ++n) {
            if constexpr (kTwo) dv[n][d] = mma(go, lp[n], dv[n][d]);
            dv[n][d] = mma(go, fp[n], dv[n][d]);
            if constexpr (sizeof(T) == 2) dk[n][d] = mma(gq, lo[n], dk[n][d]);
            dk[n][d] = mma(gq, fs[n], dk[n][d]);
          }
        }
      }
    }
  }
  __syncthreads();
  if constexpr (KS > 1) {
    float* const s = (float*)(s_mem + key_wave * handover_bytes<2 * DT>(0));
    if (share == 1) hand_over(s, dk[0]), hand_over(s + DT * 16 * 64, dv[0]);
    __syncthreads();
    if (share == 0) take_over(s, dk[0], 1.f, 1.f), take_over(s + DT * 16 * 64, dv[0], 1.f, 1.f);
    __syncthreads();
    if (share == 1) return;
  }
  void* const s_out = s_mem + key_wave * (32 * (DP + 4) * 4);
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    int64_t row = key[n] < 0 ? -1 : key[n] * a.kv_heads + kh;
    if (!keep[n]) {
#pragma unroll
      for (int t = 0; t < DT; ++t) dk[n][t] = zero16(), dv[n][t] = zero16();
    }
    if (WIN && sinks) {
      // A sink's share: to far, but for the parts of an axis that is split, which lie with the other keys'.
      const int64_t j = key[n] - k0, at = a.far_by_key ? key[n] : (int64_t)b * a.win.sinks + j;
      const int64_t to_far = key[n] >= 0 && j < a.win.sinks ? at * a.kv_heads + kh : -1;
      if (far || a.splits == 1) {
        float* const out = a.far + (far ? 1 + split : 0) * a.far_rows * a.kv_heads * a.dim;
        store_tile<float, DP>(out, s_out, dk[n], a.scale, to_far, a.dim, a.dim % 4 == 0);
        store_tile<float, DP>(out + (1 + a.far_parts) * a.far_rows * a.kv_heads * a.dim, s_out, dv[n], 1.f, to_far, a.dim,
                              a.dim % 4 == 0);
        if (to_far >= 0) row = -1;
      }
      if (far) continue;
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
// their sums are added in order (up to eight parts: one thread takes them all, to the same bits). Two results of n values each (blockIdx.y). With one thread for all parts of an
// element, 128 parts of 77 keys x 256 channels took 31 us.
template <typename T, int V, int G>
__global__ __launch_bounds__(kNT) void k_attn_sum(const float* __restrict__ part0, const float* __restrict__ part1,
                                                  int splits, const int32_t* __restrict__ off, int batch, int64_t rows,
                                                  int64_t width, T* __restrict__ out0, T* __restrict__ out1) {
  constexpr int EL = kNT / G;
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

// Gradients of the sinks: the window's share (of a split axis: of its parts) and the far parts', in order. A thread for
// each row, key head and channel in turn, dk and dv as blockIdx.y.
template <typename T>
__device__ __forceinline__ void sum_sink(const AttnArgs& a, int64_t e) {
  const int64_t width = (int64_t)a.kv_heads * a.dim, r = e / width, c = e % width;
  int b = 0;
  if (a.far_by_key) {
    for (int hi = a.batch; a.ko && hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (a.ko[mid] <= r) b = mid;
      else hi = mid;
    }
  } else {
    b = (int)(r / a.win.sinks);
  }
  int64_t k0, k1;
  seq_rows(a.ko, b, a.nk, k0, k1);
  const int64_t j = a.far_by_key ? r - k0 : r % a.win.sinks;
  if (j < 0 || j >= a.win.sinks || k0 + j >= k1) return;
  const float* far = a.far + (blockIdx.y ? (1 + a.far_parts) * a.far_rows * width : 0) + e;
  float sum = 0.f;
  if (a.splits > 1) {
    const float* part = (blockIdx.y ? a.part_b : a.part_a) + (k0 + j) * width + c;
    for (int s = 0; s < a.splits; ++s) sum += part[(int64_t)s * a.nk * width];
  } else {
    sum = *far;
  }
#pragma unroll 8
  for (int p = 1; p <= a.far_parts; ++p) sum += far[p * a.far_rows * width];
  ((T*)(blockIdx.y ? a.dv : a.dk))[(k0 + j) * width + c] = (T)sum;
}
template <typename T>
__global__ __launch_bounds__(kNT) void k_attn_sinks(AttnArgs a) {
  const int64_t n = a.far_rows * a.kv_heads * a.dim;
  for (int64_t e = (int64_t)blockIdx.x * kNT + threadIdx.x; e < n; e += (int64_t)gridDim.x * kNT) sum_sink<T>(a, e);
}

template <typename T>
void sum_go(const float* part0, const float* part1, int splits, const int32_t* off, int batch, int64_t rows, int heads,
            int dim, bool vec, void* out0, void* out1, hipStream_t s) {
  const int64_t width = (int64_t)heads * dim, n = rows * width;
  const int v = vec && dim % 4 == 0 ? 4 : 1, per = v * (splits <= 8 ? kNT : kNT / 8);  // values of a workgroup
  const dim3 grid((unsigned)((n + per - 1) / per), out1 ? 2 : 1);
  auto go = [&](auto kernel) { kernel<<<grid, kNT, 0, s>>>(part0, part1, splits, off, batch, rows, width, (T*)out0, (T*)out1); };
  if (splits <= 8) go(v == 4 ? k_attn_sum<T, 4, 1> : k_attn_sum<T, 1, 1>);
  else go(v == 4 ? k_attn_sum<T, 4, 8> : k_attn_sum<T, 1, 8>);
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
// Window attention: for dq rows, waves per SIMD, keys of a tile and waves of a workgroup, then the same for dk and dv (chosen with p rounded once for
// dv, as the figures are). One tile of rows
// and three waves per SIMD for dq, since the masks of two spill. us, dq (1, 3, 32, 4) / (2, 2, 32, 4) / (1, 2, 64, 4): 100,003 rows, 512
// to either side, masked, 4 heads on 2 of 64: 605 / 672 / 622; 100,003 rows, 256 to either side, 4 heads: 388 / 491 / 387. Heads of 32
// (200,003 rows, 8 heads, 256 to either side): 901, with the shapes without windows 996; of 96 (100,003 rows, 4 heads) 645 and 705.
// fp32, heads of 32, two waves / four waves: 50,003 rows, 4 heads, 256 to either side 358 / 359, 7,131 rows, 2 heads, 64: 44 / 54.
// Registers that the compiler spills: dk and dv of fp32 heads over 96 73 to 76 (6 without windows), of eight waves 19 to 22; dq of bf16 heads over
// 96 at addresses that are no multiple of 16 bytes 33 to 66 (34 without windows).
template <int Q, int QE, int QN, int QW, int K, int KE, int KN, int KW, int S = 1>
struct Shape {
  static constexpr int NQ = Q, QWPE = QE, QB = QN, QNW = QW, NK = K, KWPE = KE, KB = KN, KNW = KW, KS = S;
  static constexpr int kRows = 32 * Q * QW / S, kKeys = 32 * K * KW / S;
};
template <typename T, int DP>
struct WinShape : Shape<1, 1, 32, 4, 1, 1, 32, 4> {};
template <>
struct WinShape<bf16_t, 32> : Shape<1, 3, 64, 4, 1, 3, 64, 4> {};
template <>
struct WinShape<bf16_t, 64> : Shape<1, 3, 32, 4, 1, 2, 64, 4> {};
template <>
struct WinShape<bf16_t, 96> : Shape<1, 2, 64, 4, 1, 2, 32, 4> {};
template <>
struct WinShape<bf16_t, 128> : Shape<1, 2, 64, 4, 1, 1, 64, 4> {};
template <>
struct WinShape<float, 32> : Shape<1, 2, 32, 2, 1, 2, 32, 2> {};
template <>
struct WinShape<float, 64> : Shape<1, 2, 32, 4, 1, 1, 32, 4> {};
// The same where tiles are few (see window_few): two waves share the walked axis. Heads over 64 in fp32 have no room for its tiles.
template <typename T, int DP>
struct WinFewShape : Shape<1, 2, 64, 4, 1, 2, 64, 4, 2> {};
template <>
struct WinFewShape<bf16_t, 96> : Shape<1, 2, 64, 4, 1, 1, 64, 4, 2> {};
template <>
struct WinFewShape<bf16_t, 128> : Shape<1, 2, 64, 4, 1, 1, 64, 4, 2> {};
template <>
struct WinFewShape<float, 64> : Shape<1, 1, 64, 4, 1, 1, 64, 4, 2> {};
template <>
struct WinFewShape<float, 96> : WinShape<float, 96> {};
template <>
struct WinFewShape<float, 128> : WinShape<float, 128> {};
typedef Shape<1, 2, 64, 8, 1, 2, 64, 8, 2> WinMidShape;  // of fp32 heads of 64
struct BwdTiles {
  int q, k;          // rows and keys of a workgroup's tile
  int few_q, few_k;  // see window_few
  int k_threads;     // of a workgroup of keys
};
template <typename T, int DP>
BwdTiles tiles_of(const AttnArgs& a) {
  typedef BwdShape<T, DP> B;
  typedef WinShape<T, DP> W;
  typedef WinFewShape<T, DP> F;
  if (!a.windowed) return {128 * B::NQ, 128 * B::NK, 0, 0, kNT};
  const int dtype = sizeof(T) == 2 ? IGC_BF16 : IGC_F32;
  const int q = window_few(dtype, a.dim, (a.nq + a.batch - 1) / a.batch * a.group, a.batch, a.kv_heads);
  const int k = window_few(dtype, a.dim, (a.nk + a.batch - 1) / a.batch, a.batch, a.kv_heads);
  return {q == 2 ? WinMidShape::kRows : q ? F::kRows : W::kRows, k == 2 ? WinMidShape::kKeys : k ? F::kKeys : W::kKeys, q, k,
          64 * (k == 2 ? WinMidShape::KNW : k ? F::KNW : W::KNW)};
}
template <typename T>
BwdTiles tiles_t(const AttnArgs& a) {
  if (a.dim <= 32) return tiles_of<T, 32>(a);
  if (a.dim <= 64) return tiles_of<T, 64>(a);
  if (a.dim <= 96) return tiles_of<T, 96>(a);
  return tiles_of<T, 128>(a);
}
BwdTiles bwd_tiles(int dtype, const AttnArgs& a) { return dtype == IGC_BF16 ? tiles_t<bf16_t>(a) : tiles_t<float>(a); }

// Key tiles of `bm` that may hold sinks.
int64_t far_tiles(const AttnArgs& a, bool by_key, int bm) {
  return a.win.sinks == 0 ? 0 : by_key ? a.nk / bm + a.batch : (int64_t)a.batch * ((a.win.sinks + bm - 1) / bm);
}

// Workgroups of the launch for dk and dv: those of the key tiles, and before them those of the sinks' far rows.
int64_t dkv_wgs(const AttnArgs& a, const AttnBwdPlan& p, int bm) { return (a.nk / bm + a.batch) * a.kv_heads * p.dkv_splits; }
int64_t far_wgs(const AttnArgs& a, const AttnBwdPlan& p, int bm) {
  return p.far_rows > 0 ? far_tiles(a, p.far_by_key, bm) * a.kv_heads * p.far_parts : 0;
}

// f(shape) with the shape of window attention that window_few chose.
template <typename T, int DP, typename F>
void with_win_shape(int few, F f) {
  if constexpr (sizeof(T) == 4 && DP == 64) {
    if (few == 2) return f(WinMidShape{});
  }
  if (few) f(WinFewShape<T, DP>{});
  else f(WinShape<T, DP>{});
}
template <typename T, int DP, typename W>
void win_dq(const AttnArgs& a, unsigned wgs, bool vec, hipStream_t s) {
  constexpr int NT = 64 * W::QNW;
  if (a.mask) {
    if (vec) k_attn_dq<T, DP, W::NQ, W::QB, W::QWPE, true, 2, W::QNW, W::KS><<<wgs, NT, 0, s>>>(a);
    else k_attn_dq<T, DP, W::NQ, W::QB, W::QWPE, false, 2, W::QNW, W::KS><<<wgs, NT, 0, s>>>(a);
  } else {
    if (vec) k_attn_dq<T, DP, W::NQ, W::QB, W::QWPE, true, 1, W::QNW, W::KS><<<wgs, NT, 0, s>>>(a);
    else k_attn_dq<T, DP, W::NQ, W::QB, W::QWPE, false, 1, W::QNW, W::KS><<<wgs, NT, 0, s>>>(a);
  }
}
template <typename T, int DP, typename W>
void win_dkv(const AttnArgs& a, unsigned wgs, bool vec, hipStream_t s) {
  if (vec) k_attn_dkv<T, DP, W::NK, W::KB, W::KWPE, true, 1, W::KNW, W::KS><<<wgs, 64 * W::KNW, 0, s>>>(a);
  else k_attn_dkv<T, DP, W::NK, W::KB, W::KWPE, false, 1, W::KNW, W::KS><<<wgs, 64 * W::KNW, 0, s>>>(a);
}

template <typename T, int DP>
void bwd_go(AttnArgs a, const AttnBwdPlan& p, float* ws, hipStream_t s) {
  typedef BwdShape<T, DP> S;
  const BwdTiles tile = tiles_of<T, DP>(a);
  const bool vec = a.qvec && a.kvec && a.ovec;
  a.delta = ws;
  ws += (a.nq * a.heads + 63) / 64 * 64;
  if (a.nq > 0) {
    AttnArgs d = a;
    d.splits = a.dq ? p.dq_splits : 1;
    d.part_a = ws;
    const unsigned wgs = (unsigned)((a.nq * a.group / tile.q + a.batch) * a.kv_heads * d.splits);
    if (!a.windowed) {
      if (vec) k_attn_dq<T, DP, S::NQ, S::QB, S::QWPE, true, 0, 4, 1><<<wgs, kNT, 0, s>>>(d);
      else k_attn_dq<T, DP, S::NQ, S::QB, S::QWPE, false, 0, 4, 1><<<wgs, kNT, 0, s>>>(d);
    } else {
      with_win_shape<T, DP>(tile.few_q, [&](auto w) { win_dq<T, DP, decltype(w)>(d, wgs, vec, s); });
    }
    if (a.dq && d.splits > 1)
      sum_go<T>(ws, nullptr, d.splits, a.qo, a.batch, a.nq, a.heads, a.dim, a.ovec, a.dq, nullptr, s);
  }
  if (a.dk && a.nk > 0) {
    const int64_t n = a.nk * a.kv_heads * a.dim;
    a.splits = p.dkv_splits;
    a.part_a = ws;
    a.part_b = ws + (p.dkv_splits > 1 ? p.dkv_splits * n : 0);
    const unsigned wgs = (unsigned)dkv_wgs(a, p, tile.k);
    if (a.windowed) {
      a.far_parts = p.far_parts, a.far_by_key = p.far_by_key, a.far_rows = p.far_rows;
      a.far = a.delta + p.far_at;
      a.far_wgs = (unsigned)far_wgs(a, p, tile.k);
      with_win_shape<T, DP>(tile.few_k, [&](auto w) { win_dkv<T, DP, decltype(w)>(a, wgs + a.far_wgs, vec, s); });
    } else {
      if (vec) k_attn_dkv<T, DP, S::NK, S::KB, S::KWPE, true, 0, 4, 1><<<wgs, kNT, 0, s>>>(a);
      else k_attn_dkv<T, DP, S::NK, S::KB, S::KWPE, false, 0, 4, 1><<<wgs, kNT, 0, s>>>(a);
    }
    if (a.splits > 1)
      sum_go<T>(a.part_a, a.part_b, a.splits, a.ko, a.batch, a.nk, a.kv_heads, a.dim, a.ovec, a.dk, a.dv, s);
    if (a.far_rows > 0) {
      const int64_t n = a.far_rows * a.kv_heads * a.dim;
      k_attn_sinks<T><<<dim3((unsigned)std::min<int64_t>((n + kNT - 1) / kNT, kMaxWgs), 2), kNT, 0, s>>>(a);
    }
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
int parts(int64_t wgs, int64_t axis, int64_t least, int64_t fill = 512) {
  const int64_t want = wgs >= fill ? 1 : fill / std::max<int64_t>(1, wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 128), axis / least));
}

}  // namespace

AttnBwdPlan attn_bwd_plan(int dtype, const AttnArgs& a) {
  const int64_t nq = a.nq, nk = a.nk;
  const int batch = a.batch, heads = a.heads, kv_heads = a.kv_heads, dim = a.dim;
  AttnBwdPlan p;
  const BwdTiles t = bwd_tiles(dtype, a);
  const int64_t rows = (nq + batch - 1) / batch * (heads / kv_heads), keys = (nk + batch - 1) / batch;
  int64_t seen_keys = keys, seen_rows = rows;  // that a tile walks
  const int64_t fill = a.windowed && dtype == IGC_F32 && dim > 32 ? 256 : 512;  // the former: one workgroup a CU
  if (a.windowed && a.win.left >= 0 && a.win.right >= 0) {
    seen_keys = std::min<int64_t>(keys, a.win.left + a.win.right + t.q / a.group + a.win.sinks);
    seen_rows = std::min<int64_t>(rows, (a.win.left + a.win.right + t.k) * a.group);
  }
  p.dq_splits = parts(batch * ((rows + t.q - 1) / t.q) * kv_heads, seen_keys, a.windowed ? kWindowPart : 256, fill);
  p.dkv_splits = parts(batch * ((keys + t.k - 1) / t.k) * kv_heads, seen_rows, a.windowed ? kWindowPart : 64, fill);
  const size_t dq = p.dq_splits > 1 ? (size_t)p.dq_splits * nq * heads * dim : 0;
  const size_t dkv = p.dkv_splits > 1 ? (size_t)2 * p.dkv_splits * nk * kv_heads * dim : 0;
  // The two kernels run one after the other, so their partial results share the space.
  p.floats = (size_t)(nq * heads + 63) / 64 * 64 + std::max(dq, dkv);
  if (a.windowed && a.win.sinks > 0 && nk > 0) {
    // Rows behind the window of a tile with sinks: parts about as long as what the others walk, while they are few.
    p.far_by_key = (int64_t)batch * a.win.sinks >= nk;
    p.far_rows = p.far_by_key ? nk : (int64_t)batch * a.win.sinks;
    const int64_t tiles = far_tiles(a, p.far_by_key, t.k) * kv_heads;
    p.far_parts = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(64, 1024 / tiles), rows * p.dkv_splits / std::max<int64_t>(128, seen_rows)));
    p.far_at = (p.floats + 3) / 4 * 4;
    p.floats = p.far_at + (size_t)2 * (1 + p.far_parts) * p.far_rows * kv_heads * dim;
  }
  p.dkv_threads = (dkv_wgs(a, p, t.k) + far_wgs(a, p, t.k)) * t.k_threads;
  return p;
}

int launch_attn_bwd(const AttnArgs& a, int dtype, const AttnBwdPlan& p, void* ws, hipStream_t s) {
  if (dtype == IGC_BF16) bwd_t<bf16_t>(a, p, (float*)ws, s);
  else bwd_t<float>(a, p, (float*)ws, s);
  IGC_HIP(hipGetLastError(), a.fn);
  return IGC_OK;
}

}  // namespace igc
