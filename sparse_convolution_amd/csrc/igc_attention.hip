// Cross attention of voxel (or object) queries to an encoder's states, and window attention among rows in order (WIN), forward
// pass.
//
//   s_ij = scale q_i . k_j over the keys j of the query's sequence that the mask keeps
//   lse_i = log sum_j exp s_ij, out_i = sum_j exp(s_ij - lse_i) v_j
//
// One pass over the keys with a running maximum and sum (online softmax); scores never leave
// registers. A row without keys gives out = 0, lse = -infinity.
//
// Long against long, the vector unit bounds it beside the matrix cores: 425 vector instructions (exponentials,
// sums, maxima, rounding) for the 32 matrix instructions of a wave's 64 x 64 scores with heads of 64, at two waves
// per SIMD. bf16, 215,003 queries on 5 x ~1024 keys, 4 heads of 64: 278 to 309 us by the GPU's clock, 715 to 795 TFLOP/s.
// fp32, 300 queries on 43,217 keys, 8 heads of 32: 110 to 123 us in all, 108 to 121 TFLOP/s. Single tokens (k_attn_few) read
// K and V once: 64 sequences of one query and 4,096 keys, 8 heads of 64, bf16 117 us, 4.6 TB/s, fp32 194 us, 5.5 TB/s. 64
// queries on 262,147 keys where half of the sequences have no query and one has 33: 39 us and 5 to join; the 81,157 keys
// in use are 166 MB, 4.3 TB/s, and that one sequence's keys are read 33 times, once for each row (see fwd_rows).
//
// Windows: the same bound, with what narrow windows add: staging, prologue and edges, and the second part of p, are half of the vector
// instructions of a block of 32 x 32 scores (174 of them, 28 for that part; 85 without windows). 200,003 rows, 256 to either side and 8 sinks, 4
// heads of 64 bf16: 261 to 273 us by the GPU's clock, 391 to 409 TFLOP/s of visible pairs, vector unit busy 66%, matrix cores 33%, the last
// of 6.1 rounds of workgroups. 64 tokens with 1,028 visible keys each, 8 heads on 4 of 64: 28 us, 2.4 TB/s: latency of a workgroup
// on every CU.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "igc_attn.h"
#include "igc_host.h"

namespace igc {
namespace {

constexpr int kNT = 256;
// How far (in base 2) a row's scores may pass its reference before the reference is raised to them.
// Probabilities up to 2^8 lose nothing in floating point, in bf16 neither, and the result so far is
// rescaled a few times per row instead of in nearly every tile: of 64 lanes some row's maximum grows
// almost always. 215,003 queries on 5 x ~1024 keys, 4 heads of 64, measured in turn: 306 us without, 293 with.
constexpr float kSlack = 8.f;

// NW waves of 32 NQ query rows each over tiles of BN keys. A row is a (query, head of the group
// that shares the key head) pair, so few queries with shared key heads still fill a tile.
// splits > 1: each workgroup takes one part of the sequence's keys and leaves an unnormalised result.
// WIN 1: a query sees the keys of a window and a few first ones (see igc_ragged.h); 2: and a key mask keeps some. The workgroup walks the
// keys that any of its queries sees; a wave passes over those that none of its own sees, and masks by rows only where an
// edge runs through, 32 keys at a time. The key mask enters as a bias.
// KS 2 (WIN): pairs of waves share their rows, each takes every second block of 32 keys, and one adds up: half the
// latency where there are too few rows to fill the GPU.
template <typename T, int DP, int NQ, int BN, int WPE, bool VEC, int WIN, int NW, int KS>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_fwd(AttnArgs a) {
  typedef Frag<T> frag;
  constexpr int NT = 64 * NW;
  constexpr int LD = lds_ld<DP>(), PS = BN * LD;
  constexpr int BM = 32 * NQ * NW / KS;
  constexpr int KT = BN / 32, DT = DP / 32;
  static_assert(KS == 1 || (NQ == 1 && KT == KS && handover_bytes<DP / 32>(2) * NW / KS <= lds_bytes<T, DP>(4 * kParts<T> * PS, NW)), "KS");
  constexpr uint64_t kAll = BN == 64 ? ~0ull : (1ull << (BN & 63)) - 1;
  constexpr int TILE = kParts<T> * PS;
  __shared__ __attribute__((aligned(16))) char s_mem[lds_bytes<T, DP>(4 * TILE, NW)];
  __shared__ __attribute__((aligned(16))) float s_bias[WIN == 2 ? 2 : 1][WIN == 2 ? BN : 1];
  auto s_k = [&](int buf) { return (bf16_t*)s_mem + buf * TILE; };
  auto s_v = [&](int buf) { return (bf16_t*)s_mem + (2 + buf) * TILE; };

  const int lane = lane_id(), wave = threadIdx.x >> 6, h = lane >> 5;
  const int row_wave = wave / KS, share = wave % KS;
  const int kh = blockIdx.x % a.kv_heads;
  const int split = (blockIdx.x / a.kv_heads) % a.splits;
  int b;
  const int64_t tile = tile_of<WIN != 0>(a.qo, a.batch, a.nq, a.group, BM, blockIdx.x / (a.kv_heads * a.splits), b);
  int64_t q0, q1, k0, k1;
  seq_rows(a.qo, b, a.nq, q0, q1);
  seq_rows(a.ko, b, a.nk, k0, k1);
  if (WIN && a.kl) k1 = clamp64(k0 + a.kl[b], k0, k1);
  const int64_t rows = (q1 - q0) * a.group;
  if (tile * BM >= rows) return;
  // WIN: the tile's keys as one axis, of which this workgroup takes places x0 .. x0 + keys.
  WindowAxis axis = {};
  const int64_t lq = q1 - q0, lk = k1 - k0;
  int64_t x0 = 0, x1 = 0, i0 = 0;
  WindowTile tile_sees = {};
  if constexpr (WIN) {
    i0 = row_query(tile * BM, a.group);
    axis = window_axis(a.win, i0, row_query(((tile + 1) * BM < rows ? (tile + 1) * BM : rows) - 1, a.group), lq, lk);
    split_axis(axis.keys, a.splits, split, BN, x0, x1);
    tile_sees = window_tile(a.win, axis, x0, i0, lq, lk);
  } else if (a.splits > 1) {
    const int64_t part = ((k1 - k0 + a.splits - 1) / a.splits + BN - 1) / BN * BN;
    k0 = k0 + split * part < k1 ? k0 + split * part : k1;
    k1 = k0 + part < k1 ? k0 + part : k1;
  }
  int keys = WIN ? (int)(x1 - x0) : (int)(k1 - k0);

  Stage<T, BN, DP, NT, VEC> sk, sv;
  sk.start((const T*)a.k + kh * a.ks[1] + k0 * a.ks[0], 0, a.ks[0], 0, 1, a.dim);
  sv.start((const T*)a.v + kh * a.vs[1] + k0 * a.vs[0], 0, a.vs[0], 0, 1, a.dim);
  // Whether key j + lane exists and the mask keeps it. The ballot of these comes a tile later: at once it would wait for
  // the tile's loads too.
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

  // This lane's query rows (one per 32-column tile), and their values as second operands.
  int64_t row[NQ];  // row of out and lse, -1: none
  frag fq[NQ][DP / 16];
  WindowRow see[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t r = tile * BM + (row_wave * NQ + n) * 32 + (lane & 31);
    int64_t qi;
    int head;
    // WIN: rows behind the last one see what it sees.
    split_row(r < rows ? r : WIN ? rows - 1 : 0, a.group, qi, head);
    if constexpr (WIN) see[n] = tile_sees.row((int)(qi - i0));
    qi += q0;
    head += kh * a.group;
    row[n] = r < rows ? qi * a.heads + head : -1;
    const T* p = (const T*)a.q + qi * a.qs[0] + head * a.qs[1];
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      const int d = kk * 16 + h * 8;
      fq[n][kk] = to_parts(load8<T>(p + d, r < rows ? a.dim - d : 0, VEC));
    }
  }
  WindowWave wave_sees;
  if constexpr (WIN) wave_sees.start(see[0], see[NQ - 1]);

  // WIN 2: a masked key's score has to be -infinity whatever the query is, but a bias added to NaN is NaN. Rows that are not
  // finite are walked as zeros, and give NaN in the end if they saw a key.
  bool not_finite[NQ] = {};
  if constexpr (WIN == 2) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      f32x16 nan = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) nan = mma(bf16x8v{}, fq[n][kk].p[0], nan);  // 0 times the row: 0 or NaN
      not_finite[n] = nan[0] != 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
        if (not_finite[n]) fq[n][kk] = frag{};
    }
  }

  // Finite, so that the first reference (-infinity) is passed whatever the scale.
  const float c = a.scale * kLog2e, slack = fminf(kSlack / c, 3.4e38f);
  f32x16 o[NQ][DT];
  float m[NQ], l[NQ];  // references (in the scores' units) and this lane's part of the sums
  float from[NQ];      // what scores are counted from: m, 0 before there is one
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    from[n] = 0.f;
    l[n] = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[n][t] = zero16();
  }

  int buf = 0, j = 0;
  uint64_t bits = kAll;
  // The tile's blocks of 32 keys from t0 on, C of them: scores, softmax and the product with v.
  auto blocks = [&](auto count, int t0) {
    constexpr int C = decltype(count)::value;
    f32x16 s[NQ][C];
#pragma unroll
    for (int t = 0; t < C; ++t) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n][t] = zero16();
      if constexpr (WIN == 2) {
        s[0][t] = from_bias(s_bias[buf] + (t0 + t) * 32);
#pragma unroll
        for (int n = 1; n < NQ; ++n) s[n][t] = s[0][t];
      }
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const frag fk = load_row<T, PS>(s_k(buf) + ((t0 + t) * 32 + (lane & 31)) * LD + kk * 16 + h * 8);
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][t] = mma(fk, fq[n][kk], s[n][t]);
      }
    }
    if (WIN && !wave_sees.all(j + 32 * t0, 32 * C)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int t = 0; t < C; ++t) clear_unseen(s[n][t], see[n], wave_sees, j + 32 * (t0 + t), -INFINITY);
    } else if (!WIN && bits != kAll) {
#pragma unroll
      for (int t = 0; t < C; ++t) {
        const uint32_t w = (uint32_t)(bits >> (32 * t)) >> (4 * h);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool keep = w & (1u << (8 * (r >> 2) + (r & 3)));
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][t][r] = keep ? s[n][t][r] : -INFINITY;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = max16(s[n][0]);
#pragma unroll
      for (int t = 1; t < C; ++t) top = fmaxf(top, max16(s[n][t]));
      const float m_new = fmaxf(m[n], halves_max(top));
      if (__any(m_new > m[n] + slack)) {
        asm volatile("");  // a branch: the compiler would multiply always and select
        const float f = m[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[n] - m_new) * c);
        l[n] *= f;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[n][t][r] *= f;
        m[n] = m_new;
        if constexpr (WIN) from[n] = m_new == -INFINITY ? 0.f : m_new;
      }
      const float base = WIN ? from[n] : m[n] == -INFINITY ? 0.f : m[n];
#pragma unroll
      for (int t = 0; t < C; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          // bf16 data: one instruction. fp32: the difference first, which is exact near the reference.
          s[n][t][r] = __builtin_amdgcn_exp2f(sizeof(T) == 2 ? fmaf(s[n][t][r], c, -base * c) : (s[n][t][r] - base) * c);
          l[n] += s[n][t][r];
        }
    }
#pragma unroll
    for (int t = 0; t < C; ++t)
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        // bf16 data: p rounded once, since the matrix cores take bf16. out is then off by 1.26 to 1.39 times what its own
        // rounding costs (30 to 1,500 keys, heads of 64, rms against 64 bits). In two parts it is off by 1.00, but a second
        // product and the remainders cost 30 to 33% (215,003 x 5 x ~1024, 4 heads of 64: 291 and 382 us; 60,000 x 1,500, 256
        // channels, heads of 32, 64 and 128: 167 and 222, 125 and 165, 118 and 154). With windows, whose
        // rows end in few roundings besides, p has two parts: out is off by 1.00 (rounded once 1.20 to 1.41), for 7 to 22% (us,
        // once and in two parts: 200,003 rows, 256 to either side, 4 heads of 64, 225 and 273; 100,003 rows, 64 to either side, 4
        // heads of 128, 126 and 138; 30,001 rows, 1,023 before, 8 heads of 32, 84 and 100).
        constexpr bool kTwo = WIN != 0 && sizeof(T) == 2;
        frag p[NQ], lo[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          if constexpr (kTwo) to_frag2<T>(s[n][t], mm, p[n], lo[n]);
          else p[n] = to_frag<T>(s[n][t], mm);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const frag fv = load_tr<T, LD, PS>(s_v(buf), (t0 + t) * 32 + mm * 16, d * 32);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            if constexpr (kTwo) o[n][d] = mma(fv, lo[n], o[n][d]);
            o[n][d] = mma(fv, p[n], o[n][d]);
          }
        }
      }
  };
  for (; j < keys; j += BN, buf ^= 1) {
    if constexpr (WIN != 1) bits = __ballot(next_ok != 0);
    if (WIN != 1 && a.mask) {  // what a masked place holds must not meet a zero probability
      sk.template store<LD, PS>(s_k(buf), bits);
      sv.template store<LD, PS>(s_v(buf), bits);
      if (WIN == 2 && wave == 0 && lane < BN) s_bias[buf][lane] = next_ok ? 0.f : -INFINITY;
    } else {
      sk.template store<LD, PS>(s_k(buf));
      sv.template store<LD, PS>(s_v(buf));
    }
    if (j + BN < keys) next_ok = fetch(j + BN);
    // Two buffers: the barrier of the last tile already had every wave past reading this one.
    __syncthreads();
    if constexpr (!WIN) {
      blocks(std::integral_constant<int, KT>{}, 0);
    } else {
#pragma unroll 1
      for (int t = share; t < KT; t += KS)
        if (!wave_sees.none(j + 32 * t, 32)) blocks(std::integral_constant<int, 1>{}, t);
    }
  }

  __syncthreads();  // every wave is past reading the tiles: their space takes the results
  if constexpr (KS > 1) {
    float* const s = (float*)(s_mem + row_wave * handover_bytes<DT>(2));
    float* const s_ml = s + DT * 16 * 64 + lane;
    if (share == 1) {
      hand_over(s, o[0]);
      s_ml[0] = m[0], s_ml[64] = l[0];
    }
    __syncthreads();
    if (share == 0) {
      // Two references, counted from 0 where there is none: its results are then 0.
      const float m1 = s_ml[0], top = fmaxf(m[0], m1), base = top == -INFINITY ? 0.f : top;
      const float f = __builtin_amdgcn_exp2f((m[0] - base) * c), g = __builtin_amdgcn_exp2f((m1 - base) * c);
      l[0] = fmaf(s_ml[64], g, l[0] * f);
      take_over(s, o[0], f, g);
      m[0] = top;
    }
    __syncthreads();
    if (share == 1) return;
  }
  void* const s_out = s_mem + row_wave * (32 * (DP + 4) * 4);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float total = l[n] + __shfl_xor(l[n], 32, 64);
    if (WIN == 2 && not_finite[n] && total > 0.f) total = NAN;
    if (a.splits > 1) {
      const int64_t first = (int64_t)split * a.nq * a.heads;
      store_tile<float, DP>(a.part_a + first * a.dim, s_out, o[n], 1.f, row[n], a.dim, a.dim % 4 == 0);
      if (row[n] >= 0 && h == 0) {
        a.part_b[(first + row[n]) * 2] = m[n] * c;
        a.part_b[(first + row[n]) * 2 + 1] = total;
      }
    } else {
      const float f = total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;
      store_tile<T, DP>((T*)a.out, s_out, o[n], f, row[n], a.dim, a.ovec);
      if (row[n] >= 0 && h == 0) a.lse[row[n]] = total == 0.f ? -INFINITY : kLn2 * (m[n] * c + log2f(total));
    }
  }
}

// Few query rows per sequence and key head (single tokens): reading K and V once is all the time, and a
// matrix tile would be mostly empty rows and its waves would wait on barriers. LPK lanes hold one key, 8
// channels each, with a share of U keys in flight and as many being worked on; every group of LPK lanes keeps
// its own running maximum, sum and output over its keys, and they are joined at the end (lanes, waves, then
// k_attn_join for the parts of the key axis).
template <typename T, int LPK, int R, bool VEC, bool WIN>
__global__ __launch_bounds__(kNT) void k_attn_few(AttnArgs a) {
  typedef typename Raw8<T>::type frag;
  constexpr int U = 4, KPW = 64 / LPK, STEP = 4 * KPW * U;  // keys of a wave's round: KPW * U; STEP: see few_keys
  __shared__ float s_o[4][R][LPK * 8 + 2];

  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int g = lane / LPK, d = (lane % LPK) * 8;
  const int kh = blockIdx.x % a.kv_heads;
  const int split = (blockIdx.x / a.kv_heads) % a.splits;
  int b;
  const int64_t tile = tile_of<WIN != 0>(a.qo, a.batch, a.nq, a.group, R, blockIdx.x / (a.kv_heads * a.splits), b);
  int64_t q0, q1, k0, k1;
  seq_rows(a.qo, b, a.nq, q0, q1);
  seq_rows(a.ko, b, a.nk, k0, k1);
  if (WIN && a.kl) k1 = clamp64(k0 + a.kl[b], k0, k1);
  const int64_t rows = (q1 - q0) * a.group;
  if (tile * R >= rows) return;
  WindowAxis axis = {};  // as in k_attn_fwd
  const int64_t lq = q1 - q0, lk = k1 - k0;
  int64_t x0 = 0, x1 = 0, i0 = 0;
  WindowTile tile_sees = {};
  if constexpr (WIN) {
    i0 = row_query(tile * R, a.group);
    axis = window_axis(a.win, i0, row_query(((tile + 1) * R < rows ? (tile + 1) * R : rows) - 1, a.group), lq, lk);
    split_axis(axis.keys, a.splits, split, 1, x0, x1);
    tile_sees = window_tile(a.win, axis, x0, i0, lq, lk);
  } else if (a.splits > 1) {
    const int64_t part = (k1 - k0 + a.splits - 1) / a.splits;
    k0 = k0 + split * part < k1 ? k0 + split * part : k1;
    k1 = k0 + part < k1 ? k0 + part : k1;
  }
  const int keys = WIN ? (int)(x1 - x0) : (int)(k1 - k0);
  const T* kp = (const T*)a.k + kh * a.ks[1] + k0 * a.ks[0] + d;
  const T* vp = (const T*)a.v + kh * a.vs[1] + k0 * a.vs[0] + d;
  frag fk[U], fv[U];
  uint32_t ok = 0;
  auto fetch = [&](int j) {
    ok = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = j + u * KPW + g;
      int64_t key = x;
      if constexpr (WIN) key = axis.key(x0 + x);
      const bool in = x < keys && (!a.mask || a.mask[k0 + key]);
      fk[u] = load8<T>(kp + key * a.ks[0], in ? a.dim - d : 0, VEC);
      fv[u] = load8<T>(vp + key * a.vs[0], in ? a.dim - d : 0, VEC);
      ok |= (in ? 1u : 0u) << u;
    }
  };
  fetch(wave * KPW * U);

  float q[R][8], o[R][8], m[R], l[R];
  WindowRow see[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t x = tile * R + r;
    int64_t qi;
    int head;
    split_row(x < rows ? x : WIN ? rows - 1 : 0, a.group, qi, head);
    if constexpr (WIN) see[r] = tile_sees.row((int)(qi - i0));
    const frag f = load8<T>((const T*)a.q + (q0 + qi) * a.qs[0] + (kh * a.group + head) * a.qs[1] + d,
                            x < rows ? a.dim - d : 0, VEC);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[r][i] = (float)f[i] * (a.scale * kLog2e);
      o[r][i] = 0.f;
    }
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  for (int j = wave * KPW * U; j < keys; j += STEP) {
    float k[U][8], v[U][8];
    const uint32_t now = ok;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) k[u][i] = (float)fk[u][i], v[u][i] = (float)fv[u][i];
    if (j + STEP < keys) fetch(j + STEP);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s[U], top = m[r];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[u] = fmaf(q[r][i], k[u][i], s[u]);
        s[u] = lanes_sum<LPK>(s[u]);
        bool keep = now >> u & 1;
        if constexpr (WIN) {
          const int x = j + u * KPW + g;
          keep = keep && (x < see[r].first || (x >= see[r].low && x < see[r].high));
        }
        s[u] = keep ? s[u] : -INFINITY;
        top = fmaxf(top, s[u]);
      }
      const float base = top == -INFINITY ? 0.f : top;
      const float f = __builtin_amdgcn_exp2f(m[r] - base);
      m[r] = top;
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[r][i] *= f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float p = __builtin_amdgcn_exp2f(s[u] - base);
        l[r] += p;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[r][i] = fmaf(p, v[u][i], o[r][i]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float top = m[r];
#pragma unroll
    for (int x = LPK; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
    const float f = __builtin_amdgcn_exp2f(m[r] - (top == -INFINITY ? 0.f : top));
    l[r] *= f;
#pragma unroll
    for (int x = LPK; x < 64; x <<= 1) l[r] += __shfl_xor(l[r], x, 64);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[r][i] *= f;
#pragma unroll
      for (int x = LPK; x < 64; x <<= 1) o[r][i] += __shfl_xor(o[r][i], x, 64);
      if (g == 0) s_o[wave][r][d + i] = o[r][i];
    }
    if (lane == 0) s_o[wave][r][LPK * 8] = top, s_o[wave][r][LPK * 8 + 1] = l[r];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R * LPK * 8; e += kNT) {
    const int r = e / (LPK * 8), c = e % (LPK * 8);
    const int64_t x = tile * R + r;
    if (x >= rows || c >= a.dim) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, s_o[w][r][LPK * 8]);
    float total = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_o[w][r][LPK * 8] - (top == -INFINITY ? 0.f : top));
      total += f * s_o[w][r][LPK * 8 + 1];
      sum += f * s_o[w][r][c];
    }
    int64_t qi;
    int head;
    split_row(x, a.group, qi, head);
    const int64_t row = (q0 + qi) * a.heads + kh * a.group + head;
    if (a.splits > 1) {
      const int64_t at = (int64_t)split * a.nq * a.heads + row;
      a.part_a[at * a.dim + c] = sum;
      if (c == 0) a.part_b[at * 2] = top, a.part_b[at * 2 + 1] = total;
    } else {
      const float f = total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;
      ((T*)a.out)[row * a.dim + c] = (T)(sum * f);
      if (c == 0) a.lse[row] = total == 0.f ? -INFINITY : kLn2 * (top + log2f(total));
    }
  }
}

constexpr int kMaxParts = 128;
// Rows from which on a wave joins each (k_attn_join_rows), if it has up to eight parts, instead of a workgroup: 18,002 rows of 2
// parts 8 us instead of 18; 512 rows of 4 parts 0.5 us slower, 2,400 rows of 32 parts 4.
constexpr int64_t kJoinRows = 1024;

// Joins the parts of a split key axis, one workgroup per row of a sequence: a lane per part weighs it, then the waves
// share the parts and the lanes the channels.
template <typename T>
__global__ __launch_bounds__(kNT) void k_attn_join(AttnArgs a) {
  __shared__ float s_w[kMaxParts], s_o[4][kAttnMaxDim];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int64_t rows = a.nq * a.heads, row = blockIdx.x;
  int64_t q0, q1;
  covered_rows(a.qo, a.batch, a.nq, q0, q1);
  if (row < q0 * a.heads || row >= q1 * a.heads) return;
  float m[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int part = lane + 64 * i;
    const float2 ml = part < a.splits ? ((const float2*)a.part_b)[part * rows + row] : make_float2(-INFINITY, 0.f);
    m[i] = ml.x;
    l[i] = ml.y;
  }
  const float top = lanes_reduce<64>(fmaxf(m[0], m[1]), [](float x, float y) { return fmaxf(x, y); });
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float w = __builtin_amdgcn_exp2f(m[i] - base);
    total += w * l[i];
    if (wave == 0) s_w[lane + 64 * i] = w;
  }
  total = lanes_sum<64>(total);
  __syncthreads();
  const float* po = a.part_a + row * a.dim;
  float o0 = 0.f, o1 = 0.f;
#pragma unroll 8
  for (int part = wave; part < a.splits; part += 4) {
    const float* p = po + part * rows * a.dim;
    if (lane < a.dim) o0 += s_w[part] * p[lane];
    if (lane + 64 < a.dim) o1 += s_w[part] * p[lane + 64];
  }
  s_o[wave][lane] = o0;
  s_o[wave][lane + 64] = o1;
  __syncthreads();
  const float f = total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;
  for (int c = threadIdx.x; c < a.dim; c += kNT)
    ((T*)a.out)[row * a.dim + c] = (T)(((s_o[0][c] + s_o[1][c]) + (s_o[2][c] + s_o[3][c])) * f);
  if (threadIdx.x == 0) a.lse[row] = total == 0.f ? -INFINITY : kLn2 * (top + log2f(total));
}

template <typename T, int DP>
struct FwdShape;  // NQ, BN
template <int DP>
struct FwdShape<bf16_t, DP> {
  static constexpr int NQ = DP <= 64 ? 2 : 1, BN = 64, WPE = DP <= 32 ? 3 : 2;
};
template <int DP>
struct FwdShape<float, DP> {
  static constexpr int NQ = 1, BN = 32, WPE = DP <= 64 ? 2 : 1;
};

// Shapes of window attention: 32 NQ rows of a wave, keys of a tile, waves per SIMD, waves of a workgroup (chosen with p rounded once, as the
// figures are). Other than without windows, where heads of 64 do best with two tiles of rows a wave and two waves per SIMD: a wave's rows see few keys each and
// more of them beside its own rows' windows, so one tile of rows and more waves do better. us, bf16, heads of 64, windows of 256
// to either side over 200,003 rows / 64 over 200,003 / 2,047 before over 60,000, 4 heads: (1, 32, 4, 4) 207, 108, 186; (1, 64, 3,
// 4) 228, 108, 196; (2, 64, 2, 4) 273, 149, 199; (2, 32, 2, 2) 240, 126, 207; (1, 32, 4, 2) 304, 138, 265. Heads of 32, 256 to
// either side, 8 heads: (1, 64, 3, 4) 292, (1, 64, 2, 4) 298, (2, 64, 3, 4) 334. fp32, 50,003 rows, 4 heads, 256 to either side, heads
// of 32 and the small case of 7,131 rows, 64 to either side: (1, 32, 2, 2) 123 and 14.1, (1, 32, 3, 4) 119 and 17.5; heads of 64: (1,
// 32, 3, 4) 205, (1, 32, 2, 4) 213, (1, 32, 2, 2) 309.
template <int Q, int N, int E, int W, int S = 1>
struct Shape {
  static constexpr int NQ = Q, BN = N, WPE = E, NW = W, KS = S, kRows = 32 * Q * W / S;
};
template <typename T, int DP>
struct WinShape : Shape<1, 32, 1, 4> {};
template <int DP>
struct WinShape<bf16_t, DP> : Shape<1, 64, 2, 4> {};
template <>
struct WinShape<bf16_t, 32> : Shape<1, 64, 3, 4> {};
template <>
struct WinShape<bf16_t, 64> : Shape<1, 32, 4, 4> {};
template <>
struct WinShape<float, 32> : Shape<1, 32, 2, 2> {};
template <>
struct WinShape<float, 64> : Shape<1, 32, 3, 4> {};
// The same where rows are few (see window_few): a key axis shared by two waves. Heads over 64 in fp32 have no room for its tiles.
template <typename T, int DP>
struct WinFewShape : Shape<1, 64, 2, 4, 2> {};
template <>
struct WinFewShape<float, 64> : Shape<1, 64, 1, 4, 2> {};
template <>
struct WinFewShape<float, 96> : WinShape<float, 96> {};
template <>
struct WinFewShape<float, 128> : WinShape<float, 128> {};
typedef Shape<1, 64, 2, 8, 2> WinMidShape;  // of fp32 heads of 64
template <typename T>
int win_rows(int dim, int few) {
  if (few == 2) return WinMidShape::kRows;
  auto rows = [&](auto s, auto f) { return few ? f.kRows : s.kRows; };
  return dim <= 32   ? rows(WinShape<T, 32>{}, WinFewShape<T, 32>{})
         : dim <= 64 ? rows(WinShape<T, 64>{}, WinFewShape<T, 64>{})
         : dim <= 96 ? rows(WinShape<T, 96>{}, WinFewShape<T, 96>{})
                     : rows(WinShape<T, 128>{}, WinFewShape<T, 128>{});
}

constexpr int kFewRows = 4;
// Keys that a workgroup of k_attn_few takes in a round.
constexpr int few_keys(int dim) { return 1024 / (dim <= 32 ? 4 : dim <= 64 ? 8 : 16); }

// Query rows of a tile: a few (k_attn_few) or those of the matrix kernel. Decided from the average number of rows
// that share a key head in a sequence; either kernel takes any number of rows. The whole batch takes one form: a sequence of
// many rows among empty ones runs through tiles of a few, its keys read again for each. us a call, few / matrix, with 1, 2
// and 4 rows:
//                                bf16                                    fp32
//   64 x 4096 keys, 8 heads
//     of 32                      88 / 123   93 / 123   104 / 124         118 / 209   121 / 210   128 / 211
//     of 64                      117 / 151  120 / 151  129 / 152         195 / 336   199 / 339   204 / 344
//     of 128                     199 / 193  202 / 193  217 / 193         382 / 728   386 / 729   393 / 730
//   100,000 keys, 8 heads
//     of 32                      49 / 59    54 / 59    60 / 60           59 / 83     61 / 83     69 / 84
//     of 64                      60 / 71    63 / 72    70 / 72           88 / 136    91 / 137    95 / 138
//     of 128                     102 / 93   100 / 94   106 / 94          164 / 303   164 / 302   165 / 301
//   32 x 2048 keys, 2 heads
//     of 32                      20 / 19    24 / 19    30 / 19           21 / 24     23 / 24     30 / 24
//     of 64                      20 / 21    24 / 21    32 / 21           23 / 31     26 / 31     33 / 31
//     of 128                     25 / 24    29 / 24    37 / 24           33 / 64     35 / 64     42 / 65
// So a few rows take k_attn_few, but for bf16 heads over 64, where the matrix kernel is ahead throughout. What the rule
// gives away is up to 11 us a call on small problems, bf16 in the main, whose parts of 256 keys leave the GPU half empty.
// 8 rows of bf16, 64 x 4096 keys, 8 heads of 64: 184 / 101.
int fwd_rows(int dtype, int dim, int64_t nq, int batch, int group, int kv_heads, bool windowed) {
  const int64_t rows = (nq + batch - 1) / batch * group;
  if (dtype == IGC_F32 || dim <= 64) {
    for (int r = 1; r <= kFewRows; r *= 2)
      if (rows <= r) return r;
  }
  if (windowed) {
    const int few = window_few(dtype, dim, (nq + batch - 1) / batch * group, batch, kv_heads);
    return dtype == IGC_BF16 ? win_rows<bf16_t>(dim, few) : win_rows<float>(dim, few);
  }
  return dtype == IGC_BF16 && dim <= 64 ? 256 : 128;
}

// The same, a wave for each row: for many rows, whose parts are few. Sums in k_attn_join's order, so the same bits.
template <typename T>
__global__ __launch_bounds__(kNT) void k_attn_join_rows(AttnArgs a) {
  const int lane = lane_id();
  const int64_t rows = a.nq * a.heads, row = (int64_t)blockIdx.x * (kNT / 64) + (threadIdx.x >> 6);
  int64_t q0, q1;
  covered_rows(a.qo, a.batch, a.nq, q0, q1);
  if (row < q0 * a.heads || row >= q1 * a.heads) return;
  float m[2], l[2], w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int part = lane + 64 * i;
    const float2 ml = part < a.splits ? ((const float2*)a.part_b)[part * rows + row] : make_float2(-INFINITY, 0.f);
    m[i] = ml.x;
    l[i] = ml.y;
  }
  const float top = lanes_reduce<64>(fmaxf(m[0], m[1]), [](float x, float y) { return fmaxf(x, y); });
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __builtin_amdgcn_exp2f(m[i] - base);
    total += w[i] * l[i];
  }
  total = lanes_sum<64>(total);
  const float* po = a.part_a + row * a.dim;
  float o[4][2] = {};
  for (int first = 0; first < a.splits; first += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int part = first + i;
      if (part >= a.splits) break;
      const float x = __shfl(part < 64 ? w[0] : w[1], part & 63, 64);
      const float* p = po + part * rows * a.dim;
      if (lane < a.dim) o[i][0] += x * p[lane];
      if (lane + 64 < a.dim) o[i][1] += x * p[lane + 64];
    }
  }
  const float f = total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64 * i < a.dim) ((T*)a.out)[row * a.dim + lane + 64 * i] = (T)(((o[0][i] + o[1][i]) + (o[2][i] + o[3][i])) * f);
  if (lane == 0) a.lse[row] = total == 0.f ? -INFINITY : kLn2 * (top + log2f(total));
}

template <typename T>
void join(const AttnArgs& a, hipStream_t s) {
  if (a.splits == 1) return;
  const int64_t rows = a.nq * a.heads;
  if (rows > kJoinRows && a.splits <= 8) k_attn_join_rows<T><<<(unsigned)((rows + kNT / 64 - 1) / (kNT / 64)), kNT, 0, s>>>(a);
  else k_attn_join<T><<<(unsigned)rows, kNT, 0, s>>>(a);
}

template <typename T, int DP, typename W>
void win_go(const AttnArgs& a, unsigned wgs, bool vec, hipStream_t s) {
  if (a.mask) {
    if (vec) k_attn_fwd<T, DP, W::NQ, W::BN, W::WPE, true, 2, W::NW, W::KS><<<wgs, 64 * W::NW, 0, s>>>(a);
    else k_attn_fwd<T, DP, W::NQ, W::BN, W::WPE, false, 2, W::NW, W::KS><<<wgs, 64 * W::NW, 0, s>>>(a);
  } else {
    if (vec) k_attn_fwd<T, DP, W::NQ, W::BN, W::WPE, true, 1, W::NW, W::KS><<<wgs, 64 * W::NW, 0, s>>>(a);
    else k_attn_fwd<T, DP, W::NQ, W::BN, W::WPE, false, 1, W::NW, W::KS><<<wgs, 64 * W::NW, 0, s>>>(a);
  }
}

template <typename T, int DP>
void fwd_go(const AttnArgs& a, unsigned wgs, hipStream_t s) {
  typedef FwdShape<T, DP> F;
  const bool vec = a.qvec && a.kvec;
  if (!a.windowed) {
    if (vec) k_attn_fwd<T, DP, F::NQ, F::BN, F::WPE, true, 0, 4, 1><<<wgs, kNT, 0, s>>>(a);
    else k_attn_fwd<T, DP, F::NQ, F::BN, F::WPE, false, 0, 4, 1><<<wgs, kNT, 0, s>>>(a);
    return;
  }
  const int few = window_few(sizeof(T) == 2 ? IGC_BF16 : IGC_F32, a.dim, (a.nq + a.batch - 1) / a.batch * a.group, a.batch, a.kv_heads);
  if constexpr (sizeof(T) == 4 && DP == 64) {
    if (few == 2) return win_go<T, DP, WinMidShape>(a, wgs, vec, s);
  }
  if (few) win_go<T, DP, WinFewShape<T, DP>>(a, wgs, vec, s);
  else win_go<T, DP, WinShape<T, DP>>(a, wgs, vec, s);
}

template <typename T, int LPK, int R>
void few_go(const AttnArgs& a, unsigned wgs, hipStream_t s) {
  const bool vec = a.qvec && a.kvec;
  if (a.windowed) {
    if (vec) k_attn_few<T, LPK, R, true, true><<<wgs, kNT, 0, s>>>(a);
    else k_attn_few<T, LPK, R, false, true><<<wgs, kNT, 0, s>>>(a);
  } else {
    if (vec) k_attn_few<T, LPK, R, true, false><<<wgs, kNT, 0, s>>>(a);
    else k_attn_few<T, LPK, R, false, false><<<wgs, kNT, 0, s>>>(a);
  }
}
template <typename T, int LPK>
void few_r(const AttnArgs& a, int rows, unsigned wgs, hipStream_t s) {
  if (rows == 1) return few_go<T, LPK, 1>(a, wgs, s);
  if (rows == 2) return few_go<T, LPK, 2>(a, wgs, s);
  few_go<T, LPK, 4>(a, wgs, s);
}

template <typename T>
void fwd_t(const AttnArgs& a, int dtype, hipStream_t s) {
  const int rows = fwd_rows(dtype, a.dim, a.nq, a.batch, a.group, a.kv_heads, a.windowed);
  const unsigned wgs = (unsigned)((a.nq * a.group / rows + a.batch) * a.kv_heads * a.splits);
  if (rows <= kFewRows) {
    if (a.dim <= 32) few_r<T, 4>(a, rows, wgs, s);
    else if (a.dim <= 64) few_r<T, 8>(a, rows, wgs, s);
    else if constexpr (sizeof(T) == 4) few_r<T, 16>(a, rows, wgs, s);
  } else {
    if (a.dim <= 32) fwd_go<T, 32>(a, wgs, s);
    else if (a.dim <= 64) fwd_go<T, 64>(a, wgs, s);
    else if (a.dim <= 96) fwd_go<T, 96>(a, wgs, s);
    else fwd_go<T, 128>(a, wgs, s);
  }
  join<T>(a, s);
}

}  // namespace

int attn_fwd_splits(int dtype, const AttnArgs& a) {
  const int64_t nq = a.nq, nk = a.nk;
  const int batch = a.batch, heads = a.heads, kv_heads = a.kv_heads, dim = a.dim;
  // Parts of the key axis: none while the query tiles alone fill the GPU, else enough for that, each of
  // at least 256 keys.
  const int bm = fwd_rows(dtype, dim, nq, batch, heads / kv_heads, kv_heads, a.windowed);
  const int64_t per_seq = (nq + batch - 1) / batch * (heads / kv_heads);
  const int64_t wgs = batch * ((per_seq + bm - 1) / bm) * kv_heads;
  // Workgroups that fill it: two a CU of the matrix kernel, three of its fp32 form for short heads, which is small enough
  // and waits more. 300 queries on 43,217 keys, 256 channels, us with 512 / 768 / 1024: fp32 heads of 32 119 / 112 / 114, of 64
  // 102 / 118 / 111, of 128 125 / 145 / 145; bf16 56 / 58 / 68, 44 / 56 / 57 and 49 / 59 / 60. fp32 heads of 32 at other sizes: 900
  // queries on 8,000 keys, 8 heads, 68 / 65 / 67; 500 on 20,000, 4 heads, 47 / 47 / 48; 100 on 40,000, 8 heads, 48 / 50 / 52;
  // heads of 16, the first three of these sizes: 117 / 104 / 106, 68 / 62 / 63 and 46 / 45 / 45.
  const bool wide = a.windowed && dtype == IGC_F32 && dim > 32;  // one or two workgroups a CU
  const int64_t fill = bm <= kFewRows ? 2048 : wide ? 256 : dtype == IGC_F32 && dim <= 32 ? 768 : 512;
  const int64_t want = wgs >= fill ? 1 : fill / std::max<int64_t>(1, wgs);
  int64_t keys = nk / batch;  // that a tile walks
  if (a.windowed && a.win.left >= 0 && a.win.right >= 0)
    keys = std::min<int64_t>(keys, a.win.left + a.win.right + bm / a.group + a.win.sinks);
  // Single tokens: with a workgroup on every CU, few rounds of the key axis (few_keys) take less time than its parts and their
  // join: up to 8, and 2 more for each row, which costs arithmetic of its own in every round and its part of the join. us whole / in parts for
  // 2,048 workgroups, windows of as many rounds:
  //                            6            10           14           23
  //   256 workgroups, a row, bf16 heads of 64
  //                            20 / 21      31 / 29      40 / 34      63 / 46
  //   the same, fp32 heads of 32, 64 and 128, 12, 10 and 11 rounds: 64 / 53, 55 / 48, 54 / 49
  //   256 workgroups, 4 rows, bf16 heads of 64
  //                            32 / 42      47 / 62      60 / 74      92 / 85
  //   384, 2 rows, bf16 heads of 64, 8 and 16: 39 / 41, 70 / 61; fp32 64 / 60, 119 / 97 (heads of 128 16: 110 / 94, 32: 215 / 164)
  // Over 240 such problems of 256 to 900 workgroups this is 2.4% from the better of both on average (a limit of 2,048 keys 5.0%), and up to
  // 30% with 250 sequences and 2 key heads, where the whole axis stays ahead for longer.
  if (a.windowed && bm <= kFewRows && wgs >= 256 && keys <= (8 + 2 * bm) * few_keys(dim)) return 1;
  // Rows of windows are many, and so is what their parts leave to be joined. Parts of at least 256 / 384 / 1,024 keys, us: 9,001
  // rows of 2 sequences, 2 heads of 64, bf16, 511 keys before: 26 / 19 / 19; 4,000 rows, 1,999 before: 27 / 26 / 32.
  const int64_t least = a.windowed && bm > kFewRows ? kWindowPart : 256;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, kMaxParts), keys / least));
}

int launch_attn_fwd(const AttnArgs& a, int dtype, hipStream_t s) {
  if (dtype == IGC_BF16) fwd_t<bf16_t>(a, dtype, s);
  else fwd_t<float>(a, dtype, s);
  IGC_HIP(hipGetLastError(), a.fn);
  return IGC_OK;
}

}  // namespace igc
