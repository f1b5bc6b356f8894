// Cross attention of voxel (or object) queries to an encoder's states, forward pass.
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

// Four waves of 32 NQ query rows each over tiles of BN keys. A row is a (query, head of the group
// that shares the key head) pair, so few queries with shared key heads still fill a tile.
// splits > 1: each workgroup takes one part of the sequence's keys and leaves an unnormalised result.
template <typename T, int DP, int NQ, int BN, int WPE, bool VEC>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_fwd(AttnArgs a) {
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
  if (a.splits > 1) {
    const int64_t part = ((k1 - k0 + a.splits - 1) / a.splits + BN - 1) / BN * BN;
    k0 = k0 + split * part < k1 ? k0 + split * part : k1;
    k1 = k0 + part < k1 ? k0 + part : k1;
  }
  int keys = (int)(k1 - k0);

  Stage<T, BN, DP, kNT, VEC> sk, sv;
  sk.start((const T*)a.k + kh * a.ks[1] + k0 * a.ks[0], 0, a.ks[0], 0, 1, a.dim);
  sv.start((const T*)a.v + kh * a.vs[1] + k0 * a.vs[0], 0, a.vs[0], 0, 1, a.dim);
  // Whether key j + lane exists and the mask keeps it. The ballot of these comes a tile later: at once it would wait for
  // the tile's loads too.
  auto key_ok = [&](int j) -> int { return lane < BN && j + lane < keys ? (a.mask ? a.mask[k0 + j + lane] : 1) : 0; };
  sk.load(keys);
  sv.load(keys);
  int next_ok = key_ok(0);

  // This lane's query rows (one per 32-column tile), and their values as second operands.
  int64_t row[NQ];  // row of out and lse, -1: none
  frag fq[NQ][DP / 16];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t r = tile * BM + (wave * NQ + n) * 32 + (lane & 31);
    int64_t qi;
    int head;
    split_row(r < rows ? r : 0, a.group, qi, head);
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

  // Finite, so that the first reference (-infinity) is passed whatever the scale.
  const float c = a.scale * kLog2e, slack = fminf(kSlack / c, 3.4e38f);
  f32x16 o[NQ][DT];
  float m[NQ], l[NQ];  // references (in the scores' units) and this lane's part of the sums
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[n][t] = zero16();
  }

  int buf = 0;
  for (int j = 0; j < keys; j += BN, buf ^= 1) {
    const uint64_t bits = __ballot(next_ok != 0);
    if (a.mask) {  // what a masked place holds must not meet a zero probability
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
    // Two buffers: the barrier of the last tile already had every wave past reading this one.
    __syncthreads();
    f32x16 s[NQ][KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n][t] = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const frag fk = load_row<T, PS>(s_k(buf) + (t * 32 + (lane & 31)) * LD + kk * 16 + h * 8);
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][t] = mma(fk, fq[n][kk], s[n][t]);
      }
    }
    if (bits != kAll) {
#pragma unroll
      for (int t = 0; t < KT; ++t) {
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
      for (int t = 1; t < KT; ++t) top = fmaxf(top, max16(s[n][t]));
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
      }
      const float base = m[n] == -INFINITY ? 0.f : m[n];
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          // bf16 data: one instruction. fp32: the difference first, which is exact near the reference.
          s[n][t][r] = __builtin_amdgcn_exp2f(sizeof(T) == 2 ? fmaf(s[n][t][r], c, -base * c) : (s[n][t][r] - base) * c);
          l[n] += s[n][t][r];
        }
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        // bf16 data: p rounded once, since the matrix cores take bf16. out is then off by 1.26 to 1.39 times what its own
        // rounding costs (30 to 1,500 keys, heads of 64, rms against 64 bits). In two parts it is off by 1.00, but a second
        // product and the remainders cost 30 to 33% (215,003 x 5 x ~1024, 4 heads of 64: 291 and 382 us; 60,000 x 1,500, 256
        // channels, heads of 32, 64 and 128: 167 and 222, 125 and 165, 118 and 154).
        frag p[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) p[n] = to_frag<T>(s[n][t], mm);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const frag fv = load_tr<T, LD, PS>(s_v(buf), t * 32 + mm * 16, d * 32);
#pragma unroll
          for (int n = 0; n < NQ; ++n) o[n][d] = mma(fv, p[n], o[n][d]);
        }
      }
  }

  __syncthreads();  // every wave is past reading the tiles: their space takes the results
  void* const s_out = s_mem + wave * (32 * (DP + 4) * 4);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float total = l[n] + __shfl_xor(l[n], 32, 64);
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
template <typename T, int LPK, int R, bool VEC>
__global__ __launch_bounds__(kNT) void k_attn_few(AttnArgs a) {
  typedef typename Raw8<T>::type frag;
  constexpr int U = 4, KPW = 64 / LPK, STEP = 4 * KPW * U;  // keys of a wave's round: KPW * U
  __shared__ float s_o[4][R][LPK * 8 + 2];

  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int g = lane / LPK, d = (lane % LPK) * 8;
  const int kh = blockIdx.x % a.kv_heads;
  const int split = (blockIdx.x / a.kv_heads) % a.splits;
  int b;
  const int64_t tile = find_tile(a.qo, a.batch, a.nq, a.group, R, blockIdx.x / (a.kv_heads * a.splits), b);
  int64_t q0, q1, k0, k1;
  seq_rows(a.qo, b, a.nq, q0, q1);
  seq_rows(a.ko, b, a.nk, k0, k1);
  const int64_t rows = (q1 - q0) * a.group;
  if (tile * R >= rows) return;
  if (a.splits > 1) {
    const int64_t part = (k1 - k0 + a.splits - 1) / a.splits;
    k0 = k0 + split * part < k1 ? k0 + split * part : k1;
    k1 = k0 + part < k1 ? k0 + part : k1;
  }
  const int keys = (int)(k1 - k0);
  const T* kp = (const T*)a.k + kh * a.ks[1] + k0 * a.ks[0] + d;
  const T* vp = (const T*)a.v + kh * a.vs[1] + k0 * a.vs[0] + d;
  frag fk[U], fv[U];
  uint32_t ok = 0;
  auto fetch = [&](int j) {
    ok = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = j + u * KPW + g;
      const bool in = x < keys && (!a.mask || a.mask[k0 + x]);
      fk[u] = load8<T>(kp + (int64_t)x * a.ks[0], in ? a.dim - d : 0, VEC);
      fv[u] = load8<T>(vp + (int64_t)x * a.vs[0], in ? a.dim - d : 0, VEC);
      ok |= (in ? 1u : 0u) << u;
    }
  };
  fetch(wave * KPW * U);

  float q[R][8], o[R][8], m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t x = tile * R + r;
    int64_t qi;
    int head;
    split_row(x < rows ? x : 0, a.group, qi, head);
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
        s[u] = now >> u & 1 ? s[u] : -INFINITY;
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

constexpr int kFewRows = 4;

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
int fwd_rows(int dtype, int dim, int64_t nq, int batch, int group) {
  const int64_t rows = (nq + batch - 1) / batch * group;
  if (dtype == IGC_F32 || dim <= 64) {
    for (int r = 1; r <= kFewRows; r *= 2)
      if (rows <= r) return r;
  }
  return dtype == IGC_BF16 && dim <= 64 ? 256 : 128;
}

template <typename T>
void join(const AttnArgs& a, hipStream_t s) {
  if (a.splits > 1) k_attn_join<T><<<(unsigned)(a.nq * a.heads), kNT, 0, s>>>(a);
}

template <typename T, int DP>
void fwd_go(const AttnArgs& a, unsigned wgs, hipStream_t s) {
  constexpr int NQ = FwdShape<T, DP>::NQ, BN = FwdShape<T, DP>::BN, WPE = FwdShape<T, DP>::WPE;
  if (a.qvec && a.kvec) k_attn_fwd<T, DP, NQ, BN, WPE, true><<<wgs, kNT, 0, s>>>(a);
  else k_attn_fwd<T, DP, NQ, BN, WPE, false><<<wgs, kNT, 0, s>>>(a);
}

template <typename T, int LPK, int R>
void few_go(const AttnArgs& a, unsigned wgs, hipStream_t s) {
  if (a.qvec && a.kvec) k_attn_few<T, LPK, R, true><<<wgs, kNT, 0, s>>>(a);
  else k_attn_few<T, LPK, R, false><<<wgs, kNT, 0, s>>>(a);
}
template <typename T, int LPK>
void few_r(const AttnArgs& a, int rows, unsigned wgs, hipStream_t s) {
  if (rows == 1) return few_go<T, LPK, 1>(a, wgs, s);
  if (rows == 2) return few_go<T, LPK, 2>(a, wgs, s);
  few_go<T, LPK, 4>(a, wgs, s);
}

template <typename T>
void fwd_t(const AttnArgs& a, int dtype, hipStream_t s) {
  const int rows = fwd_rows(dtype, a.dim, a.nq, a.batch, a.group);
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

int attn_fwd_splits(int dtype, int64_t nq, int64_t nk, int batch, int heads, int kv_heads, int dim) {
  // Parts of the key axis: none while the query tiles alone fill the GPU, else enough for that, each of
  // at least 256 keys.
  const int bm = fwd_rows(dtype, dim, nq, batch, heads / kv_heads);
  const int64_t per_seq = (nq + batch - 1) / batch * (heads / kv_heads);
  const int64_t wgs = batch * ((per_seq + bm - 1) / bm) * kv_heads;
  // Workgroups that fill it: two a CU of the matrix kernel, three of its fp32 form for short heads, which is small enough
  // and waits more. 300 queries on 43,217 keys, 256 channels, us with 512 / 768 / 1024: fp32 heads of 32 119 / 112 / 114, of 64
  // 102 / 118 / 111, of 128 125 / 145 / 145; bf16 56 / 58 / 68, 44 / 56 / 57 and 49 / 59 / 60. fp32 heads of 32 at other sizes: 900
  // queries on 8,000 keys, 8 heads, 68 / 65 / 67; 500 on 20,000, 4 heads, 47 / 47 / 48; 100 on 40,000, 8 heads, 48 / 50 / 52;
  // heads of 16, the first three of these sizes: 117 / 104 / 106, 68 / 62 / 63 and 46 / 45 / 45.
  const int64_t fill = bm <= kFewRows ? 2048 : dtype == IGC_F32 && dim <= 32 ? 768 : 512;
  const int64_t want = wgs >= fill ? 1 : fill / std::max<int64_t>(1, wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, kMaxParts), nk / batch / 256));
}

int launch_attn_fwd(const AttnArgs& a, int dtype, hipStream_t s) {
  if (dtype == IGC_BF16) fwd_t<bf16_t>(a, dtype, s);
  else fwd_t<float>(a, dtype, s);
  IGC_HIP(hipGetLastError(), a.fn);
  return IGC_OK;
}

}  // namespace igc
