// Cross attention, backward pass.
//
//   p_ij = exp(s_ij - lse_i), delta_i = dout_i . out_i, ds_ij = p_ij (dout_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j
//   dk_j = scale sum_i ds_ij q_i, dv_j = sum_i p_ij dout_i, over the queries of the sequence and the
//          query heads that share the key head
//
// Two kernels, each keeping its output in registers while it walks the other axis: k_attn_dq owns
// query rows and walks keys, k_attn_dkv owns keys and walks query rows, so nothing is added by atomics
// and reruns are bit-identical. Scores are computed again in both (seven products instead of five).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "igc_attn.h"
#include "igc_host.h"

namespace igc {
namespace {

constexpr int kNT = 256;

// lse in base 2; +infinity for rows without keys, whose probabilities are then exp2(-infinity) = 0.
__device__ __forceinline__ float lse_base2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// dq and delta: four waves of 32 query rows over tiles of BN keys (see k_attn_fwd for rows).
template <typename T, int DP, int BN, int WPE, bool VEC>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_dq(AttnArgs a) {
  typedef typename Frag<T>::type frag;
  constexpr int LD = lds_ld<T, DP>();
  constexpr int BM = 128;
  constexpr int KT = BN / 32, DT = DP / 32;
  constexpr uint64_t kAll = BN == 64 ? ~0ull : (1ull << (BN & 63)) - 1;
  __shared__ __attribute__((aligned(16))) T s_k[2][BN * LD];
  __shared__ __attribute__((aligned(16))) T s_v[2][BN * LD];

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

  const int64_t r = tile * BM + wave * 32 + (lane & 31);
  const bool live = r < rows;
  int64_t qi;
  int head;
  split_row(live ? r : 0, a.group, qi, head);
  qi += q0;
  head += kh * a.group;
  const int64_t row = qi * a.heads + head;
  frag fq[DP / 16], fo[DP / 16];
  float delta = 0.f;
  {
    const T* p = (const T*)a.q + qi * a.qs[0] + head * a.qs[1];
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      const int d = kk * 16 + h * 8, have = live ? a.dim - d : 0;
      fq[kk] = load8<T>(p + d, have, VEC);
      fo[kk] = load8<T>((const T*)a.dout + row * a.dim + d, have, VEC);
      const frag f = load8<T>((const T*)a.out_in + row * a.dim + d, have, VEC);
#pragma unroll
      for (int i = 0; i < 8; ++i) delta = fmaf((float)fo[kk][i], (float)f[i], delta);
    }
    delta += __shfl_xor(delta, 32, 64);
    if (live && h == 0 && split == 0) a.delta[row] = delta;
  }
  const float lse = lse_base2(live ? a.lse_in[row] : -INFINITY);
  const float c = a.scale * kLog2e;
  f32x16 dq[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) dq[t] = zero16();

  int keys = (int)(k1 - k0);
  Stage<T, BN, DP, kNT, VEC> sk, sv;
  sk.start((const T*)a.k + kh * a.ks[1] + k0 * a.ks[0], 0, a.ks[0], 0, 1, a.dim);
  sv.start((const T*)a.v + kh * a.vs[1] + k0 * a.vs[0], 0, a.vs[0], 0, 1, a.dim);
  auto key_bits = [&](int j) -> uint64_t {
    bool ok = lane < BN && j + lane < keys;
    if (ok && a.mask) ok = a.mask[k0 + j + lane];
    return __ballot(ok);
  };
  sk.load(keys);
  sv.load(keys);
  uint64_t next_bits = key_bits(0);
  int buf = 0;
  for (int j = 0; j < keys; j += BN, buf ^= 1) {
    const uint64_t bits = next_bits;
    if (a.mask) {
      sk.template store<LD>(s_k[buf], bits);
      sv.template store<LD>(s_v[buf], bits);
    } else {
      sk.template store<LD>(s_k[buf]);
      sv.template store<LD>(s_v[buf]);
    }
    if (j + BN < keys) {
      sk.load(keys - j - BN);
      sv.load(keys - j - BN);
      next_bits = key_bits(j + BN);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const int at = (t * 32 + (lane & 31)) * LD + kk * 16 + h * 8;
        s = mma(load_row<T>(&s_k[buf][at]), fq[kk], s);
        dp = mma(load_row<T>(&s_v[buf][at]), fo[kk], dp);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse)) * (dp[i] - delta);
      if (bits != kAll) {
        const uint32_t w = (uint32_t)(bits >> (32 * t)) >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = w & (1u << (8 * (i >> 2) + (i & 3))) ? s[i] : 0.f;
      }
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        frag f;
        to_frag(s, mm, f);
#pragma unroll
        for (int d = 0; d < DT; ++d) dq[d] = mma(load_tr<LD>(s_k[buf], t * 32 + mm * 16, d * 32), f, dq[d]);
      }
    }
  }
  if (!live || !a.dq) return;
  if (a.splits > 1) {
    float* p = a.part_a + ((int64_t)split * a.nq * a.heads + row) * a.dim;
#pragma unroll
    for (int d = 0; d < DT; ++d) store_col<float>(p, d * 32, a.dim, dq[d], a.scale, a.dim % 4 == 0);
  } else {
#pragma unroll
    for (int d = 0; d < DT; ++d) store_col<T>((T*)a.dq + row * a.dim, d * 32, a.dim, dq[d], a.scale, a.ovec);
  }
}

// dk and dv: four waves of 32 keys each over tiles of BQ query rows of the sequence.
template <typename T, int DP, int BQ, int WPE, bool VEC>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_dkv(AttnArgs a) {
  typedef typename Frag<T>::type frag;
  constexpr int LD = lds_ld<T, DP>();
  constexpr int BM = 128;
  constexpr int QT = BQ / 32, DT = DP / 32;
  __shared__ __attribute__((aligned(16))) T s_q[2][BQ * LD];
  __shared__ __attribute__((aligned(16))) T s_o[2][BQ * LD];
  __shared__ __attribute__((aligned(16))) float s_lse[2][BQ], s_delta[2][BQ];

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

  const int64_t j = k0 + tile * BM + wave * 32 + (lane & 31);
  const bool live = j < k1;
  const bool keep = live && (!a.mask || a.mask[j]);
  frag fk[DP / 16], fv[DP / 16];
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    const int d = kk * 16 + h * 8, have = keep ? a.dim - d : 0;
    fk[kk] = load8<T>((const T*)a.k + (keep ? j : 0) * a.ks[0] + kh * a.ks[1] + d, have, VEC);
    fv[kk] = load8<T>((const T*)a.v + (keep ? j : 0) * a.vs[0] + kh * a.vs[1] + d, have, VEC);
  }
  const float c = a.scale * kLog2e;
  f32x16 dk[DT], dv[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) dk[t] = zero16(), dv[t] = zero16();

  // Rows of the tile at t0 + x; with shared key heads a tile's rows step through the group's heads.
  const int n_rows = (int)(r1 - r0);
  Stage<T, BQ, DP, kNT, VEC> sq, so;
  sq.start((const T*)a.q + q0 * a.qs[0] + kh * a.group * a.qs[1], r0, a.qs[0], a.qs[1], a.group, a.dim);
  so.start((const T*)a.dout + (q0 * a.heads + kh * a.group) * a.dim, r0, (int64_t)a.heads * a.dim, a.dim, a.group, a.dim);
  float n_lse = 0.f, n_delta = 0.f;
  auto fetch = [&](int t0) {
    sq.load(n_rows - t0);
    so.load(n_rows - t0);
    if (threadIdx.x < BQ) {
      n_lse = INFINITY;
      n_delta = 0.f;
      if (t0 + (int)threadIdx.x < n_rows) {
        int64_t qi;
        int g;
        split_row(r0 + t0 + threadIdx.x, a.group, qi, g);
        const int64_t at = (q0 + qi) * a.heads + kh * a.group + g;
        n_lse = lse_base2(a.lse_in[at]);
        n_delta = a.delta[at];
      }
    }
  };
  if (n_rows > 0) fetch(0);
  int buf = 0;
  for (int t0 = 0; t0 < n_rows; t0 += BQ, buf ^= 1) {
    sq.template store<LD>(s_q[buf]);
    so.template store<LD>(s_o[buf]);
    if (threadIdx.x < BQ) s_lse[buf][threadIdx.x] = n_lse, s_delta[buf][threadIdx.x] = n_delta;
    if (t0 + BQ < n_rows) fetch(t0 + BQ);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const int at = (t * 32 + (lane & 31)) * LD + kk * 16 + h * 8;
        s = mma(load_row<T>(&s_q[buf][at]), fk[kk], s);
        dp = mma(load_row<T>(&s_o[buf][at]), fv[kk], dp);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4v lse = *(const f32x4v*)&s_lse[buf][t * 32 + 8 * g + 4 * h];
        const f32x4v delta = *(const f32x4v*)&s_delta[buf][t * 32 + 8 * g + 4 * h];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = keep ? __builtin_amdgcn_exp2f(fmaf(s[4 * g + i], c, -lse[i])) : 0.f;
          dp[4 * g + i] = p * (dp[4 * g + i] - delta[i]);
          s[4 * g + i] = p;
        }
      }
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        frag fp, fs;
        to_frag(s, mm, fp);
        to_frag(dp, mm, fs);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          dv[d] = mma(load_tr<LD>(s_o[buf], t * 32 + mm * 16, d * 32), fp, dv[d]);
          dk[d] = mma(load_tr<LD>(s_q[buf], t * 32 + mm * 16, d * 32), fs, dk[d]);
        }
      }
    }
  }
  if (!live) return;
  const int64_t row = j * a.kv_heads + kh;
  if (a.splits > 1) {
    const int64_t at = ((int64_t)split * a.nk * a.kv_heads + row) * a.dim;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      store_col<float>(a.part_a + at, d * 32, a.dim, dk[d], a.scale, a.dim % 4 == 0);
      store_col<float>(a.part_b + at, d * 32, a.dim, dv[d], 1.f, a.dim % 4 == 0);
    }
  } else {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      store_col<T>((T*)a.dk + row * a.dim, d * 32, a.dim, dk[d], a.scale, a.ovec);
      store_col<T>((T*)a.dv + row * a.dim, d * 32, a.dim, dv[d], 1.f, a.ovec);
    }
  }
}

// out[e] = sum over splits of part[split][e], in order.
template <typename T>
__global__ __launch_bounds__(kNT) void k_attn_sum(const float* __restrict__ part, int splits, int64_t n,
                                                  T* __restrict__ out) {
  for (int64_t e = (int64_t)blockIdx.x * kNT + threadIdx.x; e < n; e += (int64_t)gridDim.x * kNT) {
    float t = 0.f;
    for (int s = 0; s < splits; ++s) t += part[(int64_t)s * n + e];
    out[e] = (T)t;
  }
}

template <typename T>
void sum_go(const float* part, int splits, int64_t n, void* out, hipStream_t s) {
  k_attn_sum<T><<<(unsigned)std::min<int64_t>((n + kNT - 1) / kNT, 8192), kNT, 0, s>>>(part, splits, n, (T*)out);
}

template <typename T, int DP>
void bwd_go(AttnArgs a, const AttnBwdPlan& p, float* ws, hipStream_t s) {
  constexpr int B = sizeof(T) == 2 ? 64 : 32, W = DP <= 64 ? 2 : 1;
  const bool vec = a.qvec && a.kvec && a.ovec;
  a.delta = ws;
  ws += (a.nq * a.heads + 63) / 64 * 64;
  if (a.nq > 0) {
    AttnArgs d = a;
    d.splits = a.dq ? p.dq_splits : 1;
    d.part_a = ws;
    const unsigned wgs = (unsigned)((a.nq * a.group / 128 + a.batch) * a.kv_heads * d.splits);
    if (vec) k_attn_dq<T, DP, B, W, true><<<wgs, kNT, 0, s>>>(d);
    else k_attn_dq<T, DP, B, W, false><<<wgs, kNT, 0, s>>>(d);
    if (a.dq && d.splits > 1) sum_go<T>(ws, d.splits, a.nq * a.heads * a.dim, a.dq, s);
  }
  if (a.dk && a.nk > 0) {
    const int64_t n = a.nk * a.kv_heads * a.dim;
    a.splits = p.dkv_splits;
    a.part_a = ws;
    a.part_b = ws + (p.dkv_splits > 1 ? p.dkv_splits * n : 0);
    const unsigned wgs = (unsigned)((a.nk / 128 + a.batch) * a.kv_heads * a.splits);
    if (vec) k_attn_dkv<T, DP, B, W, true><<<wgs, kNT, 0, s>>>(a);
    else k_attn_dkv<T, DP, B, W, false><<<wgs, kNT, 0, s>>>(a);
    if (a.splits > 1) {
      sum_go<T>(a.part_a, a.splits, n, a.dk, s);
      sum_go<T>(a.part_b, a.splits, n, a.dv, s);
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

int parts(int64_t wgs, int64_t axis) {
  const int64_t want = wgs >= 512 ? 1 : 512 / std::max<int64_t>(1, wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 128), axis / 256));
}

}  // namespace

AttnBwdPlan attn_bwd_plan(int64_t nq, int64_t nk, int batch, int heads, int kv_heads, int dim) {
  AttnBwdPlan p;
  const int64_t rows = (nq / batch) * (heads / kv_heads), keys = nk / batch;
  p.dq_splits = parts(batch * ((rows + 127) / 128) * kv_heads, keys);
  p.dkv_splits = parts(batch * ((keys + 127) / 128) * kv_heads, rows);
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
