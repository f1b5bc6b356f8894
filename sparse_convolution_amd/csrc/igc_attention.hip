// Cross attention of voxel (or object) queries to an encoder's states, forward pass.
//
//   s_ij = scale q_i . k_j over the keys j of the query's sequence that the mask keeps
//   lse_i = log sum_j exp s_ij, out_i = sum_j exp(s_ij - lse_i) v_j
//
// One pass over the keys with a running maximum and sum (online softmax); scores never leave
// registers. A row without keys gives out = 0, lse = -infinity.
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
// almost always. 215,003 queries on 5 x ~1024 keys, 4 heads of 64: 306 us without, 293 with.
constexpr float kSlack = 8.f;

// Four waves of 32 NQ query rows each over tiles of BN keys. A row is a (query, head of the group
// that shares the key head) pair, so few queries with shared key heads still fill a tile.
// splits > 1: each workgroup takes one part of the sequence's keys and leaves an unnormalised result.
template <typename T, int DP, int NQ, int BN, int WPE, bool VEC>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(WPE))) void k_attn_fwd(AttnArgs a) {
  typedef typename Frag<T>::type frag;
  constexpr int LD = lds_ld<T, DP>();
  constexpr int BM = 128 * NQ;
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
  if (a.splits > 1) {
    const int64_t part = ((k1 - k0 + a.splits - 1) / a.splits + BN - 1) / BN * BN;
    k0 = k0 + split * part < k1 ? k0 + split * part : k1;
    k1 = k0 + part < k1 ? k0 + part : k1;
  }
  int keys = (int)(k1 - k0);

  Stage<T, BN, DP, kNT, VEC> sk, sv;
  sk.start((const T*)a.k + kh * a.ks[1] + k0 * a.ks[0], 0, a.ks[0], 0, 1, a.dim);
  sv.start((const T*)a.v + kh * a.vs[1] + k0 * a.vs[0], 0, a.vs[0], 0, 1, a.dim);
  // Keys of the tile from k0 + j on that exist and that the mask keeps.
  auto key_bits = [&](int j) -> uint64_t {
    bool ok = lane < BN && j + lane < keys;
    if (ok && a.mask) ok = a.mask[k0 + j + lane];
    return __ballot(ok);
  };
  sk.load(keys);
  sv.load(keys);
  uint64_t next_bits = key_bits(0);

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
      fq[n][kk] = load8<T>(p + d, r < rows ? a.dim - d : 0, VEC);
    }
  }

  const float c = a.scale * kLog2e;
  f32x16 o[NQ][DT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[n][t] = zero16();
  }

  int buf = 0;
  for (int j = 0; j < keys; j += BN, buf ^= 1) {
    const uint64_t bits = next_bits;
    if (a.mask) {  // what a masked place holds must not meet a zero probability
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
    // Two buffers: the barrier of the last tile already had every wave past reading this one.
    __syncthreads();
    f32x16 s[NQ][KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n][t] = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const frag fk = load_row<T>(&s_k[buf][(t * 32 + (lane & 31)) * LD + kk * 16 + h * 8]);
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
      top = halves_max(top) * c;
      const float m_new = fmaxf(m[n], top);
      if (__any(m_new > m[n] + kSlack)) {
        asm volatile("");  // a branch: the compiler would multiply always and select
        const float f = m[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[n] - m_new);
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
          s[n][t][r] = __builtin_amdgcn_exp2f(fmaf(s[n][t][r], c, -base));
          l[n] += s[n][t][r];
        }
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        frag p[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) to_frag(s[n][t], mm, p[n]);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const frag fv = load_tr<LD>(s_v[buf], t * 32 + mm * 16, d * 32);
#pragma unroll
          for (int n = 0; n < NQ; ++n) o[n][d] = mma(fv, p[n], o[n][d]);
        }
      }
  }

#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float total = l[n] + __shfl_xor(l[n], 32, 64);
    if (row[n] < 0) continue;
    if (a.splits > 1) {
      const int64_t at = (int64_t)split * a.nq * a.heads + row[n];
#pragma unroll
      for (int d = 0; d < DT; ++d) store_col<float>(a.part_a + at * a.dim, d * 32, a.dim, o[n][d], 1.f, a.dim % 4 == 0);
      if (h == 0) {
        a.part_b[at * 2] = m[n];
        a.part_b[at * 2 + 1] = total;
      }
    } else {
      const float f = total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;
#pragma unroll
      for (int d = 0; d < DT; ++d)
        store_col<T>((T*)a.out + row[n] * a.dim, d * 32, a.dim, o[n][d], f, a.ovec);
      if (h == 0) a.lse[row[n]] = total == 0.f ? -INFINITY : kLn2 * (m[n] + log2f(total));
    }
  }
}

// Joins the parts of a split key axis: one wave per row.
template <typename T>
__global__ __launch_bounds__(kNT) void k_attn_join(AttnArgs a) {
  const int lane = lane_id();
  const int64_t rows = a.nq * a.heads;
  const int64_t row = (int64_t)blockIdx.x * (kNT / 64) + (threadIdx.x >> 6);
  if (row >= rows) return;
  float top = -INFINITY;
  for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, a.part_b[((int64_t)s * rows + row) * 2]);
  top = lanes_reduce<64>(top, [](float x, float y) { return fmaxf(x, y); });
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f, o0 = 0.f, o1 = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const int64_t at = (int64_t)s * rows + row;
    const float f = __builtin_amdgcn_exp2f(a.part_b[at * 2] - base);
    total += f * a.part_b[at * 2 + 1];
    const float* po = a.part_a + at * a.dim;
    if (lane < a.dim) o0 += f * po[lane];
    if (lane + 64 < a.dim) o1 += f * po[lane + 64];
  }
  const float f = total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;
  T* out = (T*)a.out + row * a.dim;
  if (lane < a.dim) out[lane] = (T)(o0 * f);
  if (lane + 64 < a.dim) out[lane + 64] = (T)(o1 * f);
  if (lane == 0) a.lse[row] = total == 0.f ? -INFINITY : kLn2 * (top + log2f(total));
}

template <typename T, int DP>
struct FwdShape;  // NQ, BN
template <int DP>
struct FwdShape<bf16_t, DP> {
  static constexpr int NQ = DP <= 64 ? 2 : 1, BN = 64, WPE = 2;
};
template <int DP>
struct FwdShape<float, DP> {
  static constexpr int NQ = 1, BN = 32, WPE = DP <= 64 ? 2 : 1;
};

int64_t fwd_slots(const AttnArgs& a, int bm) { return a.nq * a.group / bm + a.batch; }

// Row tiles of the forward kernel for this problem.
int fwd_bm(int dtype, int dim) { return dtype == IGC_BF16 && dim <= 64 ? 256 : 128; }

template <typename T, int DP>
void fwd_go(const AttnArgs& a, hipStream_t s) {
  constexpr int NQ = FwdShape<T, DP>::NQ, BN = FwdShape<T, DP>::BN;
  const int64_t wgs = fwd_slots(a, 128 * NQ) * a.kv_heads * a.splits;
  constexpr int WPE = FwdShape<T, DP>::WPE;
  if (a.qvec && a.kvec) k_attn_fwd<T, DP, NQ, BN, WPE, true><<<(unsigned)wgs, kNT, 0, s>>>(a);
  else k_attn_fwd<T, DP, NQ, BN, WPE, false><<<(unsigned)wgs, kNT, 0, s>>>(a);
  if (a.splits > 1) k_attn_join<T><<<(unsigned)((a.nq * a.heads + kNT / 64 - 1) / (kNT / 64)), kNT, 0, s>>>(a);
}

template <typename T>
void fwd_t(const AttnArgs& a, hipStream_t s) {
  if (a.dim <= 32) return fwd_go<T, 32>(a, s);
  if (a.dim <= 64) return fwd_go<T, 64>(a, s);
  if (a.dim <= 96) return fwd_go<T, 96>(a, s);
  fwd_go<T, 128>(a, s);
}

}  // namespace

int attn_fwd_splits(int dtype, int64_t nq, int64_t nk, int batch, int heads, int kv_heads, int dim) {
  // Parts of the key axis: none while the query tiles alone fill the GPU twice over, else enough for
  // that, each of at least 256 keys.
  const int bm = fwd_bm(dtype, dim);
  const int64_t per_seq = (nq / batch) * (heads / kv_heads);
  const int64_t wgs = batch * ((per_seq + bm - 1) / bm) * kv_heads;
  const int64_t want = wgs >= 512 ? 1 : 512 / std::max<int64_t>(1, wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 128), nk / batch / 256));
}

int launch_attn_fwd(const AttnArgs& a, int dtype, hipStream_t s) {
  if (dtype == IGC_BF16) fwd_t<bf16_t>(a, s);
  else fwd_t<float>(a, s);
  IGC_HIP(hipGetLastError(), a.fn);
  return IGC_OK;
}

}  // namespace igc
