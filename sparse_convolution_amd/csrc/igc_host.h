// Host-side internals of libigconv: the grid object, error reporting and allocation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "../../include/igconv.h"
#include "igc_internal.h"
#include "igc_ragged.h"

struct igc_grid {
  int device = 0;
  hipStream_t stream = nullptr;  // stream the grid was built on (destroy waits for it)
  int64_t n_input = 0, n_voxels = 0, n_leaf = 0, n_lower = 0, n_upper = 0;
  int32_t sort_passes = 0;
  int32_t host_syncs = 0;  // host synchronisations the build took
  uint32_t root_cap = 0;
  size_t bytes = 0;
  void* block = nullptr;  // one device allocation holding every array below
  igc_allocator alloc{};  // the caller's memory provider (alloc.alloc == nullptr: the library's pool)

  uint64_t* root_keys = nullptr;   // [root_cap]
  int32_t* root_vals = nullptr;    // [root_cap]
  uint64_t* root_list = nullptr;   // [U] tile keys in upper-node order
  int4* upper_origin = nullptr;    // [U]
  uint64_t* upper_mask = nullptr;  // [U*512]
  uint16_t* upper_pre = nullptr;   // [U*512]
  uint32_t* upper_first = nullptr; // [U]
  int4* lower_origin = nullptr;    // [Lw]
  uint64_t* lower_mask = nullptr;  // [Lw*64]
  uint16_t* lower_pre = nullptr;   // [Lw*64]
  uint32_t* lower_first = nullptr; // [Lw]
  igc::LeafRec* leaf = nullptr;    // [F]
  int4* leaf_origin = nullptr;     // [F]
  int32_t* leaf_nbr = nullptr;     // [F*27] neighbour leaves (the 3x3x3 block around each leaf)

  igc::GridView view() const {
    igc::GridView v;
    v.root_keys = root_keys;
    v.root_vals = root_vals;
    v.root_mask = root_cap ? root_cap - 1u : 0u;
    v.upper_mask = upper_mask;
    v.upper_pre = upper_pre;
    v.upper_first = upper_first;
    v.lower_mask = lower_mask;
    v.lower_pre = lower_pre;
    v.lower_first = lower_first;
    v.leaf = leaf;
    v.leaf_origin = leaf_origin;
    v.leaf_nbr = leaf_nbr;
    v.n_voxels = n_voxels;
    v.n_leaf = n_leaf;
    return v;
  }
};

namespace igc {

// Records the message for igc_last_error and returns the status.
int set_error(int status, const std::string& msg);
void clear_error();

// Status from a HIP call, with the call site named in the message.
int hip_status(hipError_t e, const char* what);

#define IGC_HIP(call, what)                                   \
  do {                                                        \
    hipError_t e_ = (call);                                   \
    if (e_ != hipSuccess) return ::igc::hip_status(e_, what); \
  } while (0)

// The memory provider of a grid, or nullptr for the library's own pool.
inline const igc_allocator* grid_alloc(const igc_grid* g) { return g && g->alloc.alloc ? &g->alloc : nullptr; }

// Stream-ordered device allocation: through `a` when given, else from the library's private
// per-device memory pool (free blocks kept across calls until igc_release_memory).
int dev_alloc(void** p, size_t bytes, hipStream_t s, const char* what, const igc_allocator* a = nullptr);
void dev_free(void* p, size_t bytes, hipStream_t s, const igc_allocator* a = nullptr);

// Pinned host staging buffer (per host thread) of at least `bytes` for small device -> host
// reads; *device_view (if given) receives the address kernels write it through.
void* host_staging(size_t bytes, void** device_view = nullptr);

// Temporary device workspace of one call. With a caller's allocator it is allocated through it
// and returned at release. Otherwise each device keeps one block that is handed to one call at
// a time and grows to the largest request (a call that finds it taken allocates its own): a
// stream-ordered allocation and free cost tens of microseconds of host time per call, and the
// block makes the common case free of both. On release an event is recorded on the caller's
// stream, and the next user's stream waits for it, so work still reading the block finishes
// first.
struct Workspace {
  void* p = nullptr;
  size_t bytes = 0;
  int dev = -1;
  bool cached = false;
  const igc_allocator* a = nullptr;
};
int ws_acquire(Workspace* w, size_t bytes, hipStream_t s, const char* what, const igc_allocator* a = nullptr);
void ws_release(Workspace* w, hipStream_t s);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Host-side checks shared by igc_sparse_conv and igc_sparse_conv_noalloc (fn names the call in
// messages); *path is the requested path on entry and the one to run on success.
int check_conv_args(const char* fn, const igc_grid* g, const int32_t* d_map, const void* d_feats, int32_t dtype,
                    int32_t cin, const void* d_w, int32_t cout, void* d_out, int32_t* path);
// Active voxels from which a leaf takes the leaf window under per-leaf dispatch.
uint32_t mixed_dense_rows(int32_t cin);

// Launchers (defined in the .hip files).
int build_grid(const int32_t* d_ijk, int64_t n_in, hipStream_t s, igc_grid* g);
// Output grids of a chain of strided / transposed 3x3x3 convolutions (stage k reads stage
// k-1's output), built from leaves with the counts on the device and one host synchronisation.
// strides [n][3]; outs[k] are allocated igc_grid objects (device, stream, allocator set) whose
// topology this fills. derive_supported: whether one stage over `in` fits the derived build
// (at most 4096 root tiles, record indices within the sort key).
bool derive_supported(const igc_grid* in, const int32_t* stride, int32_t transposed);
int derive_chain(const igc_grid* in, int n, const int32_t* strides, const int32_t* transposed, hipStream_t s,
                 igc_grid** outs);
int launch_active_ijk(const igc_grid* g, int32_t* d_out, hipStream_t s);
int launch_ijk_to_index(const igc_grid* g, const int32_t* d_q, int64_t m, int32_t* d_idx, hipStream_t s);
int launch_kernel_map(const igc_grid* g, const int32_t* h_offsets, int32_t K, int32_t* d_map, uint32_t* d_nbmask,
                      hipStream_t s);
bool leaf_conv_supported(int32_t dtype, int32_t cin, int32_t cout);
bool ggs_conv_supported(int32_t dtype, int32_t cin, int32_t cout);
// General-shape path (any channel counts up to kGatherMaxChannels, fp32 or bf16).
constexpr int32_t kGatherMaxChannels = 4096;
bool gather_conv_supported(int32_t dtype, int32_t cin, int32_t cout);
// d_map int32[27, N]; entries outside [0, n_in) read as absent. scratch (may be null): at least
// gather_scratch_bytes() of device memory used instead of a workspace from g's allocator.
int launch_conv_gather(const igc_grid* g, const int32_t* d_map, int64_t N, int64_t n_in, const void* d_feats,
                       int32_t dtype, int32_t cin, const void* d_w, int32_t cout, void* d_out, hipStream_t s,
                       void* scratch = nullptr);
size_t gather_scratch_bytes(int32_t cin, int32_t cout);
int launch_wgrad_gather(const igc_grid* g, const int32_t* d_map, const void* d_feats, int32_t dtype, int32_t cin,
                        const void* d_dout, int32_t cout, float* d_dw, hipStream_t s);
// dw[e] = sum over c < chunks of part[c * E + e] in fp64, in a fixed order (weight gradients).
int launch_wgrad_reduce(const float* part, int64_t chunks, int64_t E, float* dw, hipStream_t s);

// Row order of the gather-GEMM-scatter plan for one layer: rows sorted by neighbour mask within
// spans of `span` rows (256, 1024 or 4096), key bit order 0 = natural, 1 = class (corners,
// edges, faces, centre); from the rules igc_tuning_load read (default: 256, natural).
struct GgsTuning {
  int span = 256;
  int order = 0;
  int bn = 0;  // output channels per workgroup tile (0: the widest the shape allows)
  int kc = 0;  // input channels per chunk: 32 forces 32-channel chunks (0: 64 where cin allows)
  int rows = 0;  // output rows per workgroup: 128 takes half of a 256-row plan tile (0: whole)
};
GgsTuning ggs_tuning(int32_t cin, int32_t cout, int64_t n_voxels, int64_t n_leaf);
// min_count > 0 (bf16 only): leaves with fewer active voxels are skipped (their rows untouched).
// scratch (may be null): caller-provided device memory of at least leaf_scratch_bytes() used
// instead of a workspace (nothing is allocated then).
int launch_conv_leaf(const igc_grid* g, const void* d_feats, int32_t dtype, int32_t cin, const void* d_w, int32_t cout,
                     void* d_out, hipStream_t s, uint32_t min_count = 0, void* scratch = nullptr);
size_t leaf_scratch_bytes(int32_t dtype, int32_t cin, int32_t cout);
// dense_min > 0: rows of leaves with at least dense_min active voxels get no pairs (zero output).
// n_in: rows of d_feats (map entries outside [0, n_in) read as absent); -1 = the grid's N.
// scratch (may be null): caller-provided device memory of at least ggs_scratch_bytes() used
// instead of a workspace (nothing is allocated then).
int launch_conv_ggs(const igc_grid* g, const int32_t* d_map, const void* d_feats, int32_t dtype, int32_t cin,
                    const void* d_w, int32_t cout, void* d_out, hipStream_t s, uint32_t dense_min = 0,
                    int64_t n_in = -1, void* scratch = nullptr);
size_t ggs_scratch_bytes(int64_t N, int32_t cin, int32_t cout, bool with_skip);
// Mask-sorted tiles of 256 output rows (row order perm, 16-row blocks with pairs per offset blk);
// rows with skip[row] != 0 (if skip is given) count as having no neighbours.
int launch_ggs_plan(const int32_t* d_map, int64_t N, int32_t* perm, uint16_t* blk, hipStream_t s,
                    const uint8_t* skip = nullptr);
// Leaf-local fp32 weight gradient: `groups` partial dW blocks [groups][27][cin][cout] in `part`.
bool wgrad_leaf_supported(int32_t cin, int32_t cout);
int64_t wgrad_leaf_groups(const igc_grid* g);
int launch_wgrad_leaf(const igc_grid* g, const void* d_feats, int32_t cin, const void* d_dout, int32_t cout,
                      float* part, int64_t groups, hipStream_t s);
// Output grids of strided / transposed 3x3x3 convolutions and the map between two grids.
int conv_grid_slots(const int32_t* stride, int32_t transposed, int* n);
int build_conv_grid(const igc_grid* in, const int32_t* stride, int32_t transposed, hipStream_t s, igc_grid* out);
int launch_conv_map(const igc_grid* in, const igc_grid* out, const int32_t* stride, int32_t transposed,
                    int32_t* d_map, hipStream_t s);
// Fills n 32-bit words with v on stream s (a kernel, so it can sit in captured work).
int fill_u32(uint32_t* p, int64_t n, uint32_t v, hipStream_t s);
bool wgrad_supported(int32_t dtype, int32_t cin, int32_t cout);
bool wgrad_tuned_supported(int32_t dtype, int32_t cin, int32_t cout);
// A convolution's saved input: the features themselves, or an 8-bit checkpoint of them.
struct FeatsIn {
  const void* x = nullptr;
  const int8_t* codes = nullptr;
  const float* scales = nullptr;
};
int launch_conv_backward(const igc_grid* g, const int32_t* d_map, const FeatsIn& feats, int32_t dtype, int32_t cin,
                         const void* d_w, int32_t cout, const void* d_dout, void* d_dfeats, float* d_dw,
                         int32_t dgrad_path, hipStream_t s);

// Workgroups of 256 threads that a kernel striding over its work is launched with at most: a launch takes fewer than
// 2^32 threads along an axis.
constexpr int64_t kMaxWgs = (int64_t)1 << 23;

// 8-bit activation checkpoints (igc_checkpoint.hip).
int launch_pack(const void* x, int32_t dtype, int64_t n, int32_t c, int8_t* codes, float* scales, hipStream_t s);
int launch_unpack(const int8_t* codes, const float* scales, int64_t n, int32_t c, int32_t dtype, void* x, hipStream_t s);

// Layer norm over n rows of c channels. codes != nullptr: the forward pass writes an 8-bit checkpoint
// of the normalised rows and no mean, the backward pass reads it instead of x and mean.
constexpr int32_t kNormMaxChannels = 4096;
struct NormArgs {
  const char* fn = "";  // the call named in messages
  int32_t dtype = 0, c = 0;
  int64_t n = 0;
  const void *x = nullptr, *dy = nullptr, *w = nullptr, *b = nullptr;
  int wf32 = 0;  // w and b are fp32 (else the features' type)
  float eps = 0.f;
  void* y = nullptr;  // y, or dx
  float *mean = nullptr, *rstd = nullptr, *scales = nullptr, *dw = nullptr, *db = nullptr;
  int8_t* codes = nullptr;
};
int launch_norm(const NormArgs& a, hipStream_t s);
// Workgroups of the backward pass; ws holds 2 c floats for each where dw is wanted.
int norm_bwd_parts(int64_t n, int32_t c);
int launch_norm_bwd(const NormArgs& a, void* ws, hipStream_t s);
// first[e] and second[e] (null: skipped), e < c: the sums of part[chunk][e] and part[chunk][c + e] in fp64, in a fixed order.
int launch_pair_sum(const char* fn, const float* part, int chunks, int c, float* first, float* second, hipStream_t s);

// Dropout with a counter-based generator (igc_dropout.hip).
struct DropoutArgs {
  int32_t dtype = 0;
  const void *x = nullptr, *residual = nullptr;
  void* y = nullptr;
  int64_t count = 0;
  uint32_t drop = 0;  // elements with fewer than this in 16 bits are dropped
  float scale = 1.f;
  uint64_t seed = 0, offset = 0;
  const uint64_t* d_offset = nullptr;  // added to offset
};
int launch_dropout(const DropoutArgs& a, hipStream_t s);

// Norm and rotation of queries (0) and keys (1) for each head (igc_qk.hip); strides in elements.
struct QkArgs {
  const char* fn = "";
  int32_t dtype = 0;
  int64_t n = 0;
  int dim = 0, heads[2] = {0, 0}, heads_each = 0;
  const void *x[2] = {nullptr, nullptr}, *dy[2] = {nullptr, nullptr}, *w[2] = {nullptr, nullptr};
  int64_t xs[2][2] = {{0, 0}, {0, 0}};  // row and head strides of x; y and dy are dense
  void* y[2] = {nullptr, nullptr};      // y, or dx
  int wf32 = 0;                         // w is fp32 (else the data's type)
  const int32_t* positions = nullptr;   // [n, axes]
  const float* frequencies = nullptr;   // [axes, pairs]
  int axes = 0, pairs = 0, interleaved = 0, norm = 0;
  float eps = 0.f, amplitude = 1.f;
  float *part = nullptr, *dw[2] = {nullptr, nullptr};
};
// Partial weight gradients of the backward pass, 2 dim floats each.
int qk_parts(int32_t dtype, int64_t n, int32_t heads, int32_t dim);
int launch_qk(const QkArgs& a, bool backward, hipStream_t s);

// One attention problem on the device; strides in elements.
struct AttnArgs {
  const char* fn = "";
  const void *q = nullptr, *k = nullptr, *v = nullptr, *dout = nullptr, *out_in = nullptr;
  const float* lse_in = nullptr;
  void *out = nullptr, *dq = nullptr, *dk = nullptr, *dv = nullptr;
  float *lse = nullptr, *delta = nullptr;
  float *part_a = nullptr, *part_b = nullptr;  // partial results of a split axis
  const int32_t *qo = nullptr, *ko = nullptr;  // row offsets of the sequences (null: one sequence)
  const uint8_t* mask = nullptr;               // [nk], 0 = key left out
  int64_t nq = 0, nk = 0;
  int64_t qs[2] = {0, 0}, ks[2] = {0, 0}, vs[2] = {0, 0};  // row and head strides
  int batch = 1, heads = 1, kv_heads = 1, group = 1, dim = 0;
  int splits = 1;
  int qvec = 0, kvec = 0, ovec = 0;  // 16-byte loads of q, of k and v, of the dense outputs allowed
  float scale = 1.f;
  // Window attention (windowed != 0). The first `sinks` keys of a sequence, which later queries see too, get their gradients from
  // far_parts further workgroups for each of their tiles, whose results are added up in `far`: [1 + far_parts][rows][kv_heads]
  // [dim] for dk, then dv. Row b * sinks + j is key j of sequence b, or, where that takes more rows than keys
  // (far_by_key), row r is key row r.
  int windowed = 0, far_parts = 0, far_by_key = 0;
  unsigned far_wgs = 0;
  int64_t far_rows = 0;
  float* far = nullptr;
  Window win = {-1, -1, 0};
  const int32_t* kl = nullptr;  // forward: keys of each sequence in use (null: all)
};
constexpr int32_t kAttnMaxDim = 128;
// Keys, and query rows (queries times the heads that share a key head), of a problem at most: the kernels count those of a
// sequence in 32 bits and step up to 256 past its end.
constexpr int64_t kAttnMaxRows = INT32_MAX - 1023;
// Whether window attention's tiles of 64 rows (or keys) are so few that all their workgroups run at a time anyway: two
// waves then share each row's axis, for half the latency. Of wide heads only one workgroup fits a CU. us, without and with, windows of 255
// before, 2 heads, n rows, forward / gradients: bf16, heads of 64, 300 11.4, 8.3 / 28.7, 22.1; 7,000 15.7, 11.3 / 39.4, 32.5;
// 14,000 16.5, 13.9 / 45.9, 47.0; 28,000 (limits twice as high) 25.4, 31.0 / 84.9, 81.4; heads of 128, 2,000 17.1, 13.1 / 50.0, 39.6; 14,000
// 21.1, 19.9 / 79.5, 86.3; fp32, heads of 40, 2,000 27.0, 17.9 / 73.2, 49.8; 14,000 31.6, 40.8 / 119, 128.
// Counted are the launch's workgroups (one more than its rows fill for each sequence, see find_tile), not tiles: those without
// rows hold a CU on their way out too, and come in a rhythm that leaves some XCDs without work. Sequences of 64 rows, 2 heads, gradients, with
// and without: 241 of bf16 heads of 64 39 and 24, 113 of fp32 heads of 64 52 and 33. What this gives away: 120 of 128 rows, bf16 heads
// of 64, 27 and 33.
// 2: fp32 heads of 33 to 64 channels, where one workgroup fits a CU: eight waves take two tiles where one a workgroup are too many.
// 1 / 2 / 0, 255 before, 2 heads of 40, forward and gradients: 9,001 rows of 2 sequences 40 / 26 / 31 and 104 / 76 / 83; 14,000 rows 41 /
// 26 / 32 and 132 / 105 / 123; 16,200 rows of 2 sequences (256 workgroups) 43 / 27 / 32 and 133 / 107 / 125. Above 256 workgroups, heads of 64: 200
// sequences of 64 rows 36 / 21 / 15 and 116 / 78 / 63, 96 of 100 rows 2: 24 and 74, 0: 18 and 65; given away: 48 of 256 rows 2: 19 and
// 61, 0: 22 and 65.
inline int window_few(int dtype, int dim, int64_t rows, int batch, int kv_heads) {
  auto wgs = [&](int bm) { return (rows * batch / bm + batch) * kv_heads; };
  if (wgs(64) <= (dim > (dtype == IGC_F32 ? 32 : 64) ? 256 : 512)) return 1;
  return dtype == IGC_F32 && dim > 32 && dim <= 64 && wgs(128) <= 256 ? 2 : 0;
}
// Keys, or query rows, of a part of a split axis at least, for window attention's tiles.
constexpr int64_t kWindowPart = 384;
// Parts the key axis is split into; where there is more than one, the forward workspace holds dim partial results and two
// statistics for each part, query and head.
int attn_fwd_splits(int dtype, const AttnArgs& a);
int launch_attn_fwd(const AttnArgs& a, int dtype, hipStream_t s);
struct AttnBwdPlan {
  int dq_splits = 1, dkv_splits = 1;
  int far_parts = 0, far_by_key = 0;  // as in AttnArgs
  int64_t far_rows = 0;
  size_t floats = 0, far_at = 0;  // workspace, and where `far` starts in it
  int64_t dkv_threads = 0;        // of the launch for dk and dv, which takes fewer than 2^32
};
AttnBwdPlan attn_bwd_plan(int dtype, const AttnArgs& a);
int launch_attn_bwd(const AttnArgs& a, int dtype, const AttnBwdPlan& p, void* ws, hipStream_t s);

}  // namespace igc
