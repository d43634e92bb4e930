// kernels.h -- host-side launchers of the libvsa kernels (internal to the library).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace vsa {

cudaError_t launch_permute(const void* src, bool src_f32, void* dst, const uint8_t* kinds, const Geom& g, int BH,
                           int d, int* err, cudaStream_t stream);
cudaError_t launch_unpermute(const void* src, const float* src_lse, void* dst, bool dst_f32, float* dst_lse,
                             const uint8_t* kinds, const Geom& g, int BH, int d, int* err, cudaStream_t stream);

cudaError_t launch_pattern_mask(const uint8_t* kinds, const Geom& g, int BH, int w_s, int w_t, uint32_t* bits,
                                int32_t* kv_idx, int32_t* kv_cnt, int max_kv, int* err, cudaStream_t stream);
// Workspace: 2 * BH * ncubes * d doubles.
size_t cube_mask_workspace_bytes(const Geom& g, int BH, int d);
cudaError_t launch_cube_mask(const uint8_t* kinds, const void* q_cube, const void* k_cube, const Geom& g, int BH, int d,
                             int topk, uint32_t* bits, int32_t* kv_idx, int32_t* kv_cnt, int max_kv, void* ws,
                             int* err, cudaStream_t stream);

// Attention work order per head (query blocks sorted by their first kept key block).
cudaError_t launch_block_order(const uint8_t* kinds, const Geom& g, int BH, const int32_t* kv_idx,
                               const int32_t* kv_cnt, int max_kv, int32_t* order, cudaStream_t stream);

// Semantic-aware permutation (see semantic.cu).  At most kMaxClusters clusters per tensor.
constexpr int kMaxClusters = 1024;
// k-means of x [BH, N, d] bf16: cent [BH, C, d] f32, label [BH, N], counts [BH, C], perm [BH, N]
// (slot -> token, cluster-major).  ws (kmeans_workspace_bytes): the cluster offsets and
// partial-sum chunk offsets [BH, C + 1], the centroids' squared norms [BH, C], their bf16
// halves [BH, C, d] twice, the update's chunk sums [BH, ceil(N / 128) + C, d], and the
// sort's segment histograms [BH, 8, C] with one flag per head, and the chunks' clusters.
size_t kmeans_workspace_bytes(int BH, int N, int C, int d);
cudaError_t launch_kmeans(const void* x, int BH, int N, int d, int C, int iters, float* cent, int32_t* label,
                          int32_t* counts, int32_t* perm, void* ws, int* err, cudaStream_t stream);
// Workspace of launch_semantic_mask: the cluster range of every query and key block.
size_t semantic_mask_workspace_bytes(int BH, int N, int block);
cudaError_t launch_semantic_mask(const float* cent_q, const int32_t* counts_q, const int32_t* label_q,
                                 const int32_t* perm_q, int Cq, const float* cent_k, const int32_t* counts_k,
                                 const int32_t* label_k, const int32_t* perm_k, int Ck, int BH, int N, int d,
                                 int block, double scale, double top_p, uint32_t* keep, uint32_t* bits,
                                 int32_t* kv_idx, int32_t* kv_cnt, int max_kv, void* ws, int* err,
                                 cudaStream_t stream);
cudaError_t launch_gather_rows(const void* src, const int32_t* perm, void* dst, int BH, int N, int d, int* err,
                               cudaStream_t stream);
cudaError_t launch_scatter_rows(const void* src, const float* src_lse, const int32_t* perm, void* dst, float* dst_lse,
                                int BH, int N, int d, int* err, cudaStream_t stream);

// Tensor maps of one attention problem (3D: d, rows, B*H).
struct AttnMaps {
  CUtensorMap q, k, v, o;
};

struct AttnArgs {
  const uint8_t* kinds;
  const int32_t* kv_idx;
  const int32_t* kv_cnt;
  const int32_t* order;  // [B*H, nblk] query-block order, or null for natural order
  float* lse_nat;
  float* lse_perm;
  int* err;
  int BH;
  int max_kv;
  int has_perm;
  int nat_rows;  // rows per head of the natural buffers (N, or R when they hold every layout)
  int ucap;      // capacity of the per-CTA union list: min(nblk, 2 * max_kv)
  float scale_log2;
  Geom g;
  // In-kernel layout: temporal heads read Q, K, V and write O in natural order through the
  // frame-major slot map (no permuted copies); only with has_perm == 0.
  int gather;
  // e4m3 Q and K (null for bf16): per (head, block) power-of-two exponents of their scales
  const int32_t* qexp;
  const int32_t* kexp;
  const void* nat_q;
  const void* nat_k;
  const void* nat_v;
  void* nat_o;
  // What rounding O to bf16 left over, as bf16 rows beside O's (null: not wanted)
  void* lo_nat;
  void* lo_perm;
};

cudaError_t launch_sparse_attn(const AttnMaps& nat, const AttnMaps& perm, const AttnArgs& a, int d,
                               cudaStream_t stream);

// Shared memory of a CTA on sm_100a.
constexpr int kMaxSmem = 232448;

// Lets launches of a kernel ask for up to `most` bytes of dynamic shared memory.  The limit is the kernel's, for every
// thread of the process: `most` is what its largest launch takes, never the size of the launch at hand, which another
// thread's launch of the same kernel might then exceed.
template <typename K>
cudaError_t allow_smem(K* kern, int most) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// Gradient of the attention (see attn_bwd.cu): tensor maps of one set, the row terms and row
// bitsets, and the main kernel's arguments.
struct BwdMaps {
  CUtensorMap q, k, v, g, dq, dk, dv;  // g: dO
};

struct BwdPrep {
  const uint8_t* kinds;
  const int32_t* kv_idx;
  const int32_t* kv_cnt;
  const void *o_nat, *o_perm, *do_nat, *do_perm;
  const void *lo_nat, *lo_perm;  // O's rounding errors, or null
  const float *lse_nat, *lse_perm, *dlse_nat, *dlse_perm;
  uint32_t* rbits;  // [BH, nblk, ceil(nblk / 32)] kept key blocks of every query block
  float* target;    // [BH, nblk, block]: what the sum of dS over the row is, or null
  float* terms;     // [BH, nblk, 2, block]: -lse * log2 e (-inf: the row sees nothing), then -delta
  int* err;
  int BH, d, max_kv, has_perm, nat_rows;
  int by_token;     // O, dO and LSE are in natural order for every head (the whole call)
  int f32;          // O and dO are fp32 rows
  int mask_ctas;    // set by the launcher
  Geom g;
};

struct BwdArgs {
  const uint8_t* kinds;
  const uint32_t* rbits;
  const float* terms;
  const float* target;
  int* err;
  void *nat_dq, *nat_dk, *nat_dv;  // zeroed for a head with an invalid kind byte
  int BH, has_perm, nat_rows;
  int nx;                          // ring stages, set by the launcher
  int exact;                       // delta comes from the unrounded O: the rows' sums of dS are `target`
  float scale, scale_log2;
  Geom g;
};

// Whether the shape's bitsets fit the kernel's shared memory and its grid.
bool sparse_attn_bwd_fits(const Geom& g, int BH);
cudaError_t launch_sparse_attn_bwd(const BwdMaps& nat, const BwdMaps& perm, BwdPrep prep, const BwdArgs& a, int d,
                                   cudaStream_t stream);

// Profiling (see profile.cu).
struct ProfilePlan {
  int r;        // sampled rows
  int r_pad;    // rounded up to the 128-row tile
  int tiles;    // r_pad / 128
  int splits;   // key-range splits per tile
  size_t off_qs, off_ranges, off_order, off_opart, off_ml, off_rowerr, bytes;
};
ProfilePlan profile_plan(const Geom& g, int BH, int d, double frac);
// Same layout as profile_plan but with an explicit number of key-range splits (>= 1).
ProfilePlan profile_plan_splits(const Geom& g, int BH, int d, double frac, int splits);
cudaError_t launch_profile(const void* q, const void* k, const void* v, const Geom& g, int BH, int d, int w_s,
                           int w_t, float scale_log2, const ProfilePlan& plan, void* ws, uint8_t* kinds_out,
                           float* mse_out, int* err, cudaStream_t stream);

// Root-mean-square norm of rows (norm.cu): B*H heads of N rows of d elements, outputs contiguous.
struct NormArgs {
  const void *x, *res;      // rows at b * stride[0] + h * stride[1] + n * stride[2]; res may be null
  const void* w;            // d weights, or null for ones
  void *sum, *y;            // either may be null
  uint8_t* codes;           // e4m3 codes with their exponents, or null
  int32_t* exps;
  float* rstd;              // written (may be null); read by the gradient
  int64_t x_stride[3], res_stride[3];
  int w_kind;               // 0 none, 1 fp32, 2 bf16
  int BH, H, N, d;
  int block;                // rows per exponent
  int chunks;               // chunks of rows per head, set by the launcher
  float eps;
};
struct NormBwdArgs {
  NormArgs n;               // x: the normalised rows' input (the sum), rstd, weights, shape; res_stride: dx's
  const void *dy, *d_sum;   // contiguous; d_sum may be null
  void* dx;
  float* partial;           // [CTAs, d] fp32, or null when dw is not wanted
};
// Rows of d floats that the gradient's partial sums take at most.
size_t rms_norm_bwd_partials(long long rows, int d, bool f32);
cudaError_t launch_rms_norm(NormArgs a, bool f32, cudaStream_t stream);
cudaError_t launch_rms_norm_bwd(NormBwdArgs a, bool f32, float* dw, cudaStream_t stream);

// Tensor-map encoding through the driver entry point (no link-time libcuda dependency).
cudaError_t encode_rows_map(CUtensorMap* map, const void* base, int d, int rows, int BH, int box_rows);
// The same for rows of d = 128 one-byte elements (e4m3 codes): one 128-byte box per row.
cudaError_t encode_rows_map_u8(CUtensorMap* map, const void* base, int d, int rows, int BH, int box_rows);

// Per-block e4m3 quantisation (fp8.cu): dst [BH, R, d] codes, exps [BH, nblk].
cudaError_t launch_quantize_e4m3(const void* nat, const void* perm, const uint8_t* kinds, const Geom& g, int BH,
                                 int d, int nat_rows, uint8_t* dst, int32_t* exps, int* err, cudaStream_t stream);

}  // namespace vsa
