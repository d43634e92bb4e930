// api.cu -- the C ABI of libvsa.so (declared in include/vsa.h): host-side validation,
// planning helpers, TMA descriptor encoding and the launch sequence of one attention call.
// No device memory is allocated here; every buffer comes from the caller.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <vector>

#include "common.cuh"
#include "kernels.h"
#include "vsa.h"

namespace vsa {

// ---------------------------------------------------------------------------------------
// TMA descriptor encoding through the driver entry point
// ---------------------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Encodes one map.  A thread that has only called the runtime has no context of the driver's yet: the current device's
// is made its own, as a launch would.
static cudaError_t encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, const cuuint64_t (&dims)[3],
                              const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3]) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&] {
    return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  int dev = 0;
  if ((r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) && cudaGetDevice(&dev) == cudaSuccess &&
      cudaSetDevice(dev) == cudaSuccess)
    r = encode();
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// 3D view (d, rows, B*H) of a [B*H, rows, d] bf16 tensor; box = 64 columns x box_rows rows,
// 128-byte swizzle; out-of-range rows read as zero and are clipped on store.
cudaError_t encode_rows_map(CUtensorMap* map, const void* base, int d, int rows, int BH, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(BH)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(rows) * d * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, dims, strides, box);
}

cudaError_t encode_rows_map_u8(CUtensorMap* map, const void* base, int d, int rows, int BH, int box_rows) {
  if (d != 128) return cudaErrorInvalidValue;  // one 128-byte swizzled row per box row
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(BH)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows) * d};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), 1};
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, dims, strides, box);
}

static size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every non-null pointer is device (or managed) memory.  Kernels and TMA copies fault on a
// pageable host address, so a host pointer is refused here, before anything is launched.
static bool on_device(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs) {
    if (p == nullptr) continue;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return false;
  }
  return true;
}

// on_device, and on the device that is current: a kernel launched on one device must not be given
// another one's memory.
static bool on_current_device(std::initializer_list<const void*> ptrs) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  for (const void* p : ptrs) {
    if (p == nullptr) continue;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    if (at.type != cudaMemoryTypeManaged && (at.type != cudaMemoryTypeDevice || at.device != dev)) return false;
  }
  return true;
}

// One buffer of a call.
struct Span {
  const void* p;
  size_t bytes;
};

// Whether every output lies apart from every input and from the other outputs: some CTAs write while others read.
static bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  auto meet = [](const Span& x, const Span& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return a != 0 && b != 0 && (a <= b ? b - a < x.bytes : a - b < y.bytes);
  };
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* x = o + 1; x != outs.end(); ++x)
      if (meet(*o, *x)) return false;
    for (const Span& x : ins)
      if (meet(*o, x)) return false;
  }
  return true;
}

// Validate the shape and derive the geometry.
static vsa_status make_geom(const vsa_shape* s, Geom* g) {
  if (s == nullptr || g == nullptr) return VSA_ERR_INVALID_ARG;
  if (s->B <= 0 || s->H <= 0 || s->F <= 0 || s->Hl <= 0 || s->Wl <= 0 || s->d <= 0 || s->block <= 0)
    return VSA_ERR_INVALID_ARG;
  if (s->d != 64 && s->d != 128) return VSA_ERR_UNSUPPORTED;
  if (s->block != 64 && s->block != 128) return VSA_ERR_UNSUPPORTED;
  const long long N = static_cast<long long>(s->F) * s->Hl * s->Wl;
  if (N > (1LL << 28)) return VSA_ERR_UNSUPPORTED;
  const bool cubes = s->cube_f != 0 || s->cube_h != 0 || s->cube_w != 0;
  Geom r{};
  r.F = s->F;
  r.Hl = s->Hl;
  r.Wl = s->Wl;
  r.S = s->Hl * s->Wl;
  r.N = static_cast<int>(N);
  r.block = s->block;
  if (cubes) {
    if (s->cube_f <= 0 || s->cube_h <= 0 || s->cube_w <= 0) return VSA_ERR_INVALID_ARG;
    if (s->cube_f * s->cube_h * s->cube_w != s->block) return VSA_ERR_UNSUPPORTED;
    r.cf = s->cube_f;
    r.ch = s->cube_h;
    r.cw = s->cube_w;
    r.vol = r.cf * r.ch * r.cw;
    r.ncf = (r.F + r.cf - 1) / r.cf;
    r.nch = (r.Hl + r.ch - 1) / r.ch;
    r.ncw = (r.Wl + r.cw - 1) / r.cw;
    const long long nc = static_cast<long long>(r.ncf) * r.nch * r.ncw;
    if (nc * r.vol > (1LL << 28)) return VSA_ERR_UNSUPPORTED;
    r.ncubes = static_cast<int>(nc);
    r.R = r.ncubes * r.vol;
  } else {
    r.cf = r.ch = r.cw = r.vol = 1;  // unused; keeps the cube arithmetic division-safe
    r.ncf = r.nch = r.ncw = 1;
    r.ncubes = 0;
    r.R = r.N;
  }
  r.nblk = (r.R + r.block - 1) / r.block;
  *g = r;
  return VSA_OK;
}

static float scale_log2_of(float scale, int d) {
  const float s = scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(d));
  return s * 1.4426950408889634f;
}

// ---------------------------------------------------------------------------------------
// Window planning on the host: per-query-block kept ranges are contiguous, so the kept
// count for window w is a sum of range lengths found by binary search.
// ---------------------------------------------------------------------------------------
struct BlockIntervals {
  std::vector<int> a, b;  // group interval [a_i, b_i] of block i
};

static BlockIntervals intervals(const Geom& g, int kind) {
  const int G = kind == kSpatial ? g.S : g.F;
  const int nb = (g.N + g.block - 1) / g.block;
  BlockIntervals iv;
  iv.a.resize(nb);
  iv.b.resize(nb);
  for (int i = 0; i < nb; ++i) {
    iv.a[i] = (i * g.block) / G;
    iv.b[i] = (std::min(g.N, (i + 1) * g.block) - 1) / G;
  }
  return iv;
}

// Kept blocks of row i: j with a_j <= b_i + w and b_j >= a_i - w (both sequences nondecreasing).
static int kept_in_row(const BlockIntervals& iv, int i, long long w) {
  const int nb = static_cast<int>(iv.a.size());
  const long long hi_val = iv.b[i] + w, lo_val = iv.a[i] - w;
  int lo = 0, hi = nb;  // first j with b_j >= lo_val
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (iv.b[mid] >= lo_val) hi = mid; else lo = mid + 1;
  }
  const int j0 = lo;
  lo = 0;
  hi = nb;  // first j with a_j > hi_val
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (iv.a[mid] > hi_val) hi = mid; else lo = mid + 1;
  }
  const int j1 = lo;  // exclusive
  return j1 > j0 ? j1 - j0 : 0;
}

static long long kept_total(const BlockIntervals& iv, long long w, int* row_max) {
  long long tot = 0;
  int mx = 0;
  for (int i = 0; i < static_cast<int>(iv.a.size()); ++i) {
    const int k = kept_in_row(iv, i, w);
    tot += k;
    mx = std::max(mx, k);
  }
  if (row_max) *row_max = mx;
  return tot;
}

}  // namespace vsa

using namespace vsa;

extern "C" {

const char* vsa_status_string(vsa_status s) {
  switch (s) {
    case VSA_OK: return "ok";
    case VSA_ERR_INVALID_ARG: return "invalid argument";
    case VSA_ERR_UNSUPPORTED: return "unsupported configuration";
    case VSA_ERR_WORKSPACE: return "workspace too small";
    case VSA_ERR_CUDA: return "CUDA call failed";
    case VSA_ERR_DEVICE: return "device-side error flagged";
    case VSA_ERR_TIMEOUT: return "device-side wait timed out";
  }
  return "unknown status";
}

int vsa_version(void) { return 100; }

vsa_status vsa_layout_rows(const vsa_shape* shape, int64_t* rows) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (rows == nullptr) return VSA_ERR_INVALID_ARG;
  *rows = g.R;
  return VSA_OK;
}

vsa_status vsa_num_blocks(const vsa_shape* shape, int* nblk) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (nblk == nullptr) return VSA_ERR_INVALID_ARG;
  *nblk = g.nblk;
  return VSA_OK;
}

vsa_status vsa_pattern_window(const vsa_shape* shape, vsa_kind kind, double target, int* w, double* kept) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (w == nullptr || (kind != VSA_SPATIAL && kind != VSA_TEMPORAL) || !(target >= 0.0) || target > 1.0)
    return VSA_ERR_INVALID_ARG;
  const BlockIntervals iv = intervals(g, kind);
  const double nb = static_cast<double>(iv.a.size());
  const long long wmax = kind == VSA_SPATIAL ? g.F - 1 : g.S - 1;
  long long lo = 0, hi = wmax;  // smallest w in [0, wmax] with kept(w)/nb^2 >= target
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (static_cast<double>(kept_total(iv, mid, nullptr)) / (nb * nb) >= target) hi = mid; else lo = mid + 1;
  }
  *w = static_cast<int>(lo);
  if (kept) *kept = static_cast<double>(kept_total(iv, lo, nullptr)) / (nb * nb);
  return VSA_OK;
}

vsa_status vsa_max_kv(const vsa_shape* shape, const vsa_params* params, int* max_kv) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (params == nullptr || max_kv == nullptr || params->w_s < 0 || params->w_t < 0) return VSA_ERR_INVALID_ARG;
  int mx = 0, m1 = 0;
  kept_total(intervals(g, kSpatial), params->w_s, &m1);
  mx = std::max(mx, m1);
  kept_total(intervals(g, kTemporal), params->w_t, &m1);
  mx = std::max(mx, m1);
  if (g.ncubes > 0) {
    if (params->topk < 0) return VSA_ERR_INVALID_ARG;
    mx = std::max(mx, std::min(params->topk + 1, g.ncubes));
  }
  *max_kv = mx;
  return VSA_OK;
}

vsa_status vsa_profile_rows(const vsa_shape* shape, const vsa_params* params, int* rows) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (params == nullptr || rows == nullptr || !(params->profile_frac > 0.0) || params->profile_frac > 1.0)
    return VSA_ERR_INVALID_ARG;
  *rows = profile_plan(g, shape->B * shape->H, shape->d, params->profile_frac).r;
  return VSA_OK;
}

size_t vsa_profile_workspace_size(const vsa_shape* shape, const vsa_params* params) {
  Geom g;
  if (make_geom(shape, &g) != VSA_OK || params == nullptr || !(params->profile_frac > 0.0)) return 0;
  return profile_plan(g, shape->B * shape->H, shape->d, params->profile_frac).bytes;
}

size_t vsa_mask_workspace_size(const vsa_shape* shape, const vsa_params* params) {
  Geom g;
  if (make_geom(shape, &g) != VSA_OK || params == nullptr) return 0;
  return g.ncubes > 0 ? cube_mask_workspace_bytes(g, shape->B * shape->H, shape->d) : 0;
}

vsa_status vsa_permute(const void* src, vsa_dtype src_dtype, void* dst, const uint8_t* d_kind, const vsa_shape* shape,
                       int* d_err, cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!src || !dst || !d_kind || !d_err || !aligned16(src) || !aligned16(dst)) return VSA_ERR_INVALID_ARG;
  if (src_dtype != VSA_F32 && src_dtype != VSA_BF16) return VSA_ERR_INVALID_ARG;
  if (!on_device({src, dst, d_kind, d_err})) return VSA_ERR_INVALID_ARG;
  const cudaError_t e =
      launch_permute(src, src_dtype == VSA_F32, dst, d_kind, g, shape->B * shape->H, shape->d, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status vsa_unpermute(const void* src, const float* src_lse, void* dst, vsa_dtype dst_dtype, float* dst_lse,
                         const uint8_t* d_kind, const vsa_shape* shape, int* d_err, cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!src || !dst || !d_kind || !d_err || !aligned16(src) || !aligned16(dst)) return VSA_ERR_INVALID_ARG;
  if ((src_lse == nullptr) != (dst_lse == nullptr)) return VSA_ERR_INVALID_ARG;
  if (dst_dtype != VSA_F32 && dst_dtype != VSA_BF16) return VSA_ERR_INVALID_ARG;
  if (!on_device({src, src_lse, dst, dst_lse, d_kind, d_err})) return VSA_ERR_INVALID_ARG;
  const cudaError_t e = launch_unpermute(src, src_lse, dst, dst_dtype == VSA_F32, dst_lse, d_kind, g,
                                         shape->B * shape->H, shape->d, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status vsa_profile_heads(const void* q, const void* k, const void* v, const vsa_shape* shape,
                             const vsa_params* params, uint8_t* d_kind, float* d_mse, void* ws, size_t ws_bytes,
                             int* d_err, cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!q || !k || !v || !params || !d_kind || !d_mse || !ws || !d_err) return VSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(ws)) return VSA_ERR_INVALID_ARG;
  if (!(params->profile_frac > 0.0) || params->profile_frac > 1.0 || params->w_s < 0 || params->w_t < 0)
    return VSA_ERR_INVALID_ARG;
  const int BH = shape->B * shape->H;
  const ProfilePlan plan = profile_plan(g, BH, shape->d, params->profile_frac);
  if (ws_bytes < plan.bytes) return VSA_ERR_WORKSPACE;
  if (!on_device({q, k, v, d_kind, d_mse, ws, d_err})) return VSA_ERR_INVALID_ARG;
  const cudaError_t e = launch_profile(q, k, v, g, BH, shape->d, params->w_s, params->w_t,
                                       scale_log2_of(params->scale, shape->d), plan, ws, d_kind, d_mse, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status vsa_build_mask(const uint8_t* d_kind, const void* q_cube, const void* k_cube, const vsa_shape* shape,
                          const vsa_params* params, uint32_t* d_bits, int32_t* d_kv_idx, int32_t* d_kv_cnt, int max_kv,
                          void* ws, size_t ws_bytes, int* d_err, cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!d_kind || !params || !d_bits || !d_kv_idx || !d_kv_cnt || !d_err || max_kv <= 0) return VSA_ERR_INVALID_ARG;
  if (params->w_s < 0 || params->w_t < 0) return VSA_ERR_INVALID_ARG;
  const int BH = shape->B * shape->H;
  if (!on_device({d_kind, d_bits, d_kv_idx, d_kv_cnt, d_err})) return VSA_ERR_INVALID_ARG;
  if (g.ncubes > 0 && !on_device({q_cube, k_cube, ws})) return VSA_ERR_INVALID_ARG;
  cudaError_t e = launch_pattern_mask(d_kind, g, BH, params->w_s, params->w_t, d_bits, d_kv_idx, d_kv_cnt, max_kv,
                                      d_err, stream);
  if (e != cudaSuccess) return VSA_ERR_CUDA;
  if (g.ncubes > 0) {
    if (!q_cube || !k_cube || !ws || !aligned16(q_cube) || !aligned16(k_cube) || !aligned16(ws) || params->topk < 0)
      return VSA_ERR_INVALID_ARG;
    if (ws_bytes < cube_mask_workspace_bytes(g, BH, shape->d)) return VSA_ERR_WORKSPACE;
    e = launch_cube_mask(d_kind, q_cube, k_cube, g, BH, shape->d, params->topk, d_bits, d_kv_idx, d_kv_cnt, max_kv,
                         ws, d_err, stream);
    if (e != cudaSuccess) return VSA_ERR_CUDA;
  }
  return VSA_OK;
}

static vsa_status check_qkvo(const vsa_qkvo* t) {
  if (t == nullptr || !t->q || !t->k || !t->v || !t->o) return VSA_ERR_INVALID_ARG;
  if (!aligned16(t->q) || !aligned16(t->k) || !aligned16(t->v) || !aligned16(t->o)) return VSA_ERR_INVALID_ARG;
  return VSA_OK;
}

static vsa_status encode_set(AttnMaps* m, const vsa_qkvo* t, const Geom& g, int rows, int BH, int d) {
  if (encode_rows_map(&m->q, t->q, d, rows, BH, 128) != cudaSuccess) return VSA_ERR_CUDA;
  if (encode_rows_map(&m->k, t->k, d, rows, BH, g.block) != cudaSuccess) return VSA_ERR_CUDA;
  if (encode_rows_map(&m->v, t->v, d, rows, BH, g.block) != cudaSuccess) return VSA_ERR_CUDA;
  if (encode_rows_map(&m->o, t->o, d, rows, BH, g.block) != cudaSuccess) return VSA_ERR_CUDA;
  return VSA_OK;
}

vsa_status vsa_block_order(const uint8_t* d_kind, const int32_t* d_kv_idx, const int32_t* d_kv_cnt, int max_kv,
                           const vsa_shape* shape, int32_t* d_order, cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!d_kind || !d_kv_idx || !d_kv_cnt || !d_order || max_kv <= 0) return VSA_ERR_INVALID_ARG;
  if (g.nblk > 32768) return VSA_ERR_UNSUPPORTED;
  if (!on_device({d_kind, d_kv_idx, d_kv_cnt, d_order})) return VSA_ERR_INVALID_ARG;
  const cudaError_t e = launch_block_order(d_kind, g, shape->B * shape->H, d_kv_idx, d_kv_cnt, max_kv, d_order,
                                           stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

// e4m3 Q and K for vsa_sparse_attn_fwd_fp8qk (all null for bf16).
struct Fp8QK {
  const uint8_t* q8;
  const int32_t* qexp;
  const uint8_t* k8;
  const int32_t* kexp;
};

static vsa_status sparse_attn_fwd_impl(const vsa_qkvo* natural, const vsa_qkvo* permuted, const Fp8QK& f8,
                                       const uint8_t* d_kind, const int32_t* d_kv_idx, const int32_t* d_kv_cnt,
                                       int max_kv, const int32_t* d_order, const vsa_shape* shape, float scale,
                                       int* d_err, cudaStream_t stream, void* lo_nat = nullptr,
                                       void* lo_perm = nullptr) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if ((st = check_qkvo(natural)) != VSA_OK) return st;
  if (permuted != nullptr && (st = check_qkvo(permuted)) != VSA_OK) return st;
  if (!d_kind || !d_kv_idx || !d_kv_cnt || !d_err || max_kv <= 0 || !(scale >= 0.f)) return VSA_ERR_INVALID_ARG;
  const bool qk8 = f8.q8 != nullptr;
  if (qk8) {
    if (!f8.qexp || !f8.k8 || !f8.kexp || !aligned16(f8.q8) || !aligned16(f8.k8)) return VSA_ERR_INVALID_ARG;
    if (shape->d != 128 || shape->block != 128) return VSA_ERR_UNSUPPORTED;
    if (!on_device({f8.q8, f8.qexp, f8.k8, f8.kexp})) return VSA_ERR_INVALID_ARG;
  }
  const int BH = shape->B * shape->H;
  if (!on_device({natural->q, natural->k, natural->v, natural->o, natural->lse, d_kind, d_kv_idx, d_kv_cnt, d_order,
                  d_err}))
    return VSA_ERR_INVALID_ARG;
  if (permuted != nullptr &&
      !on_device({permuted->q, permuted->k, permuted->v, permuted->o, permuted->lse}))
    return VSA_ERR_INVALID_ARG;
  AttnMaps nat, perm;
  // Without a permuted set every head reads the `natural` buffers, whose rows must then
  // cover every head's layout (R rows per head).
  const int nat_rows = permuted != nullptr ? g.N : g.R;
  if ((st = encode_set(&nat, natural, g, nat_rows, BH, shape->d)) != VSA_OK) return st;
  if (permuted != nullptr) {
    if ((st = encode_set(&perm, permuted, g, g.R, BH, shape->d)) != VSA_OK) return st;
  } else {
    perm = nat;
  }
  if (qk8) {  // every head's Q and K come from the e4m3 buffers (R rows per head, its own layout)
    if (encode_rows_map_u8(&nat.q, f8.q8, shape->d, g.R, BH, 128) != cudaSuccess) return VSA_ERR_CUDA;
    if (encode_rows_map_u8(&nat.k, f8.k8, shape->d, g.R, BH, g.block) != cudaSuccess) return VSA_ERR_CUDA;
    perm.q = nat.q;
    perm.k = nat.k;
  }
  AttnArgs a;
  a.kinds = d_kind;
  a.kv_idx = d_kv_idx;
  a.kv_cnt = d_kv_cnt;
  a.order = d_order;
  a.lse_nat = natural->lse;
  a.lse_perm = permuted != nullptr ? permuted->lse : natural->lse;
  a.err = d_err;
  a.BH = BH;
  a.max_kv = max_kv;
  a.has_perm = permuted != nullptr ? 1 : 0;
  a.scale_log2 = scale_log2_of(scale, shape->d);
  a.g = g;
  a.nat_rows = nat_rows;
  a.ucap = std::min(g.nblk, 2 * max_kv);
  a.gather = 0;
  a.qexp = qk8 ? f8.qexp : nullptr;
  a.kexp = qk8 ? f8.kexp : nullptr;
  a.nat_q = a.nat_k = a.nat_v = nullptr;
  a.nat_o = natural->o;  // written only for a head with an invalid kind byte (zero rows)
  a.lo_nat = lo_nat;
  a.lo_perm = permuted != nullptr ? lo_perm : lo_nat;
  const cudaError_t e = launch_sparse_attn(nat, perm, a, shape->d, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status vsa_sparse_attn_fwd(const vsa_qkvo* natural, const vsa_qkvo* permuted, const uint8_t* d_kind,
                               const int32_t* d_kv_idx, const int32_t* d_kv_cnt, int max_kv,
                               const int32_t* d_order, const vsa_shape* shape, float scale, int* d_err,
                               cudaStream_t stream) {
  return sparse_attn_fwd_impl(natural, permuted, Fp8QK{nullptr, nullptr, nullptr, nullptr}, d_kind, d_kv_idx,
                              d_kv_cnt, max_kv, d_order, shape, scale, d_err, stream);
}

vsa_status vsa_sparse_attn_fwd_fp8qk(const vsa_qkvo* natural, const vsa_qkvo* permuted, const uint8_t* q8,
                                     const int32_t* d_qexp, const uint8_t* k8, const int32_t* d_kexp,
                                     const uint8_t* d_kind, const int32_t* d_kv_idx, const int32_t* d_kv_cnt,
                                     int max_kv, const int32_t* d_order, const vsa_shape* shape, float scale,
                                     int* d_err, cudaStream_t stream) {
  if (!q8) return VSA_ERR_INVALID_ARG;
  return sparse_attn_fwd_impl(natural, permuted, Fp8QK{q8, d_qexp, k8, d_kexp}, d_kind, d_kv_idx, d_kv_cnt, max_kv,
                              d_order, shape, scale, d_err, stream);
}

vsa_status vsa_quantize_fp8(const void* natural, const void* permuted, const uint8_t* d_kind,
                            const vsa_shape* shape, uint8_t* dst, int32_t* d_exp, int* d_err, cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!natural || !d_kind || !dst || !d_exp || !d_err) return VSA_ERR_INVALID_ARG;
  if (!aligned16(natural) || (permuted && !aligned16(permuted)) || !aligned16(dst)) return VSA_ERR_INVALID_ARG;
  if (shape->d != 128) return VSA_ERR_UNSUPPORTED;
  if (!on_device({natural, permuted, d_kind, dst, d_exp, d_err})) return VSA_ERR_INVALID_ARG;
  const int nat_rows = permuted != nullptr ? g.N : g.R;
  const cudaError_t e = launch_quantize_e4m3(natural, permuted, d_kind, g, shape->B * shape->H, shape->d, nat_rows,
                                             dst, d_exp, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

static vsa_status sparse_attn_fwd_natural_impl(const vsa_qkvo* natural, const uint8_t* d_kind,
                                               const int32_t* d_kv_idx, const int32_t* d_kv_cnt, int max_kv,
                                               const int32_t* d_order, const vsa_shape* shape, float scale, int* d_err,
                                               cudaStream_t stream, void* lo) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (g.ncubes > 0) return VSA_ERR_UNSUPPORTED;  // cube heads read cube-major copies
  if ((st = check_qkvo(natural)) != VSA_OK) return st;
  if (!d_kind || !d_kv_idx || !d_kv_cnt || !d_err || max_kv <= 0 || !(scale >= 0.f)) return VSA_ERR_INVALID_ARG;
  const int BH = shape->B * shape->H;
  if (!on_device({natural->q, natural->k, natural->v, natural->o, natural->lse, d_kind, d_kv_idx, d_kv_cnt, d_order,
                  d_err}))
    return VSA_ERR_INVALID_ARG;
  AttnMaps nat;
  if ((st = encode_set(&nat, natural, g, g.N, BH, shape->d)) != VSA_OK) return st;
  AttnArgs a;
  a.kinds = d_kind;
  a.kv_idx = d_kv_idx;
  a.kv_cnt = d_kv_cnt;
  a.order = d_order;
  a.lse_nat = natural->lse;
  a.lse_perm = natural->lse;
  a.err = d_err;
  a.BH = BH;
  a.max_kv = max_kv;
  a.has_perm = 0;
  a.scale_log2 = scale_log2_of(scale, shape->d);
  a.g = g;
  a.nat_rows = g.N;
  a.ucap = std::min(g.nblk, 2 * max_kv);
  a.gather = 1;
  a.qexp = a.kexp = nullptr;
  a.nat_q = natural->q;
  a.nat_k = natural->k;
  a.nat_v = natural->v;
  a.nat_o = natural->o;
  a.lo_nat = a.lo_perm = lo;
  const cudaError_t e = launch_sparse_attn(nat, nat, a, shape->d, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status vsa_sparse_attn_fwd_natural(const vsa_qkvo* natural, const uint8_t* d_kind, const int32_t* d_kv_idx,
                                       const int32_t* d_kv_cnt, int max_kv, const int32_t* d_order,
                                       const vsa_shape* shape, float scale, int* d_err, cudaStream_t stream) {
  return sparse_attn_fwd_natural_impl(natural, d_kind, d_kv_idx, d_kv_cnt, max_kv, d_order, shape, scale, d_err, stream,
                                      nullptr);
}

// ---------------------------------------------------------------------------------------
// Gradient of the attention
// ---------------------------------------------------------------------------------------
// Workspace of vsa_sparse_attn_bwd: one bitset of every query block, two terms and the sum of dS of every row.
struct BwdLayout {
  size_t off_bits, off_terms, off_target, bytes;
};

static BwdLayout bwd_layout(const Geom& g, int BH) {
  BwdLayout L;
  const size_t rows = static_cast<size_t>(BH) * g.nblk;
  L.off_bits = 0;
  L.off_terms = align256(rows * ((g.nblk + 31) / 32) * 4);
  L.off_target = L.off_terms + align256(rows * g.block * 8);
  L.bytes = L.off_target + align256(rows * g.block * 4);
  return L;
}

static vsa_status check_grad(const vsa_qkvo_grad* t) {
  if (t == nullptr) return VSA_ERR_INVALID_ARG;
  for (const void* p : {t->q, t->k, t->v, t->o, t->d_o, static_cast<const void*>(t->lse),
                        static_cast<const void*>(t->dq), static_cast<const void*>(t->dk),
                        static_cast<const void*>(t->dv)})
    if (p == nullptr || !aligned16(p)) return VSA_ERR_INVALID_ARG;
  if (t->dq == t->dk || t->dq == t->dv || t->dk == t->dv) return VSA_ERR_INVALID_ARG;
  for (const void* in : {t->q, t->k, t->v, t->o, t->d_o, t->o_lo})  // other CTAs still read them
    if (in == t->dq || in == t->dk || in == t->dv) return VSA_ERR_INVALID_ARG;
  return VSA_OK;
}

static bool grad_on_device(const vsa_qkvo_grad* t) {
  return aligned16(t->o_lo) &&
         on_current_device({t->q, t->k, t->v, t->o, t->d_o, t->lse, t->d_lse, t->dq, t->dk, t->dv, t->o_lo});
}

// The set's gradients (rows of d elements of es bytes) and the workspace apart from what else the set holds.
static bool grad_apart(const vsa_qkvo_grad* t, size_t rows, int d, int es, const void* ws, size_t ws_bytes) {
  const size_t n = rows * d * es, l = rows * 4;
  return apart({{t->dq, n}, {t->dk, n}, {t->dv, n}, {ws, ws_bytes}},
               {{t->q, n}, {t->k, n}, {t->v, n}, {t->o, n}, {t->d_o, n}, {t->o_lo, n}, {t->lse, l}, {t->d_lse, l}});
}

static vsa_status encode_bwd_set(BwdMaps* m, const vsa_qkvo_grad* t, const Geom& g, int rows, int BH, int d) {
  const struct {
    CUtensorMap* map;
    const void* p;
  } all[] = {{&m->q, t->q}, {&m->k, t->k}, {&m->v, t->v}, {&m->g, t->d_o}, {&m->dq, t->dq}, {&m->dk, t->dk}, {&m->dv, t->dv}};
  for (const auto& x : all)
    if (encode_rows_map(x.map, x.p, d, rows, BH, g.block) != cudaSuccess) return VSA_ERR_CUDA;
  return VSA_OK;
}

// The row terms from `rows` (O, dO, LSE: each head's layout, or natural order when by_token), then the
// gradients of the two sets.  Arguments are checked by the callers.
static vsa_status sparse_attn_bwd_impl(const vsa_qkvo_grad* natural, const vsa_qkvo_grad* permuted,
                                       const vsa_qkvo_grad* rows, bool by_token, bool f32, const uint8_t* d_kind,
                                       const int32_t* d_kv_idx, const int32_t* d_kv_cnt, int max_kv, const Geom& g,
                                       int BH, int d, float scale, void* ws, int* d_err, cudaStream_t stream) {
  vsa_status st;
  BwdMaps nat, perm;
  const int nat_rows = permuted != nullptr ? g.N : g.R;
  if ((st = encode_bwd_set(&nat, natural, g, nat_rows, BH, d)) != VSA_OK) return st;
  perm = nat;
  if (permuted != nullptr && (st = encode_bwd_set(&perm, permuted, g, g.R, BH, d)) != VSA_OK) return st;
  const BwdLayout L = bwd_layout(g, BH);
  uint8_t* w = static_cast<uint8_t*>(ws);
  BwdPrep p{};
  p.kinds = d_kind;
  p.kv_idx = d_kv_idx;
  p.kv_cnt = d_kv_cnt;
  p.o_nat = rows->o;
  p.do_nat = rows->d_o;
  p.lse_nat = rows->lse;
  p.dlse_nat = rows->d_lse;
  if (permuted != nullptr) {
    p.o_perm = permuted->o;
    p.do_perm = permuted->d_o;
    p.lse_perm = permuted->lse;
    p.dlse_perm = permuted->d_lse;
  }
  p.rbits = reinterpret_cast<uint32_t*>(w + L.off_bits);
  p.terms = reinterpret_cast<float*>(w + L.off_terms);
  // with O's rounding errors from every set that is read, delta is exact
  const bool exact = rows->o_lo != nullptr && (by_token || permuted == nullptr || permuted->o_lo != nullptr);
  p.lo_nat = exact ? rows->o_lo : nullptr;
  p.lo_perm = exact && permuted != nullptr ? permuted->o_lo : nullptr;
  p.target = exact ? reinterpret_cast<float*>(w + L.off_target) : nullptr;
  p.err = d_err;
  p.BH = BH;
  p.d = d;
  p.max_kv = max_kv;
  p.has_perm = permuted != nullptr;
  p.nat_rows = nat_rows;
  p.by_token = by_token;
  p.f32 = f32;
  p.g = g;
  BwdArgs a{};
  a.kinds = d_kind;
  a.rbits = p.rbits;
  a.terms = p.terms;
  a.target = p.target;
  a.exact = exact;
  a.err = d_err;
  a.nat_dq = natural->dq;
  a.nat_dk = natural->dk;
  a.nat_dv = natural->dv;
  a.BH = BH;
  a.has_perm = permuted != nullptr;
  a.nat_rows = nat_rows;
  a.scale_log2 = scale_log2_of(scale, d);
  a.scale = scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(d));
  a.g = g;
  return launch_sparse_attn_bwd(nat, perm, p, a, d, stream) == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

size_t vsa_sparse_attn_bwd_workspace_size(const vsa_shape* shape) {
  Geom g;
  if (make_geom(shape, &g) != VSA_OK || !sparse_attn_bwd_fits(g, shape->B * shape->H)) return 0;
  return bwd_layout(g, shape->B * shape->H).bytes;
}

vsa_status vsa_sparse_attn_bwd(const vsa_qkvo_grad* natural, const vsa_qkvo_grad* permuted, const uint8_t* d_kind,
                               const int32_t* d_kv_idx, const int32_t* d_kv_cnt, int max_kv, const vsa_shape* shape,
                               float scale, void* ws, size_t ws_bytes, int* d_err, cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if ((st = check_grad(natural)) != VSA_OK) return st;
  if (permuted != nullptr && (st = check_grad(permuted)) != VSA_OK) return st;
  if (!d_kind || !d_kv_idx || !d_kv_cnt || !d_err || max_kv <= 0 || !(scale >= 0.f) || !ws || !aligned16(ws))
    return VSA_ERR_INVALID_ARG;
  const int BH = shape->B * shape->H;
  if (!sparse_attn_bwd_fits(g, BH)) return VSA_ERR_UNSUPPORTED;
  const size_t need = bwd_layout(g, BH).bytes;
  if (ws_bytes < need) return VSA_ERR_WORKSPACE;
  const size_t perm_rows = static_cast<size_t>(BH) * g.R, nat_rows = permuted != nullptr ? static_cast<size_t>(BH) * g.N : perm_rows;
  if (!grad_apart(natural, nat_rows, shape->d, 2, ws, need) ||
      (permuted != nullptr && !grad_apart(permuted, perm_rows, shape->d, 2, ws, need)))
    return VSA_ERR_INVALID_ARG;
  if (!grad_on_device(natural) || (permuted != nullptr && !grad_on_device(permuted)) ||
      !on_current_device({d_kind, d_kv_idx, d_kv_cnt, ws, d_err}))
    return VSA_ERR_INVALID_ARG;
  return sparse_attn_bwd_impl(natural, permuted, natural, false, false, d_kind, d_kv_idx, d_kv_cnt, max_kv, g, BH,
                              shape->d, scale, ws, d_err, stream);
}

// ---------------------------------------------------------------------------------------
// Root-mean-square norm
// ---------------------------------------------------------------------------------------
static bool known_dtype(vsa_dtype t) { return t == VSA_F32 || t == VSA_BF16; }

static bool on_elements(const void* p, vsa_dtype t) {
  return reinterpret_cast<uintptr_t>(p) % (t == VSA_F32 ? 4 : 2) == 0;
}

// Strides of a [B, H, N] array of rows: as given, or contiguous where all three are 0.
static vsa_status norm_strides(const vsa_norm_shape* s, const int64_t (&given)[3], int64_t (&out)[3]) {
  const int64_t most = INT64_C(1) << 46, size[3] = {s->B, s->H, s->N};
  for (int i = 0; i < 3; ++i)
    if (given[i] < 0 || given[i] > most / size[i]) return VSA_ERR_INVALID_ARG;
  const bool contiguous = given[0] == 0 && given[1] == 0 && given[2] == 0;
  const int64_t d = s->d;
  out[0] = contiguous ? d * s->N * s->H : given[0];
  out[1] = contiguous ? d * s->N : given[1];
  out[2] = contiguous ? d : given[2];
  return VSA_OK;
}

static vsa_status norm_args(const vsa_norm_shape* s, NormArgs* a) {
  if (s == nullptr) return VSA_ERR_INVALID_ARG;
  if (s->B <= 0 || s->H <= 0 || s->N <= 0 || s->d <= 0 || !(s->eps >= 0.f) || !std::isfinite(s->eps))
    return VSA_ERR_INVALID_ARG;
  if (s->d > 16384 || s->N > (1 << 28)) return VSA_ERR_UNSUPPORTED;
  const long long heads = static_cast<long long>(s->B) * s->H;
  if (heads > 0x7fffffffLL || heads * s->N > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;  // one CTA per row at most
  vsa_status st;
  if ((st = norm_strides(s, s->x_stride, a->x_stride)) != VSA_OK) return st;
  if ((st = norm_strides(s, s->res_stride, a->res_stride)) != VSA_OK) return st;
  a->BH = static_cast<int>(heads);
  a->H = s->H;
  a->N = s->N;
  a->d = s->d;
  a->block = 1;
  a->eps = s->eps;
  return VSA_OK;
}

vsa_status vsa_rms_norm(const void* x, const void* residual, vsa_dtype dtype, const void* weight,
                        vsa_dtype weight_dtype, const vsa_norm_shape* shape, void* sum, void* y, uint8_t* codes,
                        int32_t* d_exp, float* rstd, cudaStream_t stream) {
  NormArgs a{};
  vsa_status st = norm_args(shape, &a);
  if (st != VSA_OK) return st;
  if (!x || !known_dtype(dtype) || (weight && !known_dtype(weight_dtype))) return VSA_ERR_INVALID_ARG;
  if (!y && !codes) return VSA_ERR_INVALID_ARG;
  if ((sum && !residual) || (codes == nullptr) != (d_exp == nullptr)) return VSA_ERR_INVALID_ARG;
  if (!on_elements(x, dtype) || !on_elements(residual, dtype)) return VSA_ERR_INVALID_ARG;
  if (!aligned16(weight) || !aligned16(sum) || !aligned16(y) || !aligned16(codes) || !aligned16(d_exp) ||
      !aligned16(rstd))
    return VSA_ERR_INVALID_ARG;
  for (const void* out : {static_cast<const void*>(sum), static_cast<const void*>(y), static_cast<const void*>(codes)})
    if (out && (out == x || out == residual || out == weight)) return VSA_ERR_INVALID_ARG;
  if (sum && (sum == y || sum == codes)) return VSA_ERR_INVALID_ARG;
  if (codes) {
    if (shape->block != 1 && shape->block != 64 && shape->block != 128) return VSA_ERR_UNSUPPORTED;
    if (shape->block > 1 && shape->d != 64 && shape->d != 128) return VSA_ERR_UNSUPPORTED;
    a.block = shape->block;
  }
  if (!on_current_device({x, residual, weight, sum, y, codes, d_exp, rstd})) return VSA_ERR_INVALID_ARG;
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.w_kind = weight == nullptr ? 0 : weight_dtype == VSA_F32 ? 1 : 2;
  a.sum = sum;
  a.y = y;
  a.codes = codes;
  a.exps = d_exp;
  a.rstd = rstd;
  return launch_rms_norm(a, dtype == VSA_F32, stream) == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

size_t vsa_rms_norm_bwd_workspace_size(const vsa_norm_shape* shape, vsa_dtype dtype) {
  NormArgs a{};
  if (norm_args(shape, &a) != VSA_OK || !known_dtype(dtype)) return 0;
  return align256(rms_norm_bwd_partials(static_cast<long long>(a.BH) * a.N, a.d, dtype == VSA_F32) * a.d * 4);
}

vsa_status vsa_rms_norm_bwd(const void* dy, const void* d_sum, const void* s, vsa_dtype dtype, const void* weight,
                            vsa_dtype weight_dtype, const float* rstd, const vsa_norm_shape* shape, void* dx,
                            float* d_weight, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NormBwdArgs a{};
  vsa_status st = norm_args(shape, &a.n);
  if (st != VSA_OK) return st;
  if (!dy || !s || !rstd || !dx || !known_dtype(dtype) || (weight && !known_dtype(weight_dtype)))
    return VSA_ERR_INVALID_ARG;
  if (!on_elements(s, dtype) || !on_elements(dx, dtype) || !aligned16(dy) || !aligned16(d_sum) || !aligned16(weight) ||
      !aligned16(rstd) || !aligned16(d_weight) || !aligned16(ws))
    return VSA_ERR_INVALID_ARG;
  if (dx == dy || dx == d_sum || dx == s) return VSA_ERR_INVALID_ARG;
  // rows of dx must not overlap: each stride has to step over everything the smaller ones span
  struct {
    int64_t stride, size;
  } dims[3] = {{a.n.res_stride[0], shape->B}, {a.n.res_stride[1], shape->H}, {a.n.res_stride[2], shape->N}};
  std::sort(dims, dims + 3, [](const auto& p, const auto& q) { return p.stride < q.stride; });
  int64_t span = a.n.d;
  for (const auto& m : dims) {
    if (m.size == 1) continue;
    if (m.stride < span) return VSA_ERR_INVALID_ARG;
    span += m.stride * (m.size - 1);
  }
  if (d_weight) {
    if (!ws) return VSA_ERR_INVALID_ARG;
    if (ws_bytes < vsa_rms_norm_bwd_workspace_size(shape, dtype)) return VSA_ERR_WORKSPACE;
  }
  if (!on_current_device({dy, d_sum, s, weight, rstd, dx, d_weight, d_weight ? ws : nullptr})) return VSA_ERR_INVALID_ARG;
  a.n.x = s;
  a.n.w = weight;
  a.n.w_kind = weight == nullptr ? 0 : weight_dtype == VSA_F32 ? 1 : 2;
  a.n.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.d_sum = d_sum;
  a.dx = dx;
  a.partial = d_weight ? static_cast<float*>(ws) : nullptr;
  return launch_rms_norm_bwd(a, dtype == VSA_F32, d_weight, stream) == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

// ---------------------------------------------------------------------------------------
// Semantic-aware permutation ("Sparse VideoGen2" page, abstract)
// ---------------------------------------------------------------------------------------
// Shapes of the semantic path: no cube dims (every head has N rows).
static vsa_status semantic_geom(const vsa_shape* shape, Geom* g) {
  vsa_status st = make_geom(shape, g);
  if (st != VSA_OK) return st;
  if (g->ncubes > 0) return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}

static bool clusters_ok(const Geom& g, int C) { return C >= 1 && C <= kMaxClusters && C <= g.N; }

size_t vsa_kmeans_workspace_size(const vsa_shape* shape, int n_clusters) {
  Geom g;
  if (semantic_geom(shape, &g) != VSA_OK || !clusters_ok(g, n_clusters)) return 0;
  return kmeans_workspace_bytes(shape->B * shape->H, g.N, n_clusters, shape->d);
}

vsa_status vsa_kmeans(const void* x, const vsa_shape* shape, int n_clusters, int iters, float* d_centroids,
                      int32_t* d_labels, int32_t* d_counts, int32_t* d_perm, void* ws, size_t ws_bytes, int* d_err,
                      cudaStream_t stream) {
  Geom g;
  vsa_status st = semantic_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!clusters_ok(g, n_clusters) || iters < 1 || iters > 1000) return VSA_ERR_INVALID_ARG;
  if (!x || !d_centroids || !d_labels || !d_counts || !d_perm || !ws || !d_err || !aligned16(x) ||
      !aligned16(d_centroids))
    return VSA_ERR_INVALID_ARG;
  if (ws_bytes < vsa_kmeans_workspace_size(shape, n_clusters)) return VSA_ERR_WORKSPACE;
  if (!on_device({x, d_centroids, d_labels, d_counts, d_perm, ws, d_err})) return VSA_ERR_INVALID_ARG;
  const cudaError_t e = launch_kmeans(x, shape->B * shape->H, g.N, shape->d, n_clusters, iters, d_centroids,
                                      d_labels, d_counts, d_perm, ws, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

size_t vsa_semantic_mask_workspace_size(const vsa_shape* shape) {
  Geom g;
  if (semantic_geom(shape, &g) != VSA_OK) return 0;
  return align256(semantic_mask_workspace_bytes(shape->B * shape->H, g.N, g.block));
}

vsa_status vsa_semantic_mask(const float* d_cent_q, const int32_t* d_counts_q, const int32_t* d_labels_q,
                             const int32_t* d_perm_q, int cq, const float* d_cent_k, const int32_t* d_counts_k,
                             const int32_t* d_labels_k, const int32_t* d_perm_k, int ck, const vsa_shape* shape,
                             float top_p, float scale, uint32_t* d_keep, uint32_t* d_bits, int32_t* d_kv_idx,
                             int32_t* d_kv_cnt, int max_kv, void* ws, size_t ws_bytes, int* d_err,
                             cudaStream_t stream) {
  Geom g;
  vsa_status st = semantic_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!clusters_ok(g, cq) || !clusters_ok(g, ck)) return VSA_ERR_INVALID_ARG;
  if (!(top_p > 0.f && top_p <= 1.f) || !(scale >= 0.f) || max_kv <= 0) return VSA_ERR_INVALID_ARG;
  if (!d_cent_q || !d_counts_q || !d_labels_q || !d_perm_q || !d_cent_k || !d_counts_k || !d_labels_k ||
      !d_perm_k || !d_keep || !d_bits || !d_kv_idx || !d_kv_cnt || !ws || !d_err || !aligned16(ws))
    return VSA_ERR_INVALID_ARG;
  if (ws_bytes < vsa_semantic_mask_workspace_size(shape)) return VSA_ERR_WORKSPACE;
  if (!on_device({d_cent_q, d_counts_q, d_labels_q, d_perm_q, d_cent_k, d_counts_k, d_labels_k, d_perm_k, d_keep,
                  d_bits, d_kv_idx, d_kv_cnt, ws, d_err}))
    return VSA_ERR_INVALID_ARG;
  const double sc = scale > 0.f ? static_cast<double>(scale) : 1.0 / std::sqrt(static_cast<double>(shape->d));
  const cudaError_t e = launch_semantic_mask(d_cent_q, d_counts_q, d_labels_q, d_perm_q, cq, d_cent_k, d_counts_k,
                                             d_labels_k, d_perm_k, ck, shape->B * shape->H, g.N, shape->d, g.block,
                                             sc, static_cast<double>(top_p), d_keep, d_bits, d_kv_idx, d_kv_cnt,
                                             max_kv, ws, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status vsa_gather_rows(const void* src, const int32_t* d_perm, void* dst, const vsa_shape* shape, int* d_err,
                           cudaStream_t stream) {
  Geom g;
  vsa_status st = semantic_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!src || !d_perm || !dst || !d_err || !aligned16(src) || !aligned16(dst)) return VSA_ERR_INVALID_ARG;
  if (!on_device({src, d_perm, dst, d_err})) return VSA_ERR_INVALID_ARG;
  const cudaError_t e = launch_gather_rows(src, d_perm, dst, shape->B * shape->H, g.N, shape->d, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status vsa_scatter_rows(const void* src, const float* src_lse, const int32_t* d_perm, void* dst, float* dst_lse,
                            const vsa_shape* shape, int* d_err, cudaStream_t stream) {
  Geom g;
  vsa_status st = semantic_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!src || !d_perm || !dst || !d_err || !aligned16(src) || !aligned16(dst)) return VSA_ERR_INVALID_ARG;
  if ((src_lse == nullptr) != (dst_lse == nullptr)) return VSA_ERR_INVALID_ARG;
  if (!on_device({src, src_lse, d_perm, dst, dst_lse, d_err})) return VSA_ERR_INVALID_ARG;
  const cudaError_t e =
      launch_scatter_rows(src, src_lse, d_perm, dst, dst_lse, shape->B * shape->H, g.N, shape->d, d_err, stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

// Workspace of the whole semantic call.
struct SemLayout {
  size_t kinds, cent_q, lab_q, cnt_q, perm_q, cent_k, lab_k, cnt_k, perm_k, offs, keep, bits, idx, cnt, mws, pq, pk,
      pv, po, plse, bytes;
  int max_kv;
};

static vsa_status semantic_layout(const vsa_shape* shape, const vsa_semantic_params* sp, SemLayout* L) {
  Geom g;
  vsa_status st = semantic_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (sp == nullptr || L == nullptr) return VSA_ERR_INVALID_ARG;
  if (!clusters_ok(g, sp->cq) || !clusters_ok(g, sp->ck) || sp->iters < 1 || sp->iters > 1000) return VSA_ERR_INVALID_ARG;
  if (!(sp->top_p > 0.f && sp->top_p <= 1.f) || !(sp->scale >= 0.f)) return VSA_ERR_INVALID_ARG;
  const size_t BH = static_cast<size_t>(shape->B) * shape->H, N = g.N, d = shape->d, nb = g.nblk;
  const size_t kwords = (sp->ck + 31) / 32, bwords = (nb + 31) / 32;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  L->kinds = take(BH);
  L->cent_q = take(BH * sp->cq * d * 4);
  L->lab_q = take(BH * N * 4);
  L->cnt_q = take(BH * sp->cq * 4);
  L->perm_q = take(BH * N * 4);
  L->cent_k = take(BH * sp->ck * d * 4);
  L->lab_k = take(BH * N * 4);
  L->cnt_k = take(BH * sp->ck * 4);
  L->perm_k = take(BH * N * 4);
  L->offs = take(kmeans_workspace_bytes(static_cast<int>(BH), g.N, std::max(sp->cq, sp->ck), static_cast<int>(d)));
  L->keep = take(BH * sp->cq * kwords * 4);
  L->bits = take(BH * nb * bwords * 4);
  L->idx = take(BH * nb * nb * 4);
  L->cnt = take(BH * nb * 4);
  L->mws = take(semantic_mask_workspace_bytes(static_cast<int>(BH), g.N, g.block));
  L->pq = take(BH * N * d * 2);
  L->pk = take(BH * N * d * 2);
  L->pv = take(BH * N * d * 2);
  L->po = take(BH * N * d * 2);
  L->plse = take(BH * N * 4);
  L->bytes = off;
  L->max_kv = static_cast<int>(nb);
  return VSA_OK;
}

size_t vsa_semantic_workspace_size(const vsa_shape* shape, const vsa_semantic_params* params) {
  SemLayout L;
  return semantic_layout(shape, params, &L) == VSA_OK ? L.bytes : 0;
}

vsa_status vsa_semantic_attention(const vsa_qkvo* io, const vsa_shape* shape, const vsa_semantic_params* params,
                                  void* ws, size_t ws_bytes, int* d_err, cudaStream_t stream) {
  SemLayout L;
  vsa_status st = semantic_layout(shape, params, &L);
  if (st != VSA_OK) return st;
  if ((st = check_qkvo(io)) != VSA_OK) return st;
  if (!ws || !d_err || !aligned16(ws)) return VSA_ERR_INVALID_ARG;
  if (ws_bytes < L.bytes) return VSA_ERR_WORKSPACE;
  if (!on_device({io->q, io->k, io->v, io->o, io->lse, ws, d_err})) return VSA_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto f32 = [&](size_t off) { return reinterpret_cast<float*>(w + off); };
  auto i32 = [&](size_t off) { return reinterpret_cast<int32_t*>(w + off); };
  const size_t kmws = L.keep - L.offs;  // bytes reserved for the k-means scratch
  // 1. clusters and cluster-major orders of Q and of K
  if ((st = vsa_kmeans(io->q, shape, params->cq, params->iters, f32(L.cent_q), i32(L.lab_q), i32(L.cnt_q),
                       i32(L.perm_q), w + L.offs, kmws, d_err, stream)) != VSA_OK)
    return st;
  if ((st = vsa_kmeans(io->k, shape, params->ck, params->iters, f32(L.cent_k), i32(L.lab_k), i32(L.cnt_k),
                       i32(L.perm_k), w + L.offs, kmws, d_err, stream)) != VSA_OK)
    return st;
  // 2. rows in cluster-major order: Q by its clusters, K and V by the key clusters
  void *pq = w + L.pq, *pk = w + L.pk, *pv = w + L.pv, *po = w + L.po;
  if ((st = vsa_gather_rows(io->q, i32(L.perm_q), pq, shape, d_err, stream)) != VSA_OK) return st;
  if ((st = vsa_gather_rows(io->k, i32(L.perm_k), pk, shape, d_err, stream)) != VSA_OK) return st;
  if ((st = vsa_gather_rows(io->v, i32(L.perm_k), pv, shape, d_err, stream)) != VSA_OK) return st;
  // 3. top-p cluster budget and the block mask over the two layouts
  if ((st = vsa_semantic_mask(f32(L.cent_q), i32(L.cnt_q), i32(L.lab_q), i32(L.perm_q), params->cq, f32(L.cent_k),
                              i32(L.cnt_k), i32(L.lab_k), i32(L.perm_k), params->ck, shape, params->top_p,
                              params->scale, reinterpret_cast<uint32_t*>(w + L.keep),
                              reinterpret_cast<uint32_t*>(w + L.bits), i32(L.idx), i32(L.cnt), L.max_kv, w + L.mws,
                              ws_bytes - L.mws, d_err, stream)) != VSA_OK)
    return st;
  // 4. attention on the permuted rows.  The kernel reads a VSA_TEMPORAL head's N rows from the
  // permuted set; which permutation produced them does not matter to it.
  uint8_t* kinds = w + L.kinds;
  if (cudaMemsetAsync(kinds, kTemporal, static_cast<size_t>(shape->B) * shape->H, stream) != cudaSuccess)
    return VSA_ERR_CUDA;
  float* plse = io->lse ? f32(L.plse) : nullptr;
  const vsa_qkvo perm_set{pq, pk, pv, po, plse};
  if ((st = vsa_sparse_attn_fwd(io, &perm_set, kinds, i32(L.idx), i32(L.cnt), L.max_kv, nullptr, shape,
                                params->scale, d_err, stream)) != VSA_OK)
    return st;
  // 5. output rows back to token order through the query permutation
  return vsa_scatter_rows(po, plse, i32(L.perm_q), io->o, io->lse, shape, d_err, stream);
}

// ---------------------------------------------------------------------------------------
// Whole call
// ---------------------------------------------------------------------------------------
struct AttnLayout {
  size_t off_bits, off_idx, off_cnt, off_order, off_q, off_k, off_v, off_o, off_lse, off_prof, off_mask;
  size_t off_q8, off_k8, off_qe, off_ke, bytes;
  int max_kv;
};

static vsa_status attention_layout(const vsa_shape* shape, const vsa_params* params, vsa_dtype dtype,
                                   vsa_select select, AttnLayout* L) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (params == nullptr || L == nullptr) return VSA_ERR_INVALID_ARG;
  if (select != VSA_SELECT_PROFILE && select != VSA_SELECT_GIVEN && select != VSA_SELECT_CUBE)
    return VSA_ERR_INVALID_ARG;
  if (select == VSA_SELECT_CUBE && g.ncubes == 0) return VSA_ERR_INVALID_ARG;
  if (select == VSA_SELECT_PROFILE && dtype != VSA_BF16) return VSA_ERR_UNSUPPORTED;
  const bool qk8 = params->qk_fp8 != 0;
  if (qk8 && (dtype != VSA_BF16 || shape->d != 128 || shape->block != 128 || params->layout_in_kernel != 0))
    return VSA_ERR_UNSUPPORTED;
  int max_kv = 0;
  if ((st = vsa_max_kv(shape, params, &max_kv)) != VSA_OK) return st;
  if (max_kv <= 0) max_kv = 1;
  const size_t BH = static_cast<size_t>(shape->B) * shape->H, d = shape->d;
  const size_t nwords = (g.nblk + 31) / 32;
  size_t off = 0;
  L->off_bits = off;
  off = align256(off + BH * g.nblk * nwords * 4);
  L->off_idx = off;
  off = align256(off + BH * g.nblk * max_kv * 4);
  L->off_cnt = off;
  off = align256(off + BH * g.nblk * 4);
  L->off_order = off;
  if (g.ncubes > 0) off = align256(off + BH * g.nblk * 4);
  const bool fused = params->layout_in_kernel != 0 && dtype == VSA_BF16 && g.ncubes == 0;
  const size_t tbytes = fused ? 0 : BH * g.R * d * 2;  // permuted copies (none when fused)
  L->off_q = off;
  off = align256(off + tbytes);
  L->off_k = off;
  off = align256(off + tbytes);
  L->off_v = off;
  off = align256(off + tbytes);
  L->off_o = off;
  off = align256(off + tbytes);
  L->off_lse = off;
  off = align256(off + (fused ? BH * 2 * 4 : BH * g.R * 4));  // fused: only the profiling MSE scratch
  L->off_prof = off;
  if (select == VSA_SELECT_PROFILE) off = align256(off + vsa_profile_workspace_size(shape, params));
  L->off_mask = off;
  off = align256(off + vsa_mask_workspace_size(shape, params));
  // e4m3 Q and K with their per-block scale exponents
  L->off_q8 = off;
  if (qk8) off = align256(off + BH * g.R * d);
  L->off_k8 = off;
  if (qk8) off = align256(off + BH * g.R * d);
  L->off_qe = off;
  if (qk8) off = align256(off + BH * g.nblk * 4);
  L->off_ke = off;
  if (qk8) off = align256(off + BH * g.nblk * 4);
  L->bytes = off;
  L->max_kv = max_kv;
  return VSA_OK;
}

size_t vsa_attention_workspace_size(const vsa_shape* shape, const vsa_params* params, vsa_dtype dtype,
                                    vsa_select select) {
  AttnLayout L;
  return attention_layout(shape, params, dtype, select, &L) == VSA_OK ? L.bytes : 0;
}

vsa_status vsa_attention_workspace_layout(const vsa_shape* shape, const vsa_params* params, vsa_dtype dtype,
                                          vsa_select select, size_t* off_bits, size_t* off_kv_idx,
                                          size_t* off_kv_cnt, int* max_kv) {
  AttnLayout L;
  vsa_status st = attention_layout(shape, params, dtype, select, &L);
  if (st != VSA_OK) return st;
  if (off_bits) *off_bits = L.off_bits;
  if (off_kv_idx) *off_kv_idx = L.off_idx;
  if (off_kv_cnt) *off_kv_cnt = L.off_cnt;
  if (max_kv) *max_kv = L.max_kv;
  return VSA_OK;
}

// o_lo: O's rounding errors in natural order (dtype rows), or null; their permuted rows follow vsa_attention's own
// workspace.
static vsa_status attention_impl(const vsa_qkvo* io, void* o_lo, vsa_dtype dtype, const vsa_shape* shape,
                                 const vsa_params* params, vsa_select select, uint8_t* d_kind, float* d_mse, void* ws,
                                 size_t ws_bytes, int* d_err, cudaStream_t stream) {
  AttnLayout L;
  vsa_status st = attention_layout(shape, params, dtype, select, &L);
  if (st != VSA_OK) return st;
  void* plo = static_cast<uint8_t*>(ws) + L.bytes;
  if (o_lo != nullptr) L.bytes = vsa_attention_train_workspace_size(shape, params, dtype, select);
  if ((st = check_qkvo(io)) != VSA_OK) return st;
  if (!d_kind || !ws || !d_err || !aligned16(ws)) return VSA_ERR_INVALID_ARG;
  if (ws_bytes < L.bytes) return VSA_ERR_WORKSPACE;
  if (dtype != VSA_F32 && dtype != VSA_BF16) return VSA_ERR_INVALID_ARG;
  if (!on_device({io->q, io->k, io->v, io->o, io->lse, d_kind, d_mse, ws, d_err})) return VSA_ERR_INVALID_ARG;
  Geom g;
  make_geom(shape, &g);
  const int BH = shape->B * shape->H;
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint32_t* bits = reinterpret_cast<uint32_t*>(w + L.off_bits);
  int32_t* kv_idx = reinterpret_cast<int32_t*>(w + L.off_idx);
  int32_t* kv_cnt = reinterpret_cast<int32_t*>(w + L.off_cnt);
  void *pq = w + L.off_q, *pk = w + L.off_k, *pv = w + L.off_v, *po = w + L.off_o;
  float* plse = io->lse ? reinterpret_cast<float*>(w + L.off_lse) : nullptr;

  // 1. kinds
  if (select == VSA_SELECT_PROFILE) {
    float* mse = d_mse;
    if (mse == nullptr) mse = reinterpret_cast<float*>(w + L.off_lse);  // scratch before the LSE is written
    if ((st = vsa_profile_heads(io->q, io->k, io->v, shape, params, d_kind, mse, w + L.off_prof,
                                ws_bytes - L.off_prof, d_err, stream)) != VSA_OK)
      return st;
  } else if (select == VSA_SELECT_CUBE) {
    if (cudaMemsetAsync(d_kind, kCube, BH, stream) != cudaSuccess) return VSA_ERR_CUDA;
  }
  // In-kernel layout: no permuted copies for pattern heads; the attention gathers them.
  const bool fused = params->layout_in_kernel != 0 && dtype == VSA_BF16 && g.ncubes == 0;
  if (fused) {
    if ((st = vsa_build_mask(d_kind, nullptr, nullptr, shape, params, bits, kv_idx, kv_cnt, L.max_kv, nullptr, 0,
                             d_err, stream)) != VSA_OK)
      return st;
    return sparse_attn_fwd_natural_impl(io, d_kind, kv_idx, kv_cnt, L.max_kv, nullptr, shape, params->scale, d_err,
                                        stream, o_lo);
  }
  // 2. layouts
  const vsa_dtype src_t = dtype;
  if ((st = vsa_permute(io->q, src_t, pq, d_kind, shape, d_err, stream)) != VSA_OK) return st;
  if ((st = vsa_permute(io->k, src_t, pk, d_kind, shape, d_err, stream)) != VSA_OK) return st;
  if ((st = vsa_permute(io->v, src_t, pv, d_kind, shape, d_err, stream)) != VSA_OK) return st;
  // 3. masks
  if ((st = vsa_build_mask(d_kind, pq, pk, shape, params, bits, kv_idx, kv_cnt, L.max_kv, w + L.off_mask,
                           ws_bytes - L.off_mask, d_err, stream)) != VSA_OK)
    return st;
  // 4. attention: fp32 inputs run every head from the converted buffers.  With cube heads
  // possible, query blocks are paired and scheduled by their first kept key block.
  int32_t* order = nullptr;
  if (g.ncubes > 0) {
    order = reinterpret_cast<int32_t*>(w + L.off_order);
    if ((st = vsa_block_order(d_kind, kv_idx, kv_cnt, L.max_kv, shape, order, stream)) != VSA_OK) return st;
  }
  const vsa_qkvo perm_set{pq, pk, pv, po, plse};
  if (params->qk_fp8 != 0) {  // e4m3 Q and K (bf16 inputs only, checked by attention_layout)
    uint8_t *q8 = w + L.off_q8, *k8 = w + L.off_k8;
    int32_t *qe = reinterpret_cast<int32_t*>(w + L.off_qe), *ke = reinterpret_cast<int32_t*>(w + L.off_ke);
    if ((st = vsa_quantize_fp8(io->q, pq, d_kind, shape, q8, qe, d_err, stream)) != VSA_OK) return st;
    if ((st = vsa_quantize_fp8(io->k, pk, d_kind, shape, k8, ke, d_err, stream)) != VSA_OK) return st;
    st = vsa_sparse_attn_fwd_fp8qk(io, &perm_set, q8, qe, k8, ke, d_kind, kv_idx, kv_cnt, L.max_kv, order, shape,
                                   params->scale, d_err, stream);
  } else if (dtype == VSA_F32) {
    st = sparse_attn_fwd_impl(&perm_set, nullptr, Fp8QK{nullptr, nullptr, nullptr, nullptr}, d_kind, kv_idx, kv_cnt,
                              L.max_kv, order, shape, params->scale, d_err, stream, o_lo != nullptr ? plo : nullptr);
  } else {
    st = sparse_attn_fwd_impl(io, &perm_set, Fp8QK{nullptr, nullptr, nullptr, nullptr}, d_kind, kv_idx, kv_cnt,
                              L.max_kv, order, shape, params->scale, d_err, stream, o_lo,
                              o_lo != nullptr ? plo : nullptr);
  }
  if (st != VSA_OK) return st;
  // 5. back to natural order
  if ((st = vsa_unpermute(po, plse, io->o, dtype, io->lse, d_kind, shape, d_err, stream)) != VSA_OK || o_lo == nullptr)
    return st;
  return vsa_unpermute(plo, nullptr, o_lo, dtype, nullptr, d_kind, shape, d_err, stream);
}

vsa_status vsa_attention(const vsa_qkvo* io, vsa_dtype dtype, const vsa_shape* shape, const vsa_params* params,
                         vsa_select select, uint8_t* d_kind, float* d_mse, void* ws, size_t ws_bytes, int* d_err,
                         cudaStream_t stream) {
  return attention_impl(io, nullptr, dtype, shape, params, select, d_kind, d_mse, ws, ws_bytes, d_err, stream);
}

size_t vsa_attention_train_workspace_size(const vsa_shape* shape, const vsa_params* params, vsa_dtype dtype,
                                          vsa_select select) {
  AttnLayout L;
  Geom g;
  if (attention_layout(shape, params, dtype, select, &L) != VSA_OK || make_geom(shape, &g) != VSA_OK) return 0;
  if (params->qk_fp8 != 0) return 0;
  return align256(L.bytes + static_cast<size_t>(shape->B) * shape->H * g.R * shape->d * 2);
}

vsa_status vsa_attention_train(const vsa_qkvo* io, void* o_lo, vsa_dtype dtype, const vsa_shape* shape,
                               const vsa_params* params, vsa_select select, uint8_t* d_kind, float* d_mse, void* ws,
                               size_t ws_bytes, int* d_err, cudaStream_t stream) {
  if (o_lo == nullptr || !aligned16(o_lo) || io == nullptr || io->lse == nullptr) return VSA_ERR_INVALID_ARG;
  if (params != nullptr && params->qk_fp8 != 0) return VSA_ERR_UNSUPPORTED;
  vsa_status st = check_qkvo(io);
  if (st != VSA_OK) return st;
  Geom g;
  if ((st = make_geom(shape, &g)) != VSA_OK) return st;
  const size_t rows = static_cast<size_t>(shape->B) * shape->H * g.N, n = rows * shape->d * (dtype == VSA_F32 ? 4 : 2);
  if (!apart({{o_lo, n}}, {{io->q, n}, {io->k, n}, {io->v, n}, {io->o, n}, {io->lse, rows * 4}})) return VSA_ERR_INVALID_ARG;
  if (!on_current_device({o_lo})) return VSA_ERR_INVALID_ARG;
  return attention_impl(io, o_lo, dtype, shape, params, select, d_kind, d_mse, ws, ws_bytes, d_err, stream);
}

// Workspace of vsa_attention_bwd: the masks, the permuted q, k, v, dO, dq, dk, dv, the mask and the
// gradient kernels' scratch.
struct AttnBwdLayout {
  size_t off_bits, off_idx, off_cnt, off_t[7], off_mask, mask_bytes, off_bwd, bytes;
  int max_kv;
};

static vsa_status attention_bwd_layout(const vsa_shape* shape, const vsa_params* params, vsa_dtype dtype,
                                       AttnBwdLayout* L) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (params == nullptr || !(params->scale >= 0.f)) return VSA_ERR_INVALID_ARG;
  if (dtype != VSA_F32 && dtype != VSA_BF16) return VSA_ERR_INVALID_ARG;
  if (params->qk_fp8 != 0) return VSA_ERR_UNSUPPORTED;  // the codes have no gradient
  const int BH = shape->B * shape->H;
  if (!sparse_attn_bwd_fits(g, BH)) return VSA_ERR_UNSUPPORTED;
  if ((st = vsa_max_kv(shape, params, &L->max_kv)) != VSA_OK) return st;
  L->max_kv = std::max(L->max_kv, 1);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const size_t lists = static_cast<size_t>(BH) * g.nblk;
  L->off_bits = take(lists * ((g.nblk + 31) / 32) * 4);
  L->off_idx = take(lists * L->max_kv * 4);
  L->off_cnt = take(lists * 4);
  for (size_t& t : L->off_t) t = take(static_cast<size_t>(BH) * g.R * shape->d * 2);
  L->mask_bytes = vsa_mask_workspace_size(shape, params);
  L->off_mask = take(L->mask_bytes);
  L->off_bwd = take(bwd_layout(g, BH).bytes);
  L->bytes = off;
  return VSA_OK;
}

size_t vsa_attention_bwd_workspace_size(const vsa_shape* shape, const vsa_params* params, vsa_dtype dtype) {
  AttnBwdLayout L;
  return attention_bwd_layout(shape, params, dtype, &L) == VSA_OK ? L.bytes : 0;
}

vsa_status vsa_attention_bwd(const vsa_qkvo_grad* io, vsa_dtype dtype, const vsa_shape* shape,
                             const vsa_params* params, const uint8_t* d_kind, void* ws, size_t ws_bytes, int* d_err,
                             cudaStream_t stream) {
  AttnBwdLayout L;
  vsa_status st = attention_bwd_layout(shape, params, dtype, &L);
  if (st != VSA_OK) return st;
  if ((st = check_grad(io)) != VSA_OK) return st;
  if (!d_kind || !ws || !d_err || !aligned16(ws)) return VSA_ERR_INVALID_ARG;
  if (ws_bytes < L.bytes) return VSA_ERR_WORKSPACE;
  if (!grad_on_device(io) || !on_current_device({d_kind, ws, d_err})) return VSA_ERR_INVALID_ARG;
  Geom g;
  make_geom(shape, &g);
  const int BH = shape->B * shape->H;
  if (!grad_apart(io, static_cast<size_t>(BH) * g.N, shape->d, dtype == VSA_F32 ? 4 : 2, ws, L.bytes))
    return VSA_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint32_t* bits = reinterpret_cast<uint32_t*>(w + L.off_bits);
  int32_t* kv_idx = reinterpret_cast<int32_t*>(w + L.off_idx);
  int32_t* kv_cnt = reinterpret_cast<int32_t*>(w + L.off_cnt);
  // 1. each head's layout of q, k, v and dO
  vsa_qkvo_grad set{};
  void* t[7];
  for (int i = 0; i < 7; ++i) t[i] = w + L.off_t[i];
  const void* src[4] = {io->q, io->k, io->v, io->d_o};
  for (int i = 0; i < 4; ++i)
    if ((st = vsa_permute(src[i], dtype, t[i], d_kind, shape, d_err, stream)) != VSA_OK) return st;
  set.q = t[0];
  set.k = t[1];
  set.v = t[2];
  set.d_o = t[3];
  set.dq = t[4];
  set.dk = t[5];
  set.dv = t[6];
  // 2. the call's masks
  if ((st = vsa_build_mask(d_kind, t[0], t[1], shape, params, bits, kv_idx, kv_cnt, L.max_kv, w + L.off_mask,
                           L.mask_bytes, d_err, stream)) != VSA_OK)
    return st;
  // 3. gradients: spatial heads in place for bf16, everything else through the copies
  const bool f32 = dtype == VSA_F32;
  if ((st = sparse_attn_bwd_impl(f32 ? &set : io, f32 ? nullptr : &set, io, true, f32, d_kind, kv_idx, kv_cnt, L.max_kv,
                                 g, BH, shape->d, params->scale, w + L.off_bwd, d_err, stream)) != VSA_OK)
    return st;
  // 4. back to natural order
  void* dst[3] = {io->dq, io->dk, io->dv};
  for (int i = 0; i < 3; ++i)
    if ((st = vsa_unpermute(t[4 + i], nullptr, dst[i], dtype, nullptr, d_kind, shape, d_err, stream)) != VSA_OK)
      return st;
  return VSA_OK;
}

vsa_status vsa_attention_host(const vsa_host_batch* host, int n, const vsa_qkvo* sets, vsa_dtype dtype,
                              const vsa_shape* shape, const vsa_params* params, vsa_select select, uint8_t* d_kind,
                              float* d_mse, void* ws, size_t ws_bytes, int* d_err, cudaStream_t stream_up,
                              cudaStream_t stream_compute, cudaStream_t stream_down) {
  if (host == nullptr || sets == nullptr || n < 0 || shape == nullptr) return VSA_ERR_INVALID_ARG;
  if (dtype != VSA_F32 && dtype != VSA_BF16) return VSA_ERR_INVALID_ARG;
  if (shape->B <= 0 || shape->H <= 0 || shape->F <= 0 || shape->Hl <= 0 || shape->Wl <= 0 || shape->d <= 0)
    return VSA_ERR_INVALID_ARG;
  const size_t bytes = static_cast<size_t>(shape->B) * shape->H * shape->F * shape->Hl * shape->Wl * shape->d *
                       (dtype == VSA_F32 ? 4 : 2);
  for (int i = 0; i < n; ++i)
    if (!host[i].q || !host[i].k || !host[i].v || !host[i].o) return VSA_ERR_INVALID_ARG;
  for (int s = 0; s < 2; ++s) {
    vsa_status st = check_qkvo(&sets[s]);
    if (st != VSA_OK) return st;
  }
  if (n == 0) return VSA_OK;
  // events: uploaded[i], computed[i], downloaded[i] (host-side objects)
  std::vector<cudaEvent_t> ev(3 * static_cast<size_t>(n), nullptr);
  auto cleanup = [&]() {
    for (cudaEvent_t e : ev)
      if (e) cudaEventDestroy(e);
  };
  for (auto& e : ev)
    if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) {
      cleanup();
      return VSA_ERR_CUDA;
    }
  vsa_status st = VSA_OK;
  for (int i = 0; i < n && st == VSA_OK; ++i) {
    const vsa_qkvo& d = sets[i % 2];
    cudaEvent_t up = ev[3 * i], comp = ev[3 * i + 1], down = ev[3 * i + 2];
    // upload: the set must no longer be read by batch i-2's compute
    if (i >= 2 && cudaStreamWaitEvent(stream_up, ev[3 * (i - 2) + 1], 0) != cudaSuccess) st = VSA_ERR_CUDA;
    if (st == VSA_OK &&
        (cudaMemcpyAsync(const_cast<void*>(d.q), host[i].q, bytes, cudaMemcpyHostToDevice, stream_up) != cudaSuccess ||
         cudaMemcpyAsync(const_cast<void*>(d.k), host[i].k, bytes, cudaMemcpyHostToDevice, stream_up) != cudaSuccess ||
         cudaMemcpyAsync(const_cast<void*>(d.v), host[i].v, bytes, cudaMemcpyHostToDevice, stream_up) != cudaSuccess ||
         cudaEventRecord(up, stream_up) != cudaSuccess))
      st = VSA_ERR_CUDA;
    // compute: inputs uploaded, and batch i-2's output has left this set's o
    if (st == VSA_OK && cudaStreamWaitEvent(stream_compute, up, 0) != cudaSuccess) st = VSA_ERR_CUDA;
    if (st == VSA_OK && i >= 2 && cudaStreamWaitEvent(stream_compute, ev[3 * (i - 2) + 2], 0) != cudaSuccess)
      st = VSA_ERR_CUDA;
    if (st == VSA_OK)
      st = vsa_attention(&d, dtype, shape, params, select, d_kind, d_mse, ws, ws_bytes, d_err, stream_compute);
    if (st == VSA_OK && cudaEventRecord(comp, stream_compute) != cudaSuccess) st = VSA_ERR_CUDA;
    // download
    if (st == VSA_OK && (cudaStreamWaitEvent(stream_down, comp, 0) != cudaSuccess ||
                         cudaMemcpyAsync(host[i].o, d.o, bytes, cudaMemcpyDeviceToHost, stream_down) != cudaSuccess ||
                         cudaEventRecord(down, stream_down) != cudaSuccess))
      st = VSA_ERR_CUDA;
  }
  cleanup();
  return st;
}

vsa_status vsa_get_device_error(const int* d_err, cudaStream_t stream, int* host_err) {
  if (d_err == nullptr) return VSA_ERR_INVALID_ARG;
  int h = 0;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return VSA_ERR_CUDA;
  if (cudaMemcpy(&h, d_err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return VSA_ERR_CUDA;
  if (host_err) *host_err = h;
  if (h == 0) return VSA_OK;
  return (h & VSA_DEVERR_TIMEOUT) ? VSA_ERR_TIMEOUT : VSA_ERR_DEVICE;
}

}  // extern "C"

// ---------------------------------------------------------------------------------------
// Profiling without caller-provided scratch
// ---------------------------------------------------------------------------------------
// Some callers cannot allocate device memory for a workspace: a host framework that has
// reserved all device memory for its own pool and hands out only the tensors it owns, or
// a latency-critical path where cudaMalloc's implicit device synchronisation is not
// acceptable.  For them vsa_profile_heads_static keeps its scratch in a fixed device array
// of this file (kStaticProfileScratchBytes, held by every GPU that loads the library until
// the process exits).  The array's host-side name is only a stand-in for the device
// address.  Each call asks the runtime for the array's device address in the current context
// (cudaGetSymbolAddress, a host-side lookup) and passes it to the kernels; no address is
// cached, so a context that was reset and created again gets its own array's address.
namespace vsa {
constexpr size_t kStaticProfileScratchBytes = size_t(16) << 20;
static __device__ __align__(256) uint8_t g_profile_scratch[kStaticProfileScratchBytes];

// Device address of the scratch array in the current device's context.
static cudaError_t profile_scratch_address(void** out) {
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_profile_scratch);
  if (e != cudaSuccess) return e;
  *out = p;
  return cudaSuccess;
}
}  // namespace vsa

extern "C" {

size_t vsa_profile_static_scratch_bytes(void) { return vsa::kStaticProfileScratchBytes; }

vsa_status vsa_profile_heads_static(const void* q, const void* k, const void* v, const vsa_shape* shape,
                                    const vsa_params* params, uint8_t* d_kind, float* d_mse, int* d_err,
                                    cudaStream_t stream) {
  Geom g;
  vsa_status st = make_geom(shape, &g);
  if (st != VSA_OK) return st;
  if (!q || !k || !v || !params || !d_kind || !d_mse || !d_err) return VSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return VSA_ERR_INVALID_ARG;
  if (!(params->profile_frac > 0.0) || params->profile_frac > 1.0 || params->w_s < 0 || params->w_t < 0)
    return VSA_ERR_INVALID_ARG;
  const int BH = shape->B * shape->H;
  // Fewer key-range splits need less scratch; use the largest count that fits.
  ProfilePlan plan = profile_plan(g, BH, shape->d, params->profile_frac);
  for (int s = plan.splits; s >= 1; --s) {
    plan = profile_plan_splits(g, BH, shape->d, params->profile_frac, s);
    if (plan.bytes <= kStaticProfileScratchBytes) break;
  }
  if (plan.bytes > kStaticProfileScratchBytes) return VSA_ERR_WORKSPACE;
  if (!on_device({q, k, v, d_kind, d_mse, d_err})) return VSA_ERR_INVALID_ARG;
  void* scratch = nullptr;
  if (profile_scratch_address(&scratch) != cudaSuccess) return VSA_ERR_CUDA;
  const cudaError_t e = launch_profile(q, k, v, g, BH, shape->d, params->w_s, params->w_t,
                                       scale_log2_of(params->scale, shape->d), plan, scratch, d_kind, d_mse, d_err,
                                       stream);
  return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

}  // extern "C"
