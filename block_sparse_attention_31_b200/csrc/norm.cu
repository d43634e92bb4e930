// norm.cu -- root-mean-square norm of rows (vsa_rms_norm) and its gradient (vsa_rms_norm_bwd).
//
//   s = x + residual      rstd = 1 / sqrt(mean(s^2) + eps)      y = s * rstd * w
//   codes = e4m3(y / 2^e), one e per row or per block of rows, the smallest with max |y| <= 448 * 2^e
//
//   g = dy * w      dx = rstd * (g - xh * mean(g * xh)) + d_sum      dw = sum over rows of dy * xh,  xh = s * rstd
//
// Both are bound by memory: each row is read once into registers (16 bytes a load), reduced by the
// threads that hold it, and written.  A row belongs to TPR threads of one warp, or to a whole CTA when
// it is longer than a warp's registers hold; short rows are taken several at a time so that every
// thread has several loads in flight.  At 6.5 TB/s an SM has some 12 instructions for an element, so the
// arithmetic runs on packed pairs (f32x2) and a thread holds at least 16 elements of a row where it can:
// what a row costs once (its reduction, root and exponent) is shared by them.  Measured, of the 6.54 TB/s copy:
// with L2 flushed before each: 12 heads x 32760 rows of 128 bf16 read from [B, N, H, d] 36 us (0.86), to codes per 128
// rows 34.5 us (0.67; 43 with a CTA a block, whose maximum stands between its loads and its stores), 32760 rows of 1536
// with residual, sum and codes 59 us (0.91); gradients of the first 58 us (0.80) and of rows of 1536 84 us (0.73), 2 to
// 2.5 us more without the next chunk's loads under the work on one.  All arithmetic is fp32; y, sum and dx are rounded once, when they
// are written, and y is normalised from the sum before its rounding.
#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace vsa {

namespace {

// VEC consecutive elements of a row: 16 bytes, or one element where rows are not 16-byte aligned.
template <typename T, int VEC>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(__nv_bfloat16* p, const float* f) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                              pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Chunk<float, 4> {
  float4 v;
  __device__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ void get(float* f) const {
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  }
  __device__ static void store(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Chunk<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ void load(const __nv_bfloat16* p) { v = *p; }
  __device__ void get(float* f) const { f[0] = __bfloat162float(v); }
  __device__ static void store(__nv_bfloat16* p, const float* f) { *p = __float2bfloat16_rn(f[0]); }
};
template <>
struct Chunk<float, 1> {
  float v;
  __device__ void load(const float* p) { v = *p; }
  __device__ void get(float* f) const { f[0] = v; }
  __device__ static void store(float* p, const float* f) { *p = f[0]; }
};

// ---- arithmetic on the N elements of a chunk, two at a time where N is even ----
template <int N>
__device__ __forceinline__ void v_scale(float* f, float c) {
  if constexpr (N % 2 == 0) {
    const uint64_t c2 = f2_make(c, c);
#pragma unroll
    for (int i = 0; i < N; i += 2) f2_split(f2_mul(f2_make(f[i], f[i + 1]), c2), f[i], f[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] *= c;
  }
}
template <int N>
__device__ __forceinline__ void v_mul(float* f, const float* w) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) f2_split(f2_mul(f2_make(f[i], f[i + 1]), f2_make(w[i], w[i + 1])), f[i], f[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] *= w[i];
  }
}
template <int N>
__device__ __forceinline__ void v_add(float* f, const float* o) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) f2_split(f2_add(f2_make(f[i], f[i + 1]), f2_make(o[i], o[i + 1])), f[i], f[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] += o[i];
  }
}
// f = a * b + f
template <int N>
__device__ __forceinline__ void v_fma(float* f, const float* a, const float* b) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      f2_split(f2_fma(f2_make(a[i], a[i + 1]), f2_make(b[i], b[i + 1]), f2_make(f[i], f[i + 1])), f[i], f[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fmaf(a[i], b[i], f[i]);
  }
}
// f = a * c + f
template <int N>
__device__ __forceinline__ void v_fma(float* f, const float* a, float c) {
  if constexpr (N % 2 == 0) {
    const uint64_t c2 = f2_make(c, c);
#pragma unroll
    for (int i = 0; i < N; i += 2) f2_split(f2_fma(f2_make(a[i], a[i + 1]), c2, f2_make(f[i], f[i + 1])), f[i], f[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fmaf(a[i], c, f[i]);
  }
}
template <int N>
__device__ __forceinline__ float v_dot(const float* a, const float* b) {
  if constexpr (N % 2 == 0) {
    uint64_t s = f2_mul(f2_make(a[0], a[1]), f2_make(b[0], b[1]));
#pragma unroll
    for (int i = 2; i < N; i += 2) s = f2_fma(f2_make(a[i], a[i + 1]), f2_make(b[i], b[i + 1]), s);
    float lo, hi;
    f2_split(s, lo, hi);
    return lo + hi;
  } else {
    float s = a[0] * b[0];
#pragma unroll
    for (int i = 1; i < N; ++i) s = fmaf(a[i], b[i], s);
    return s;
  }
}
template <int N>
__device__ __forceinline__ float v_top(const float* f, float top) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) top = fmax3(top, fabsf(f[i]), fabsf(f[i + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(f[i]));
  }
  return top;
}

template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, float* y, const E4m3Scale& scale) {
  v_scale<VEC>(y, scale.a);
  if (scale.twice) v_scale<VEC>(y, scale.b);
  if constexpr (VEC == 1) {
    *p = static_cast<uint8_t>(e4m3_pair(y[0], 0.f) & 0xffu);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      w[i] = e4m3_pair(y[4 * i], y[4 * i + 1]) | (e4m3_pair(y[4 * i + 2], y[4 * i + 3]) << 16);
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// How the weights are given.
enum : int { kWeightNone = 0, kWeightF32 = 1, kWeightBf16 = 2 };

// The weights of one chunk (16-byte aligned where VEC > 1, as the chunk is).
template <int VEC>
__device__ __forceinline__ void weights(const NormArgs& a, int col, float* w) {
  if (a.w_kind == kWeightNone) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = 1.f;
  } else if (a.w_kind == kWeightF32) {
    const float* f = static_cast<const float*>(a.w) + col;
    if constexpr (VEC == 1) {
      w[0] = f[0];
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(f + i);
        w[i] = v.x;
        w[i + 1] = v.y;
        w[i + 2] = v.z;
        w[i + 3] = v.w;
      }
    }
  } else {
    const __nv_bfloat16* f = static_cast<const __nv_bfloat16*>(a.w) + col;
    if constexpr (VEC == 8) {
      Chunk<__nv_bfloat16, 8> c;
      c.load(f);
      c.get(w);
    } else if constexpr (VEC == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(f);
      w[0] = __uint_as_float(v.x << 16);
      w[1] = __uint_as_float(v.x & 0xffff0000u);
      w[2] = __uint_as_float(v.y << 16);
      w[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
      w[0] = __bfloat162float(f[0]);
    }
  }
}

// Sums (or maxima) of ROWS rows over the threads that hold them: TPR of a warp, or the whole CTA (TPR = 0)
// through one barrier; callers alternate between the two buffers.
template <int TPR, int ROWS, bool kMax>
__device__ __forceinline__ void row_reduce(float (&v)[ROWS], float (*smem)[32], int& buf) {
#pragma unroll
  for (int off = (TPR == 0 ? 32 : TPR) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float o = __shfl_xor_sync(0xffffffffu, v[r], off);
      v[r] = kMax ? fmaxf(v[r], o) : v[r] + o;
    }
  if constexpr (TPR == 0) {
    float (*mine)[32] = smem + buf * ROWS;
    buf ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) mine[r][threadIdx.x >> 5] = v[r];
    __syncthreads();
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      v[r] = mine[r][0];
      for (int w = 1; w < warps; ++w) v[r] = kMax ? fmaxf(v[r], mine[r][w]) : v[r] + mine[r][w];
    }
  }
}

__device__ __forceinline__ size_t row_at(const int64_t (&stride)[3], int b, int h, int n) {
  return static_cast<size_t>(b) * stride[0] + static_cast<size_t>(h) * stride[1] + static_cast<size_t>(n) * stride[2];
}

// CTA = one chunk of consecutive rows of one head; heads run fastest so that CTAs that run together read
// neighbouring rows of a [B, N, H, d] tensor.  Thread group g takes rows g, g + groups, ...
// Rows and columns past the end load the last row or the first column again (every load is in bounds without a
// branch) and count as zero.
template <typename T, int VEC, int NV, int TPR, int ROWS, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : TPR != 0 ? 256 : 512) rms_norm_kernel(const NormArgs a) {
  __shared__ float red[2 * ROWS][32];
  int buf = 0;
  const int bh = static_cast<int>(blockIdx.x % a.BH), chunk = static_cast<int>(blockIdx.x / a.BH);
  const int b = bh / a.H, h = bh - b * a.H;
  const int tpr = TPR == 0 ? blockDim.x : TPR, groups = TPR == 0 ? 1 : blockDim.x / TPR;
  const int g = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int n0 = chunk * groups * ROWS + g;
  const T* x = static_cast<const T*>(a.x) + row_at(a.x_stride, b, h, 0);
  const bool has_res = a.res != nullptr;
  const T* res = has_res ? static_cast<const T*>(a.res) + row_at(a.res_stride, b, h, 0) : x;
  const int64_t res_n = has_res ? a.res_stride[2] : a.x_stride[2];
  const size_t out_row = static_cast<size_t>(bh) * a.N;
  Chunk<T, VEC> cx[ROWS][NV], cr[ROWS][NV];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int n = min(n0 + r * groups, a.N - 1);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * tpr + t) * VEC;
      cx[r][j].load(x + static_cast<size_t>(n) * a.x_stride[2] + (col < a.d ? col : 0));
    }
    if (has_res)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * tpr + t) * VEC;
        cr[r][j].load(res + static_cast<size_t>(n) * res_n + (col < a.d ? col : 0));
      }
  }
  const float inv_d = 1.f / static_cast<float>(a.d);
  float s[ROWS][NV * VEC], stat[ROWS], rstd[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int n = n0 + r * groups;
    stat[r] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * tpr + t) * VEC;
      float* f = s[r] + j * VEC;
      cx[r][j].get(f);
      if (has_res) {
        float o[VEC];
        cr[r][j].get(o);
        v_add<VEC>(f, o);
        if (a.sum != nullptr && n < a.N && col < a.d)
          Chunk<T, VEC>::store(static_cast<T*>(a.sum) + (out_row + n) * a.d + col, f);
      }
      const float sq = v_dot<VEC>(f, f);
      stat[r] += col < a.d ? sq : 0.f;
    }
  }
  row_reduce<TPR, ROWS, false>(stat, red, buf);
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int n = n0 + r * groups;
    rstd[r] = rsqrtf(fmaf(stat[r], inv_d, a.eps));
    if (t == 0 && n < a.N && a.rstd != nullptr) a.rstd[out_row + n] = rstd[r];
    stat[r] = 0.f;  // from here the largest |y|
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * tpr + t) * VEC;
    float w[VEC];
    weights<VEC>(a, col < a.d ? col : 0, w);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = n0 + r * groups;
      float* f = s[r] + j * VEC;
      v_scale<VEC>(f, rstd[r]);
      v_mul<VEC>(f, w);
      if (kBlock || a.codes != nullptr) stat[r] = col < a.d ? v_top<VEC>(f, stat[r]) : stat[r];
      if (a.y != nullptr && n < a.N && col < a.d)
        Chunk<T, VEC>::store(static_cast<T*>(a.y) + (out_row + n) * a.d + col, f);
    }
  }
  if (!kBlock && a.codes == nullptr) return;
  int e[ROWS];
  if constexpr (kBlock) {  // the CTA's rows are the block
    float top = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (n0 + r * groups < a.N) top = fmaxf(top, stat[r]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = top;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) top = fmaxf(top, red[0][w]);
    const int be = e4m3_block_exponent(fminf(top, FLT_MAX));
    if (threadIdx.x == 0) a.exps[static_cast<size_t>(bh) * a.chunks + chunk] = be;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) e[r] = be;
  } else {
    row_reduce<TPR, ROWS, true>(stat, red, buf);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = n0 + r * groups;
      e[r] = e4m3_block_exponent(fminf(stat[r], FLT_MAX));
      if (t == 0 && n < a.N) a.exps[out_row + n] = e[r];
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int n = n0 + r * groups;
    const E4m3Scale scale(e[r]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * tpr + t) * VEC;
      if (n < a.N && col < a.d) store_codes<VEC>(a.codes + (out_row + n) * a.d + col, s[r] + j * VEC, scale);
    }
  }
}

// Rows of 2 * TPR * VEC elements without a residual to codes with one exponent per block: a CTA's rows are a block.
// The block's maximum stands between its loads and its stores, so persistent CTAs fetch the next block (cp.async, every
// thread its own 16 bytes at a time into its own slots: no barrier for them) while they work on one.
template <typename T, int VEC, int TPR, int ROWS>
__global__ void __launch_bounds__(1024) rms_norm_block_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint4 ahead[];  // [2 stages][ROWS * 2][threads]
  __shared__ __align__(16) float red[2][32];
  const int groups = blockDim.x / TPR, g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const unsigned items = static_cast<unsigned>(a.chunks) * a.BH, heads = a.BH;  // below 2^31
  auto slot = [&](int st, int r, int j) { return ahead + ((st * ROWS + r) * 2 + j) * blockDim.x + threadIdx.x; };
  auto fetch = [&](unsigned item, int st) {
    if (item < items) {
      const int chunk = item / heads, bh = item - chunk * heads;
      const T* x = static_cast<const T*>(a.x) + row_at(a.x_stride, bh / a.H, bh % a.H, 0);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int n = min((chunk * ROWS + r) * groups + g, a.N - 1);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          cp_async_16(smem_u32(slot(st, r, j)), x + static_cast<size_t>(n) * a.x_stride[2] + (j * TPR + t) * VEC, 16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(blockIdx.x, 0);
  int st = 0;
  for (unsigned item = blockIdx.x; item < items; item += gridDim.x, st ^= 1) {
    const int chunk = item / heads, bh = item - chunk * heads;
    const int n0 = chunk * ROWS * groups + g;
    const size_t out_row = static_cast<size_t>(bh) * a.N;
    fetch(item + gridDim.x, st ^ 1);  // read two barriers ago
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    float s[ROWS][2 * VEC], stat[ROWS], top = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      stat[r] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Chunk<T, VEC> c;
        c.load(reinterpret_cast<const T*>(slot(st, r, j)));
        c.get(s[r] + j * VEC);
        stat[r] += v_dot<VEC>(s[r] + j * VEC, s[r] + j * VEC);
      }
    }
    int none = 0;
    row_reduce<TPR, ROWS, false>(stat, red, none);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = n0 + r * groups;
      stat[r] = rsqrtf(fmaf(stat[r], 1.f / (2 * TPR * VEC), a.eps));
      if (t == 0 && n < a.N && a.rstd != nullptr) a.rstd[out_row + n] = stat[r];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = (j * TPR + t) * VEC;
      float w[VEC];
      weights<VEC>(a, col, w);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int n = n0 + r * groups;
        float* f = s[r] + j * VEC;
        v_scale<VEC>(f, stat[r]);
        v_mul<VEC>(f, w);
        top = n < a.N ? v_top<VEC>(f, top) : top;
        if (a.y != nullptr && n < a.N) Chunk<T, VEC>::store(static_cast<T*>(a.y) + (out_row + n) * a.d + col, f);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if ((threadIdx.x & 31) == 0) red[st][threadIdx.x >> 5] = top;
    __syncthreads();  // the other half of red is written only behind the next one
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); w += 4) {  // at least 128 threads
      const float4 m = *reinterpret_cast<const float4*>(&red[st][w]);
      top = fmax3(fmax3(top, m.x, m.y), m.z, m.w);
    }
    const int e = e4m3_block_exponent(fminf(top, FLT_MAX));
    if (threadIdx.x == 0) a.exps[static_cast<size_t>(bh) * a.chunks + chunk] = e;
    const E4m3Scale scale(e);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = n0 + r * groups;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (n < a.N) store_codes<VEC>(a.codes + (out_row + n) * a.d + (j * TPR + t) * VEC, s[r] + j * VEC, scale);
    }
  }
}

// Persistent CTAs walk the chunks; every thread keeps the weights and the dw of its columns in registers, and the
// CTA's sum goes to one row of the workspace, which rms_norm_dw_kernel adds up in a fixed order (no atomics).
// kAhead: the next chunk is fetched (cp.async, every thread its own 16 bytes at a time into its own slots) while one
// is worked on, and read from shared memory in both passes, which leaves the registers to the columns' sums.
template <typename T, int VEC, int NV, int TPR, int ROWS, bool kAhead>
__global__ void __launch_bounds__(TPR != 0 ? 256 : sizeof(T) == 4 && VEC == 4 && NV == 4 ? 1024 : 512, TPR != 0 ? 2 : 1)
    rms_norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int C = NV * VEC;
  extern __shared__ __align__(16) uint4 ahead[];  // kAhead: [2 stages][s, dy, d_sum][ROWS][NV][threads]
  __shared__ float red[2 * ROWS][32];
  __shared__ float dw_smem[TPR == 0 ? 1 : C * TPR];
  int buf = 0;
  const int tpr = TPR == 0 ? blockDim.x : TPR, groups = TPR == 0 ? 1 : blockDim.x / TPR;
  const int g = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int d = a.n.d, N = a.n.N;
  // the weights stay in registers where there is room; elsewhere each row reads them again (from L1)
  constexpr bool kHoldW = C <= 16;
  float w[kHoldW ? C : 1], dw[C];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * tpr + t) * VEC;
    if constexpr (kHoldW) weights<VEC>(a.n, col < d ? col : 0, w + j * VEC);
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[j * VEC + i] = 0.f;
  }
  const float inv_d = 1.f / static_cast<float>(d);
  const bool has_ds = a.d_sum != nullptr;
  const T* dy = static_cast<const T*>(a.dy);
  const T* ds = has_ds ? static_cast<const T*>(a.d_sum) : dy;
  const unsigned heads = a.n.BH, items = static_cast<unsigned>(a.n.chunks) * heads;  // below 2^31
  Chunk<T, VEC> held[kAhead ? 1 : 3][ROWS][NV];
  float rstd_next[ROWS], rstd[ROWS], dot[ROWS];
  int st = 0;
  auto slot = [&](int stage, int which, int r, int j) {
    return ahead + (((stage * (has_ds ? 3 : 2) + which) * ROWS + r) * NV + j) * blockDim.x + threadIdx.x;
  };
  auto fetch = [&](unsigned item, int stage) {
    if (item < items) {
      const int chunk = item / heads, bh = item - chunk * heads;
      const size_t out_row = static_cast<size_t>(bh) * N;
      const T* s = static_cast<const T*>(a.n.x) + row_at(a.n.x_stride, bh / a.n.H, bh % a.n.H, 0);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int n = min((chunk * ROWS + r) * groups + g, N - 1);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int col = (j * tpr + t) * VEC, at = col < d ? col : 0;
          const T* from[3] = {s + static_cast<size_t>(n) * a.n.x_stride[2] + at, dy + (out_row + n) * d + at,
                              ds + (out_row + n) * d + at};
#pragma unroll
          for (int which = 0; which < 3; ++which) {
            if (which == 2 && !has_ds) continue;
            if constexpr (kAhead) cp_async_16(smem_u32(slot(stage, which, r, j)), from[which], 16);
            else held[which][r][j].load(from[which]);
          }
        }
        rstd_next[r] = a.n.rstd[out_row + n];
      }
    }
    if constexpr (kAhead) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto get = [&](int which, int r, int j, float* f) {
    if constexpr (kAhead) {
      Chunk<T, VEC> c;
      c.load(reinterpret_cast<const T*>(slot(st, which, r, j)));
      c.get(f);
    } else {
      held[which][r][j].get(f);
    }
  };
  if constexpr (kAhead) fetch(blockIdx.x, 0);
  for (unsigned item = blockIdx.x; item < items; item += gridDim.x) {
    const int chunk = item / heads, bh = item - chunk * heads;
    const int n0 = chunk * groups * ROWS + g;
    T* dx = static_cast<T*>(a.dx) + row_at(a.n.res_stride, bh / a.n.H, bh % a.n.H, 0);
    if constexpr (!kAhead) fetch(item, 0);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) rstd[r] = rstd_next[r];
    if constexpr (kAhead) {
      fetch(item + gridDim.x, st ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const bool in = n0 + r * groups < N;
      dot[r] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * tpr + t) * VEC;
        float xh[VEC], fy[VEC], wt[VEC];
        get(0, r, j, xh);
        get(1, r, j, fy);
        if constexpr (!kHoldW) weights<VEC>(a.n, col < d ? col : 0, wt);
        v_scale<VEC>(xh, rstd[r]);
        if (in) v_fma<VEC>(dw + j * VEC, fy, xh);
        v_mul<VEC>(fy, kHoldW ? w + j * VEC : wt);
        const float p = v_dot<VEC>(fy, xh);
        dot[r] += col < d ? p : 0.f;
      }
    }
    row_reduce<TPR, ROWS, false>(dot, red, buf);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = n0 + r * groups;
      // dx = rstd * (dy * w - (rstd * mean) * s): rstd^2 may be beyond the floats where dx is not
      const float c = -rstd[r] * (dot[r] * inv_d);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * tpr + t) * VEC;
        float fs[VEC], fy[VEC], out[VEC], wt[VEC];
        get(0, r, j, fs);
        get(1, r, j, fy);
        if constexpr (!kHoldW) weights<VEC>(a.n, col < d ? col : 0, wt);
        if (has_ds) {
          get(2, r, j, out);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) out[i] = 0.f;
        }
        v_scale<VEC>(fs, c);
        v_fma<VEC>(fs, fy, kHoldW ? w + j * VEC : wt);
        v_fma<VEC>(out, fs, rstd[r]);
        if (n < N && col < d) Chunk<T, VEC>::store(dx + static_cast<size_t>(n) * a.n.res_stride[2] + col, out);
      }
    }
    st ^= 1;
  }
  if (a.partial == nullptr) return;
  float* mine = a.partial + static_cast<size_t>(blockIdx.x) * d;
  if constexpr (TPR == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int col = (j * tpr + t) * VEC + i;
        if (col < d) mine[col] = dw[j * VEC + i];
      }
  } else {
#pragma unroll
    for (int off = 16; off >= TPR; off >>= 1)
#pragma unroll
      for (int i = 0; i < C; ++i) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], off);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int k = 0; k < warps; ++k) {
      if (warp == k && lane < TPR) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int col = (j * TPR + t) * VEC + i;
            dw_smem[col] = k == 0 ? dw[j * VEC + i] : dw_smem[col] + dw[j * VEC + i];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += blockDim.x) mine[c] = dw_smem[c];
  }
}

// dw[c] = sum of the CTAs' rows, in fp64 (some hundred terms): 32 threads a column, each a fixed share.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* __restrict__ partial, int rows, int d,
                                                           float* __restrict__ dw) {
  __shared__ double part[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  double s = 0.0;
  const int cc = min(c, d - 1);
#pragma unroll 4
  for (int r = k; r < rows; r += 32) s += static_cast<double>(partial[static_cast<size_t>(r) * d + cc]);
  part[k][threadIdx.x & 31] = s;
  __syncthreads();
  // warp k adds up column k
  s = part[threadIdx.x & 31][k];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + k < d) dw[blockIdx.x * 32 + k] = static_cast<float>(s);
}

// How a row of d elements is held: VEC elements a load, NV loads a thread, TPR threads of a warp (0: a whole CTA
// of as many threads as the row needs), ROWS rows at a time.
template <int V, int N, int P, int R>
struct Hold {
  static constexpr int VEC = V, NV = N, TPR = P, ROWS = R;
  // threads of a CTA for n loads a row
  static int threads(int n) { return P != 0 ? 256 : (n + N * 32 - 1) / (N * 32) * 32; }
};

// Calls f with the Hold of a forward (or gradient) row and its number of loads.  A row stays in a warp, without
// a barrier, while the warp's registers hold it: up to 256 loads forward; the gradient, which holds up to three
// rows and the sums of its columns, up to 128, then takes 64 threads and more.
template <typename T, bool kBwd, typename F>
cudaError_t with_hold(int d, bool vectors, F&& f) {
  constexpr int V = 16 / sizeof(T);
  const int n = vectors ? d / V : d;  // loads a row
  if (vectors) {
    if (n <= 8) return f(Hold<V, 2, 4, 2>(), n);
    if (n <= 16) return f(Hold<V, 2, 8, 2>(), n);
    if (n <= 32) return f(Hold<V, 2, 16, 2>(), n);
    if (n <= 64) return f(Hold<V, 2, 32, 2>(), n);
    if (n <= 128) return f(Hold<V, 4, 32, 1>(), n);
    if constexpr (kBwd) {
      if (n <= 192) return f(Hold<V, 3, 0, 1>(), n);
      return f(Hold<V, 4, 0, 1>(), n);
    } else {
      if (n <= 192) return f(Hold<V, 6, 32, 1>(), n);
      if (n <= 256) return f(Hold<V, 8, 32, 1>(), n);
      if (n <= 1024) return f(Hold<V, 4, 0, 1>(), n);
      return f(Hold<V, 8, 0, 1>(), n);
    }
  }
  if (n <= 32) return f(Hold<1, 1, 32, 4>(), n);
  if (n <= 128) return f(Hold<1, 4, 32, 4>(), n);
  if (n <= 4096) return f(Hold<1, 8, 0, 1>(), n);
  return f(Hold<1, 32, 0, 1>(), n);
}

// Whether every row starts on 16 bytes and is a whole number of 16-byte loads.
bool vector_rows(const NormArgs& a, int es) {
  const int V = 16 / es;
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  bool ok = a.d % V == 0 && on16(a.x) && on16(a.res);
  for (int i = 0; i < 3; ++i) ok = ok && a.x_stride[i] % V == 0 && (a.res == nullptr || a.res_stride[i] % V == 0);
  return ok;
}

template <typename T>
cudaError_t launch_norm_t(NormArgs a, cudaStream_t stream) {
  return with_hold<T, false>(a.d, vector_rows(a, sizeof(T)), [&](auto hold, int n) -> cudaError_t {
    using H = decltype(hold);
    const bool blocks = a.codes != nullptr && a.block > 1;
    const int threads = blocks ? a.block * H::TPR / H::ROWS : H::threads(n);
    const int rows = (H::TPR == 0 ? 1 : threads / H::TPR) * H::ROWS;
    a.chunks = static_cast<int>((static_cast<long long>(a.N) + rows - 1) / rows);
    const long long grid = static_cast<long long>(a.chunks) * a.BH;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned gr = static_cast<unsigned>(grid);
    if (!blocks) {
      rms_norm_kernel<T, H::VEC, H::NV, H::TPR, H::ROWS, false><<<gr, threads, 0, stream>>>(a);
      return cudaGetLastError();
    }
    // blocks are of rows of 64 or 128, which these hold (64 elements read one by one leave half of their 128 empty)
    constexpr int kHeld = H::NV * H::TPR * H::VEC;
    if constexpr (H::VEC > 1 && (kHeld == 64 || kHeld == 128)) {
      if (a.res == nullptr && a.d == kHeld) {
        auto kern = rms_norm_block_kernel<T, H::VEC, H::TPR, H::ROWS>;
        const int smem = 2 * H::ROWS * 2 * 16 * threads;
        const cudaError_t e = allow_smem(kern, 2 * H::ROWS * 2 * 16 * (128 * H::TPR / H::ROWS));  // blocks of 128 rows
        if (e != cudaSuccess) return e;
        const long long most = 148 * (1024 / threads);  // 64 registers a thread
        kern<<<static_cast<unsigned>(grid < most ? grid : most), threads, smem, stream>>>(a);
        return cudaGetLastError();
      }
    }
    if constexpr (kHeld == 64 || kHeld == 128) {
      rms_norm_kernel<T, H::VEC, H::NV, H::TPR, H::ROWS, true><<<gr, threads, 0, stream>>>(a);
      return cudaGetLastError();
    }
    return cudaErrorInvalidValue;
  });
}

// CTAs of the gradient: as many as 148 SMs hold at up to 128 registers a thread.
template <typename H>
int bwd_ctas(int n) {
  return 148 * (H::threads(n) < 512 ? 512 / H::threads(n) : 1);
}

template <typename T>
cudaError_t launch_norm_bwd_t(NormBwdArgs a, float* dw, cudaStream_t stream) {
  return with_hold<T, true>(a.n.d, vector_rows(a.n, sizeof(T)), [&](auto hold, int n) -> cudaError_t {
    using H = decltype(hold);
    const int threads = H::threads(n), rows = (H::TPR == 0 ? 1 : threads / H::TPR) * H::ROWS;
    a.n.chunks = static_cast<int>((static_cast<long long>(a.n.N) + rows - 1) / rows);
    const long long items = static_cast<long long>(a.n.chunks) * a.n.BH;
    const int most = bwd_ctas<H>(n), grid = static_cast<int>(items < most ? items : most);
    cudaError_t e;
    // two stages take at most 192 KB for 512 threads, as many as an SM holds; fp32 rows of over 8192 take more
    constexpr bool kVec = H::VEC > 1, kLong = sizeof(T) == 4 && H::TPR == 0 && H::NV == 4;
    constexpr int kArray = 2 * H::ROWS * H::NV * 16;  // bytes a thread for each of s, dy and d_sum
    if (kVec && threads <= 512) {
      auto kern = rms_norm_bwd_kernel<T, H::VEC, H::NV, H::TPR, H::ROWS, kVec>;
      e = allow_smem(kern, 3 * kArray * (H::TPR != 0 ? 256 : 512));
      if (e != cudaSuccess) return e;
      kern<<<grid, threads, (a.d_sum != nullptr ? 3 : 2) * kArray * threads, stream>>>(a);
    } else {
      rms_norm_bwd_kernel<T, H::VEC, H::NV, H::TPR, H::ROWS, kVec && !kLong><<<grid, threads, 0, stream>>>(a);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess || dw == nullptr) return e;
    rms_norm_dw_kernel<<<(a.n.d + 31) / 32, 1024, 0, stream>>>(a.partial, grid, a.n.d, dw);
    return cudaGetLastError();
  });
}

// One head of B*H*N rows where the rows are contiguous and no block of rows has to end with a head.
void collapse(NormArgs* a) {
  const int64_t d = a->d, hs = d * a->N, bs = hs * a->H;
  auto whole = [&](const int64_t (&s)[3]) {
    return (a->N == 1 || s[2] == d) && (a->H == 1 || s[1] == hs) && (a->BH == a->H || s[0] == bs);
  };
  const long long rows = static_cast<long long>(a->BH) * a->N;
  if (a->block > 1 || rows > 0x7fffffffLL || !whole(a->x_stride) || (a->res != nullptr && !whole(a->res_stride))) return;
  a->N = static_cast<int>(rows);
  a->BH = a->H = 1;
  a->x_stride[2] = a->res_stride[2] = d;
}

}  // namespace

size_t rms_norm_bwd_partials(long long rows, int d, bool f32) {
  // whether the rows are read as vectors shows only with the pointers: the larger of the two
  long long most = 0;
  for (const bool vectors : {false, true}) {
    if (vectors && d % (f32 ? 4 : 8) != 0) continue;
    auto count = [&](auto hold, int n) {
      const long long c = bwd_ctas<decltype(hold)>(n);
      most = c > most ? c : most;
      return cudaSuccess;
    };
    f32 ? with_hold<float, true>(d, vectors, count) : with_hold<__nv_bfloat16, true>(d, vectors, count);
  }
  return static_cast<size_t>(rows < most ? rows : most);
}

cudaError_t launch_rms_norm(NormArgs a, bool f32, cudaStream_t stream) {
  if (a.codes == nullptr) a.block = 1;
  collapse(&a);
  return f32 ? launch_norm_t<float>(a, stream) : launch_norm_t<__nv_bfloat16>(a, stream);
}

cudaError_t launch_rms_norm_bwd(NormBwdArgs a, bool f32, float* dw, cudaStream_t stream) {
  a.n.block = 1;
  a.n.res = a.dx;  // its strides and alignment count as the residual's do
  collapse(&a.n);
  return f32 ? launch_norm_bwd_t<float>(a, dw, stream) : launch_norm_bwd_t<__nv_bfloat16>(a, dw, stream);
}

}  // namespace vsa
