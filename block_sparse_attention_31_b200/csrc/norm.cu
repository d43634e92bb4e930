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
// thread has several loads in flight.  All arithmetic is fp32; y, sum and dx are rounded once, when they are
// written, and y is normalised from the sum before its rounding.
#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace vsa {

namespace {

constexpr int kCodesNone = 0, kCodesRow = 1, kCodesBlock = 2;

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

template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* y, const E4m3Scale& scale) {
  if constexpr (VEC == 1) {
    *p = static_cast<uint8_t>(e4m3_pair(scale(y[0]), 0.f) & 0xffu);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      w[i] = e4m3_pair(scale(y[4 * i]), scale(y[4 * i + 1])) | (e4m3_pair(scale(y[4 * i + 2]), scale(y[4 * i + 3])) << 16);
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// How the weights are given.
enum : int { kWeightNone = 0, kWeightF32 = 1, kWeightBf16 = 2 };

// The weights of one chunk (16-byte aligned where VEC > 1, as the chunk is).
template <int VEC, int WEIGHT>
__device__ __forceinline__ void weights(const void* p, int col, float* w) {
  if constexpr (WEIGHT == kWeightNone) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = 1.f;
  } else if constexpr (WEIGHT == kWeightF32) {
    const float* f = static_cast<const float*>(p) + col;
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
    const __nv_bfloat16* f = static_cast<const __nv_bfloat16*>(p) + col;
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

// Sum (or maximum) over the TPR threads of a row: a part of a warp, or the whole CTA.
template <int TPR, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* smem) {
#pragma unroll
  for (int off = (TPR < 32 ? TPR : 32) / 2; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  if constexpr (TPR > 32) {
    __syncthreads();  // the last reduction has been read
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    v = smem[0];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) v = kMax ? fmaxf(v, smem[w]) : v + smem[w];
  }
  return v;
}

__device__ __forceinline__ size_t row_at(const int64_t (&stride)[3], int b, int h, int n) {
  return static_cast<size_t>(b) * stride[0] + static_cast<size_t>(h) * stride[1] + static_cast<size_t>(n) * stride[2];
}

// CTA = one chunk of consecutive rows of one head; heads run fastest so that CTAs that run together read
// neighbouring rows of a [B, N, H, d] tensor.  Thread group g takes rows g, g + groups, ...
// Rows and columns past the end load the last row or the first column again (every load is in bounds without a
// branch) and count as zero.
template <typename T, int VEC, int NV, int TPR, int ROWS, int CODES, int WEIGHT>
__global__ void __launch_bounds__(CODES == kCodesBlock ? 1024 : 256) rms_norm_kernel(const NormArgs a) {
  __shared__ float red[32];
  const int bh = static_cast<int>(blockIdx.x % a.BH), chunk = static_cast<int>(blockIdx.x / a.BH);
  const int b = bh / a.H, h = bh - b * a.H;
  const int groups = blockDim.x / TPR, g = threadIdx.x / TPR, t = threadIdx.x % TPR;
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
      const int col = (j * TPR + t) * VEC;
      cx[r][j].load(x + static_cast<size_t>(n) * a.x_stride[2] + (col < a.d ? col : 0));
    }
    if (has_res)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * TPR + t) * VEC;
        cr[r][j].load(res + static_cast<size_t>(n) * res_n + (col < a.d ? col : 0));
      }
  }
  float s[ROWS][NV * VEC];
  float amax = 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int n = n0 + r * groups;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * TPR + t) * VEC;
      float* f = s[r] + j * VEC;
      cx[r][j].get(f);
      if (has_res) {
        float o[VEC];
        cr[r][j].get(o);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] += o[i];
        if (a.sum != nullptr && n < a.N && col < a.d)
          Chunk<T, VEC>::store(static_cast<T*>(a.sum) + (out_row + n) * a.d + col, f);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (col >= a.d) f[i] = 0.f;
        sq = fmaf(f[i], f[i], sq);
      }
    }
    sq = row_reduce<TPR, false>(sq, red);
    const float rstd = 1.f / sqrtf(sq / static_cast<float>(a.d) + a.eps);
    if (t == 0 && n < a.N && a.rstd != nullptr) a.rstd[out_row + n] = rstd;
    if (CODES == kCodesRow) amax = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * TPR + t) * VEC;
      float* f = s[r] + j * VEC;
      float w[VEC];
      weights<VEC, WEIGHT>(a.w, col < a.d ? col : 0, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        f[i] = col < a.d ? f[i] * rstd * w[i] : 0.f;
        if (CODES != kCodesNone && n < a.N) amax = fmaxf(amax, fabsf(f[i]));
      }
      if (a.y != nullptr && n < a.N && col < a.d)
        Chunk<T, VEC>::store(static_cast<T*>(a.y) + (out_row + n) * a.d + col, f);
    }
    if constexpr (CODES == kCodesRow) {
      const int e = e4m3_block_exponent(fminf(row_reduce<TPR, true>(amax, red), FLT_MAX));
      const E4m3Scale scale(e);
      if (n < a.N) {
        if (t == 0) a.exps[out_row + n] = e;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int col = (j * TPR + t) * VEC;
          if (col < a.d) store_codes<VEC>(a.codes + (out_row + n) * a.d + col, s[r] + j * VEC, scale);
        }
      }
    }
  }
  if constexpr (CODES == kCodesBlock) {  // the CTA's rows are the block
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) amax = fmaxf(amax, red[w]);
    const int e = e4m3_block_exponent(fminf(amax, FLT_MAX));
    const E4m3Scale scale(e);
    if (threadIdx.x == 0) a.exps[static_cast<size_t>(bh) * a.chunks + chunk] = e;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = n0 + r * groups;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * TPR + t) * VEC;
        if (n < a.N && col < a.d) store_codes<VEC>(a.codes + (out_row + n) * a.d + col, s[r] + j * VEC, scale);
      }
    }
  }
}

// Persistent CTAs walk the chunks; every thread keeps the dw of its columns in fp32 and the CTA's sum goes to
// one row of the workspace, which rms_norm_dw_kernel adds up in a fixed order (no atomics).
template <typename T, int VEC, int NV, int TPR, int ROWS, int WEIGHT>
__global__ void __launch_bounds__(256) rms_norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int C = NV * VEC;
  extern __shared__ float dw_smem[];  // d floats (TPR <= 32)
  __shared__ float red[32];
  constexpr int groups = 256 / TPR;
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  float dw[C];
#pragma unroll
  for (int i = 0; i < C; ++i) dw[i] = 0.f;
  const float inv_d = 1.f / static_cast<float>(a.n.d);
  const long long items = static_cast<long long>(a.n.chunks) * a.n.BH;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int bh = static_cast<int>(item % a.n.BH), chunk = static_cast<int>(item / a.n.BH);
    const int b = bh / a.n.H, h = bh - b * a.n.H;
    const int n0 = chunk * groups * ROWS + g;
    const size_t out_row = static_cast<size_t>(bh) * a.n.N;
    const T* s = static_cast<const T*>(a.n.x) + row_at(a.n.x_stride, b, h, 0);
    T* dx = static_cast<T*>(a.dx) + row_at(a.n.res_stride, b, h, 0);
    const T* dy = static_cast<const T*>(a.dy);
    const bool has_ds = a.d_sum != nullptr;
    const T* ds = has_ds ? static_cast<const T*>(a.d_sum) : dy;
    Chunk<T, VEC> cs[ROWS][NV], cy[ROWS][NV];
    float rstd[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = min(n0 + r * groups, a.n.N - 1);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * TPR + t) * VEC, at = col < a.n.d ? col : 0;
        cs[r][j].load(s + static_cast<size_t>(n) * a.n.x_stride[2] + at);
        cy[r][j].load(dy + (out_row + n) * a.n.d + at);
      }
      rstd[r] = a.n.rstd[out_row + n];
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int n = n0 + r * groups;
      Chunk<T, VEC> cd[NV];
      const bool in = n < a.n.N;
      if (has_ds) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int col = (j * TPR + t) * VEC;
          cd[j].load(ds + (out_row + min(n, a.n.N - 1)) * a.n.d + (col < a.n.d ? col : 0));
        }
      }
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * TPR + t) * VEC;
        float fs[VEC], fy[VEC], w[VEC];
        cs[r][j].get(fs);
        cy[r][j].get(fy);
        weights<VEC, WEIGHT>(a.n.w, col < a.n.d ? col : 0, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xh = fs[i] * rstd[r];
          if (in) dw[j * VEC + i] = fmaf(fy[i], xh, dw[j * VEC + i]);
          if (col < a.n.d) dot = fmaf(fy[i] * w[i], xh, dot);
        }
      }
      dot = row_reduce<TPR, false>(dot, red) * inv_d;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * TPR + t) * VEC;
        if (!in || col >= a.n.d) continue;
        float fs[VEC], fy[VEC], w[VEC], fd[VEC], out[VEC];
        cs[r][j].get(fs);
        cy[r][j].get(fy);
        weights<VEC, WEIGHT>(a.n.w, col, w);
        if (has_ds) cd[j].get(fd);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          out[i] = rstd[r] * (fy[i] * w[i] - fs[i] * rstd[r] * dot);
          if (has_ds) out[i] += fd[i];
        }
        Chunk<T, VEC>::store(dx + static_cast<size_t>(n) * a.n.res_stride[2] + col, out);
      }
    }
  }
  if (a.partial == nullptr) return;
  float* mine = a.partial + static_cast<size_t>(blockIdx.x) * a.n.d;
  if constexpr (TPR > 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int col = (j * TPR + t) * VEC + i;
        if (col < a.n.d) mine[col] = dw[j * VEC + i];
      }
  } else {
#pragma unroll
    for (int off = 16; off >= TPR; off >>= 1)
#pragma unroll
      for (int i = 0; i < C; ++i) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], off);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int w = 0; w < 8; ++w) {
      if (warp == w && lane < TPR) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int col = (j * TPR + t) * VEC + i;
            if (col < a.n.d) dw_smem[col] = w == 0 ? dw[j * VEC + i] : dw_smem[col] + dw[j * VEC + i];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.n.d; c += 256) mine[c] = dw_smem[c];
  }
}

// dw[c] = sum of the CTAs' rows, in fp64 (a few hundred terms): 8 threads a column, each a fixed share.
__global__ void __launch_bounds__(256) rms_norm_dw_kernel(const float* __restrict__ partial, int rows, int d,
                                                          float* __restrict__ dw) {
  __shared__ double part[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  double s = 0.0;
  if (c < d)
    for (int r = k; r < rows; r += 8) s += static_cast<double>(partial[static_cast<size_t>(r) * d + c]);
  part[k][threadIdx.x & 31] = s;
  __syncthreads();
  if (k == 0 && c < d) {
    for (int j = 1; j < 8; ++j) s += part[j][threadIdx.x];
    dw[c] = static_cast<float>(s);
  }
}

// How a row of d elements is held: VEC elements a load, NV loads a thread, TPR threads a row, ROWS rows at a
// time.  with_hold calls f with the smallest that holds it.
template <int V, int N, int P, int R>
struct Hold {
  static constexpr int VEC = V, NV = N, TPR = P, ROWS = R;
};

template <typename T, typename F>
cudaError_t with_hold(int d, bool vectors, F&& f) {
  constexpr int V = 16 / sizeof(T);
  const int n = vectors ? d / V : d;  // loads a row
  if (vectors) {
    if (n <= 8) return f(Hold<V, 1, 8, 4>());
    if (n <= 16) return f(Hold<V, 1, 16, 4>());
    if (n <= 32) return f(Hold<V, 1, 32, 4>());
    if (n <= 64) return f(Hold<V, 2, 32, 2>());
    if (n <= 128) return f(Hold<V, 4, 32, 1>());
    if (n <= 192) return f(Hold<V, 6, 32, 1>());
    if (n <= 256) return f(Hold<V, 8, 32, 1>());
    if (n <= 512) return f(Hold<V, 2, 256, 1>());
    if (n <= 1024) return f(Hold<V, 4, 256, 1>());
    if (n <= 2048) return f(Hold<V, 8, 256, 1>());
    if constexpr (V == 4)
      if (n <= 4096) return f(Hold<V, 16, 256, 1>());
  } else {
    if (n <= 32) return f(Hold<1, 1, 32, 4>());
    if (n <= 128) return f(Hold<1, 4, 32, 4>());
    if (n <= 512) return f(Hold<1, 16, 32, 1>());
    if (n <= 4096) return f(Hold<1, 16, 256, 1>());
    if (n <= 16384) return f(Hold<1, 64, 256, 1>());
  }
  return cudaErrorInvalidValue;
}

// Whether every row starts on 16 bytes and is a whole number of 16-byte loads.
bool vector_rows(const NormArgs& a, int es) {
  const int V = 16 / es;
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  bool ok = a.d % V == 0 && on16(a.x) && on16(a.res);
  for (int i = 0; i < 3; ++i) ok = ok && a.x_stride[i] % V == 0 && (a.res == nullptr || a.res_stride[i] % V == 0);
  return ok;
}

template <typename T, int WEIGHT>
cudaError_t launch_norm_t(NormArgs a, cudaStream_t stream) {
  return with_hold<T>(a.d, vector_rows(a, sizeof(T)), [&](auto hold) -> cudaError_t {
    using H = decltype(hold);
    const bool blocks = a.codes != nullptr && a.block > 1;
    const int threads = blocks ? a.block * H::TPR / H::ROWS : 256;
    const int rows = threads / H::TPR * H::ROWS;
    a.chunks = static_cast<int>((static_cast<long long>(a.N) + rows - 1) / rows);
    const long long grid = static_cast<long long>(a.chunks) * a.BH;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned gr = static_cast<unsigned>(grid);
    if (blocks) {
      if constexpr (H::TPR <= 32 && H::NV <= 4) {  // rows of 64 or 128
        rms_norm_kernel<T, H::VEC, H::NV, H::TPR, H::ROWS, kCodesBlock, WEIGHT><<<gr, threads, 0, stream>>>(a);
        return cudaGetLastError();
      }
      return cudaErrorInvalidValue;
    }
    if (a.codes != nullptr)
      rms_norm_kernel<T, H::VEC, H::NV, H::TPR, H::ROWS, kCodesRow, WEIGHT><<<gr, threads, 0, stream>>>(a);
    else
      rms_norm_kernel<T, H::VEC, H::NV, H::TPR, H::ROWS, kCodesNone, WEIGHT><<<gr, threads, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

template <typename T, int WEIGHT>
cudaError_t launch_norm_bwd_t(NormBwdArgs a, float* dw, cudaStream_t stream) {
  return with_hold<T>(a.n.d, vector_rows(a.n, sizeof(T)), [&](auto hold) -> cudaError_t {
    using H = decltype(hold);
    constexpr int ROWS = H::ROWS > 2 ? 2 : H::ROWS;
    const int rows = 256 / H::TPR * ROWS;
    a.n.chunks = static_cast<int>((static_cast<long long>(a.n.N) + rows - 1) / rows);
    const long long items = static_cast<long long>(a.n.chunks) * a.n.BH;
    const int grid = static_cast<int>(items < kNormBwdCtas ? items : kNormBwdCtas);
    const int smem = H::TPR <= 32 ? a.n.d * 4 : 0;
    rms_norm_bwd_kernel<T, H::VEC, H::NV, H::TPR, ROWS, WEIGHT><<<grid, 256, smem, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || dw == nullptr) return e;
    rms_norm_dw_kernel<<<(a.n.d + 31) / 32, 256, 0, stream>>>(a.partial, grid, a.n.d, dw);
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

cudaError_t launch_rms_norm(NormArgs a, bool f32, cudaStream_t stream) {
  if (a.codes == nullptr) a.block = 1;
  collapse(&a);
  if (a.w == nullptr)
    return f32 ? launch_norm_t<float, kWeightNone>(a, stream) : launch_norm_t<__nv_bfloat16, kWeightNone>(a, stream);
  if (a.w_f32)
    return f32 ? launch_norm_t<float, kWeightF32>(a, stream) : launch_norm_t<__nv_bfloat16, kWeightF32>(a, stream);
  return f32 ? launch_norm_t<float, kWeightBf16>(a, stream) : launch_norm_t<__nv_bfloat16, kWeightBf16>(a, stream);
}

cudaError_t launch_rms_norm_bwd(NormBwdArgs a, bool f32, float* dw, cudaStream_t stream) {
  a.n.block = 1;
  a.n.res = a.dx;  // its strides and alignment count as the residual's do
  collapse(&a.n);
  if (a.n.w == nullptr)
    return f32 ? launch_norm_bwd_t<float, kWeightNone>(a, dw, stream)
               : launch_norm_bwd_t<__nv_bfloat16, kWeightNone>(a, dw, stream);
  if (a.n.w_f32)
    return f32 ? launch_norm_bwd_t<float, kWeightF32>(a, dw, stream)
               : launch_norm_bwd_t<__nv_bfloat16, kWeightF32>(a, dw, stream);
  return f32 ? launch_norm_bwd_t<float, kWeightBf16>(a, dw, stream)
             : launch_norm_bwd_t<__nv_bfloat16, kWeightBf16>(a, dw, stream);
}

}  // namespace vsa
