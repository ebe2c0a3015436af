// Layer norm, forward and backward, over the last axis of [rows, cols].
//
//   mean = sum(x) / n,  var = sum((x - mean)^2) / n,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b, in x's type or as E4M3 codes with one
//   power-of-two scale per 1 x 128 row group (the GEMMs' operand, and the
//   8-bit checkpoint of the normed activation)
//
// Backward, with xh = (x - mean) rstd and t = w dy:
//   dx = rstd (t - mean(t) - xh mean(t xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by HBM: x (and dy) are read once and stay in registers for both the
// row's sums and its results.  All sums are FP32; the variance is summed
// around the mean, so a large mean costs no digits.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_device.cuh"
#include "dg_ops.cuh"

namespace dg {
namespace {

template <class T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// VEC elements as one access of VEC * sizeof(T) bytes (16, or one element).
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_float(__ldg(p));
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_float(e[i]);
  }
}
template <class T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_float<T>(f[0]);
  } else {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = from_float<T>(f[i]);
    *reinterpret_cast<uint4*>(p) = v;
  }
}

// Weight or bias element, FP32 or x's type (a branch every thread of the
// launch takes the same way).
template <class T>
__device__ __forceinline__ float param(const void* p, bool fp32, int64_t i) {
  return fp32 ? __ldg(static_cast<const float*>(p) + i) : to_float(__ldg(static_cast<const T*>(p) + i));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the `warps` warps of this thread's row; every thread gets it.
// `slot` alternates between calls, so one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int warps, int row_warp0, int slot) {
  v = warp_sum(v);
  if (warps == 1) return v;
  red += slot * 32;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < warps; ++w) s += red[row_warp0 + w];
  return s;
}

struct LayerNormArgs {
  const void* x;
  const void* dy;
  const void* weight;
  const void* bias;  // nullable
  void* y;           // y, codes, or dx
  uint32_t* sf;      // FP8 results only
  float* mean;
  float* rstd;
  float* part;       // backward: [2][parts][cols] partial sums
  int64_t rows, cols, ldx, lddy, rows_pad;
  int tpr;           // threads a row
  float eps;
  bool w_fp32;       // weight and bias are FP32, else x's type
};

// A row is held by tpr threads (a multiple of 32), NV vectors of VEC elements
// each; a CTA holds blockDim / tpr rows.
template <class T, int VEC, int NV, bool FP8>
__global__ void __launch_bounds__(1024) layer_norm_kernel(const LayerNormArgs p) {
  __shared__ float red[64];
  griddep_wait();
  griddep_launch_dependents();
  const int rpc = blockDim.x / p.tpr;
  const int tid = threadIdx.x % p.tpr;
  const int64_t row = (int64_t)blockIdx.x * rpc + threadIdx.x / p.tpr;
  const int warps = p.tpr / 32, warp0 = threadIdx.x / p.tpr * warps;
  const bool in = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  float v[NV][VEC];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * p.tpr + tid) * VEC;
    if (in && c < p.cols) load_vec<T, VEC>(x + c, v[i]);
    else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i][k] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) s += v[i][k];
  }
  const float n = (float)p.cols;
  const float mean = row_sum(s, red, warps, warp0, 0) / n;
  float d2 = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * p.tpr + tid) * VEC;
    if (c < p.cols) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        v[i][k] -= mean;
        d2 += v[i][k] * v[i][k];
      }
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum(d2, red, warps, warp0, 1) / n + p.eps);
  if (in && tid == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * p.tpr + tid) * VEC;
    const bool live = c < p.cols;
    if (live) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        v[i][k] = v[i][k] * rstd * param<T>(p.weight, p.w_fp32, c + k);
        if (p.bias) v[i][k] += param<T>(p.bias, p.w_fp32, c + k);
      }
    }
    if constexpr (!FP8) {
      if (in && live) store_vec<T, VEC>(static_cast<T*>(p.y) + row * p.cols + c, v[i]);
    } else {
      // 128 / VEC neighbouring threads hold a group of 128 columns, whole or not at all
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < VEC; ++k) m = max(m, abs_bits(v[i][k]));
#pragma unroll
      for (int o = 64 / VEC; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (live && row < p.rows_pad) {
        const int e = scale_exponent(__uint_as_float(m));
        const int kb = (int)(c / 128);
        if (in) {
          const float inv = pow2f(-e);
          uint32_t* q = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + row * p.cols + c);
#pragma unroll
          for (int k = 0; k < VEC; k += 4)
            q[k / 4] = e4m3x4(v[i][k] * inv, v[i][k + 1] * inv, v[i][k + 2] * inv, v[i][k + 3] * inv);
        }
        if (c % 128 == 0)
          store_scale_byte(p.sf + (int64_t)(kb >> 2) * p.rows_pad + row, kb, (int64_t)kb * 128 + 128 == p.cols,
                           in ? (uint32_t)(e + 127) : 0u);
      }
    }
  }
}

// Rows too long for registers: one CTA a row, each pass reading it again
// (from L2).
template <class T>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(const LayerNormArgs p) {
  __shared__ float red[64];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const float n = (float)p.cols;
  const int warps = blockDim.x / 32;
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) s += to_float(__ldg(x + c));
  const float mean = row_sum(s, red, warps, 0, 0) / n;
  float d2 = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float d = to_float(__ldg(x + c)) - mean;
    d2 += d * d;
  }
  const float rstd = 1.0f / sqrtf(row_sum(d2, red, warps, 0, 1) / n + p.eps);
  if (threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    float y = (to_float(__ldg(x + c)) - mean) * rstd * param<T>(p.weight, p.w_fp32, c);
    if (p.bias) y += param<T>(p.bias, p.w_fp32, c);
    static_cast<T*>(p.y)[row * p.cols + c] = from_float<T>(y);
  }
}

// Backward: a CTA walks the rows blockIdx, blockIdx + grid, ... with tpr =
// blockDim threads a row, every thread keeping the sums dw and db of its own
// columns in registers; they go to `part` once, at the end.
template <class T, int VEC, int NV>
__global__ void __launch_bounds__(1024) layer_norm_backward_kernel(const LayerNormArgs p) {
  __shared__ float red[128];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warps = blockDim.x / 32;
  float w[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int64_t c = ((int64_t)i * blockDim.x + tid) * VEC + k;
      w[i][k] = c < p.cols ? param<T>(p.weight, p.w_fp32, c) : 0.0f;
      aw[i][k] = ab[i][k] = 0.0f;
    }
  const float rn = 1.0f / (float)p.cols;
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    float xv[NV][VEC], dv[NV][VEC];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * blockDim.x + tid) * VEC;
      if (c < p.cols) {
        load_vec<T, VEC>(x + c, xv[i]);
        load_vec<T, VEC>(dy + c, dv[i]);
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          xv[i][k] = mean;
          dv[i][k] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        xv[i][k] = (xv[i][k] - mean) * rstd;
        aw[i][k] += dv[i][k] * xv[i][k];
        ab[i][k] += dv[i][k];
        dv[i][k] *= w[i][k];
        s1 += dv[i][k];
        s2 += dv[i][k] * xv[i][k];
      }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    float* r = red + slot * 64;
    slot ^= 1;
    if ((tid & 31) == 0) {
      r[tid >> 5] = s1;
      r[32 + (tid >> 5)] = s2;
    }
    __syncthreads();
    s1 = s2 = 0.0f;
    for (int i = 0; i < warps; ++i) {
      s1 += r[i];
      s2 += r[32 + i];
    }
    const float c1 = s1 * rn, c2 = s2 * rn;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * blockDim.x + tid) * VEC;
      if (c < p.cols) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) dv[i][k] = rstd * (dv[i][k] - c1 - xv[i][k] * c2);
        store_vec<T, VEC>(static_cast<T*>(p.y) + row * p.cols + c, dv[i]);
      }
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  float* partb = part + (int64_t)gridDim.x * p.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int64_t c = ((int64_t)i * blockDim.x + tid) * VEC + k;
      if (c < p.cols) {
        part[c] = aw[i][k];
        partb[c] = ab[i][k];
      }
    }
}

// Rows too long for registers: dx one CTA a row ...
template <class T>
__global__ void __launch_bounds__(1024) layer_norm_backward_long_kernel(const LayerNormArgs p) {
  __shared__ float red[64];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
  const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row), rn = 1.0f / (float)p.cols;
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float t = to_float(__ldg(dy + c)) * param<T>(p.weight, p.w_fp32, c);
    s1 += t;
    s2 += t * (to_float(__ldg(x + c)) - mean) * rstd;
  }
  const int warps = blockDim.x / 32;
  const float c1 = row_sum(s1, red, warps, 0, 0) * rn;
  const float c2 = row_sum(s2, red, warps, 0, 1) * rn;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float t = to_float(__ldg(dy + c)) * param<T>(p.weight, p.w_fp32, c);
    const float xh = (to_float(__ldg(x + c)) - mean) * rstd;
    static_cast<T*>(p.y)[row * p.cols + c] = from_float<T>(rstd * (t - c1 - xh * c2));
  }
}
// ... and the columns' sums over a slice of the rows a CTA.
template <class T>
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(const LayerNormArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float aw = 0.0f, ab = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float d = to_float(__ldg(static_cast<const T*>(p.dy) + row * p.lddy + c));
    aw += d * (to_float(__ldg(static_cast<const T*>(p.x) + row * p.ldx + c)) - __ldg(p.mean + row)) *
          __ldg(p.rstd + row);
    ab += d;
  }
  p.part[(int64_t)blockIdx.y * p.cols + c] = aw;
  p.part[((int64_t)gridDim.y + blockIdx.y) * p.cols + c] = ab;
}

// dw and db from the partial sums, added in a fixed order: a CTA takes 32
// columns of one of the two, its 32 warps every 32nd part.
__global__ void __launch_bounds__(1024) layer_norm_join_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                               float* __restrict__ db, int parts, int64_t cols) {
  __shared__ float sum[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const float* src = part + (int64_t)blockIdx.y * parts * cols;
  float s = 0.0f;
  if (c < cols)
    for (int i = warp; i < parts; i += 32) s += src[(int64_t)i * cols + c];
  sum[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sum[lane][warp]);
  const int64_t o = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && o < cols) (blockIdx.y ? db : dw)[o] = s;
}

template <class T, bool FP8>
cudaError_t forward(const LayerNormArgs& a, bool vec, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t units = vec ? (p.cols + V - 1) / V : p.cols;
  // vectors a thread: the fewest of 1, 2, 4 (x 16 bytes) or 4, 32 single
  // elements that keep a row within 1024 threads, from 128 threads on
  const int64_t most = vec ? 4 * 1024 : 32 * 1024;
  const int64_t rows = FP8 ? p.rows_pad : p.rows;
  if (units > most) {
    if (FP8) return cudaErrorInvalidValue;
    return launch_op(layer_norm_long_kernel<T>, dim3((unsigned)p.rows), 1024, 0, pdl, st, p);
  }
  auto go = [&](auto kern, int nv) {
    int64_t t = (units + nv - 1) / nv;
    t = (t + 31) / 32 * 32;
    p.tpr = (int)t;
    const int rpc = t >= 128 ? 1 : (int)(128 / t);
    return launch_op(kern, dim3((unsigned)((rows + rpc - 1) / rpc)), (unsigned)(rpc * t), 0, pdl, st, p);
  };
  if (vec) {
    if (units <= 256) return go(layer_norm_kernel<T, V, 1, FP8>, 1);
    if (units <= 512) return go(layer_norm_kernel<T, V, 2, FP8>, 2);
    return go(layer_norm_kernel<T, V, 4, FP8>, 4);
  }
  if constexpr (!FP8) {
    if (units <= 4096) return go(layer_norm_kernel<T, 1, 4, false>, 4);
    return go(layer_norm_kernel<T, 1, 32, false>, 32);
  }
  return cudaErrorInvalidValue;
}

template <class T>
cudaError_t backward(const LayerNormArgs& a, bool vec, int parts, int* used, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t units = vec ? (p.cols + V - 1) / V : p.cols;
  auto go = [&](auto kern, int nv) {
    const int64_t t = ((units + nv - 1) / nv + 31) / 32 * 32;
    *used = (int)(p.rows < parts ? p.rows : parts);
    return launch_op(kern, dim3((unsigned)*used), (unsigned)t, 0, pdl, st, p);
  };
  if (vec && units <= 1024) return go(layer_norm_backward_kernel<T, V, 1>, 1);
  if (!vec && units <= 4096) return go(layer_norm_backward_kernel<T, 1, 4>, 4);
  cudaError_t e = launch_op(layer_norm_backward_long_kernel<T>, dim3((unsigned)p.rows), 1024, 0, pdl, st, p);
  if (e != cudaSuccess) return e;
  int64_t slices = p.rows < 32 ? p.rows : 32;
  if (slices > parts) slices = parts;
  *used = (int)slices;
  return launch_op(layer_norm_columns_kernel<T>, dim3((unsigned)((p.cols + 255) / 256), (unsigned)slices), 256, 0,
                   pdl, st, p);
}

}  // namespace

cudaError_t layer_norm_launch(const void* x, int dtype, const void* weight, const void* bias,
                              bool w_fp32, void* y, void* sf, float* mean, float* rstd, int64_t rows,
                              int64_t cols, int64_t ldx, float eps, bool pdl, cudaStream_t stream) {
  LayerNormArgs p = {};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.w_fp32 = w_fp32;
  p.y = y;
  p.sf = (uint32_t*)sf;
  p.mean = mean;
  p.rstd = rstd;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.rows_pad = (rows + 3) / 4 * 4;
  p.eps = eps;
  // 16-byte accesses need every row of x and y to start on 16 bytes
  const int64_t v = dtype == DG_DTYPE_FP32 ? 4 : 8;
  const bool vec = cols % v == 0 && ldx % v == 0 && ((uintptr_t)x & 15) == 0 && ((uintptr_t)y & 15) == 0;
  if (dtype == DG_DTYPE_FP32)
    return sf ? forward<float, true>(p, vec, pdl, stream) : forward<float, false>(p, vec, pdl, stream);
  if (dtype == DG_DTYPE_BF16)
    return sf ? forward<__nv_bfloat16, true>(p, vec, pdl, stream) : forward<__nv_bfloat16, false>(p, vec, pdl, stream);
  return sf ? forward<__half, true>(p, vec, pdl, stream) : forward<__half, false>(p, vec, pdl, stream);
}

int layer_norm_backward_parts(int sms) { return 2 * sms; }

cudaError_t layer_norm_backward_launch(const void* dy, const void* x, int dtype, const void* weight,
                                       bool w_fp32, const float* mean, const float* rstd, void* dx,
                                       float* dw, float* db, float* part, int parts, int64_t rows,
                                       int64_t cols, int64_t lddy, int64_t ldx, bool pdl,
                                       cudaStream_t stream) {
  LayerNormArgs p = {};
  p.x = x;
  p.dy = dy;
  p.weight = weight;
  p.w_fp32 = w_fp32;
  p.y = dx;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.part = part;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.lddy = lddy;
  const int64_t v = dtype == DG_DTYPE_FP32 ? 4 : 8;
  const bool vec = cols % v == 0 && ldx % v == 0 && lddy % v == 0 &&
                   (((uintptr_t)x | (uintptr_t)dy | (uintptr_t)dx) & 15) == 0;
  int used = 0;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    e = dtype == DG_DTYPE_FP32   ? backward<float>(p, vec, parts, &used, pdl, stream)
        : dtype == DG_DTYPE_BF16 ? backward<__nv_bfloat16>(p, vec, parts, &used, pdl, stream)
                                 : backward<__half>(p, vec, parts, &used, pdl, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_op(layer_norm_join_kernel, dim3((unsigned)((cols + 31) / 32), 2), 1024, 0, pdl, stream,
                   (const float*)part, dw, db, used, cols);
}

}  // namespace dg
