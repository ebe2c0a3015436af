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

#include <algorithm>

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
// Rows are read once: they are kept out of L1, which holds weight and bias.
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_float(__ldg(p));
  } else {
    const uint4 v = ld_stream_u4(p);
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

// VEC neighbouring elements; `wide`: the base is 16-byte aligned.
template <class T, int VEC>
__device__ __forceinline__ void param_vec(const void* p, bool fp32, bool wide, int64_t i, float (&f)[VEC]) {
  if (VEC == 1 || !wide) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = param<T>(p, fp32, i + k);
  } else if (fp32) {
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i) + k);
      f[4 * k] = v.x;
      f[4 * k + 1] = v.y;
      f[4 * k + 2] = v.z;
      f[4 * k + 3] = v.w;
    }
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + i));
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = to_float(e[k]);
  }
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

// 1 / sqrt(v): the hardware's estimate and one Newton step.
__device__ __forceinline__ float rsqrt_newton(float v) {
  const float r = rsqrtf(v);
  return r * (1.5f - (0.5f * v * r) * r);
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
  bool w_wide;       // weight and bias are 16-byte aligned
};

// A thread's share of a row is NV vectors, held as pairs: of VEC neighbouring
// elements (one 16-byte access, whole or past the row), or, for VEC = 1, of two
// single elements tpr apart.
template <int VEC>
struct Share {
  static constexpr int W = VEC == 1 ? 2 : VEC;  // elements of a vector
  static constexpr int P = W / 2;
  // column of element e of vector i
  static __device__ __forceinline__ int col(int i, int e, int tid, int tpr) {
    return VEC == 1 ? (2 * i + e) * tpr + tid : (i * tpr + tid) * VEC + e;
  }
};

// Vector i of a row, zeros past `cols` (0 for a row that is not there).
template <class T, int VEC>
__device__ __forceinline__ void load_share(const T* x, int i, int tid, int tpr, int cols,
                                           float2 (&v)[Share<VEC>::P]) {
  using S = Share<VEC>;
  float e[S::W];
#pragma unroll
  for (int k = 0; k < S::W; ++k) e[k] = 0.0f;
  if constexpr (VEC == 1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = S::col(i, k, tid, tpr);
      if (c < cols) e[k] = to_float(__ldg(x + c));
    }
  } else {
    const int c = S::col(i, 0, tid, tpr);
    if (c < cols) load_vec<T, VEC>(x + c, e);
  }
#pragma unroll
  for (int k = 0; k < S::P; ++k) v[k] = make_float2(e[2 * k], e[2 * k + 1]);
}
template <class T, int VEC>
__device__ __forceinline__ void store_share(T* y, int i, int tid, int tpr, int cols, const float2 (&v)[Share<VEC>::P]) {
  using S = Share<VEC>;
  if constexpr (VEC == 1) {
    const int c0 = S::col(i, 0, tid, tpr), c1 = S::col(i, 1, tid, tpr);
    if (c0 < cols) y[c0] = from_float<T>(v[0].x);
    if (c1 < cols) y[c1] = from_float<T>(v[0].y);
  } else {
    const int c = S::col(i, 0, tid, tpr);
    if (c < cols) {
      float e[VEC];
#pragma unroll
      for (int k = 0; k < S::P; ++k) {
        e[2 * k] = v[k].x;
        e[2 * k + 1] = v[k].y;
      }
      store_vec<T, VEC>(y + c, e);
    }
  }
}
// The same of weight or bias, zeros past the row.
template <class T, int VEC>
__device__ __forceinline__ void param_share(const void* p, bool fp32, bool wide, int i, int tid, int tpr, int cols,
                                            float2 (&v)[Share<VEC>::P]) {
  using S = Share<VEC>;
  float e[S::W];
#pragma unroll
  for (int k = 0; k < S::W; ++k) e[k] = 0.0f;
  if constexpr (VEC == 1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = S::col(i, k, tid, tpr);
      if (c < cols) e[k] = param<T>(p, fp32, c);
    }
  } else {
    const int c = S::col(i, 0, tid, tpr);
    if (c < cols) param_vec<T, VEC>(p, fp32, wide, c, e);
  }
#pragma unroll
  for (int k = 0; k < S::P; ++k) v[k] = make_float2(e[2 * k], e[2 * k + 1]);
}

// A row is held by tpr threads (a multiple of 32), NV vectors of VEC elements
// each; a CTA holds blockDim / tpr rows.  An element costs about a dozen
// instructions, close to what HBM leaves time for, so arithmetic goes in pairs.
template <class T, int VEC, int NV, bool FP8>
__global__ void __launch_bounds__(NV * Share<VEC>::W > 8 ? 512 : 256) layer_norm_kernel(const LayerNormArgs p) {
  using S = Share<VEC>;
  constexpr int P = S::P;
  __shared__ float red[64];
  griddep_wait();
  griddep_launch_dependents();
  const int rpc = blockDim.x / p.tpr, tpr = p.tpr;
  const int tid = threadIdx.x % tpr;
  const int64_t row = (int64_t)blockIdx.x * rpc + threadIdx.x / tpr;
  const int warps = tpr / 32, warp0 = threadIdx.x / tpr * warps;
  const bool in = row < p.rows;
  const int cols = (int)p.cols;
  const T* x = static_cast<const T*>(p.x) + (in ? row : 0) * p.ldx;
  float2 v[NV][P];
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) load_share<T, VEC>(x, i, tid, tpr, in ? cols : 0, v[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) s = add2(s, v[i][k]);
  const float rn = 1.0f / (float)cols;
  const float mean = row_sum(s.x + s.y, red, warps, warp0, 0) * rn;
  const float2 nm = make_float2(-mean, -mean);
  float2 d2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (VEC == 1 || S::col(i, 0, tid, tpr) < cols) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        v[i][k] = add2(v[i][k], nm);
        if constexpr (VEC == 1) {
          if (S::col(i, 0, tid, tpr) >= cols) v[i][k].x = 0.0f;
          if (S::col(i, 1, tid, tpr) >= cols) v[i][k].y = 0.0f;
        }
        d2 = fma2(v[i][k], v[i][k], d2);
      }
    }
  }
  const float rstd = rsqrt_newton(row_sum(d2.x + d2.y, red, warps, warp0, 1) * rn + p.eps);
  if (in && tid == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float2 w[P];
    param_share<T, VEC>(p.weight, p.w_fp32, p.w_wide, i, tid, tpr, cols, w);
#pragma unroll
    for (int k = 0; k < P; ++k) v[i][k] = mul2(mul2(v[i][k], rstd), w[k]);
    if (p.bias) {
      param_share<T, VEC>(p.bias, p.w_fp32, p.w_wide, i, tid, tpr, cols, w);
#pragma unroll
      for (int k = 0; k < P; ++k) v[i][k] = add2(v[i][k], w[k]);
    }
    if constexpr (!FP8) {
      if (in) store_share<T, VEC>(static_cast<T*>(p.y) + row * p.cols, i, tid, tpr, cols, v[i]);
    } else {
      // 128 / VEC neighbouring threads hold a group of 128 columns, whole or not at all
      const int c = S::col(i, 0, tid, tpr);
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < P; ++k) m = abs_max2(m, v[i][k]);
#pragma unroll
      for (int o = 64 / VEC; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (c < cols && row < p.rows_pad) {
        const uint32_t e = scale_byte(m);
        if (in) {
          const float inv = inverse_of_byte(e);
          uint32_t q[VEC / 4];
#pragma unroll
          for (int k = 0; k < VEC / 4; ++k) q[k] = e4m3x4(mul2(v[i][2 * k], inv), mul2(v[i][2 * k + 1], inv));
          uint8_t* dst = static_cast<uint8_t*>(p.y) + row * p.cols + c;
          if constexpr (VEC == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
          else *reinterpret_cast<uint32_t*>(dst) = q[0];
        }
        if (c % 128 == 0) {
          const int kb = c / 128;
          store_scale_byte(p.sf + (int64_t)(kb >> 2) * p.rows_pad + row, kb, c + 128 == cols, in ? e : 0u);
        }
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
  const float rstd = rsqrt_newton(row_sum(d2, red, warps, 0, 1) / n + p.eps);
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

// Backward: a CTA holds blockDim / tpr rows at a time and walks on by the grid,
// every thread keeping the sums dw and db of its own columns in registers; at
// the end the CTA adds its row groups' sums up in order and writes them to
// `part`.  With 16-byte accesses the rows ahead are on their way into shared
// memory (a ring of kNormRing; each thread copies and reads only its own
// pieces, so no barrier guards them) while a row's two sums cross the CTA.
constexpr int kNormRing = 4;
constexpr int kNormParts = 4;  // most CTAs an SM that keep column sums

template <class T, int VEC, int NV>
__global__ void __launch_bounds__(512) layer_norm_backward_kernel(const LayerNormArgs p) {
  constexpr bool kRing = VEC > 1;
  using S = Share<VEC>;
  constexpr int P = S::P;
  extern __shared__ uint4 ring[];  // [kNormRing][x, dy][NV][blockDim]; at the end, the row groups' sums
  __shared__ float red[2][32];     // a warp's two sums
  griddep_wait();
  griddep_launch_dependents();
  const int rpc = blockDim.x / p.tpr, tpr = p.tpr;
  const int tid = threadIdx.x % tpr, lane = threadIdx.x % 32;
  const int warps = tpr / 32, warp0 = threadIdx.x / tpr * warps;
  const int cols = (int)p.cols;
  const int64_t step = (int64_t)gridDim.x * rpc;
  const int64_t first = (int64_t)blockIdx.x * rpc + threadIdx.x / tpr;
  float2 w[NV][P], aw[NV][P], ab[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    param_share<T, VEC>(p.weight, p.w_fp32, p.w_wide, i, tid, tpr, cols, w[i]);
#pragma unroll
    for (int k = 0; k < P; ++k) aw[i][k] = ab[i][k] = make_float2(0.0f, 0.0f);
  }
  auto slot = [&](int s, int which, int i) { return ring + ((s * 2 + which) * NV + i) * blockDim.x + threadIdx.x; };
  auto fetch = [&](int64_t row, int s) {
    if (row < p.rows) {
      const T* x = static_cast<const T*>(p.x) + row * p.ldx;
      const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + tid) * VEC;
        if (c < cols) {
          cp_async16(slot(s, 0, i), x + c);
          cp_async16(slot(s, 1, i), dy + c);
        }
      }
    }
    cp_async_commit();
  };
  if constexpr (kRing)
    for (int s = 0; s < kNormRing - 1; ++s) fetch(first + s * step, s);
  const float rn = 1.0f / (float)cols;
  int at = 0, turn = 0;
  // every row group of the CTA takes as many rounds as its first one
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < p.rows; base += step) {
    const int64_t row = base + threadIdx.x / tpr;
    const bool in = row < p.rows;
    const float mean = in ? __ldg(p.mean + row) : 0.0f, rstd = in ? __ldg(p.rstd + row) : 0.0f;
    if constexpr (kRing) {
      // the slot read in the last round is free: this thread alone read it
      fetch(row + (kNormRing - 1) * step, at == 0 ? kNormRing - 1 : at - 1);
      cp_async_wait<kNormRing - 1>();
    }
    float2 xv[NV][P], dv[NV][P];
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (kRing) {
        const bool here = in && S::col(i, 0, tid, tpr) < cols;
        const uint4 a = here ? *slot(at, 0, i) : make_uint4(0, 0, 0, 0), b = here ? *slot(at, 1, i) : make_uint4(0, 0, 0, 0);
        const T *ae = reinterpret_cast<const T*>(&a), *be = reinterpret_cast<const T*>(&b);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          xv[i][k] = make_float2(to_float(ae[2 * k]), to_float(ae[2 * k + 1]));
          dv[i][k] = make_float2(to_float(be[2 * k]), to_float(be[2 * k + 1]));
        }
      } else {
        load_share<T, VEC>(static_cast<const T*>(p.x) + (in ? row : 0) * p.ldx, i, tid, tpr, in ? cols : 0, xv[i]);
        load_share<T, VEC>(static_cast<const T*>(p.dy) + (in ? row : 0) * p.lddy, i, tid, tpr, in ? cols : 0, dv[i]);
      }
    }
    if (++at == kNormRing) at = 0;
    // past the row dy is 0, so whatever xh is there adds nothing
    const float2 nm = make_float2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < P; ++k) {
        xv[i][k] = mul2(add2(xv[i][k], nm), rstd);
        aw[i][k] = fma2(dv[i][k], xv[i][k], aw[i][k]);
        ab[i][k] = add2(ab[i][k], dv[i][k]);
        dv[i][k] = mul2(dv[i][k], w[i][k]);
        s1 = add2(s1, dv[i][k]);
        s2 = fma2(dv[i][k], xv[i][k], s2);
      }
    float c1, c2;
    const float both = warp_sum2(s1.x + s1.y, s2.x + s2.y);
    if (warps == 1) {
      c1 = __shfl_sync(0xffffffffu, both, 0) * rn;
      c2 = __shfl_sync(0xffffffffu, both, 16) * rn;
    } else {
      // alternating slots: one barrier a round is enough.  [warp][s1, s2]
      float* r = red[turn];
      turn ^= 1;
      if (lane % 16 == 0) r[(threadIdx.x / 32) * 2 + lane / 16] = both;
      __syncthreads();
      float t = 0.0f;  // lanes 0-15: s1 of the row's warps, lanes 16-31: s2
      if (lane % 16 < warps) t = r[(warp0 + lane % 16) * 2 + lane / 16];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      c1 = __shfl_sync(0xffffffffu, t, 0) * rn;
      c2 = __shfl_sync(0xffffffffu, t, 16) * rn;
    }
    const float2 nc1 = make_float2(-c1, -c1), nc2 = make_float2(-c2, -c2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < P; ++k) dv[i][k] = mul2(fma2(xv[i][k], nc2, add2(dv[i][k], nc1)), rstd);
      if (in) store_share<T, VEC>(static_cast<T*>(p.y) + row * p.cols, i, tid, tpr, cols, dv[i]);
    }
  }
  if constexpr (kRing) cp_async_wait<0>();
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  float* partb = part + (int64_t)gridDim.x * p.cols;
  float2* sums = reinterpret_cast<float2*>(ring);  // [row group][2][NV][P][tpr]
  if (rpc > 1) {
    __syncthreads();
    float2* mine = sums + (size_t)(threadIdx.x / tpr) * 2 * NV * P * tpr + tid;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < P; ++k) {
        mine[(i * P + k) * tpr] = aw[i][k];
        mine[((NV + i) * P + k) * tpr] = ab[i][k];
      }
    __syncthreads();
    if (threadIdx.x >= tpr) return;
    for (int g = 1; g < rpc; ++g) {
      mine += 2 * NV * P * tpr;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          aw[i][k] = add2(aw[i][k], mine[(i * P + k) * tpr]);
          ab[i][k] = add2(ab[i][k], mine[((NV + i) * P + k) * tpr]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < S::W; ++k) {
      const int c = S::col(i, k, tid, tpr);
      if (c < cols) {
        part[c] = k % 2 ? aw[i][k / 2].y : aw[i][k / 2].x;
        partb[c] = k % 2 ? ab[i][k / 2].y : ab[i][k / 2].x;
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
  // Vectors a thread: up to 4 of 16 bytes, or 8 or 32 single elements, the
  // fewest that keep a row within 512 threads; rows of up to 4 vectors a lane
  // are one warp's, so that they need no barrier.  CTAs of about 128 threads.
  const int64_t units = vec ? p.cols / V : p.cols;
  const int64_t rows = FP8 ? p.rows_pad : p.rows;
  auto go = [&](auto kern, int nv) {
    const int64_t t = ((units + nv - 1) / nv + 31) / 32 * 32;
    p.tpr = (int)t;
    const int rpc = t >= 128 ? 1 : (int)(128 / t);
    return launch_op(kern, dim3((unsigned)((rows + rpc - 1) / rpc)), (unsigned)(rpc * t), 0, pdl, st, p);
  };
  if (vec) {
    if (units <= 32) return go(layer_norm_kernel<T, V, 1, FP8>, 1);
    if (units <= 64) return go(layer_norm_kernel<T, V, 2, FP8>, 2);
    if (units <= 4 * 512) return go(layer_norm_kernel<T, V, 4, FP8>, 4);
    if (units <= 8 * 512) return go(layer_norm_kernel<T, V, 8, FP8>, 8);
  }
  if constexpr (FP8) return cudaErrorInvalidValue;
  else {
    if (!vec && units <= 8 * 512) return go(layer_norm_kernel<T, 1, 4, false>, 8);
    if (!vec && units <= 32 * 512) return go(layer_norm_kernel<T, 1, 16, false>, 32);
    return launch_op(layer_norm_long_kernel<T>, dim3((unsigned)p.rows), 1024, 0, pdl, st, p);
  }
}

template <class T>
cudaError_t backward(const LayerNormArgs& a, bool vec, int parts, int* used, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t units = vec ? p.cols / V : p.cols;
  // A row takes tpr threads of nv vectors (8 or 16 elements of 16-byte
  // accesses, 4 or 16 single ones); CTAs of 128 threads or one row, as many an
  // SM as its threads, registers and shared memory take, at most kNormParts.
  auto go = [&](auto kern, int nv) {
    const int64_t t = ((units + nv - 1) / nv + 31) / 32 * 32;
    p.tpr = (int)t;
    const int rpc = t >= 128 ? 1 : (int)(128 / t);
    const int64_t threads = rpc * t;
    const size_t sums = rpc > 1 ? (size_t)threads * nv * (vec ? V : 1) * 2 * sizeof(float) : 0;
    const size_t smem = std::max<size_t>(vec ? (size_t)kNormRing * 2 * nv * threads * 16 : 0, sums);
    int64_t per_sm = std::min<int64_t>(kNormParts, 65536 / 128 / threads);
    per_sm = std::max<int64_t>(1, std::min<int64_t>(per_sm, (int64_t)(220 * 1024) / (int64_t)(smem + 2048)));
    *used = (int)std::min<int64_t>((p.rows + rpc - 1) / rpc, per_sm * (parts / kNormParts));
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_op(kern, dim3((unsigned)*used), (unsigned)threads, smem, pdl, st, p);
  };
  if (vec && units <= 256) return go(layer_norm_backward_kernel<T, V, 1>, 1);
  if (vec && units <= 2 * 512) return go(layer_norm_backward_kernel<T, V, 2>, 2);
  if (!vec && units <= 4 * 256) return go(layer_norm_backward_kernel<T, 1, 2>, 4);
  if (!vec && units <= 16 * 512) return go(layer_norm_backward_kernel<T, 1, 8>, 16);
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
  p.w_wide = (((uintptr_t)weight | (uintptr_t)bias) & 15) == 0;
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

int layer_norm_backward_parts(int sms) { return kNormParts * sms; }

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
  p.w_wide = ((uintptr_t)weight & 15) == 0;
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
