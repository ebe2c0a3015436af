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
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? red[row_warp0 + lane] : 0.0f);
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

// VEC values of one row from column c on as E4M3 codes; the 128 / VEC
// neighbouring threads that hold a group of 128 columns (whole or past the
// row) share its scale.
template <int VEC>
__device__ __forceinline__ void store_codes(const LayerNormArgs& p, const float2 (&v)[Share<VEC>::P], int64_t row, int c,
                                            int cols, bool in) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < Share<VEC>::P; ++k) m = abs_max2(m, v[k]);
#pragma unroll
  for (int o = 64 / VEC; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (c >= cols || row >= p.rows_pad) return;
  const uint32_t e = scale_byte(m);
  if (in) {
    const float inv = inverse_of_byte(e);
    uint32_t q[VEC / 4];
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) q[k] = e4m3x4(mul2(v[2 * k], inv), mul2(v[2 * k + 1], inv));
    uint8_t* dst = static_cast<uint8_t*>(p.y) + row * p.cols + c;
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(dst) = q[0];
  }
  if (c % 128 == 0) {
    const int kb = c / 128;
    store_scale_byte(p.sf + (int64_t)(kb >> 2) * p.rows_pad + row, kb, c + 128 == cols, in ? e : 0u);
  }
}

// A row is held by tpr threads (a multiple of 32), NV vectors of VEC elements
// each; a CTA holds blockDim / tpr rows.  An element costs about a dozen
// instructions, close to what HBM leaves time for, so arithmetic goes in pairs.
template <class T, int VEC, int NV, bool FP8>
__global__ void __launch_bounds__(512) layer_norm_kernel(const LayerNormArgs p) {
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
      store_codes<VEC>(p, v[i], row, S::col(i, 0, tid, tpr), cols, in);
    }
  }
}

// Rows on their way into shared memory.  A warp's share of a row is 32 NV pieces
// of 16 bytes, copied by its lanes side by side and read back as each lane's
// own NV neighbouring pieces (with two, stored crosswise so that 8 lanes meet
// no bank twice).  Pieces past the row are never copied and stay zero, rows
// past the last leave what was there; only the warp itself reads its pieces,
// so __syncwarp is all that guards them.
constexpr int kNormRing = 4;

template <class T, int NV>
struct RowRing {
  static constexpr int V = 16 / (int)sizeof(T);
  static constexpr int E = NV * V;  // neighbouring columns of a lane
  uint4* mine;                      // [kNormRing][blockDim / 32][32 NV] at this warp's part
  int stage;                        // distance between stages
  const T* src;                     // this lane's first piece of the next row to copy
  int64_t step;                     // elements between the rows this thread meets
  int64_t row, rows, row_step;      // the next row to copy
  uint32_t on;                      // bit j: piece lane + 32 j lies in the row

  __device__ __forceinline__ static int place(int p) { return NV == 2 ? p ^ ((p >> 3) & 1) : p; }
  __device__ __forceinline__ void init(uint4* ring, const void* x, int64_t ld, int64_t first, int64_t every,
                                       int64_t last, int tid, int cols) {
    const int lane = threadIdx.x & 31;
    mine = ring + (threadIdx.x >> 5) * 32 * NV;
    stage = blockDim.x * NV;
    const int c0 = (tid >> 5) * 32 * E;
    src = static_cast<const T*>(x) + first * ld + c0 + lane * V;
    step = every * ld;
    row = first;
    rows = last;
    row_step = every;
    on = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (c0 + (lane + 32 * j) * V < cols) on |= 1u << j;
      else
        for (int s = 0; s < kNormRing; ++s) mine[s * stage + place(lane + 32 * j)] = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void fetch(int s) {
    if (row < rows) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on >> j & 1) cp_async16(mine + s * stage + place(lane + 32 * j), src + 32 * j * V);
    }
    src += step;
    row += row_step;
  }
  __device__ __forceinline__ void read(int s, float2 (&v)[NV][V / 2]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint4 a = mine[s * stage + place(lane * NV + j)];
      const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) v[j][k] = make_float2(to_float(e[2 * k]), to_float(e[2 * k + 1]));
    }
  }
};

// A lane's NV neighbouring pieces of a row of y; `wide`: in one access of 32 bytes.
template <class T, int NV>
__device__ __forceinline__ void store_pieces(T* y, bool wide, uint32_t on, const float2 (&v)[NV][8 / (int)sizeof(T)]) {
  constexpr int V = 16 / (int)sizeof(T);
  uint32_t w[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    T* e = reinterpret_cast<T*>(w[j]);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      e[2 * k] = from_float<T>(v[j][k].x);
      e[2 * k + 1] = from_float<T>(v[j][k].y);
    }
  }
  if (NV == 2 && wide && on == 3u) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y), "r"(w[0][0]), "r"(w[0][1]),
                 "r"(w[0][2]), "r"(w[0][3]), "r"(w[NV - 1][0]), "r"(w[NV - 1][1]), "r"(w[NV - 1][2]), "r"(w[NV - 1][3])
                 : "memory");
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (on >> j & 1) *reinterpret_cast<uint4*>(y + j * V) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
}

// Weight or bias of a lane's columns, zeros past the row.
template <class T, int NV>
__device__ __forceinline__ void param_pieces(const void* p, bool fp32, bool wide, int c, uint32_t on,
                                             float2 (&v)[NV][8 / (int)sizeof(T)]) {
  constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float e[V];
#pragma unroll
    for (int k = 0; k < V; ++k) e[k] = 0.0f;
    if (p && (on >> j & 1)) param_vec<T, V>(p, fp32, wide, c + j * V, e);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) v[j][k] = make_float2(e[2 * k], e[2 * k + 1]);
  }
}

// The forward pass for rows of up to 896 pieces of 16 bytes: a CTA keeps its
// columns' weight and bias in registers and walks over rows by the grid.
// Reading weight and bias anew for every row would move four times the row's
// own bytes through L1.
template <class T, int NV, bool FP8>
__global__ void __launch_bounds__(NV == 1 ? 256 : 448, NV == 1 ? 5 : 2) layer_norm_ring_kernel(const LayerNormArgs p) {
  using R = RowRing<T, NV>;
  constexpr int P = R::V / 2, E = R::E;
  extern __shared__ uint4 ring[];
  __shared__ float red[64];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.tpr, rpc = blockDim.x / tpr;
  const int tid = threadIdx.x % tpr;
  const int warps = tpr / 32, warp0 = threadIdx.x / tpr * warps;
  const int cols = (int)p.cols;
  const int64_t rows = FP8 ? p.rows_pad : p.rows;
  const int64_t step = (int64_t)gridDim.x * rpc;
  int64_t row = (int64_t)blockIdx.x * rpc + threadIdx.x / tpr;
  R src;
  src.init(ring, p.x, p.ldx, row, step, p.rows, tid, cols);
  const int c = tid * E;
  uint32_t on = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c + j * R::V < cols) on |= 1u << j;
  float2 w[NV][P], b[NV][P];
  param_pieces<T, NV>(p.weight, p.w_fp32, p.w_wide, c, on, w);
  param_pieces<T, NV>(p.bias, p.w_fp32, p.w_wide, c, on, b);
  const bool wide = ((p.cols * (int64_t)sizeof(T)) | (int64_t)(uintptr_t)p.y) % 32 == 0;
  const int64_t y_step = step * p.cols;
  T* y = static_cast<T*>(p.y) + row * p.cols + c;             // same-type results
  uint8_t* q = static_cast<uint8_t*>(p.y) + row * p.cols + c;  // 8-bit results
  uint32_t* sf = p.sf + (int64_t)(c / 512) * p.rows_pad + row;
  const int kb = c / 128;
  const bool sf_mine = FP8 && on && c % 128 == 0, sf_last = c + 128 == cols;
  for (int s = 0; s < kNormRing - 1; ++s) {
    src.fetch(s);
    cp_async_commit();
  }
  const float rn = 1.0f / (float)cols;
  int at = 0;
  // every row group of the CTA takes as many rounds as its first one
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < rows; base += step) {
    const bool in = row < p.rows;
    __syncwarp();  // the warp has read the slot that is filled next
    src.fetch(at == 0 ? kNormRing - 1 : at - 1);
    cp_async_commit();
    cp_async_wait<kNormRing - 1>();
    __syncwarp();
    float2 v[NV][P];
    src.read(at, v);
    if (++at == kNormRing) at = 0;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < P; ++k) s = add2(s, v[j][k]);
    const float mean = row_sum(s.x + s.y, red, warps, warp0, 0) * rn;
    float2 d2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float m = (on >> j & 1) ? -mean : 0.0f;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        v[j][k] = add2(v[j][k], make_float2(m, m));
        d2 = fma2(v[j][k], v[j][k], d2);
      }
    }
    const float rstd = rsqrt_newton(row_sum(d2.x + d2.y, red, warps, warp0, 1) * rn + p.eps);
    if (in && tid == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < P; ++k) v[j][k] = fma2(mul2(v[j][k], rstd), w[j][k], b[j][k]);
    if constexpr (!FP8) {
      if (in) store_pieces<T, NV>(y, wide, on, v);
    } else {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < P; ++k) m = abs_max2(m, v[j][k]);
#pragma unroll
      for (int o = 64 / E; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t e = scale_byte(m);
      if (in && on) {
        const float inv = inverse_of_byte(e);
        uint32_t o[E / 4];
#pragma unroll
        for (int k = 0; k < E / 4; ++k) {
          const int j = 4 * k / R::V, i = (4 * k % R::V) / 2;
          o[k] = e4m3x4(mul2(v[j][i], inv), mul2(v[j][i + 1], inv));
        }
        if constexpr (E == 16) *reinterpret_cast<uint4*>(q) = make_uint4(o[0], o[1], o[2], o[3]);
        else if constexpr (E == 8) *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
        else *reinterpret_cast<uint32_t*>(q) = o[0];
      }
      if (sf_mine && row < rows) store_scale_byte(sf, kb, sf_last, in ? e : 0u);
      sf += step;
    }
    y += y_step;
    q += y_step;
    row += step;
  }
  cp_async_wait<0>();
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
// `part`.
constexpr int kNormParts = 4;  // most CTAs an SM that keep column sums

// A row's two sums, from a thread's share of them, to every thread of the row.
__device__ __forceinline__ float2 row_sum_pair(float a, float b, float (&red)[2][32], int turn, int warps, int warp0) {
  const int lane = threadIdx.x & 31;
  float t = warp_sum2(a, b);  // lanes 0-15: a, lanes 16-31: b
  if (warps > 1) {
    float* r = red[turn];  // alternating slots: one barrier a row is enough.  [warp][a, b]
    if (lane % 16 == 0) r[(threadIdx.x / 32) * 2 + lane / 16] = t;
    __syncthreads();
    t = lane % 16 < warps ? r[(warp0 + lane % 16) * 2 + lane / 16] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  return make_float2(__shfl_sync(0xffffffffu, t, 0), __shfl_sync(0xffffffffu, t, 16));
}

// One row's share: x becomes xh, dy becomes dx; the columns' sums grow.
template <int NV, int P>
__device__ __forceinline__ float2 backward_sums(float2 (&xv)[NV][P], float2 (&dv)[NV][P], const float2 (&w)[NV][P],
                                                float2 (&aw)[NV][P], float2 (&ab)[NV][P], float mean, float rstd) {
  const float2 nm = make_float2(-mean, -mean);
  float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
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
  return make_float2(s1.x + s1.y, s2.x + s2.y);
}
template <int NV, int P>
__device__ __forceinline__ void backward_dx(const float2 (&xv)[NV][P], float2 (&dv)[NV][P], float2 c, float rn, float rstd) {
  const float2 n1 = make_float2(-c.x * rn, -c.x * rn), n2 = make_float2(-c.y * rn, -c.y * rn);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) dv[i][k] = mul2(fma2(xv[i][k], n2, add2(dv[i][k], n1)), rstd);
}
// Adds the CTA's row groups' sums up in their order; false in the threads of
// all groups but the first, which ends with the whole.
template <int NV, int P>
__device__ __forceinline__ bool join_groups(float2* sums, int tpr, float2 (&aw)[NV][P], float2 (&ab)[NV][P]) {
  const int rpc = blockDim.x / tpr;
  if (rpc == 1) return true;
  __syncthreads();
  float2* mine = sums + (size_t)(threadIdx.x / tpr) * 2 * NV * P * tpr + threadIdx.x % tpr;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) {
      mine[(i * P + k) * tpr] = aw[i][k];
      mine[((NV + i) * P + k) * tpr] = ab[i][k];
    }
  __syncthreads();
  if ((int)threadIdx.x >= tpr) return false;
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
  return true;
}

template <class T, int NV>
__global__ void __launch_bounds__(NV == 1 ? 256 : 512, NV == 1 ? 4 : 1)
    layer_norm_backward_ring_kernel(const LayerNormArgs p) {
  using R = RowRing<T, NV>;
  constexpr int P = R::V / 2;
  extern __shared__ uint4 ring[];  // x's rows, then dy's; at the end, the row groups' sums
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.tpr, rpc = blockDim.x / tpr;
  const int tid = threadIdx.x % tpr;
  const int warps = tpr / 32, warp0 = threadIdx.x / tpr * warps;
  const int cols = (int)p.cols;
  const int64_t step = (int64_t)gridDim.x * rpc;
  int64_t row = (int64_t)blockIdx.x * rpc + threadIdx.x / tpr;
  R xs, ds;
  xs.init(ring, p.x, p.ldx, row, step, p.rows, tid, cols);
  ds.init(ring + kNormRing * blockDim.x * NV, p.dy, p.lddy, row, step, p.rows, tid, cols);
  const int c = tid * R::E;
  uint32_t on = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c + j * R::V < cols) on |= 1u << j;
  float2 w[NV][P], aw[NV][P], ab[NV][P];
  param_pieces<T, NV>(p.weight, p.w_fp32, p.w_wide, c, on, w);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < P; ++k) aw[j][k] = ab[j][k] = make_float2(0.0f, 0.0f);
  const bool wide = ((p.cols * (int64_t)sizeof(T)) | (int64_t)(uintptr_t)p.y) % 32 == 0;
  const int64_t y_step = step * p.cols;
  T* y = static_cast<T*>(p.y) + row * p.cols + c;
  for (int s = 0; s < kNormRing - 1; ++s) {
    xs.fetch(s);
    ds.fetch(s);
    cp_async_commit();
  }
  const float rn = 1.0f / (float)cols;
  int at = 0, turn = 0;
  // a row's mean and rstd are loaded a round ahead
  float mean = row < p.rows ? __ldg(p.mean + row) : 0.0f, rstd = row < p.rows ? __ldg(p.rstd + row) : 0.0f;
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < p.rows; base += step) {
    const bool in = row < p.rows;
    __syncwarp();  // the warp has read the slot that is filled next
    const int next = at == 0 ? kNormRing - 1 : at - 1;
    xs.fetch(next);
    ds.fetch(next);
    cp_async_commit();
    const bool more = row + step < p.rows;
    const float mean1 = more ? __ldg(p.mean + row + step) : 0.0f, rstd1 = more ? __ldg(p.rstd + row + step) : 0.0f;
    cp_async_wait<kNormRing - 1>();
    __syncwarp();
    float2 xv[NV][P], dv[NV][P];
    xs.read(at, xv);
    ds.read(at, dv);
    if (++at == kNormRing) at = 0;
    if (!in) {  // the last round of a row group that has no row in it: an old row adds nothing
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < P; ++k) xv[j][k] = dv[j][k] = make_float2(0.0f, 0.0f);
    }
    const float2 mine = backward_sums<NV, P>(xv, dv, w, aw, ab, mean, rstd);
    const float2 sums = row_sum_pair(mine.x, mine.y, red, turn, warps, warp0);
    turn ^= 1;
    backward_dx<NV, P>(xv, dv, sums, rn, rstd);
    if (in) store_pieces<T, NV>(y, wide, on, dv);
    y += y_step;
    row += step;
    mean = mean1;
    rstd = rstd1;
  }
  cp_async_wait<0>();
  if (!join_groups<NV, P>(reinterpret_cast<float2*>(ring), tpr, aw, ab)) return;
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  float* partb = part + (int64_t)gridDim.x * p.cols;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (on >> j & 1) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int cc = c + j * R::V + 2 * k;
        part[cc] = aw[j][k].x;
        part[cc + 1] = aw[j][k].y;
        partb[cc] = ab[j][k].x;
        partb[cc + 1] = ab[j][k].y;
      }
    }
}

// The same where rows are not 16-byte aligned: single elements, read directly.
template <class T, int NV>
__global__ void __launch_bounds__(512) layer_norm_backward_kernel(const LayerNormArgs p) {
  extern __shared__ uint4 ring[];  // the row groups' sums
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.tpr, rpc = blockDim.x / tpr;
  const int tid = threadIdx.x % tpr;
  const int warps = tpr / 32, warp0 = threadIdx.x / tpr * warps;
  const int cols = (int)p.cols;
  float2 w[NV][1], aw[NV][1], ab[NV][1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    param_share<T, 1>(p.weight, p.w_fp32, p.w_wide, i, tid, tpr, cols, w[i]);
    aw[i][0] = ab[i][0] = make_float2(0.0f, 0.0f);
  }
  const float rn = 1.0f / (float)cols;
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < p.rows; base += (int64_t)gridDim.x * rpc) {
    const int64_t row = base + threadIdx.x / tpr;
    const bool in = row < p.rows;
    const float mean = in ? __ldg(p.mean + row) : 0.0f, rstd = in ? __ldg(p.rstd + row) : 0.0f;
    float2 xv[NV][1], dv[NV][1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_share<T, 1>(static_cast<const T*>(p.x) + (in ? row : 0) * p.ldx, i, tid, tpr, in ? cols : 0, xv[i]);
      load_share<T, 1>(static_cast<const T*>(p.dy) + (in ? row : 0) * p.lddy, i, tid, tpr, in ? cols : 0, dv[i]);
    }
    const float2 mine = backward_sums<NV, 1>(xv, dv, w, aw, ab, mean, rstd);  // past the row dy is 0
    const float2 sums = row_sum_pair(mine.x, mine.y, red, turn, warps, warp0);
    turn ^= 1;
    backward_dx<NV, 1>(xv, dv, sums, rn, rstd);
    if (in) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        store_share<T, 1>(static_cast<T*>(p.y) + row * p.cols, i, tid, tpr, cols, dv[i]);
    }
  }
  if (!join_groups<NV, 1>(reinterpret_cast<float2*>(ring), tpr, aw, ab)) return;
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  float* partb = part + (int64_t)gridDim.x * p.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = Share<1>::col(i, k, tid, tpr);
      if (c < cols) {
        part[c] = k ? aw[i][0].y : aw[i][0].x;
        partb[c] = k ? ab[i][0].y : ab[i][0].x;
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
cudaError_t forward(const LayerNormArgs& a, bool vec, int sms, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  // Rows of up to 896 vectors take the ring kernel: 1 or 2 vectors a thread,
  // CTAs of 128 threads or one row.  Longer ones are read into 4 or 8 vectors
  // a thread (or 8 or 32 single elements) of one CTA a row.
  const int64_t units = vec ? p.cols / V : p.cols;
  const int64_t rows = FP8 ? p.rows_pad : p.rows;
  auto shape = [&](int nv) {
    const int64_t t = ((units + nv - 1) / nv + 31) / 32 * 32;
    p.tpr = (int)t;
    return t >= 128 ? t : 128 / t * t;
  };
  auto go = [&](auto kern, int nv) {
    const int64_t threads = shape(nv), rpc = threads / p.tpr;
    return launch_op(kern, dim3((unsigned)((rows + rpc - 1) / rpc)), (unsigned)threads, 0, pdl, st, p);
  };
  auto go_ring = [&](auto kern, int nv) {
    const int64_t threads = shape(nv), rpc = threads / p.tpr;
    const size_t smem = (size_t)kNormRing * nv * threads * 16;
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>((int64_t)(220 * 1024) / (int64_t)(smem + 2048),
                                                                  (nv == 1 ? 1280 : 896) / threads));
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_op(kern, dim3((unsigned)std::min<int64_t>((rows + rpc - 1) / rpc, per_sm * sms)), (unsigned)threads,
                     smem, pdl, st, p);
  };
  if (vec) {
    if (units <= 256) return go_ring(layer_norm_ring_kernel<T, 1, FP8>, 1);
    if (units <= 2 * 448) return go_ring(layer_norm_ring_kernel<T, 2, FP8>, 2);  // 2 x 448 threads of 72 registers
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
  // A row takes tpr threads of 1 or 2 pieces of 16 bytes (4 or 16 single
  // elements); CTAs of 128 threads or one row, as many an SM as fit, at most
  // kNormParts.
  auto go = [&](auto kern, int nv, int most) {
    const int64_t t = ((units + nv - 1) / nv + 31) / 32 * 32;
    p.tpr = (int)t;
    const int64_t threads = t >= 128 ? t : 128 / t * t;
    const int64_t rpc = threads / t;
    const size_t sums = rpc > 1 ? (size_t)threads * nv * (vec ? V : 1) * 2 * sizeof(float) : 0;
    const size_t smem = std::max<size_t>(vec ? (size_t)kNormRing * 2 * nv * threads * 16 : 0, sums);
    int64_t per_sm = std::min<int64_t>(kNormParts, most / threads);
    per_sm = std::max<int64_t>(1, std::min<int64_t>(per_sm, (int64_t)(220 * 1024) / (int64_t)(smem + 2048)));
    *used = (int)std::min<int64_t>((p.rows + rpc - 1) / rpc, per_sm * (parts / kNormParts));
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_op(kern, dim3((unsigned)*used), (unsigned)threads, smem, pdl, st, p);
  };
  if (vec && units <= 256) return go(layer_norm_backward_ring_kernel<T, 1>, 1, 1024);
  if (vec && units <= 2 * 512) return go(layer_norm_backward_ring_kernel<T, 2>, 2, 512);
  if (!vec && units <= 4 * 256) return go(layer_norm_backward_kernel<T, 2>, 4, 1024);
  if (!vec && units <= 16 * 512) return go(layer_norm_backward_kernel<T, 8>, 16, 512);
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
                              int64_t cols, int64_t ldx, float eps, int sms, bool pdl, cudaStream_t stream) {
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
    return sf ? forward<float, true>(p, vec, sms, pdl, stream) : forward<float, false>(p, vec, sms, pdl, stream);
  if (dtype == DG_DTYPE_BF16)
    return sf ? forward<__nv_bfloat16, true>(p, vec, sms, pdl, stream) : forward<__nv_bfloat16, false>(p, vec, sms, pdl, stream);
  return sf ? forward<__half, true>(p, vec, sms, pdl, stream) : forward<__half, false>(p, vec, sms, pdl, stream);
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
