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
#include <type_traits>

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

// Two neighbouring 16-bit elements in one word, as FP32 and back.
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return make_float2(bf16_lo(w), bf16_hi(w));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float2 v) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return bf16x2_bits(v.x, v.y);
  else {
    const __half2 h = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// 16 bytes as pairs of FP32 and back.
template <class T>
__device__ __forceinline__ void unpack16(const uint4& a, float2* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
  } else {
    v[0] = unpack2<T>(a.x);
    v[1] = unpack2<T>(a.y);
    v[2] = unpack2<T>(a.z);
    v[3] = unpack2<T>(a.w);
  }
}
template <class T>
__device__ __forceinline__ uint4 pack16(const float2* v) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  else return make_uint4(pack2<T>(v[0]), pack2<T>(v[1]), pack2<T>(v[2]), pack2<T>(v[3]));
}

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
  int64_t ring_bytes;  // of one ring of rows
  int tpr;             // threads a row
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

// ---------------------------------------------------------------- rows in a ring
// Rows on their way into shared memory, Row::kRing of them, while others are
// worked on.  Every warp copies and reads only its own columns, so __syncwarp
// is all that guards them.  Two forms with one interface: a thread's P pairs of
// values of a row (zeros past it), the same of weight or bias, and storing them.

// Rows of whole, 16-byte aligned pieces.  A warp's share is 32 NV pieces, copied
// by its lanes side by side and read back as each lane's own NV neighbouring
// pieces (with two, stored crosswise so that 8 lanes meet no bank twice).
// Pieces past the row are never copied and stay zero; rows past the last leave
// what was there.
template <class T_, int NV_>
struct AlignedRow {
  using T = T_;
  static constexpr int NV = NV_;
  static constexpr int V = 16 / (int)sizeof(T);
  static constexpr int E = NV * V;  // neighbouring columns of a lane
  static constexpr int P = E / 2;
  static constexpr int kRing = 4;
  static constexpr bool kWide = NV == 2;  // CTAs of up to 448 or 512 threads instead of 256
  static size_t bytes(int64_t threads) { return (size_t)kRing * NV * threads * 16; }
  static constexpr size_t store_bytes(int64_t) { return 0; }
  uint4* mine;                      // [kRing][blockDim / 32][32 NV] at this warp's part
  int stage;                        // distance between stages
  const T* src;                     // this lane's first piece of the next row to copy
  int64_t step;                     // elements between the rows this thread meets
  int64_t row, rows, row_step;      // the next row to copy
  uint32_t copy, on;                // bit j: piece lane + 32 j / the lane's own piece j lies in the row
  int c;                            // the lane's first column

  __device__ __forceinline__ static int place(int p) { return NV == 2 ? p ^ ((p >> 3) & 1) : p; }
  __device__ __forceinline__ void init(void* ring, const void* x, int64_t ld, int64_t first, int64_t every,
                                       int64_t last, int tid, int cols) {
    const int lane = threadIdx.x & 31;
    mine = static_cast<uint4*>(ring) + (threadIdx.x >> 5) * 32 * NV;
    stage = blockDim.x * NV;
    const int c0 = (tid >> 5) * 32 * E;
    src = static_cast<const T*>(x) + first * ld + c0 + lane * V;
    step = every * ld;
    row = first;
    rows = last;
    row_step = every;
    c = tid * E;
    copy = on = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (c + j * V < cols) on |= 1u << j;
      if (c0 + (lane + 32 * j) * V < cols) copy |= 1u << j;
      else
        for (int s = 0; s < kRing; ++s) mine[s * stage + place(lane + 32 * j)] = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void fetch(int s) {
    if (row < rows) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (copy >> j & 1) cp_async16(mine + s * stage + place(lane + 32 * j), src + 32 * j * V);
    }
    src += step;
    row += row_step;
  }
  __device__ __forceinline__ void read(int s, float2 (&v)[P]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack16<T>(mine[s * stage + place(lane * NV + j)], &v[j * V / 2]);
    }
  }
  __device__ __forceinline__ void params(const void* p, bool fp32, bool wide, float2 (&v)[P]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float e[V];
#pragma unroll
      for (int k = 0; k < V; ++k) e[k] = 0.0f;
      if (p && (on >> j & 1)) param_vec<T, V>(p, fp32, wide, c + j * V, e);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) v[j * V / 2 + k] = make_float2(e[2 * k], e[2 * k + 1]);
    }
  }
  // Adds m to the columns inside the row.
  __device__ __forceinline__ void shift(float2 (&v)[P], float m) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float a = (on >> j & 1) ? m : 0.0f;
#pragma unroll
      for (int k = 0; k < V / 2; ++k) v[j * V / 2 + k] = add2(v[j * V / 2 + k], make_float2(a, a));
    }
  }
  // Into the row at y; `wide`: rows start on 32 bytes, so two pieces are one access.
  __device__ __forceinline__ void store(T* y, bool wide, void*, const float2 (&v)[P]) const {
    y += c;
    uint4 w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) w[j] = pack16<T>(&v[j * V / 2]);
    if (NV == 2 && wide && on == 3u) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y), "r"(w[0].x), "r"(w[0].y),
                   "r"(w[0].z), "r"(w[0].w), "r"(w[NV - 1].x), "r"(w[NV - 1].y), "r"(w[NV - 1].z), "r"(w[NV - 1].w)
                   : "memory");
      return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on >> j & 1) *reinterpret_cast<uint4*>(y + j * V) = w[j];
  }
  // A column sum per pair element.
  __device__ __forceinline__ void store_sums(float* out, const float2 (&v)[P]) const {
#pragma unroll
    for (int k = 0; k < P; ++k)
      if (on >> (2 * k / V) & 1) {
        out[c + 2 * k] = v[k].x;
        out[c + 2 * k + 1] = v[k].y;
      }
  }
};

// Rows of any width and alignment.  A warp's share is 32 N columns; the
// 16-byte granules that cover them are copied whole (from the granule's start,
// which for the first column may lie before the row but not before the tensor,
// up to the row's last byte) and the lanes read their elements at the row's own
// offset: G neighbouring ones (2 where rows start on 4 bytes), 32 G columns
// apart.  Results are collected the same way and leave as whole granules, with
// single elements at both ends.
template <class T_, int N_, int G_>
struct RaggedRow {
  using T = T_;
  static constexpr int N = N_, G = G_, P = N / 2;
  static constexpr bool kWide = N == 16;
  static constexpr int kRing = kWide && sizeof(T) == 4 ? 2 : 4;  // what shared memory holds
  static constexpr int kSize = (int)sizeof(T);
  static constexpr int kGranules = 32 * N * kSize / 16 + 1;  // a warp's
  static size_t bytes(int64_t threads) { return (size_t)kRing * kGranules * (threads / 32) * 16; }
  static size_t store_bytes(int64_t threads) { return (size_t)kGranules * (threads / 32) * 16; }
  uint4* mine;
  int stage;
  const uint8_t* src;           // this warp's first column in the next row to copy
  const uint8_t* base;          // the tensor's first byte
  int64_t step, row, rows, row_step;
  uint32_t at, at_step;         // where in its granule the next row to read starts
  int seg, live, cols;          // this warp's first column, its columns inside the row

  __device__ __forceinline__ int col(int k, int e) const {  // element e of pair k
    const int lane = threadIdx.x & 31;
    return G == 2 ? seg + (k * 32 + lane) * 2 + e : seg + (2 * k + e) * 32 + lane;
  }
  __device__ __forceinline__ void init(void* ring, const void* x, int64_t ld, int64_t first, int64_t every,
                                       int64_t last, int tid, int n) {
    mine = static_cast<uint4*>(ring) + (threadIdx.x >> 5) * kGranules;
    stage = (int)(blockDim.x >> 5) * kGranules;
    seg = (tid >> 5) * 32 * N;
    cols = n;
    live = min(32 * N, n - seg);  // < 0: none
    base = static_cast<const uint8_t*>(x);
    src = base + (first * ld + seg) * kSize;
    step = every * ld * kSize;
    row = first;
    rows = last;
    row_step = every;
    at = (uint32_t)(uintptr_t)src;
    at_step = (uint32_t)step;
  }
  __device__ __forceinline__ void fetch(int s) {
    if (row < rows && live > 0) {
      const int lane = threadIdx.x & 31;
      const int skip = (int)((uintptr_t)src & 15u);
      const uint8_t* from = src - skip;
      const int total = skip + live * kSize;
#pragma unroll
      for (int i = 0; i < (kGranules + 31) / 32; ++i) {
        const int g = lane + 32 * i;
        if (g * 16 < total) {
          uint4* to = mine + s * stage + g;
          if (from + g * 16 >= base) cp_async16_part(to, from + g * 16, min(16, total - g * 16));
          else  // the tensor's first granule, where it starts inside one
            for (int b = skip; b < min(16, total); b += kSize)
              *reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(to) + b) = *reinterpret_cast<const T*>(from + b);
        }
      }
    }
    src += step;
    row += row_step;
  }
  __device__ __forceinline__ void read(int s, float2 (&v)[P]) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(mine + s * stage) + (at & 15u);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if constexpr (G == 2) {
        v[k] = unpack2<T>(*reinterpret_cast<const uint32_t*>(p + (k * 32 + lane) * 4));
      } else {
        v[k] = make_float2(to_float(*reinterpret_cast<const T*>(p + (2 * k * 32 + lane) * kSize)),
                           to_float(*reinterpret_cast<const T*>(p + ((2 * k + 1) * 32 + lane) * kSize)));
      }
    }
    at += at_step;
    if (live < 32 * N) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        if (col(k, 0) >= cols) v[k].x = 0.0f;
        if (col(k, 1) >= cols) v[k].y = 0.0f;
      }
    }
  }
  __device__ __forceinline__ void params(const void* p, bool fp32, bool, float2 (&v)[P]) const {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int a = col(k, 0), b = col(k, 1);
      v[k] = make_float2(p && a < cols ? param<T>(p, fp32, a) : 0.0f, p && b < cols ? param<T>(p, fp32, b) : 0.0f);
    }
  }
  __device__ __forceinline__ void shift(float2 (&v)[P], float m) const {
    if (live == 32 * N) {
#pragma unroll
      for (int k = 0; k < P; ++k) v[k] = add2(v[k], make_float2(m, m));
    } else {
#pragma unroll
      for (int k = 0; k < P; ++k)
        v[k] = add2(v[k], make_float2(col(k, 0) < cols ? m : 0.0f, col(k, 1) < cols ? m : 0.0f));
    }
  }
  // Through `room` (store_bytes), which the caller's next __syncwarp frees again.
  __device__ __forceinline__ void store(T* y, bool, void* room, const float2 (&v)[P]) const {
    if (live <= 0) return;
    const int lane = threadIdx.x & 31;
    uint8_t* dst = reinterpret_cast<uint8_t*>(y + seg);
    const int skip = (int)((uintptr_t)dst & 15u);
    uint8_t* p = reinterpret_cast<uint8_t*>(static_cast<uint4*>(room) + (threadIdx.x >> 5) * kGranules);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if constexpr (G == 2) {
        *reinterpret_cast<uint32_t*>(p + skip + (k * 32 + lane) * 4) = pack2<T>(v[k]);
      } else {
        *reinterpret_cast<T*>(p + skip + (2 * k * 32 + lane) * kSize) = from_float<T>(v[k].x);
        *reinterpret_cast<T*>(p + skip + ((2 * k + 1) * 32 + lane) * kSize) = from_float<T>(v[k].y);
      }
    }
    __syncwarp();
    const int total = skip + live * kSize;
#pragma unroll
    for (int i = 0; i < (kGranules + 31) / 32; ++i) {
      const int g = lane + 32 * i;
      if (g * 16 >= skip && g * 16 + 16 <= total)
        *reinterpret_cast<uint4*>(dst - skip + g * 16) = *reinterpret_cast<const uint4*>(p + g * 16);
    }
    // the ends: bytes before the first whole granule and after the last
    const int head = min((skip + 15) / 16 * 16, total), rest = max(total / 16 * 16, head);
    for (int b = skip + lane * kSize; b < head; b += 32 * kSize)
      *reinterpret_cast<T*>(dst - skip + b) = *reinterpret_cast<const T*>(p + b);
    for (int b = rest + lane * kSize; b < total; b += 32 * kSize)
      *reinterpret_cast<T*>(dst - skip + b) = *reinterpret_cast<const T*>(p + b);
  }
  __device__ __forceinline__ void store_sums(float* out, const float2 (&v)[P]) const {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if (col(k, 0) < cols) out[col(k, 0)] = v[k].x;
      if (col(k, 1) < cols) out[col(k, 1)] = v[k].y;
    }
  }
};

// The forward pass for rows of up to about 7 KB of FP32 (448 threads of 16
// values): a CTA keeps its columns' weight and bias in registers and walks over
// rows by the grid.  Reading weight and bias anew for every row would move four
// times the row's own bytes through L1.
template <class Row, bool FP8>
__global__ void __launch_bounds__(Row::kWide ? 448 : 256, Row::kWide ? 2 : 4)
    layer_norm_ring_kernel(const LayerNormArgs p) {
  using T = typename Row::T;
  constexpr int P = Row::P, kRing = Row::kRing;
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
  Row src;
  src.init(ring, p.x, p.ldx, row, step, p.rows, tid, cols);
  void* const room = reinterpret_cast<uint8_t*>(ring) + p.ring_bytes;
  float2 w[P], b[P];
  src.params(p.weight, p.w_fp32, p.w_wide, w);
  src.params(p.bias, p.w_fp32, p.w_wide, b);
  const bool wide = ((p.cols * (int64_t)sizeof(T)) | (int64_t)(uintptr_t)p.y) % 32 == 0;
  for (int s = 0; s < kRing - 1; ++s) {
    src.fetch(s);
    cp_async_commit();
  }
  const float rn = 1.0f / (float)cols;
  int at = 0;
  // every row group of the CTA takes as many rounds as its first one
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < rows; base += step) {
    const bool in = row < p.rows;
    __syncwarp();  // the warp has read the slot that is filled next
    src.fetch(at == 0 ? kRing - 1 : at - 1);
    cp_async_commit();
    cp_async_wait<kRing - 1>();
    __syncwarp();
    float2 v[P];
    src.read(at, v);
    if (++at == kRing) at = 0;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < P; ++k) s = add2(s, v[k]);
    const float mean = row_sum(s.x + s.y, red, warps, warp0, 0) * rn;
    float2 d2 = make_float2(0.0f, 0.0f);
    src.shift(v, -mean);
#pragma unroll
    for (int k = 0; k < P; ++k) d2 = fma2(v[k], v[k], d2);
    const float rstd = rsqrt_newton(row_sum(d2.x + d2.y, red, warps, warp0, 1) * rn + p.eps);
    if (in && tid == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < P; ++k) v[k] = fma2(mul2(v[k], rstd), w[k], b[k]);
    if constexpr (!FP8) {
      if (in) src.store(static_cast<T*>(p.y) + row * p.cols, wide, room, v);
    } else {
      constexpr int E = Row::E;  // neighbouring columns of a lane
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < P; ++k) m = abs_max2(m, v[k]);
#pragma unroll
      for (int o = 64 / E; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t e = scale_byte(m);
      const int c = src.c;
      if (in && c < cols) {
        const float inv = inverse_of_byte(e);
        uint32_t o[E / 4];
#pragma unroll
        for (int k = 0; k < E / 4; ++k) o[k] = e4m3x4(mul2(v[2 * k], inv), mul2(v[2 * k + 1], inv));
        uint8_t* q = static_cast<uint8_t*>(p.y) + row * p.cols + c;
        if constexpr (E == 16) *reinterpret_cast<uint4*>(q) = make_uint4(o[0], o[1], o[2], o[3]);
        else if constexpr (E == 8) *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
        else *reinterpret_cast<uint32_t*>(q) = o[0];
      }
      // the warp's 32 E columns are a whole scale word (E = 16), a half or a
      // byte of one; the row's last warp zeroes what its word has left
      constexpr int G = 128 / E, B = E / 4;  // lanes of a group, bytes of the warp
      const int block = (c - (int)(threadIdx.x & 31) * E) / 128;
      const uint32_t part = __reduce_or_sync(
          0xffffffffu, in && c < cols && (threadIdx.x & 31) % G == 0 ? e << (8 * ((threadIdx.x & 31) / G)) : 0u);
      if ((threadIdx.x & 31) == 0 && c < cols && row < rows) {
        uint32_t* word = p.sf + (int64_t)(block >> 2) * p.rows_pad + row;
        if constexpr (B == 4) {
          *word = part;
        } else {
          uint8_t* to = reinterpret_cast<uint8_t*>(word) + (block & 3);
          if constexpr (B == 2) *reinterpret_cast<uint16_t*>(to) = (uint16_t)part;
          else *to = (uint8_t)part;
          if (c + 32 * E >= cols)
            for (int i = (block & 3) + B; i < 4; ++i) to[i - (block & 3)] = 0;
        }
      }
    }
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

template <class Row>
__global__ void __launch_bounds__(Row::kWide ? 512 : 256, Row::kWide ? 1 : 3)
    layer_norm_backward_ring_kernel(const LayerNormArgs p) {
  using T = typename Row::T;
  constexpr int P = Row::P, kRing = Row::kRing;
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
  uint8_t* const shared = reinterpret_cast<uint8_t*>(ring);
  Row xs, ds;
  xs.init(shared, p.x, p.ldx, row, step, p.rows, tid, cols);
  ds.init(shared + p.ring_bytes, p.dy, p.lddy, row, step, p.rows, tid, cols);
  void* const room = shared + 2 * p.ring_bytes;
  float2 w[P], aw[P], ab[P];
  xs.params(p.weight, p.w_fp32, p.w_wide, w);
#pragma unroll
  for (int k = 0; k < P; ++k) aw[k] = ab[k] = make_float2(0.0f, 0.0f);
  const bool wide = ((p.cols * (int64_t)sizeof(T)) | (int64_t)(uintptr_t)p.y) % 32 == 0;
  for (int s = 0; s < kRing - 1; ++s) {
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
    const int next = at == 0 ? kRing - 1 : at - 1;
    xs.fetch(next);
    ds.fetch(next);
    cp_async_commit();
    const bool more = row + step < p.rows;
    const float mean1 = more ? __ldg(p.mean + row + step) : 0.0f, rstd1 = more ? __ldg(p.rstd + row + step) : 0.0f;
    cp_async_wait<kRing - 1>();
    __syncwarp();
    float2 xv[P], dv[P];
    xs.read(at, xv);
    ds.read(at, dv);
    if (++at == kRing) at = 0;
    if (!in) {  // the last round of a row group that has no row in it: an old row adds nothing
#pragma unroll
      for (int k = 0; k < P; ++k) xv[k] = dv[k] = make_float2(0.0f, 0.0f);
    }
    // past the row dy is 0, so whatever xh is there adds nothing
    const float2 nm = make_float2(-mean, -mean);
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      xv[k] = mul2(add2(xv[k], nm), rstd);
      aw[k] = fma2(dv[k], xv[k], aw[k]);
      ab[k] = add2(ab[k], dv[k]);
      dv[k] = mul2(dv[k], w[k]);
      s1 = add2(s1, dv[k]);
      s2 = fma2(dv[k], xv[k], s2);
    }
    const float2 sums = row_sum_pair(s1.x + s1.y, s2.x + s2.y, red, turn, warps, warp0);
    turn ^= 1;
    const float2 n1 = make_float2(-sums.x * rn, -sums.x * rn), n2 = make_float2(-sums.y * rn, -sums.y * rn);
#pragma unroll
    for (int k = 0; k < P; ++k) dv[k] = mul2(fma2(xv[k], n2, add2(dv[k], n1)), rstd);
    if (in) xs.store(static_cast<T*>(p.y) + row * p.cols, wide, room, dv);
    row += step;
    mean = mean1;
    rstd = rstd1;
  }
  cp_async_wait<0>();
  if (rpc > 1) {  // the row groups' sums, added up in their order by the first group
    __syncthreads();
    float2* mine = reinterpret_cast<float2*>(ring) + (size_t)(threadIdx.x / tpr) * 2 * P * tpr + tid;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      mine[k * tpr] = aw[k];
      mine[(P + k) * tpr] = ab[k];
    }
    __syncthreads();
    if ((int)threadIdx.x >= tpr) return;
    for (int g = 1; g < rpc; ++g) {
      mine += 2 * P * tpr;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        aw[k] = add2(aw[k], mine[k * tpr]);
        ab[k] = add2(ab[k], mine[(P + k) * tpr]);
      }
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  xs.store_sums(part, aw);
  xs.store_sums(part + (int64_t)gridDim.x * p.cols, ab);
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

// Threads of a row and of a CTA (at least 128, whole rows) for n values a thread.
struct NormShape {
  int64_t tpr, threads, rpc;
  NormShape(int64_t cols, int n) {
    tpr = ((cols + n - 1) / n + 31) / 32 * 32;
    threads = tpr >= 128 ? tpr : 128 / tpr * tpr;
    rpc = threads / tpr;
  }
};

// Two neighbouring elements can be read at once where rows start on 4 bytes.
template <class T>
bool pairs_aligned(const LayerNormArgs& p, bool backward) {
  if (sizeof(T) == 4) return false;
  return ((p.ldx | p.cols | (backward ? p.lddy : 0)) & 1) == 0 &&
         (((uintptr_t)p.x | (uintptr_t)p.y | (backward ? (uintptr_t)p.dy : 0)) & 3) == 0;
}

template <class T, bool FP8>
cudaError_t forward(const LayerNormArgs& a, bool vec, int sms, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t rows = FP8 ? p.rows_pad : p.rows;
  // Rows of up to 448 threads of 16 values (8 of FP32 by pieces) take the ring
  // kernel, as many CTAs an SM as its registers and shared memory hold.
  // Longer ones are read into registers of one CTA a row, or in passes.
  auto ring = [&](auto kern, auto row, int n) {
    using Row = decltype(row);
    const NormShape s(p.cols, n);
    p.tpr = (int)s.tpr;
    p.ring_bytes = (int64_t)Row::bytes(s.threads);
    const size_t smem = Row::bytes(s.threads) + Row::store_bytes(s.threads);
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>((int64_t)(220 * 1024) / (int64_t)(smem + 2048),
                                                                  (Row::kWide ? 896 : 1024) / s.threads));
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_op(kern, dim3((unsigned)std::min<int64_t>((rows + s.rpc - 1) / s.rpc, per_sm * sms)),
                     (unsigned)s.threads, smem, pdl, st, p);
  };
  auto whole = [&](auto kern, int n) {
    const NormShape s(p.cols, n);
    p.tpr = (int)s.tpr;
    return launch_op(kern, dim3((unsigned)((rows + s.rpc - 1) / s.rpc)), (unsigned)s.threads, 0, pdl, st, p);
  };
#define DG_NORM_RING(ROW, n) ring(layer_norm_ring_kernel<ROW, FP8>, ROW(), n)
  if (vec) {
    using One = AlignedRow<T, 1>;
    using Two = AlignedRow<T, 2>;
    if (p.cols <= 256 * V) return DG_NORM_RING(One, V);
    if (p.cols <= 448 * 2 * V) return DG_NORM_RING(Two, 2 * V);
    if (p.cols <= 512 * 4 * V) return whole(layer_norm_kernel<T, V, 4, FP8>, 4 * V);
    if (p.cols <= 512 * 8 * V) return whole(layer_norm_kernel<T, V, 8, FP8>, 8 * V);
  }
  if constexpr (FP8) return cudaErrorInvalidValue;
  else {
    if (!vec && p.cols <= 448 * 16) {
      using Few1 = RaggedRow<T, 8, 1>;
      using Many1 = RaggedRow<T, 16, 1>;
      if constexpr (sizeof(T) == 2) {
        using Few2 = RaggedRow<T, 8, 2>;
        using Many2 = RaggedRow<T, 16, 2>;
        if (pairs_aligned<T>(p, false)) return p.cols <= 256 * 8 ? DG_NORM_RING(Few2, 8) : DG_NORM_RING(Many2, 16);
      }
      return p.cols <= 256 * 8 ? DG_NORM_RING(Few1, 8) : DG_NORM_RING(Many1, 16);
    }
    if (!vec && p.cols <= 32 * 512) return whole(layer_norm_kernel<T, 1, 16, false>, 32);
    return launch_op(layer_norm_long_kernel<T>, dim3((unsigned)p.rows), 1024, 0, pdl, st, p);
  }
#undef DG_NORM_RING
}

template <class T>
cudaError_t backward(const LayerNormArgs& a, bool vec, int parts, int* used, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  auto ring = [&](auto kern, auto row, int n) {
    using Row = decltype(row);
    const NormShape s(p.cols, n);
    p.tpr = (int)s.tpr;
    p.ring_bytes = (int64_t)Row::bytes(s.threads);
    const size_t sums = s.rpc > 1 ? (size_t)s.threads * 2 * Row::P * sizeof(float2) : 0;
    const size_t smem = std::max<size_t>(2 * Row::bytes(s.threads) + Row::store_bytes(s.threads), sums);
    int64_t per_sm = std::min<int64_t>(kNormParts, (Row::kWide ? 512 : 768) / s.threads);
    per_sm = std::max<int64_t>(1, std::min<int64_t>(per_sm, (int64_t)(220 * 1024) / (int64_t)(smem + 2048)));
    *used = (int)std::min<int64_t>((p.rows + s.rpc - 1) / s.rpc, per_sm * (parts / kNormParts));
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_op(kern, dim3((unsigned)*used), (unsigned)s.threads, smem, pdl, st, p);
  };
#define DG_NORM_RING(ROW, n) ring(layer_norm_backward_ring_kernel<ROW>, ROW(), n)
  if (vec) {
    using One = AlignedRow<T, 1>;
    using Two = AlignedRow<T, 2>;
    if (p.cols <= 256 * V) return DG_NORM_RING(One, V);
    if (p.cols <= 512 * 2 * V) return DG_NORM_RING(Two, 2 * V);
  } else if (p.cols <= 512 * 16) {
    using Few1 = RaggedRow<T, 8, 1>;
    using Many1 = RaggedRow<T, 16, 1>;
    if constexpr (sizeof(T) == 2) {
      using Few2 = RaggedRow<T, 8, 2>;
      using Many2 = RaggedRow<T, 16, 2>;
      if (pairs_aligned<T>(p, true)) return p.cols <= 256 * 8 ? DG_NORM_RING(Few2, 8) : DG_NORM_RING(Many2, 16);
    }
    return p.cols <= 256 * 8 ? DG_NORM_RING(Few1, 8) : DG_NORM_RING(Many1, 16);
  }
#undef DG_NORM_RING
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
