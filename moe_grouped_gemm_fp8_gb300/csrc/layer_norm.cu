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
// row's sums and its results.  All sums are FP32; the variance is summed around
// the mean or a value near it, so a large mean costs no digits.
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

// Weight or bias element, FP32 or x's type (a branch every thread of the
// launch takes the same way).
template <class T>
__device__ __forceinline__ float param(const void* p, bool fp32, int64_t i) {
  return fp32 ? __ldg(static_cast<const float*>(p) + i) : to_float(__ldg(static_cast<const T*>(p) + i));
}

// VEC neighbouring elements; `wide`: the base is 16-byte aligned.
template <class T, int VEC>
__device__ __forceinline__ void param_vec(const void* p, bool fp32, bool wide, int64_t i, float (&f)[VEC]) {
  if (!wide) {
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

// The one nearer to zero; a where b is NaN.
__device__ __forceinline__ float nearer(float a, float b) { return fabsf(b) < fabsf(a) ? b : a; }

// Sum over the CTA; every thread gets it.  Two calls use different slots.
__device__ __forceinline__ float row_sum(float v, float* red, int slot) {
  v = warp_sum(v);
  red += slot * 32;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < (int)blockDim.x / 32 ? red[lane] : 0.0f);
}

// 1 / sqrt(v): the hardware's estimate and one Newton step (which would make a
// NaN of the infinity that a row without spread has for eps = 0).
__device__ __forceinline__ float rsqrt_newton(float v) {
  const float r = rsqrtf(v);
  return v > 0.0f ? r * (1.5f - (0.5f * v * r) * r) : r;
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
  int64_t ring_bytes;  // backward: of one ring of rows
  int64_t par_at;      // where weight and bias start in shared memory
  int tpr;             // threads a row
  float eps;
  bool w_fp32;       // weight and bias are FP32, else x's type
  bool w_wide;       // weight and bias are 16-byte aligned
};

// Rows of 16-byte pieces too long for the ring kernels below: a CTA a row, all of
// it in registers (kWideVecs pieces a thread).  Its loads, two sums and stores
// follow one another: 6144 x 20480 BF16 167 us (3.0 TB/s), 4096 x 16384
// FP32 84 (6.4); to 8 bits, where 16-bit rows spill, 304 (1.2) and 138 (2.4).
constexpr int kWideThreads = 512, kWideVecs = 8;

template <class T, bool FP8>
__global__ void __launch_bounds__(kWideThreads) layer_norm_wide_kernel(const LayerNormArgs p) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2, NV = kWideVecs;
  __shared__ float red[64];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int cols = (int)p.cols, first = (int)threadIdx.x * V;
  const bool in = row < p.rows;  // else one of the scales' padding
  const T* x = static_cast<const T*>(p.x) + (in ? row : 0) * p.ldx;
  float2 v[NV][P];
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * kWideThreads * V;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (in && c < cols) raw = ld_stream_u4(x + c);
    unpack16<T>(raw, v[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) s = add2(s, v[i][k]);
  const float rn = 1.0f / (float)cols;
  const float mean = row_sum(s.x + s.y, red, 0) * rn;
  float2 d2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (first + i * kWideThreads * V < cols) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        v[i][k] = add2(v[i][k], make_float2(-mean, -mean));
        d2 = fma2(v[i][k], v[i][k], d2);
      }
    }
  }
  const float rstd = rsqrt_newton(row_sum(d2.x + d2.y, red, 1) * rn + p.eps);
  if (in && threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * kWideThreads * V;
    if (c < cols) {
      float w[V], b[V];
      param_vec<T, V>(p.weight, p.w_fp32, p.w_wide, c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) b[k] = 0.0f;
      if (p.bias) param_vec<T, V>(p.bias, p.w_fp32, p.w_wide, c, b);
#pragma unroll
      for (int k = 0; k < P; ++k)
        v[i][k] = fma2(mul2(v[i][k], rstd), make_float2(w[2 * k], w[2 * k + 1]), make_float2(b[2 * k], b[2 * k + 1]));
    }
    if constexpr (!FP8) {
      if (c < cols) *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + row * p.cols + c) = pack16<T>(v[i]);
    } else {
      // a group of 128 columns lies in 128 / V neighbouring threads, whole or past the row
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < P; ++k) m = abs_max2(m, v[i][k]);
#pragma unroll
      for (int o = 64 / V; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (c >= cols) continue;
      const uint32_t e = scale_byte(m);
      if (in) {
        const float inv = inverse_of_byte(e);
        uint32_t q[V / 4];
#pragma unroll
        for (int k = 0; k < V / 4; ++k) q[k] = e4m3x4(mul2(v[i][2 * k], inv), mul2(v[i][2 * k + 1], inv));
        uint8_t* dst = static_cast<uint8_t*>(p.y) + row * p.cols + c;
        if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
        else *reinterpret_cast<uint32_t*>(dst) = q[0];
      }
      if (c % 128 == 0) {
        const int kb = c / 128;
        store_scale_byte(p.sf + (int64_t)(kb >> 2) * p.rows_pad + row, kb, c + 128 == cols, in ? e : 0u);
      }
    }
  }
}

// ---------------------------------------------------------------- rows in a ring
// Rows on their way into shared memory, in a ring of slots, while others are
// worked on (two slots are enough for lanes of 32 elements: more rows in flight
// make HBM no faster).  Every warp copies and reads only its own columns, so __syncwarp
// is all that guards them.  Two forms with one interface: a thread's P pairs of
// values of a row (zeros past it), the same of weight or bias, and storing them.

// Rows of whole, 16-byte aligned pieces.  A warp's share is 32 NV pieces, copied
// by its lanes side by side and read back as each lane's own NV neighbouring
// pieces (stored crosswise so that 8 lanes meet no bank twice): they hold whole
// groups' maxima in few lanes, and the E4M3 codes leave 32 bytes a lane.
// Pieces past the row are never copied and stay zero; rows past the last leave
// what was there.
template <class T_, int NV_>
struct AlignedRow {
  using T = T_;
  static constexpr int NV = NV_;
  static constexpr int V = 16 / (int)sizeof(T);
  static constexpr int E = NV * V;  // neighbouring columns of a lane
  static constexpr int P = E / 2;
  static constexpr int kRing = E == 32 ? 2 : 4, kBackRing = E == 16 && sizeof(T) == 4 ? 3 : 4;
  static int64_t bytes(int64_t threads) { return (int64_t)NV * threads * 16; }  // of a slot
  uint32_t put, get;  // shared address of the lane's first piece to copy / to read in slot 0
  int stage;          // bytes between slots
  const T* src;       // this lane's first piece of the next row to copy
  int64_t step;       // elements between the rows this thread meets
  bool full;          // the warp's columns all lie in the row
  int copy, on;       // pieces that do: of those the lane copies, of its own
  int c;              // the lane's first column

  __device__ __forceinline__ static int place(int p) { return p ^ ((p >> 3) & (NV - 1)); }
  __device__ __forceinline__ void init(void* ring, int slots, const void* x, int64_t ld, int64_t first, int64_t every,
                                       int tid, int cols) {
    const int lane = threadIdx.x & 31;
    const uint32_t mine = smem_u32(ring) + (threadIdx.x >> 5) * 32 * NV * 16;
    put = mine + place(lane) * 16;
    get = mine + place(lane * NV) * 16;
    stage = blockDim.x * NV * 16;
    const int c0 = (tid >> 5) * 32 * E;
    src = static_cast<const T*>(x) + first * ld + c0 + lane * V;
    step = every * ld;
    c = tid * E;
    full = c0 + 32 * E <= cols;
    on = min(max((cols - c + V - 1) / V, 0), NV);
    copy = min(max(((cols - c0 + V - 1) / V - lane + 31) / 32, 0), NV);
    for (int j = copy; j < NV; ++j)
      for (int s = 0; s < slots; ++s)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(place_of(j) + s * stage), "r"(0) : "memory");
  }
  // Where piece lane + 32 j goes: with eight pieces a lane every second one is crossed once more.
  __device__ __forceinline__ uint32_t place_of(int j) const { return (NV == 8 && (j & 1) ? put ^ 64 : put) + j * 512; }
  // The next row into the slot at `off`; nothing where there is none.
  __device__ __forceinline__ void fetch(int off, bool there) {
    if (there) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (full || j < copy) cp_async16(place_of(j) + off, src + 32 * j * V);
    }
    src += step;
  }
  __device__ __forceinline__ void read(int off, float2 (&v)[P]) {
    const uint32_t from = get + off;  // slots start on multiples of the lane's 16 NV bytes
#pragma unroll
    for (int j = 0; j < NV; ++j) unpack16<T>(ld_shared_u4(from ^ (j * 16)), &v[j * V / 2]);
  }
  // Pairs of a lane whose means can stand for the warp's; one over how many of
  // their first and of their second values lie inside the row (past it they are 0).
  static constexpr int kPilot = P < 8 ? P : 8;
  __device__ __forceinline__ float2 pilot_weights() const {
    const float r = 1.0f / (float)max(min(on * V / 2, kPilot), 1);
    return make_float2(r, r);
  }
  __device__ __forceinline__ void params(const void* p, bool fp32, bool wide, float2 (&v)[P]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float e[V];
#pragma unroll
      for (int k = 0; k < V; ++k) e[k] = 0.0f;
      if (p && j < on) param_vec<T, V>(p, fp32, wide, c + j * V, e);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) v[j * V / 2 + k] = make_float2(e[2 * k], e[2 * k + 1]);
    }
  }
  // Adds m to the columns inside the row.
  __device__ __forceinline__ void shift(float2 (&v)[P], float m) const {
    if (full) {
#pragma unroll
      for (int k = 0; k < P; ++k) v[k] = add2(v[k], make_float2(m, m));
      return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float a = j < on ? m : 0.0f;
#pragma unroll
      for (int k = 0; k < V / 2; ++k) v[j * V / 2 + k] = add2(v[j * V / 2 + k], make_float2(a, a));
    }
  }
  // Into the row at y; `wide`: rows start on 32 bytes, so two pieces are one access.
  __device__ __forceinline__ void store(T* y, bool wide, int, const float2 (&v)[P]) const {
    y += c;
    if (NV > 1 && wide && on == NV) {
#pragma unroll
      for (int j = 0; j + 1 < NV; j += 2)
        st_global_32(y + j * V, pack16<T>(&v[j * V / 2]), pack16<T>(&v[(j + 1) % NV * V / 2]));
      return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j < on) *reinterpret_cast<uint4*>(y + j * V) = pack16<T>(&v[j * V / 2]);
  }
  // A column sum per pair element.
  __device__ __forceinline__ void store_sums(float* out, const float2 (&v)[P]) const {
#pragma unroll
    for (int k = 0; k < P; ++k)
      if (2 * k / V < on) {
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
  static constexpr int kRing = N == 32 ? 2 : 4, kBackRing = N == 16 && sizeof(T) == 4 ? 3 : 4;
  static constexpr int kSize = (int)sizeof(T);
  static constexpr int kGranules = 32 * N * kSize / 16 + 1;  // a warp's
  static int64_t bytes(int64_t threads) { return (int64_t)kGranules * (threads / 32) * 16; }
  uint4* mine;
  int stage;
  const uint8_t* src;           // this warp's first column in the next row to copy
  const uint8_t* base;          // the tensor's first byte
  int64_t step;
  uint32_t at, at_step;         // where in its granule the next row to read starts
  int seg, live, cols;          // this warp's first column, its columns inside the row

  __device__ __forceinline__ int col(int k, int e) const {  // element e of pair k
    const int lane = threadIdx.x & 31;
    return G == 2 ? seg + (k * 32 + lane) * 2 + e : seg + (2 * k + e) * 32 + lane;
  }
  __device__ __forceinline__ void init(void* ring, int, const void* x, int64_t ld, int64_t first, int64_t every, int tid,
                                       int n) {
    mine = static_cast<uint4*>(ring) + (threadIdx.x >> 5) * kGranules;
    stage = (int)(blockDim.x >> 5) * kGranules * 16;
    seg = (tid >> 5) * 32 * N;
    cols = n;
    live = min(32 * N, n - seg);  // < 0: none
    base = static_cast<const uint8_t*>(x);
    src = base + (first * ld + seg) * kSize;
    step = every * ld * kSize;
    at = (uint32_t)(uintptr_t)src;
    at_step = (uint32_t)step;
  }
  __device__ __forceinline__ void fetch(int off, bool there) {
    if (there && live > 0) {
      const int lane = threadIdx.x & 31;
      const int skip = (int)((uintptr_t)src & 15u);
      const uint8_t* from = src - skip;
      const int total = skip + live * kSize;
#pragma unroll
      for (int i = 0; i < (kGranules + 31) / 32; ++i) {
        const int g = lane + 32 * i;
        if (g * 16 < total) {
          uint4* to = mine + off / 16 + g;
          if (from + g * 16 >= base) cp_async16_part(to, from + g * 16, min(16, total - g * 16));
          else  // the tensor's first granule, where it starts inside one
            for (int b = skip; b < min(16, total); b += kSize)
              *reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(to) + b) = *reinterpret_cast<const T*>(from + b);
        }
      }
    }
    src += step;
  }
  static constexpr int kPilot = 2;  // (eight cost 16384 x 7167 BF16 5%)
  __device__ __forceinline__ float2 pilot_weights() const {
    int a = 0, b = 0;
#pragma unroll
    for (int k = 0; k < kPilot; ++k) {
      a += col(k, 0) < cols;
      b += col(k, 1) < cols;
    }
    return make_float2(1.0f / (float)max(a, 1), 1.0f / (float)b);  // none: 0 inf, which is never nearer
  }
  __device__ __forceinline__ void read(int off, float2 (&v)[P]) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(mine) + off + (at & 15u);
    at += at_step;
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
  // By way of the slot at `off`, which the warp has read and fills again only
  // after the caller's next __syncwarp.
  __device__ __forceinline__ void store(T* y, bool, int off, const float2 (&v)[P]) const {
    __syncwarp();
    if (live <= 0) return;
    const int lane = threadIdx.x & 31;
    uint8_t* dst = reinterpret_cast<uint8_t*>(y + seg);
    const int skip = (int)((uintptr_t)dst & 15u);
    uint8_t* p = reinterpret_cast<uint8_t*>(mine) + off;
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

// The forward pass: a CTA works on as many rows at once as its threads and
// shared memory hold, every row by its own threads with a barrier of their own,
// and walks on by the grid.  Both sums of a row are exchanged at once.
//
// Weight and bias wait in shared memory, as pairs of float4 a lane: read anew
// for every row from L1 they would move four times the row's own bytes, and in
// registers they leave room for 14 warps a SM only (16384 x 7168 BF16 to 8 bits
// 77 us instead of 71).  A warp's work on a row is about as much outside its
// elements as eight elements a lane are, so lanes take many: 16384 x 7168 BF16 to
// 8 bits 92 us with 16 a lane, 71 with 32 (5.0 TB/s; issue slots 60% busy, the
// latency of the sums between), to BF16 73 us (6.4 TB/s); 114688 x 1024 to 8 bits
// 57 us (6.1 TB/s).
constexpr int kNormThreads = 768;
constexpr int64_t kNormMaxSmem = 220 * 1024;  // dynamic shared memory of a CTA, at most (forward and backward)

template <class Row, bool FP8>
__global__ void __launch_bounds__(kNormThreads, 1) layer_norm_ring_kernel(const LayerNormArgs p) {
  using T = typename Row::T;
  constexpr int P = Row::P, kRing = Row::kRing;
  extern __shared__ __align__(128) uint4 ring[];  // rows, then weight and bias
  __shared__ float2 red[2][kNormThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.tpr, rpc = blockDim.x / tpr, warps = tpr / 32;
  const int group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr, lane = threadIdx.x & 31;
  const int cols = (int)p.cols;
  const int step = (int)gridDim.x * rpc;
  const int64_t first = (int64_t)blockIdx.x * rpc + group;
  auto count = [&](int64_t rows) { return first < rows ? (int)((rows - first - 1) / step) + 1 : 0; };
  const int live = count(p.rows);                         // rows of this group,
  const int rounds = FP8 ? count(p.rows_pad) : live;      // with those of the scales' padding
  Row src;
  src.init(ring, kRing, p.x, p.ldx, first, step, tid, cols);
  float4* const par = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(ring) + p.par_at) + (tid >> 5) * (P * 32) + lane;
  if (group == 0) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      float2 v[P];
      src.params(i ? p.bias : p.weight, p.w_fp32, p.w_wide, v);
#pragma unroll
      for (int k = 0; k < P; k += 2) par[(k + i) * 32] = make_float4(v[k].x, v[k].y, v[k + 1].x, v[k + 1].y);
    }
  }
  const bool wide = ((p.cols * (FP8 ? 1 : (int64_t)sizeof(T))) | (int64_t)(uintptr_t)p.y) % 32 == 0;
  const int last = (kRing - 1) * src.stage;
  for (int s = 0; s < kRing - 1; ++s) {
    src.fetch(s * src.stage, s < live);
    cp_async_commit();
  }
  __syncthreads();
  const float rn = 1.0f / (float)cols;
  const float2 r_pilot = src.pilot_weights();
  const float r_warp = 1.0f / (float)max(min(cols - (tid - lane) * 2 * P, 64 * P), 1);
  const int peer = lane & (warps > 8 ? 15 : 7);  // the warp whose part of the row's sums the lane takes
  const float n_peer = (float)max(min(cols - peer * 64 * P, 64 * P), 0);
  int64_t row = first;
  int at = 0;
  for (int round = 0; round < rounds; ++round) {
    const bool in = round < live;
    __syncwarp();  // the warp has read the slot that is filled next
    src.fetch(at == 0 ? last : at - src.stage, round + kRing - 1 < live);
    cp_async_commit();
    cp_async_wait<kRing - 1>();
    __syncwarp();
    float2 v[P];
    src.read(at, v);
    const int slot = at;
    at = at == last ? 0 : at + src.stage;
    // Both sums at once, around a value near the warp's mean: the mean of a few
    // values of its first lane, or of as many others where those are nearer to
    // zero, so that one loud channel does not move it (every value is rounded at
    // the size of its distance from it).
    float2 s = v[0];
#pragma unroll
    for (int k = 1; k < Row::kPilot; ++k) s = add2(s, v[k]);
    s = mul2(s, r_pilot);
    const float pilot = __shfl_sync(0xffffffffu, nearer(s.x, s.y), 0);
    src.shift(v, -pilot);
    s = v[0];
    float2 d2 = mul2(v[0], v[0]);
#pragma unroll
    for (int k = 1; k < P; ++k) {
      s = add2(s, v[k]);
      d2 = fma2(v[k], v[k], d2);
    }
    float s1 = s.x + s.y, s2 = d2.x + d2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    // The warp's mean and sum of squares around it; the row's from the warps',
    // around the reader's own pilot (so two warps' may differ in the last bit).
    float mean = pilot + s1 * r_warp;
    s2 -= s1 * s1 * r_warp;
    if (warps > 1) {
      float2* r = red[round & 1] + group * warps;  // alternating: one barrier a row is enough
      if (lane == 0) r[tid >> 5] = make_float2(mean, s2);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
      const float2 of = r[min(peer, warps - 1)];
      const float d = of.x - pilot;
      s1 = n_peer * d;
      s2 = peer < warps ? s1 * d + of.y : 0.0f;
      if (warps > 8) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, 8);
        s2 += __shfl_xor_sync(0xffffffffu, s2, 8);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
      mean = pilot + s1 * rn;
      s2 -= s1 * s1 * rn;
    }
    const float rstd = rsqrt_newton((s2 < 0.0f ? 0.0f : s2) * rn + p.eps);
    if (in && tid == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    const float shift = (pilot - mean) * rstd;
#pragma unroll
    for (int k = 0; k < P; k += 2) {
      const float4 w = par[k * 32], b = par[(k + 1) * 32];
      v[k] = fma2(fma2(v[k], make_float2(rstd, rstd), make_float2(shift, shift)), make_float2(w.x, w.y),
                  make_float2(b.x, b.y));
      v[k + 1] = fma2(fma2(v[k + 1], make_float2(rstd, rstd), make_float2(shift, shift)), make_float2(w.z, w.w),
                      make_float2(b.z, b.w));
    }
    if constexpr (!FP8) {
      if (in) src.store(static_cast<T*>(p.y) + row * cols, wide, slot, v);
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
        uint8_t* q = static_cast<uint8_t*>(p.y) + row * cols + c;
        if constexpr (E == 32) {
          const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
          if (wide) {
            st_global_32(q, lo, hi);
          } else {
            *reinterpret_cast<uint4*>(q) = lo;
            *reinterpret_cast<uint4*>(q + 16) = hi;
          }
        } else if constexpr (E == 16) *reinterpret_cast<uint4*>(q) = make_uint4(o[0], o[1], o[2], o[3]);
        else if constexpr (E == 8) *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
        else *reinterpret_cast<uint32_t*>(q) = o[0];
      }
      // the warp's 32 E columns are two scale words, one (E = 16), a half or a
      // byte of one; the row's last warp zeroes what its word has left
      constexpr int G = 128 / E, B = E / 4;  // lanes of a group, bytes of the warp
      const uint32_t mine = in && c < cols && lane % G == 0 ? e << (8 * (lane / G % 4)) : 0u;
      const uint32_t part = __reduce_or_sync(0xffffffffu, B == 8 && lane >= 16 ? 0u : mine);
      uint32_t upper = 0;
      if constexpr (B == 8) upper = __reduce_or_sync(0xffffffffu, lane >= 16 ? mine : 0u);
      if (lane == 0 && c < cols) {
        uint32_t* sf = p.sf + (int64_t)(c / 512) * p.rows_pad + row;
        if constexpr (B >= 4) {
          *sf = part;
          if (B == 8 && c + 16 * E < cols) sf[p.rows_pad] = upper;
        } else {
          uint8_t* word = reinterpret_cast<uint8_t*>(sf);
          const int byte = c / 128 & 3;
          if constexpr (B == 2) *reinterpret_cast<uint16_t*>(word + byte) = (uint16_t)part;
          else word[byte] = (uint8_t)part;
          if (c + 32 * E >= cols)
            for (int i = byte + B; i < 4; ++i) word[i] = 0;
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
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) s += to_float(__ldg(x + c));
  const float mean = row_sum(s, red, 0) / n;
  float d2 = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float d = to_float(__ldg(x + c)) - mean;
    d2 += d * d;
  }
  const float rstd = rsqrt_newton(row_sum(d2, red, 1) / n + p.eps);
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

// Backward: as many rows at once as fit, as in the forward pass; every thread
// keeps the sums dw and db of its own columns in registers (E of 16: 14 to 16
// warps an SM; with 8 and 28 warps 197 us at 16384 x 7168 where this takes 133),
// and at the end the CTA adds its row groups' sums up in order and writes them to
// `part`.  BF16 with its join: 16384 x 7168 133 us (5.3 TB/s), where one row at a
// time leaves the sums' latency open, 28672 x 4096 118 us, 114688 x 1024 114 us
// (6.2 TB/s).  Reading the row once more from shared memory a round later, to
// wait for no sums, cost 25% more instructions: 140, 121 and 116 us.
constexpr int kNormBackThreads = 512;

template <class Row>
__global__ void __launch_bounds__(kNormBackThreads, 1) layer_norm_backward_ring_kernel(const LayerNormArgs p) {
  using T = typename Row::T;
  constexpr int P = Row::P, kRing = Row::kBackRing;
  extern __shared__ __align__(128) uint4 ring[];  // x's rows, dy's, weight; at the end, the row groups' sums
  __shared__ float red[2][kNormBackThreads / 16];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.tpr, rpc = blockDim.x / tpr, warps = tpr / 32;
  const int group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr, lane = threadIdx.x & 31;
  const int cols = (int)p.cols;
  const int step = (int)gridDim.x * rpc;
  int64_t row = (int64_t)blockIdx.x * rpc + group;
  const int live = row < p.rows ? (int)((p.rows - row - 1) / step) + 1 : 0;  // rows of this group
  uint8_t* const shared = reinterpret_cast<uint8_t*>(ring);
  Row xs, ds;
  xs.init(shared, kRing, p.x, p.ldx, row, step, tid, cols);
  ds.init(shared + p.ring_bytes, kRing, p.dy, p.lddy, row, step, tid, cols);
  float4* const par = reinterpret_cast<float4*>(shared + p.par_at) + (tid >> 5) * (P * 16) + lane;
  float2 aw[P], ab[P];
  if (group == 0) {
    xs.params(p.weight, p.w_fp32, p.w_wide, aw);
#pragma unroll
    for (int k = 0; k < P; k += 2) par[k * 16] = make_float4(aw[k].x, aw[k].y, aw[k + 1].x, aw[k + 1].y);
  }
#pragma unroll
  for (int k = 0; k < P; ++k) aw[k] = ab[k] = make_float2(0.0f, 0.0f);
  const bool wide = ((p.cols * (int64_t)sizeof(T)) | (int64_t)(uintptr_t)p.y) % 32 == 0;
  const int stage = xs.stage;
  const int last = (kRing - 1) * stage;
  for (int s = 0; s < kRing - 1; ++s) {
    xs.fetch(s * stage, s < live);
    ds.fetch(s * stage, s < live);
    cp_async_commit();
  }
  __syncthreads();
  const float rn = 1.0f / (float)cols;
  int at = 0;
  // a row's mean and rstd are loaded a round ahead
  float mean = live > 0 ? __ldg(p.mean + row) : 0.0f, rstd = live > 0 ? __ldg(p.rstd + row) : 0.0f;
  for (int round = 0; round < live; ++round) {
    __syncwarp();  // the warp has read the slot that is filled next
    const int next = at == 0 ? last : at - stage;
    xs.fetch(next, round + kRing - 1 < live);
    ds.fetch(next, round + kRing - 1 < live);
    cp_async_commit();
    const bool more = round + 1 < live;
    const float mean1 = more ? __ldg(p.mean + row + step) : 0.0f, rstd1 = more ? __ldg(p.rstd + row + step) : 0.0f;
    cp_async_wait<kRing - 1>();
    __syncwarp();
    float2 xv[P], dv[P];
    xs.read(at, xv);
    ds.read(at, dv);
    // past the row dy is 0, so whatever xh is there adds nothing
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
    for (int k = 0; k < P; k += 2) {
      const float4 w = par[k * 16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        xv[k + i] = mul2(add2(xv[k + i], make_float2(-mean, -mean)), rstd);
        aw[k + i] = fma2(dv[k + i], xv[k + i], aw[k + i]);
        ab[k + i] = add2(ab[k + i], dv[k + i]);
        dv[k + i] = mul2(dv[k + i], i ? make_float2(w.z, w.w) : make_float2(w.x, w.y));
        s1 = add2(s1, dv[k + i]);
        s2 = fma2(dv[k + i], xv[k + i], s2);
      }
    }
    // lanes 0-15 sum(t), lanes 16-31 sum(t xh), the warps' in their order
    float t = warp_sum2(s1.x + s1.y, s2.x + s2.y);
    if (warps > 1) {
      float* const r = red[round & 1] + group * warps * 2;  // alternating: one barrier a row is enough
      if (lane % 16 == 0) r[(tid >> 5) * 2 + lane / 16] = t;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
      t = lane % 16 < warps ? r[lane % 16 * 2 + lane / 16] : 0.0f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    const float c1 = -__shfl_sync(0xffffffffu, t, 0) * rn * rstd;
    const float c2 = -__shfl_sync(0xffffffffu, t, 16) * rn * rstd;
#pragma unroll
    for (int k = 0; k < P; ++k)
      dv[k] = fma2(dv[k], make_float2(rstd, rstd), fma2(xv[k], make_float2(c2, c2), make_float2(c1, c1)));
    xs.store(static_cast<T*>(p.y) + row * cols, wide, at, dv);
    at = at == last ? 0 : at + stage;
    row += step;
    mean = mean1;
    rstd = rstd1;
  }
  cp_async_wait<0>();
  if (rpc > 1) {  // the row groups' sums, added up in their order by the first group
    __syncthreads();
    float2* mine = reinterpret_cast<float2*>(ring) + (size_t)group * 2 * P * tpr + tid;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      mine[k * tpr] = aw[k];
      mine[(P + k) * tpr] = ab[k];
    }
    __syncthreads();
    if (group > 0) return;
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
  const float c1 = row_sum(s1, red, 0) * rn;
  const float c2 = row_sum(s2, red, 1) * rn;
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
// columns of one of the two, its warps every kJoinWarps-th part, eight loads in
// flight a lane.  At 16384 x 7168 it adds about 4 us to the kernel before it.
constexpr int kJoinWarps = 16;

__global__ void __launch_bounds__(32 * kJoinWarps) layer_norm_join_kernel(const float* __restrict__ part,
                                                                          float* __restrict__ dw,
                                                                          float* __restrict__ db, int parts,
                                                                          int64_t cols) {
  __shared__ float sum[kJoinWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const float* src = part + (int64_t)blockIdx.y * parts * cols;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int i = warp; i < parts; i += kJoinWarps) s += src[(int64_t)i * cols + c];
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp > 0 || c >= cols) return;
#pragma unroll
  for (int i = 1; i < kJoinWarps; ++i) s += sum[i][lane];
  (blockIdx.y ? db : dw)[c] = s;
}

// Two neighbouring elements can be read at once where rows start on 4 bytes.
template <class T>
bool pairs_aligned(const LayerNormArgs& p, bool backward) {
  if (sizeof(T) == 4) return false;
  return ((p.ldx | p.cols | (backward ? p.lddy : 0)) & 1) == 0 &&
         (((uintptr_t)p.x | (uintptr_t)p.y | (backward ? (uintptr_t)p.dy : 0)) & 3) == 0;
}

// Values a thread of the ring kernels takes: a row costs its warps about
// as many instructions as E + 8 values a warp do.
int norm_values(int64_t cols) {
  int best = 32;
  for (int e : {16, 8})
    if ((cols + 32 * e - 1) / (32 * e) * (e + 8) < (cols + 32 * best - 1) / (32 * best) * (best + 8)) best = e;
  return best;
}

template <class T, bool FP8>
cudaError_t forward(const LayerNormArgs& a, bool vec, int sms, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t rows = FP8 ? p.rows_pad : p.rows;
  // As many rows a CTA as its threads and shared memory hold, but no more than
  // give every SM a CTA.  0: not even one fits.
  auto groups = [&](auto row, int n) {
    using Row = decltype(row);
    const int64_t tpr = (p.cols + 32 * n - 1) / (32 * n) * 32;
    const int64_t par = tpr * Row::P * 16, each = Row::kRing * Row::bytes(tpr);
    if (tpr > 512 || par + each > kNormMaxSmem) return (int64_t)0;
    return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(kNormThreads / tpr, (kNormMaxSmem - par) / each),
                                                  (rows + sms - 1) / sms));
  };
  auto ring = [&](auto kern, auto row, int n) {
    using Row = decltype(row);
    const int64_t rpc = groups(row, n);
    p.tpr = (int)((p.cols + 32 * n - 1) / (32 * n) * 32);
    const int64_t threads = rpc * p.tpr;
    p.par_at = Row::kRing * Row::bytes(threads);
    const size_t smem = (size_t)(p.par_at + (int64_t)p.tpr * Row::P * 16);
    cudaError_t e = set_smem(kern, smem, kNormMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_op(kern, dim3((unsigned)std::min<int64_t>((rows + rpc - 1) / rpc, sms)), (unsigned)threads, smem, pdl,
                     st, p);
  };
  int best = norm_values(p.cols);
  // While there are not 12 warps an SM, more threads a row (1 x 7168 to 8 bits 4.1
  // us instead of 4.9, 600 x 2048 4.0 and 4.5; asked for 24 warps, the latter 4.9).
  while (best > 8 && best * 256 >= p.cols && (p.cols + 32 * best - 1) / (32 * best) * rows < 12 * sms) best /= 2;
#define DG_NORM_RING(ROW, n) ring(layer_norm_ring_kernel<ROW, FP8>, ROW(), n)
  if (vec) {
    using E8 = AlignedRow<T, 8 / V>;
    using E16 = AlignedRow<T, 16 / V>;
    using E32 = AlignedRow<T, 32 / V>;
    // Results in x's type leave faster with E = 16 where three rows fit at a time
    // (235 MB in and out, 16 bits: up to 4096 columns 74-75 us, with E = 32 82-84;
    // 7168 columns 98 and 73), FP32 always (2048 columns 82 and 88, 7168 70 and 94).
    if (!FP8 && best == 32 && groups(E16(), 16) >= std::min<int64_t>(sizeof(T) == 2 ? 3 : 1, (rows + sms - 1) / sms)) best = 16;
    if (best == 8) return DG_NORM_RING(E8, 8);
    if (best == 16) return DG_NORM_RING(E16, 16);
    if (groups(E32(), 32)) return DG_NORM_RING(E32, 32);
    if (p.cols <= kWideThreads * kWideVecs * V)
      return launch_op(layer_norm_wide_kernel<T, FP8>, dim3((unsigned)rows), kWideThreads, 0, pdl, st, p);
  }
  if constexpr (FP8) return cudaErrorInvalidValue;
  else {
    if (!vec) {
      using Few1 = RaggedRow<T, 8, 1>;
      using Many1 = RaggedRow<T, 32, 1>;
      const bool few = best == 8;
      if (few || groups(Many1(), 32)) {
        if constexpr (sizeof(T) == 2) {
          using Few2 = RaggedRow<T, 8, 2>;
          using Many2 = RaggedRow<T, 32, 2>;
          if (pairs_aligned<T>(p, false)) return few ? DG_NORM_RING(Few2, 8) : DG_NORM_RING(Many2, 32);
        }
        return few ? DG_NORM_RING(Few1, 8) : DG_NORM_RING(Many1, 32);
      }
    }
    return launch_op(layer_norm_long_kernel<T>, dim3((unsigned)p.rows), 1024, 0, pdl, st, p);
  }
#undef DG_NORM_RING
}

template <class T>
cudaError_t backward(const LayerNormArgs& a, bool vec, int parts, int* used, bool pdl, cudaStream_t st) {
  LayerNormArgs p = a;
  constexpr int V = 16 / (int)sizeof(T);
  const int sms = parts;
  auto groups = [&](auto row, int n) {  // as in forward
    using Row = decltype(row);
    const int64_t tpr = (p.cols + 32 * n - 1) / (32 * n) * 32;
    const int64_t par = tpr * Row::P * 8, each = 2 * Row::kBackRing * Row::bytes(tpr);
    if (tpr > kNormBackThreads || par + each > kNormMaxSmem) return (int64_t)0;
    return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(kNormBackThreads / tpr, (kNormMaxSmem - par) / each),
                                                  (p.rows + sms - 1) / sms));
  };
  auto ring = [&](auto kern, auto row, int n) {
    using Row = decltype(row);
    const int64_t rpc = groups(row, n);
    p.tpr = (int)((p.cols + 32 * n - 1) / (32 * n) * 32);
    const int64_t threads = rpc * p.tpr;
    p.ring_bytes = Row::kBackRing * Row::bytes(threads);
    p.par_at = 2 * p.ring_bytes;
    const int64_t sums = rpc > 1 ? threads * 2 * Row::P * (int64_t)sizeof(float2) : 0;
    const size_t smem = (size_t)std::max<int64_t>(p.par_at + (int64_t)p.tpr * Row::P * 8, sums);
    *used = (int)std::min<int64_t>((p.rows + rpc - 1) / rpc, sms);
    cudaError_t e = set_smem(kern, smem, kNormMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_op(kern, dim3((unsigned)*used), (unsigned)threads, smem, pdl, st, p);
  };
#define DG_NORM_RING(ROW, n) ring(layer_norm_backward_ring_kernel<ROW>, ROW(), n)
  const bool few = norm_values(p.cols) == 8;
  if (vec) {
    using E8 = AlignedRow<T, 8 / V>;
    using E16 = AlignedRow<T, 16 / V>;
    if (few) return DG_NORM_RING(E8, 8);
    if (groups(E16(), 16)) return DG_NORM_RING(E16, 16);
  } else {
    using Few1 = RaggedRow<T, 8, 1>;
    using Many1 = RaggedRow<T, 16, 1>;
    if (few || groups(Many1(), 16)) {
      if constexpr (sizeof(T) == 2) {
        using Few2 = RaggedRow<T, 8, 2>;
        using Many2 = RaggedRow<T, 16, 2>;
        if (pairs_aligned<T>(p, true)) return few ? DG_NORM_RING(Few2, 8) : DG_NORM_RING(Many2, 16);
      }
      return few ? DG_NORM_RING(Few1, 8) : DG_NORM_RING(Many1, 16);
    }
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

int layer_norm_backward_parts(int sms) { return sms; }  // a CTA an SM

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
  return launch_op(layer_norm_join_kernel, dim3((unsigned)((cols + 31) / 32), 2), 32 * kJoinWarps, 0, pdl, stream,
                   (const float*)part, dw, db, used, cols);
}

}  // namespace dg
