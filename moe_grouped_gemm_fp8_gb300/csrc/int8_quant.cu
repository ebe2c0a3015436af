// Rows to 8-bit integers: scale = amax / 127, code = the integer nearest to
// 127 x / amax, ties to even, of the exact quotient (so the codes do not depend
// on how a division or a reciprocal rounds).
//
// Bound by HBM.  A row is read once and stays in registers between its maximum
// and its codes.  127 / amax is bracketed by two FP32 numbers, 2^-22 below and above
// its rounded value; where x times both rounds to one integer, so does the exact
// quotient.  Elsewhere a 16-bit value's quotient is a half integer; of FP32 values (6
// in 100,000) 254 |x| and (2 n + 1) amax are compared, exactly (all values in FP64: 307
// us where this takes 53).  Measured in a graph: 16384 x 7168 of BF16 53.2 us, 6.6 TB/s,
// 98% of the copy's rate (FP16 57.5, FP32 85.6: 101%); one row 1.9 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "int8_gemm.h"

namespace dg {
namespace {

constexpr int kQiWidest = 32;  // warps of the longest rows
constexpr int kQiItems = 32;  // values a thread keeps (16-bit types; FP32: 16)

// Values 4 i to 4 i + 3 of a thread's words.
template <class T>
__device__ __forceinline__ void qi_unpack(const uint32_t* w, int i, float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[4 * i + j]);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t b = w[2 * i + j];
      if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      } else {
        v[2 * j] = bf16_lo(b);
        v[2 * j + 1] = bf16_hi(b);
      }
    }
  }
}

// max(m, |v|), NaN where either is
__device__ __forceinline__ float qi_max(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

// The code of v where the bracket holds a half integer: 254 |v| against (2 n + 1)
// amax, n the lower integer.  Both products are kept exactly as an FP32 and its
// rounding error; near each other, their difference is exact too.
__device__ __forceinline__ int qi_settle(float v, float amax, float low) {
  // (2^-8 of both: 255 amax may be too large; every bit stays above 2^-149, as amax >= kQiTiny)
  const float n = rintf(fabsf(v) * low), odd = fmaf(2.0f, n, 1.0f);
  const float a = fabsf(v) * 0.00390625f;
  amax *= 0.00390625f;
  const float p = __fmul_rn(254.0f, a), m = __fmul_rn(odd, amax);
  const float d = (p - m) + (fmaf(254.0f, a, -p) - fmaf(odd, amax, -m));
  const int c = (int)n;
  const int code = d > 0.0f || (d == 0.0f && (c & 1)) ? c + 1 : c;
  return v < 0.0f ? -code : code;
}
// The code of v where 127 / amax may overflow: the quotient in FP64, whose
// rounding cannot reach a half integer (a 31-bit number over one of 24).
__device__ __noinline__ int qi_tiny(float v, float amax) { return (int)rint(127.0 * (double)v / (double)amax); }

// Adding it rounds to an integer, which the low bits hold.
constexpr float kQiMagic = 12582912.0f;  // 1.5 2^23

// The low bytes of four FP32 numbers.
__device__ __forceinline__ uint32_t qi_pack(float2 a, float2 b) {
  const uint32_t x = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
  const uint32_t y = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
  return __byte_perm(x, y, 0x5410);
}

// Four values -> four codes in a word. FP32: open is nonzero where the bracket's
// ends round to different integers. Of 16-bit types they do at halves alone: a
// quotient 127 V / (2^k M), V and M of 11 bits at most, that is no half is 1 / (254 V)
// > 2^-19 of itself away from one, and the bracket 2^-21 wide. So the even one is the
// code. (Half of a BF16 row's maximum, 63.5 exactly, is in most warps' values:
// settling them one by one took 16384 x 7168 from 60 to 82 us.)
template <class T>
__device__ __forceinline__ uint32_t qi_four(const float (&v)[4], float low, float high, uint32_t& open) {
  const float2 magic = make_float2(kQiMagic, kQiMagic), l = make_float2(low, low), h = make_float2(high, high);
  const float2 a = make_float2(v[0], v[1]), b = make_float2(v[2], v[3]);
  const float2 al = fma2(a, l, magic), ah = fma2(a, h, magic), bl = fma2(b, l, magic), bh = fma2(b, h, magic);
  const uint32_t codes = qi_pack(al, bl);
  if constexpr (sizeof(T) == 4) {
    open |= __float_as_uint(al.x) ^ __float_as_uint(ah.x);
    open |= __float_as_uint(al.y) ^ __float_as_uint(ah.y);
    open |= __float_as_uint(bl.x) ^ __float_as_uint(bh.x);
    open |= __float_as_uint(bl.y) ^ __float_as_uint(bh.y);
    return codes;
  } else {
    const uint32_t odd = (codes & 0x01010101u) * 0xFFu;
    return (codes & ~odd) | (qi_pack(ah, bh) & odd);
  }
}

// max(m, magnitudes of a word's values), NaN where one is: pairs of halves, or an FP32.
template <class T>
__device__ __forceinline__ void qi_max_word(uint32_t& m, uint32_t w) {
  if constexpr (sizeof(T) == 4) {
    m = __float_as_uint(qi_max(__uint_as_float(m), __uint_as_float(w), 0.0f));
  } else if constexpr (std::is_same<T, __half>::value) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&m), __habs2(*reinterpret_cast<const __half2*>(&w)));
    m = *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    m = *reinterpret_cast<const uint32_t*>(&r);
  }
}

constexpr float kQiTiny = 1e-30f;  // below it 127 / amax may overflow

// How a row lies in W warps: words of 16 bytes one lane after the other.
template <class T, int W>
struct QiPlan {
  static constexpr int E = 16 / sizeof(T), V = kQiItems * 2 / sizeof(T) / E, PER = E * V;
  static constexpr int kThreads = W <= 8 ? 256 : 32 * W, kCtas = W <= 8 ? 4 : 32 / W, kRows = kThreads / (32 * W);
  static constexpr int kWide = 32 * W * PER;  // columns at once
  static constexpr int kRing = 2;             // rows a CTA has on their way or in work
  static constexpr size_t kSmem = (size_t)kRing * V * kThreads * 16;
};

// The maximum of a row's magnitudes, from its threads' words; NaN where a value is. part: one a warp.
template <class T, int W, int N>
__device__ __forceinline__ float qi_row_max(uint32_t most, const uint32_t (&x4)[N], float* part) {
#pragma unroll
  for (int i = 0; i < N; ++i) qi_max_word<T>(most, x4[i]);
  float m;
  if constexpr (sizeof(T) == 4) {
    m = __uint_as_float(most);
  } else {
    const uint32_t pair[2] = {most, 0};
    float v[4];
    qi_unpack<T>(pair, 0, v);
    m = qi_max(0.0f, v[0], v[1]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = qi_max(m, __shfl_xor_sync(0xffffffffu, m, o), 0.0f);
  if constexpr (W > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = m;
    __syncthreads();
    const int first = warp / W * W;
#pragma unroll
    for (int i = 0; i < W; ++i) m = qi_max(m, part[first + i], 0.0f);
  }
  return m;
}

// The scale of a row whose maximum is m; no number where that is not finite.
__device__ __forceinline__ float qi_scale(float m) { return m < INFINITY ? m / 127.0f : __uint_as_float(0x7FC00000u); }

// What brackets 127 / m; 0 where it may overflow or m is not finite.
struct QiBracket {
  float low, high;
  __device__ __forceinline__ explicit QiBracket(float m) {
    const float inv = m < INFINITY && !(m < kQiTiny) ? 127.0f / m : 0.0f;
    low = inv * (1.0f - 0x1p-22f);
    high = inv * (1.0f + 0x1p-22f);
  }
};

// Codes of a thread's words, all 0 where m is not finite.
template <class T, int N, int CODES>
__device__ __forceinline__ void qi_codes(uint32_t (&x4)[N], float m, const QiBracket& b, uint32_t (&w)[CODES]) {
  if (!(m < INFINITY)) {
#pragma unroll
    for (int i = 0; i < N; ++i) x4[i] = 0;
  }
  uint32_t open = 0;
#pragma unroll
  for (int i = 0; i < CODES; ++i) {
    float v[4];
    qi_unpack<T>(x4, i, v);
    w[i] = qi_four<T>(v, b.low, b.high, open);
  }
  if (sizeof(T) == 4 && open) {
#pragma unroll
    for (int i = 0; i < CODES; ++i) {
      float v[4];
      qi_unpack<T>(x4, i, v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (fmaf(v[j], b.low, kQiMagic) != fmaf(v[j], b.high, kQiMagic))
          w[i] = (w[i] & ~(0xFFu << (8 * j))) | ((uint32_t)qi_settle(v[j], m, b.low) & 0xFFu) << (8 * j);
    }
  }
  if (m < kQiTiny && m > 0.0f) {
#pragma unroll
    for (int i = 0; i < CODES; ++i) {
      float v[4];
      qi_unpack<T>(x4, i, v);
      w[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i] |= ((uint32_t)qi_tiny(v[j], m) & 0xFFu) << (8 * j);
    }
  }
}

// 4 E codes of a 16-byte word of E values.
template <int E, int CODES>
__device__ __forceinline__ void qi_store(int8_t* to, const uint32_t (&w)[CODES], int i) {
  if constexpr (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[2 * i], w[2 * i + 1]);
  else *reinterpret_cast<uint32_t*>(to) = w[i];
}

// Rows on 16 bytes, of at most kWide columns: a CTA takes every gridDim.x-th, the next
// on its way by asynchronous copies while one is in work.  A thread copies what it
// will read itself, so nothing waits for another's copies.
template <class T, int W>
__global__ void __launch_bounds__(QiPlan<T, W>::kThreads, QiPlan<T, W>::kCtas)
    quantize_int8_ring_kernel(const T* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scales, int64_t rows,
                              int cols, int64_t ldx) {
  using Plan = QiPlan<T, W>;
  constexpr int E = Plan::E, V = Plan::V, RING = Plan::kRing, kThreads = Plan::kThreads;
  extern __shared__ uint4 ring[];  // [slot][word][thread]
  __shared__ float part[2][kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int at = threadIdx.x % (32 * W);  // in the row's threads
  const int64_t mine = (int64_t)blockIdx.x * Plan::kRows + (threadIdx.x >> 5) / W, step = (int64_t)gridDim.x * Plan::kRows;
  const int64_t first = (int64_t)blockIdx.x * Plan::kRows;  // the CTA's: its threads make the same rounds
  int64_t ahead = mine;
  int put = 0;
  auto next = [&]() {
    const bool on = ahead < rows;
    const T* xr = x + (on ? ahead : 0) * ldx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * 32 * W + at) * E;
      const bool in = on && c < cols;
      cp_async16_or_zero(ring + (put * V + i) * kThreads + threadIdx.x, xr + (in ? c : 0), in);
    }
    cp_async_commit();
    put = put + 1 == RING ? 0 : put + 1;
    ahead += step;
  };
#pragma unroll
  for (int i = 0; i < RING - 1; ++i) next();
  int get = 0;
  uint32_t turn = 0;
  int64_t row = mine;
  for (int64_t r = first; r < rows; r += step, row += step) {
    next();
    cp_async_wait<RING - 1>();
    uint32_t x4[V * 4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint4 v = ring[(get * V + i) * kThreads + threadIdx.x];
      x4[4 * i] = v.x;
      x4[4 * i + 1] = v.y;
      x4[4 * i + 2] = v.z;
      x4[4 * i + 3] = v.w;
    }
    get = get + 1 == RING ? 0 : get + 1;
    const float m = qi_row_max<T, W>(0u, x4, part[turn]);
    turn ^= 1u;
    if (row >= rows) continue;
    if (at == 0) scales[row] = qi_scale(m);
    uint32_t w[Plan::PER / 4];
    qi_codes<T>(x4, m, QiBracket(m), w);
    int8_t* qr = q + row * cols;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * 32 * W + at) * E;
      if (c < cols) qi_store<E>(qr + c, w, i);
    }
  }
  cp_async_wait<0>();
}

// Other rows, W warps each.  VEC: rows of x on 16 bytes and of codes on 16 /
// sizeof(T), longer than the ring's; else a value at a time.
template <class T, int W, bool VEC>
__global__ void __launch_bounds__(QiPlan<T, W>::kThreads, QiPlan<T, W>::kCtas)
    quantize_int8_kernel(const T* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scales, int64_t rows,
                         int cols, int64_t ldx) {
  using Plan = QiPlan<T, W>;
  constexpr int E = Plan::E, V = Plan::V, PER = Plan::PER, kThreads = Plan::kThreads, kRows = Plan::kRows;
  __shared__ float part[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int at = threadIdx.x % (32 * W);  // in the row's threads
  const int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 5) / W;
  const bool on = row < rows;
  const T* xr = x + (on ? row : 0) * ldx;
  const int n = on ? cols : 0;
  constexpr int kWide = Plan::kWide;  // columns of a pass; more than one only at the widest W
  uint32_t x4[V * 4];  // the values as they came
  uint32_t most = 0;
  auto load = [&](int c0) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + (i * 32 * W + at) * E;
        const uint4 w = c < n ? ld_stream_u4(xr + c) : make_uint4(0, 0, 0, 0);
        x4[4 * i] = w.x;
        x4[4 * i + 1] = w.y;
        x4[4 * i + 2] = w.z;
        x4[4 * i + 3] = w.w;
      }
    } else {
      using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
      const Bits* bits = reinterpret_cast<const Bits*>(xr);
      constexpr int kPack = 4 / sizeof(T);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = c0 + i * 32 * W + at;
        const uint32_t one = c < n ? (uint32_t)bits[c] : 0u;
        if (i % kPack == 0) x4[i / kPack] = one;
        else x4[i / kPack] |= one << 16;
      }
    }
  };
  const bool once = cols <= kWide;
  for (int c0 = 0; c0 + kWide < cols; c0 += kWide) {
    load(c0);
#pragma unroll
    for (int i = 0; i < V * 4; ++i) qi_max_word<T>(most, x4[i]);
  }
  load((cols - 1) / kWide * kWide);
  const float m = qi_row_max<T, W>(most, x4, part);
  if (!on) return;
  if (at == 0) scales[row] = qi_scale(m);
  const QiBracket bracket(m);
  int8_t* qr = q + row * cols;
  for (int c0 = 0; c0 == 0 || c0 < cols; c0 += kWide) {
    if (!once) load(c0);
    uint32_t w[PER / 4];
    qi_codes<T>(x4, m, bracket, w);
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + (i * 32 * W + at) * E;
        if (c < n) qi_store<E>(qr + c, w, i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = c0 + i * 32 * W + at;
        if (c < n) qr[c] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

template <class T, int W>
cudaError_t qi_launch(const void* x, int8_t* q, float* scales, int64_t rows, int64_t cols, int64_t ldx, int sms, bool pdl,
                      cudaStream_t stream) {
  using Plan = QiPlan<T, W>;
  const bool vec = cols % Plan::E == 0 && ldx % Plan::E == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(q) % Plan::E == 0;
  const int64_t ctas = (rows + Plan::kRows - 1) / Plan::kRows, at_once = (int64_t)sms * Plan::kCtas;
  const T* xt = static_cast<const T*>(x);
  // (by a CTA a row 16384 x 7168 of BF16 takes 68.5 us, the ring 53.2; 4096 rows 18.3 / 14.8, 600 rows 4.5 / 4.2, one
  // 1.9 / 2.0)
  if (vec && cols <= Plan::kWide) {
    cudaError_t e = set_smem(quantize_int8_ring_kernel<T, W>, Plan::kSmem, Plan::kSmem);
    if (e != cudaSuccess) return e;
    return launch_op(quantize_int8_ring_kernel<T, W>, dim3((unsigned)std::min(ctas, at_once)), Plan::kThreads, Plan::kSmem, pdl,
                     stream, xt, q, scales, rows, (int)cols, ldx);
  }
  const dim3 grid((unsigned)ctas);
  if constexpr (W == kQiWidest)
    if (vec)
      return launch_op(quantize_int8_kernel<T, W, true>, grid, Plan::kThreads, 0, pdl, stream, xt, q, scales, rows, (int)cols, ldx);
  // (off 16 bytes two passes of 16 warps are quicker than one of 32: 4096 x 20001 126 us and 147; on them the ring's one
  // pass: 4096 x 20480 56 and 76)
  constexpr int kOff = std::min(W, kQiWidest / 2);
  return launch_op(quantize_int8_kernel<T, kOff, false>, grid, QiPlan<T, kOff>::kThreads, 0, pdl, stream, xt, q, scales, rows,
                   (int)cols, ldx);
}

template <class T>
cudaError_t qi_dispatch(const void* x, int8_t* q, float* scales, int64_t rows, int64_t cols, int64_t ldx, int sms,
                        bool pdl, cudaStream_t stream) {
  constexpr int kPer = kQiItems * 2 / sizeof(T) * 32;  // columns of a warp
  if (cols <= kPer) return qi_launch<T, 1>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
  if (cols <= 2 * kPer) return qi_launch<T, 2>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
  if (cols <= 4 * kPer) return qi_launch<T, 4>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
  if (cols <= 8 * kPer) return qi_launch<T, 8>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
  if (cols <= 16 * kPer) return qi_launch<T, 16>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
  return qi_launch<T, kQiWidest>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
}

}  // namespace

cudaError_t quantize_int8_launch(const void* x, int dtype, int8_t* q, float* scales, int64_t rows, int64_t cols,
                                 int64_t ldx, int sms, bool pdl, cudaStream_t stream) {
  if (dtype == DG_DTYPE_FP32) return qi_dispatch<float>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
  if (dtype == DG_DTYPE_FP16) return qi_dispatch<__half>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
  return qi_dispatch<__nv_bfloat16>(x, q, scales, rows, cols, ldx, sms, pdl, stream);
}

}  // namespace dg
