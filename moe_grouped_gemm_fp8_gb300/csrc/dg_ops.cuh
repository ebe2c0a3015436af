// Pieces shared by the kernels around the GEMMs (8-bit checkpoints, the gated
// feed-forward's backward pass, layer norm): E4M3 and BF16 conversions, the
// activations, scale bytes and launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_device.cuh"

namespace dg {

// 16 bytes read once, not kept in L1.
__device__ __forceinline__ uint4 ld_stream_u4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Asynchronous 16-byte copy into shared memory, past L1, in groups.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {  // dst: a shared address
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
// 32 bytes as one access (32-byte aligned).
__device__ __forceinline__ void st_global_32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
// The first `bytes` (1 to 16) of them, zeros after.
__device__ __forceinline__ void cp_async16_part(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
// The same with zeros in the place of the source where `live` is false (the
// source is not read).
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async8_or_zero(void* dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4_or_zero(void* dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Four values (already divided by their scale) -> four E4M3 codes, first lowest.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Four E4M3 codes -> halves and FP32, exactly (every E4M3 value is a half).
__device__ __forceinline__ void e4m3x4_to_half(uint32_t codes, __half2& a, __half2& b) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
  a = *reinterpret_cast<__half2*>(&lo);
  b = *reinterpret_cast<__half2*>(&hi);
}
// Four halves -> E4M3 codes, rounded to nearest even.
__device__ __forceinline__ uint32_t half_to_e4m3x4(__half2 a, __half2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "r"(*reinterpret_cast<uint32_t*>(&a)), "r"(*reinterpret_cast<uint32_t*>(&b)));
  return r;
}
// (2^k, 2^k) for k <= 15, 0 below 2^-24.
__device__ __forceinline__ __half2 half_pow2(int k) {
  const uint32_t h = k >= -14 ? (uint32_t)(k + 15) << 10 : (k >= -24 ? 1u << (k + 24) : 0u);
  const uint32_t w = h * 0x10001u;
  return *reinterpret_cast<const __half2*>(&w);
}
__device__ __forceinline__ void e4m3x4_to_float(uint32_t codes, float (&f)[4]) {
  __half2 lo, hi;
  e4m3x4_to_half(codes, lo, hi);
  const float2 a = __half22float2(lo);
  const float2 b = __half22float2(hi);
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// scale_exponent(amax) + 127 without branches: adding 0x1FFFFF carries into the
// exponent exactly when the fraction is above 1.75; an infinity gets 2^127.
// amax: the maximum of magnitudes that passes over NaN (abs_max2, abs_max3).
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const int t = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
  const uint32_t b = amax > 0.0f ? (uint32_t)max(t, 0) : 127u;
  return amax == INFINITY ? 254u : b;
}
// 2^(127 - byte), the factor that brings a group into E4M3's range (byte <= 254,
// where it is the subnormal 2^-127).
__device__ __forceinline__ float inverse_of_byte(uint32_t byte) {
  return __uint_as_float(max((254u - byte) << 23, 1u << 22));
}

// Pairs of FP32 (one instruction for two).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float b) { return __fmul2_rn(a, make_float2(b, b)); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
// max(|m|, |a|, |b|) of those that are numbers
__device__ __forceinline__ float abs_max3(float m, float a, float b) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float abs_max2(float m, float2 a) { return abs_max3(m, a.x, a.y); }
// The bits of |v|, 0 for NaN: ordered like the magnitudes.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(fmaxf(fabsf(v), 0.0f)); }
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) { return e4m3x4(a.x, a.y, b.x, b.y); }
// Two FP32 sums over the warp in one butterfly: lanes 0-15 end with a's, lanes
// 16-31 with b's.
__device__ __forceinline__ float warp_sum2(float a, float b) {
  const bool hi = (threadIdx.x & 16) != 0;
  float v = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// UE8M0 byte -> its scale 2^(b - 127) (b = 0: 2^-127, a subnormal).
__device__ __forceinline__ float scale_of_byte(uint32_t b) { return pow2f((int)b - 127); }

// Byte `block % 4` of a packed scale word; the last block of the axis also
// writes the word's unused bytes as 0.
__device__ __forceinline__ void store_scale_byte(uint32_t* word, int block, bool last, uint32_t byte) {
  uint8_t* p = reinterpret_cast<uint8_t*>(word);
  const int t = block & 3;
  p[t] = (uint8_t)byte;
  if (last)
    for (int i = t + 1; i < 4; ++i) p[i] = 0;
}

// The hardware's base-2 exponential and reciprocal (about 2^-22 relative each;
// results below 2^-126 become 0, which the logistic function does not notice).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The logistic function uses the fast exponential and
// reciprocal: together about 2^-21 relative, well below the 2^-9 (BF16) or
// 2^-4 (E4M3) at which every result of these kernels is rounded.  For large
// negative g exp(-g) is inf and s is 0, so silu and its derivative are 0.
__device__ __forceinline__ float logistic(float z) { return rcp_approx(1.0f + exp2_approx(z * -1.4426950408889634f)); }

// silu(g) = g s with s = logistic(g); its derivative s + g s (1 - s).
// gelu in its tanh form, g (1 + tanh t) / 2 with t = c (g + 0.044715 g^3),
// c = sqrt(2 / pi): (1 + tanh t) / 2 is logistic(2 t), so it is g s with
// s = logistic(2 t), and its derivative s + g s (1 - s) 2 t'.
template <int ACT>
__device__ __forceinline__ float gate_logistic(float g) {
  if constexpr (ACT == DG_ACT_SILU) return logistic(g);
  constexpr float c2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  return logistic(g * (c2 + (c2 * 0.044715f) * g * g));
}
template <int ACT>
__device__ __forceinline__ float gate_act(float g) {
  return g * gate_logistic<ACT>(g);
}
// act(g) and act'(g) of a pair.
template <int ACT>
__device__ __forceinline__ void gate_act_grad2(float2 g, float2& a, float2& da) {
  float2 z = g;  // logistic's argument times -log2(e)
  float2 dz = make_float2(1.0f, 1.0f);
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (ACT == DG_ACT_SILU) {
    z = mul2(g, -kLog2e);
  } else {
    constexpr float c2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float2 gg = mul2(g, g);
    z = mul2(mul2(g, -kLog2e), fma2(gg, make_float2(c2 * 0.044715f, c2 * 0.044715f), make_float2(c2, c2)));
    // finite where g^2 is not: there a or 1 - s is 0, and 0 dz has to be too
    const float2 most = make_float2(fminf(gg.x, 1e30f), fminf(gg.y, 1e30f));
    dz = fma2(most, make_float2(3.0f * c2 * 0.044715f, 3.0f * c2 * 0.044715f), make_float2(c2, c2));
  }
  const float2 q = add2(make_float2(exp2_approx(z.x), exp2_approx(z.y)), make_float2(1.0f, 1.0f));
  const float2 s = make_float2(rcp_approx(q.x), rcp_approx(q.y));
  a = mul2(g, s);
  float2 t = fma2(s, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
  if constexpr (ACT != DG_ACT_SILU) t = mul2(t, dz);
  da = fma2(a, t, s);
}

// Raises a kernel's dynamic shared-memory limit where a launch of `smem` bytes
// may need more than 48 KB with the (few) bytes of its static arrays: always to
// `most`, the largest a launch of this kernel asks for. The limit belongs to the
// kernel, not to the launch: set to each launch's own size, a host thread with a
// small launch would lower it between another's call here and its launch.
template <class Kern>
static cudaError_t set_smem(Kern kern, size_t smem, size_t most) {
  if (smem > most) return cudaErrorInvalidValue;
  if (smem <= 40 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

// The (row block, column block) of tiles t, t + grid, ...: one division per CTA.
struct TileWalk {
  int t, rb, cb;
  __device__ __forceinline__ void init(int first, int blocks) {
    t = first;
    rb = first / blocks;
    cb = first - rb * blocks;
  }
  // drb = grid / blocks, dcb = grid % blocks
  __device__ __forceinline__ void next(int blocks, int drb, int dcb) {
    t += gridDim.x;
    rb += drb;
    cb += dcb;
    if (cb >= blocks) {
      cb -= blocks;
      ++rb;
    }
  }
};

// Launches with programmatic stream serialisation when pdl is set.
template <class Kern, class... Args>
static cudaError_t launch_op(Kern kern, dim3 grid, unsigned threads, size_t smem, bool pdl,
                             cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace dg
