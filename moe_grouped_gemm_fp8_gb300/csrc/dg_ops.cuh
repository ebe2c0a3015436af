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

// 8 bytes read once, not kept in L1.
__device__ __forceinline__ uint2 ld_stream_u2(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Magnitudes compare as unsigned integers of their bits (NaN above all).
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t abs_bits_max4(float a, float b, float c, float d) {
  return max(max(abs_bits(a), abs_bits(b)), max(abs_bits(c), abs_bits(d)));
}

// Four values (already divided by their scale) -> four E4M3 codes, first lowest.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)cvt_e4m3x2(a, b) | ((uint32_t)cvt_e4m3x2(c, d) << 16);
}
// Four E4M3 codes -> FP32, exactly (every E4M3 value is a half).
__device__ __forceinline__ void e4m3x4_to_float(uint32_t codes, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
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

// act(g) and act'(g).  The logistic function uses the fast exponential and
// reciprocal: together about 2^-21 relative, well below the 2^-9 (BF16) or
// 2^-4 (E4M3) at which every result of these kernels is rounded.  For large
// negative g exp(-g) is inf and s is 0, so silu and its derivative are 0.
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

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
template <int ACT>
__device__ __forceinline__ void gate_act_grad(float g, float& a, float& da) {
  const float s = gate_logistic<ACT>(g);
  a = g * s;
  if constexpr (ACT == DG_ACT_SILU) {
    da = s + a * (1.0f - s);
  } else {
    constexpr float c2 = 1.5957691216057308f;
    da = s + a * (1.0f - s) * (c2 + (3.0f * c2 * 0.044715f) * g * g);
  }
}

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
