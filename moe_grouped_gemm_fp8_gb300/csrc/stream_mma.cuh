// 8-bit weights as halves in registers, and mma m16n8k16 of halves with FP32 sums:
// every E4M3 value and every 8-bit integer is a half exactly.
#pragma once

#include "dg_device.cuh"
#include "dg_ops.cuh"

namespace dg {

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four E4M3 codes -> two words of halves.
struct DecodeE4m3 {
  static __device__ __forceinline__ void four(uint32_t c, uint32_t& lo, uint32_t& hi) {
    __half2 a, b;
    e4m3x4_to_half(c, a, b);
    lo = *reinterpret_cast<uint32_t*>(&a);
    hi = *reinterpret_cast<uint32_t*>(&b);
  }
};
// Four 8-bit integers -> two words of halves: 1024 + (c + 128) is the half with
// that byte in its low bits.
struct DecodeInt8 {
  static __device__ __forceinline__ void four(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = c ^ 0x80808080u, magic = 0x64646464u;
    const uint32_t l = __byte_perm(u, magic, 0x4140), h = __byte_perm(u, magic, 0x4342);
    const uint32_t off = 0xE480E480u;  // -1152
    const __half2 o = *reinterpret_cast<const __half2*>(&off);
    const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&l), o), b = __hadd2(*reinterpret_cast<const __half2*>(&h), o);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  }
};

}  // namespace dg
