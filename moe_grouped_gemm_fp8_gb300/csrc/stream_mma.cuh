// Products of many weight rows with a few tokens, as a warp's stream: 16 rows of
// 8-bit weights, 128 columns at a time, go by asynchronous copies through the
// warp's own ring in shared memory, are decoded to halves in registers (exact:
// every E4M3 value and every 8-bit integer is a half) and multiplied with the
// tokens' halves by mma m16n8k16 with FP32 sums.
//
// Which 4 columns of the 128 a lane holds for a product is free as long as
// weights and tokens agree.  Lane (r, q) = (lane / 4, lane % 4) takes, of rows r
// and r + 8, the 16 bytes at columns 16 q and at 64 + 16 q: whole 64-byte pieces
// a row and instruction.  Product j (0..7) multiplies columns
//   64 (j / 4) + 16 q + 4 (j % 4) + 0..3
// of every q.  The tokens' halves are stored in that order: of each 128 columns
#pragma once

#include "dg_device.cuh"
#include "dg_ops.cuh"

namespace dg {

constexpr int kStreamCols = 128;                       // columns of a stage

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

// The lane's codes of half a stage (h = 0, 1: 64 columns), decoded: a[i] are the
// A registers of product 4 h + i.
template <class Decode>
__device__ __forceinline__ void stream_decode(const uint8_t* stage, int h, int lane, uint32_t (&a)[4][4]) {
  const uint4 g = *reinterpret_cast<const uint4*>(stage + h * 1024 + lane * 16);
  const uint4 u = *reinterpret_cast<const uint4*>(stage + h * 1024 + 512 + lane * 16);
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Decode::four(gw[i], a[i][0], a[i][2]);
    Decode::four(uw[i], a[i][1], a[i][3]);
  }
}

}  // namespace dg
