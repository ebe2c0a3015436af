// Operands of the 8-bit integer product for the tensor cores: codes loaded,
// widened to halves in registers and stored in the MMA's 128-byte swizzle.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "int8_gemm.h"
#include "stream_mma.cuh"

namespace dg {

constexpr int kIgWiden = 16;  // producer warps, from warp 8 on
constexpr int kIgThreads = 32 * (8 + kIgWiden);
constexpr int kIgPass = 4 * kIgWiden;  // rows that they load at a time
constexpr int kIgK = 128;       // columns of a stage: two swizzle atoms of 64 halves
constexpr int kIgAhead = 2;     // stages whose loads are in flight

// FP32 D (bits 4-5 = 1), FP16 A and B (format 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
template <bool PAIR>
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 codes at the 16-byte chunks 2 q and 2 q + 1 of a row of 128 bytes of halves;
// in the second atom the other way round (in a and b alike, so the products'
// sum is the same), which lets 8 lanes hold a row's 128 columns, a whole line of
// memory, and still store to all banks.
__device__ __forceinline__ void ig_widen(uint32_t tile, int row, int q, int atom, const uint4& c) {
  uint32_t h[8];
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) DecodeInt8::four(w[i], h[2 * i], h[2 * i + 1]);
  const uint32_t at = tile + row * 128 + (((2 * q + atom) ^ (row & 7)) << 4);
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
               : "memory");
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ 16u), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
               : "memory");
}

// A producer thread's share of a stage: 16 codes of each kIgPass-th row.  A warp
// covers 4 rows' 128 columns.
template <int ROWS>
struct IgRows {
  static constexpr int kPieces = (ROWS + kIgPass - 1) / kIgPass;
  const int8_t* src;  // the thread's first row, from its first column on
  uint32_t on;        // bit i: row kIgPass i + row exists
  __device__ __forceinline__ void aim(const int8_t* base, int64_t ld, int first, int end, int row, int col) {
    on = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (kIgPass * i + row < ROWS && first + kIgPass * i + row < end) on |= 1u << i;
    src = base + (int64_t)(on ? first + row : 0) * ld + col;
  }
  __device__ __forceinline__ void load(uint4 (&v)[kPieces], int64_t ld, int k, bool in) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      v[i] = in && (on >> i & 1u) ? __ldg(reinterpret_cast<const uint4*>(src + i * kIgPass * ld + k)) : make_uint4(0, 0, 0, 0);
  }
  static __device__ __forceinline__ void store(const uint4 (&v)[kPieces], uint32_t tile, int row, int atom, int q) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (ROWS % kIgPass == 0 || kIgPass * i + row < ROWS)
        ig_widen(tile + atom * (ROWS * 128), kIgPass * i + row, q, atom, v[i]);
  }
};

}  // namespace dg
