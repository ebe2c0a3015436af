// 8-bit activation checkpoints: an activation is kept between the passes as
// E4M3 codes with one power-of-two scale per 1 x 128 row group (the layout
// the NT GEMMs read), and the backward pass uses it as it is.
//
//   save:  BF16 rows -> codes + packed scales (3 bytes moved per element)
//   use:   codes + row scales -> codes + scales per 128 rows of each column,
//          the K-grouped GEMM's operand of a weight gradient (2 bytes)
//   restore: codes + row scales -> BF16 or FP32
//
// All three are bound by HBM.  Quantising a given number is exact arithmetic
// (a power of two times the number, rounded once), so results are bitwise
// those of the formula.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_device.cuh"
#include "dg_ops.cuh"

namespace dg {
namespace {

// One warp per (group, row, 512-column pack), lane l on columns 4l .. 4l+3 of
// each 128-column block; warps ordered row-fastest so that the scale words of
// neighbouring warps are adjacent.
__global__ void __launch_bounds__(256) save_rows_kernel(const __nv_bfloat16* __restrict__ x,
                                                        uint8_t* __restrict__ q,
                                                        uint32_t* __restrict__ sf, int64_t groups,
                                                        int64_t rows, int64_t rows_pad,
                                                        int64_t cols, int kblocks, int kpacks) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (w >= groups * rows_pad * kpacks) return;
  const int64_t r = w % rows_pad;
  const int64_t j = (w / rows_pad) % kpacks;
  const int64_t g = w / (rows_pad * kpacks);
  uint32_t word = 0;
  if (r < rows) {
    const int64_t at = (g * rows + r) * cols + 4 * j * 128 + lane * 4;
    uint2 v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (4 * j + t < kblocks) v[t] = ld_stream_u2(x + at + t * 128);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (4 * j + t >= kblocks) break;
      const float a = bf16_lo(v[t].x), b = bf16_hi(v[t].x), c = bf16_lo(v[t].y), d = bf16_hi(v[t].y);
      const uint32_t m = __reduce_max_sync(0xffffffffu, abs_bits_max4(a, b, c, d));
      const int e = scale_exponent(__uint_as_float(m));
      const float inv = pow2f(-e);
      *reinterpret_cast<uint32_t*>(q + at + t * 128) = e4m3x4(a * inv, b * inv, c * inv, d * inv);
      word |= (uint32_t)(e + 127) << (8 * t);
    }
  }
  if (lane == 0) sf[(g * kpacks + j) * rows_pad + r] = word;
}

// Same walk; each lane turns 4 codes of each block into BF16 or FP32.
template <class OUT>
__global__ void __launch_bounds__(256) restore_rows_kernel(const uint8_t* __restrict__ q,
                                                           const uint32_t* __restrict__ sf,
                                                           OUT* __restrict__ x, int64_t groups,
                                                           int64_t rows, int64_t rows_pad,
                                                           int64_t cols, int kblocks, int kpacks) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (w >= groups * rows * kpacks) return;
  const int64_t r = w % rows;
  const int64_t j = (w / rows) % kpacks;
  const int64_t g = w / (rows * kpacks);
  const uint32_t word = __ldg(sf + (g * kpacks + j) * rows_pad + r);
  const int64_t at = (g * rows + r) * cols + 4 * j * 128 + lane * 4;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (4 * j + t >= kblocks) break;
    const float s = scale_of_byte((word >> (8 * t)) & 0xFFu);
    float f[4];
    e4m3x4_to_float(__ldg(reinterpret_cast<const uint32_t*>(q + at + t * 128)), f);
    if constexpr (sizeof(OUT) == 4) {
      *reinterpret_cast<float4*>(x + at + t * 128) = make_float4(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
    } else {
      *reinterpret_cast<uint2*>(x + at + t * 128) =
          make_uint2(bf16x2_bits(f[0] * s, f[1] * s), bf16x2_bits(f[2] * s, f[3] * s));
    }
  }
}

// One CTA per 128 x 128 tile, 512 threads: warp w holds rows 8w .. 8w+7, lane
// l columns 4l .. 4l+3.  Column maxima go through shared memory once.
__global__ void __launch_bounds__(512) use_cols_kernel(const uint8_t* __restrict__ q,
                                                       const uint32_t* __restrict__ sf,
                                                       const int32_t* __restrict__ m_indices,
                                                       uint8_t* __restrict__ qc,
                                                       uint32_t* __restrict__ sfc, int64_t rows,
                                                       int64_t rows_pad, int64_t cols, int rblocks) {
  __shared__ uint4 cmax[16][32];
  __shared__ float4 cinv[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kblocks = (int)(cols / 128);
  const int rb = blockIdx.x / kblocks, kb = blockIdx.x % kblocks;
  const int64_t row0 = (int64_t)rb * 128 + warp * 8;
  const int64_t col = (int64_t)kb * 128 + lane * 4;
  float v[8][4];
  uint4 m = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + i;
    const bool live = r < rows && (!m_indices || __ldg(m_indices + r) >= 0);
    uint32_t codes = 0;
    float s = 0.0f;
    if (live) {
      codes = __ldg(reinterpret_cast<const uint32_t*>(q + r * cols + col));
      s = scale_of_byte((__ldg(sf + (int64_t)(kb >> 2) * rows_pad + r) >> (8 * (kb & 3))) & 0xFFu);
    }
    e4m3x4_to_float(codes, v[i]);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[i][c] *= s;
    m.x = max(m.x, abs_bits(v[i][0]));
    m.y = max(m.y, abs_bits(v[i][1]));
    m.z = max(m.z, abs_bits(v[i][2]));
    m.w = max(m.w, abs_bits(v[i][3]));
  }
  cmax[warp][lane] = m;
  __syncthreads();
  if (threadIdx.x < 128) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(&cmax[0][0]) + threadIdx.x;
    uint32_t a = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) a = max(a, p[w * 128]);
    const int e = scale_exponent(__uint_as_float(a));
    reinterpret_cast<float*>(cinv)[threadIdx.x] = pow2f(-e);
    store_scale_byte(sfc + (int64_t)(rb >> 2) * cols + (int64_t)kb * 128 + threadIdx.x, rb, rb == rblocks - 1,
                     (uint32_t)(e + 127));
  }
  __syncthreads();
  const float4 inv = cinv[lane];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint32_t*>(qc + (row0 + i) * cols + col) =
        e4m3x4(v[i][0] * inv.x, v[i][1] * inv.y, v[i][2] * inv.z, v[i][3] * inv.w);
}

}  // namespace

cudaError_t save_rows_launch(const void* x, void* q, void* sf, int64_t groups, int64_t rows,
                             int64_t cols, bool pdl, cudaStream_t stream) {
  const int kblocks = (int)(cols / 128), kpacks = (kblocks + 3) / 4;
  const int64_t rows_pad = (rows + 3) / 4 * 4;
  const int64_t blocks = (groups * rows_pad * kpacks + 7) / 8;
  return launch_op(save_rows_kernel, dim3((unsigned)blocks), 256, 0, pdl, stream,
                   (const __nv_bfloat16*)x, (uint8_t*)q, (uint32_t*)sf, groups, rows, rows_pad, cols,
                   kblocks, kpacks);
}

cudaError_t restore_rows_launch(const void* q, const void* sf, void* x, int dtype, int64_t groups,
                                int64_t rows, int64_t cols, bool pdl, cudaStream_t stream) {
  const int kblocks = (int)(cols / 128), kpacks = (kblocks + 3) / 4;
  const int64_t rows_pad = (rows + 3) / 4 * 4;
  const dim3 grid((unsigned)((groups * rows * kpacks + 7) / 8));
  if (dtype == DG_DTYPE_FP32)
    return launch_op(restore_rows_kernel<float>, grid, 256, 0, pdl, stream, (const uint8_t*)q,
                     (const uint32_t*)sf, (float*)x, groups, rows, rows_pad, cols, kblocks, kpacks);
  return launch_op(restore_rows_kernel<__nv_bfloat16>, grid, 256, 0, pdl, stream, (const uint8_t*)q,
                   (const uint32_t*)sf, (__nv_bfloat16*)x, groups, rows, rows_pad, cols, kblocks, kpacks);
}

cudaError_t use_cols_launch(const void* q, const void* sf, const int32_t* m_indices, void* qc,
                            void* sfc, int64_t rows, int64_t cols, bool pdl, cudaStream_t stream) {
  const int rblocks = (int)((rows + 127) / 128);
  return launch_op(use_cols_kernel, dim3((unsigned)(cols / 128 * rblocks)), 512, 0, pdl, stream,
                   (const uint8_t*)q, (const uint32_t*)sf, m_indices, (uint8_t*)qc, (uint32_t*)sfc, rows,
                   (rows + 3) / 4 * 4, cols, rblocks);
}

}  // namespace dg
