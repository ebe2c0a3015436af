// Product of 8-bit integers for a few tokens: D = c + sa sb (a b^T).
//
// Bound by reading b once: its rows go through the tensor cores 16 at a time
// with all tokens, 128 columns a stage, by asynchronous copies through the warp's own
// ring in shared memory; several warps share the columns of 16 rows and join their
// sums in shared memory in a fixed order.  A code is exact as
// a half, so is every product in FP32.  Up to 32 tokens: mma.sync with its columns of
// 8 tokens takes what there is, where a tile of tcgen05 would spend 128 lanes or
// a cluster's joining of sums on them.  One token, 7168 x 2048: 7.3 us in a graph, 2.0
// TB/s (2.2 us at the copy's rate; a launch and the first loads' latency are 5).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "int8_gemm.h"
#include "stream_mma.cuh"

namespace dg {
namespace {

constexpr int kIsWarps = 16;
constexpr int kIsThreads = 32 * kIsWarps;
constexpr int kStreamCols = 128;             // columns of a stage
constexpr int kIsStage = 16 * kStreamCols;
constexpr int is_ring(int nb) { return nb <= 2 ? 6 : 4; }
constexpr size_t is_smem(int nb) { return (size_t)kIsWarps * (is_ring(nb) * kIsStage + nb * 512); }

// Which 4 columns of the 128 a lane holds for a product is free as long as b and a
// agree.  Lane (r, q) = (lane / 4, lane % 4) takes, of rows r and r + 8, the 16 bytes
// at columns 16 q and at 64 + 16 q: whole 64-byte pieces a row and instruction.
// Product j (0..7) multiplies columns 64 (j / 4) + 16 q + 4 (j % 4) + 0..3 of every q.
//
// The lane's codes of half a stage (h = 0, 1: 64 columns), decoded: a[i] are the A
// registers of product 4 h + i.
__device__ __forceinline__ void stream_decode(const uint8_t* stage, int h, int lane, uint32_t (&a)[4][4]) {
  const uint4 g = *reinterpret_cast<const uint4*>(stage + h * 1024 + lane * 16);
  const uint4 u = *reinterpret_cast<const uint4*>(stage + h * 1024 + 512 + lane * 16);
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    DecodeInt8::four(gw[i], a[i][0], a[i][2]);
    DecodeInt8::four(uw[i], a[i][1], a[i][3]);
  }
}

template <int NB>
__global__ void __launch_bounds__(kIsThreads, 1) int8_stream_kernel(const Int8Args p, const int split) {
  constexpr int RING = is_ring(NB);
  extern __shared__ uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q = lane & 3;
  uint8_t* const ring = smem + warp * RING * kIsStage;
  float4* const exchange = reinterpret_cast<float4*>(smem + kIsWarps * RING * kIsStage) + lane;  // [warp][NB][lane]
  griddep_wait();
  griddep_launch_dependents();

  const int chunks = (p.k + kStreamCols - 1) / kStreamCols, units = (p.n + 15) / 16;
  const int groups = kIsWarps / split, group = warp / split, rank = warp % split;
  const int c0 = (int)((int64_t)chunks * rank / split), c1 = (int)((int64_t)chunks * (rank + 1) / split);
  const int begin = blockIdx.x + gridDim.x * group, step = gridDim.x * groups;

  int put = 0, stage = 0;
  int ahead = c0 < c1 ? begin : units, ac = c0;
  const int8_t *g = p.b, *u = p.b;
  bool g_on = false, u_on = false;
  auto aim = [&]() {
    const int row = ahead * 16 + r;
    g_on = ahead < units && row < p.n;
    u_on = ahead < units && row + 8 < p.n;
    g = p.b + (int64_t)(g_on ? row : 0) * p.ldb;
    u = p.b + (int64_t)(u_on ? row + 8 : 0) * p.ldb;
  };
  aim();
  auto next = [&]() {
    if (ahead < units) {
      uint8_t* to = ring + put * kIsStage + lane * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = ac * kStreamCols + h * 64 + q * 16;
        const bool in = k < p.k;
        cp_async16_or_zero(to + h * 1024, g + (in ? k : 0), in && g_on);
        cp_async16_or_zero(to + h * 1024 + 512, u + (in ? k : 0), in && u_on);
      }
      put = put + 1 == RING ? 0 : put + 1;
      if (++ac == c1) {
        ac = c0;
        ahead += step;
        aim();
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < RING - 1; ++i) next();

  for (int unit = begin; unit < units; unit += step) {
    float acc[NB][4] = {};
    for (int c = c0; c < c1; ++c) {
      next();
      uint4 x[NB <= 2 ? NB : 1][2];  // the tokens' codes, on their way while b's are waited for
      auto tokens = [&](int nb, uint4 (&to)[2]) {
        const int n = nb * 8 + r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = c * kStreamCols + h * 64 + q * 16;
          to[h] = n < p.m && k < p.k ? __ldg(reinterpret_cast<const uint4*>(p.a + (int64_t)n * p.lda + k))
                                     : make_uint4(0, 0, 0, 0);
        }
      };
      if constexpr (NB <= 2)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) tokens(nb, x[nb]);
      cp_async_wait<RING - 1>();
      const uint8_t* at = ring + stage * kIsStage;
      stage = stage + 1 == RING ? 0 : stage + 1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[4][4];
        stream_decode(at, h, lane, w);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (NB > 2) tokens(nb, x[0]);
          const uint4 xs = x[NB <= 2 ? nb : 0][h];
          const uint32_t xw[4] = {xs.x, xs.y, xs.z, xs.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            DecodeInt8::four(xw[i], b0, b1);
            mma_f16(acc[nb], w[i], b0, b1);
          }
        }
      }
    }
    if (split > 1) {
      if (rank)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          exchange[(warp * NB + nb) * 32] = make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * split) : "memory");
      if (rank == 0)
        for (int i = 1; i < split; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float4 v = exchange[((warp + i) * NB + nb) * 32];
            acc[nb][0] += v.x;
            acc[nb][1] += v.y;
            acc[nb][2] += v.z;
            acc[nb][3] += v.w;
          }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * split) : "memory");
    }
    if (rank == 0) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = nb * 8 + 2 * q + (i & 1), n = unit * 16 + r + 8 * (i >> 1);
          if (m < p.m && n < p.n) {
            float v = acc[nb][i] * __ldg(p.sa + m);
            const float s = __ldg(p.sb + n);
            const int64_t at = (int64_t)m * p.ldd + n, from = (int64_t)m * p.ldc + n;
            if (p.fp16) {
              v = p.c ? fmaf(v, s, __half2float(static_cast<const __half*>(p.c)[from])) : v * s;
              static_cast<__half*>(p.d)[at] = __float2half_rn(v);
            } else {
              v = p.c ? fmaf(v, s, __bfloat162float(static_cast<const __nv_bfloat16*>(p.c)[from])) : v * s;
              static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16_rn(v);
            }
          }
        }
    }
  }
  cp_async_wait<0>();
}

template <int NB>
cudaError_t is_launch(const Int8Args& p, bool pdl, cudaStream_t stream) {
  cudaError_t e = set_smem(int8_stream_kernel<NB>, is_smem(NB), is_smem(NB));
  if (e != cudaSuccess) return e;
  const int units = (p.n + 15) / 16, chunks = (p.k + kStreamCols - 1) / kStreamCols;
  // warps that share 16 rows: as many as keep all warps of the device busy
  int split = 1;
  while (split < kIsWarps && (int64_t)units * split * 2 <= (int64_t)p.sms * kIsWarps && split < chunks) split *= 2;
  const int grid = std::min(units, p.sms);
  return launch_op(int8_stream_kernel<NB>, dim3((unsigned)grid), kIsThreads, is_smem(NB), pdl, stream, p, split);
}

}  // namespace

// Measured against the kernel with swapped operand roles (us in a graph, weights
// from HBM, this kernel / that one): 4096 x 7168 (256 units of 16 rows): 8 tokens
// 11.9 / 18.9, 32 17.2 / 19.6, 64 26.6 / 20.3; 7168 x 2048: 32 tokens 11.0 / 14.5,
// 64 17.5 / 15.8; 1001 x 1552: 32 tokens 6.1 / 7.0, 64 9.9 / 7.6; 24576 x 1536: 32
// tokens 19.0 / 34.2, 64 34.0 / 37.5.
bool int8_stream_takes(const Int8Args& p) { return p.m <= 32; }

cudaError_t int8_stream_launch(const Int8Args& p, bool pdl, cudaStream_t stream) {
  if (p.m <= 8) return is_launch<1>(p, pdl, stream);
  if (p.m <= 16) return is_launch<2>(p, pdl, stream);
  return is_launch<4>(p, pdl, stream);
}

}  // namespace dg
