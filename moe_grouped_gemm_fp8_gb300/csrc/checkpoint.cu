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

#include <algorithm>

#include "dg_device.cuh"
#include "dg_ops.cuh"

namespace dg {
namespace {

// One warp per (group, pair of rows, 512-column pack), lane l on columns 16l ..
// 16l+15, so a 128-column group is eight lanes and a scale word one store; warps
// ordered row-fastest so that the scale words of neighbouring warps are adjacent.
// Both rows' loads are in flight together: 16384 x 7168 in 56 us (6.3 TB/s), 4096
// x 7168 in 12.5, where a row a warp took 17.9.
__global__ void __launch_bounds__(256) save_rows_kernel(const __nv_bfloat16* __restrict__ x,
                                                        uint8_t* __restrict__ q,
                                                        uint32_t* __restrict__ sf, int64_t groups,
                                                        int64_t rows, int64_t rows_pad,
                                                        int64_t cols, int kpacks) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int64_t pairs = rows_pad / 2;
  if (w >= groups * pairs * kpacks) return;
  const int64_t r0 = w % pairs * 2;
  const int64_t j = (w / pairs) % kpacks;
  const int64_t g = w / (pairs * kpacks);
  const int64_t c = j * 512 + lane * 16;
  const int64_t at = (g * rows + r0) * cols + c;
  uint4 v[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (r0 + i < rows && c < cols) {
      v[i][0] = ld_stream_u4(x + at + i * cols);
      v[i][1] = ld_stream_u4(x + at + i * cols + 8);
    }
  }
  uint32_t word[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t raw[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    float2 f[8];
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = make_float2(bf16_lo(raw[k]), bf16_hi(raw[k]));
      m = abs_max2(m, f[k]);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t e = scale_byte(m);
    const bool in = r0 + i < rows && c < cols;
    if (in) {
      const float inv = inverse_of_byte(e);
      *reinterpret_cast<uint4*>(q + at + i * cols) =
          make_uint4(e4m3x4(mul2(f[0], inv), mul2(f[1], inv)), e4m3x4(mul2(f[2], inv), mul2(f[3], inv)),
                     e4m3x4(mul2(f[4], inv), mul2(f[5], inv)), e4m3x4(mul2(f[6], inv), mul2(f[7], inv)));
    }
    word[i] = __reduce_or_sync(0xffffffffu, in ? e << (8 * (lane / 8)) : 0u);
  }
  if (lane == 0) *reinterpret_cast<uint2*>(sf + (g * kpacks + j) * rows_pad + r0) = make_uint2(word[0], word[1]);
}

// One warp per (group, four rows, 512-column pack), lane l on columns 16l .. 16l+15
// of each row: 16 bytes of codes in, 32 or 64 of values out, all four rows' loads
// in flight together.  16384 x 7168 to BF16 in 55.5 us (6.3 TB/s), to
// FP32 in 90 (6.5 TB/s); a row a warp, four codes a lane at a time, took 89 and 115.
template <class OUT>
__global__ void __launch_bounds__(256) restore_rows_kernel(const uint8_t* __restrict__ q,
                                                           const uint32_t* __restrict__ sf,
                                                           OUT* __restrict__ x, int64_t groups,
                                                           int64_t rows, int64_t rows_pad,
                                                           int64_t cols, int kpacks, bool wide) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int64_t quads = rows_pad / 4;
  if (w >= groups * quads * kpacks) return;
  const int64_t r0 = w % quads * 4;
  const int64_t j = (w / quads) % kpacks;
  const int64_t g = w / (quads * kpacks);
  const int64_t c = j * 512 + lane * 16;
  if (c >= cols) return;
  const int64_t at = (g * rows + r0) * cols + c;
  const uint4 words = __ldg(reinterpret_cast<const uint4*>(sf + (g * kpacks + j) * rows_pad + r0));
  const uint32_t word[4] = {words.x, words.y, words.z, words.w};
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i < rows) v[i] = ld_stream_u4(q + at + i * cols);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (r0 + i >= rows) break;
    const float s = scale_of_byte((word[i] >> (8 * (lane / 8))) & 0xFFu);
    const uint32_t codes[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint4 out[sizeof(OUT)];  // 16 values
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float f[4];
      e4m3x4_to_float(codes[t], f);
      if constexpr (sizeof(OUT) == 4) {
        out[t] = make_uint4(__float_as_uint(f[0] * s), __float_as_uint(f[1] * s), __float_as_uint(f[2] * s),
                            __float_as_uint(f[3] * s));
      } else {
        const uint32_t lo = bf16x2_bits(f[0] * s, f[1] * s), hi = bf16x2_bits(f[2] * s, f[3] * s);
        if (t % 2) out[t / 2].z = lo, out[t / 2].w = hi;
        else out[t / 2].x = lo, out[t / 2].y = hi;
      }
    }
    OUT* dst = x + at + i * cols;
#pragma unroll
    for (int t = 0; t < (int)sizeof(OUT); t += 2) {
      uint4* to = reinterpret_cast<uint4*>(dst) + t;
      if (wide) {
        st_global_32(to, out[t], out[t + 1]);
      } else {
        to[0] = out[t];
        to[1] = out[t + 1];
      }
    }
  }
}

// Persistent CTAs of 4 warps, kUseCtas a SM, over 128 x 128 tiles.  Warp w
// holds rows 32w .. 32w+31: lane l columns 16 (l % 8) .. +15 (one 16-byte
// access) of rows 4i + l / 8.  The next tile is on its way into shared
// memory while one is worked on (rows that count as zero are filled with zeros
// instead of being read).  The codes are read from there and decoded twice, for
// the columns' maxima and to encode them; where the exponents allow it the
// arithmetic is exact in pairs of halves, half as many instructions as in FP32
// (21k x 7168 with routed rows in 53.6 us, 5.6 TB/s; in FP32 alone 68).  Six CTAs
// with one tile on its way each do better than four with two (57.5 us).
constexpr int kUseRing = 2;
constexpr int kUseCtas = 6;

struct UseShared {
  uint4 codes[kUseRing][8][128];
  uint32_t words[kUseRing][128];  // the rows' scale words
  float cmax[4][128];
  int cexp[128];                  // the columns' exponents
};

__global__ void __launch_bounds__(128, kUseCtas) use_cols_kernel(const uint8_t* __restrict__ q,
                                                          const uint32_t* __restrict__ sf,
                                                          const int32_t* __restrict__ m_indices,
                                                          uint8_t* __restrict__ qc,
                                                          uint32_t* __restrict__ sfc, int64_t rows,
                                                          int64_t rows_pad, int64_t cols, int kblocks,
                                                          int rblocks) {
  extern __shared__ uint4 smem[];
  UseShared& sh = *reinterpret_cast<UseShared*>(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int tiles = kblocks * rblocks;
  // m_indices of the lane's row of tile t, negative where it counts as zero;
  // loaded a round before the fetch that needs it.
  auto row_index = [&](const TileWalk& w) {
    int index = -1;
    if (w.t < tiles) {
      const int64_t row = (int64_t)w.rb * 128 + warp * 32 + lane;
      if (row < rows) index = m_indices ? __ldg(m_indices + row) : 0;
    }
    return index;
  };
  // live: which of the warp's 32 rows hold data, bit l for row 32 warp + l.
  auto fetch = [&](const TileWalk& w, int s, int index, uint32_t& live) {
    const bool in = index >= 0;
    live = __ballot_sync(0xffffffffu, in);
    if (w.t < tiles) {
      const int rb = w.rb, kb = w.cb;
      const int64_t row = (int64_t)rb * 128 + warp * 32 + lane;
      cp_async4_or_zero(&sh.words[s][tid], in ? sf + (int64_t)(kb >> 2) * rows_pad + row : sf, in);
      const uint8_t* src = q + ((int64_t)rb * 128 + warp * 32 + lane / 8) * cols + (int64_t)kb * 128 + (lane % 8) * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool on = live >> (4 * i + lane / 8) & 1;
        cp_async16_or_zero(&sh.codes[s][i][tid], on ? src : q, on);
        src += 4 * cols;
      }
    }
    cp_async_commit();
  };
  uint32_t live[kUseRing];
  const int drb = gridDim.x / kblocks, dcb = gridDim.x % kblocks;
  TileWalk now, ahead;  // the tile worked on; the tile whose rows are looked up next
  now.init(blockIdx.x, kblocks);
  ahead = now;
#pragma unroll
  for (int s = 0; s < kUseRing - 1; ++s) {
    fetch(ahead, s, row_index(ahead), live[s]);
    ahead.next(kblocks, drb, dcb);
  }
  int index = row_index(ahead);
  int at = 0;
  for (; now.t < tiles; now.next(kblocks, drb, dcb)) {
    const int rb = now.rb, kb = now.cb;
    fetch(ahead, at == 0 ? kUseRing - 1 : at - 1, index, live[kUseRing - 1]);
    ahead.next(kblocks, drb, dcb);
    index = row_index(ahead);
    cp_async_wait<kUseRing - 1>();
    __syncwarp();  // a warp's scale words are copied by its own lanes
    // The warp's rows' exponents, one a lane, and their largest.
    const uint32_t wd = sh.words[at][tid];
    const bool on = live[0] >> lane & 1;
    const int e_row = on ? (int)((wd >> (8 * (kb & 3))) & 0xFFu) - 127 : -1000;
    const int e_max = __reduce_max_sync(0xffffffffu, e_row), e_min = __reduce_min_sync(0xffffffffu, on ? e_row : 1000);
    const int e_ref = live[0] ? e_max : 0;
    // Values relative to 2^e_ref are exact halves while the rows' exponents lie
    // within 15 of one another: 4 significant bits from 2^-9 2^-15 to 448.
    const bool halves = !live[0] || e_max - e_min <= 15;
    float m[16];
    if (halves) {
      __half2 mh[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) mh[c] = __half2half2(__ushort_as_half(0));
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {
        const uint4 ci = sh.codes[at][i][tid];
        const __half2 f = half_pow2(__shfl_sync(0xffffffffu, e_row, 4 * i + lane / 8) - e_ref);
        const uint32_t w[4] = {ci.x, ci.y, ci.z, ci.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          __half2 lo, hi;
          e4m3x4_to_half(w[c], lo, hi);
          mh[2 * c] = __hmax2(mh[2 * c], __habs2(__hmul2(lo, f)));
          mh[2 * c + 1] = __hmax2(mh[2 * c + 1], __habs2(__hmul2(hi, f)));
        }
      }
      const float ref = pow2f(e_ref);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        mh[c] = __hmax2(mh[c], __shfl_xor_sync(0xffffffffu, mh[c], 8));
        mh[c] = __hmax2(mh[c], __shfl_xor_sync(0xffffffffu, mh[c], 16));
        const float2 v = __half22float2(mh[c]);
        m[2 * c] = v.x * ref;
        m[2 * c + 1] = v.y * ref;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) m[c] = 0.0f;
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const uint4 ci = sh.codes[at][i][tid];
        const int e = __shfl_sync(0xffffffffu, e_row, 4 * i + lane / 8);
        const float s = e >= -127 ? pow2f(e) : 0.0f;
        const uint32_t w[4] = {ci.x, ci.y, ci.z, ci.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float f[4];
          e4m3x4_to_float(w[c], f);
#pragma unroll
          for (int k = 0; k < 4; ++k) m[4 * c + k] = fmaxf(m[4 * c + k], fabsf(f[k] * s));
        }
      }
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        m[c] = fmaxf(m[c], __shfl_xor_sync(0xffffffffu, m[c], 8));
        m[c] = fmaxf(m[c], __shfl_xor_sync(0xffffffffu, m[c], 16));
      }
    }
    if (lane < 8) {
#pragma unroll
      for (int c = 0; c < 16; c += 4)
        *reinterpret_cast<float4*>(&sh.cmax[warp][lane * 16 + c]) = make_float4(m[c], m[c + 1], m[c + 2], m[c + 3]);
    }
    __syncthreads();
    {
      const float a = fmaxf(fmaxf(sh.cmax[0][tid], sh.cmax[1][tid]), fmaxf(sh.cmax[2][tid], sh.cmax[3][tid]));
      const uint32_t b = scale_byte(a);
      sh.cexp[tid] = (int)b - 127;
      store_scale_byte(sfc + (int64_t)(rb >> 2) * cols + (int64_t)kb * 128 + tid, rb, rb == rblocks - 1, b);
    }
    __syncthreads();
    int e_col[16];
    int least = 1000;
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
      const int4 x = *reinterpret_cast<const int4*>(&sh.cexp[(lane % 8) * 16 + c]);
      e_col[c] = x.x;
      e_col[c + 1] = x.y;
      e_col[c + 2] = x.z;
      e_col[c + 3] = x.w;
      least = min(min(least, min(x.x, x.y)), min(x.z, x.w));
    }
    uint8_t* dst = qc + ((int64_t)rb * 128 + warp * 32 + lane / 8) * cols + (int64_t)kb * 128 + (lane % 8) * 16;
    // A column's factor 2^(e_ref - e_col) is a half up to 2^15.  Below 2^-24 it
    // becomes 0, as its products, at most 448 2^-25, do in E4M3; and a product
    // that still reaches a code (2^-10) has all its bits above 2^-24.
    if (halves && __all_sync(0xffffffffu, e_ref - least <= 15)) {
      __half2 f2[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        f2[c] = __halves2half2(__low2half(half_pow2(e_ref - e_col[2 * c])), __low2half(half_pow2(e_ref - e_col[2 * c + 1])));
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {
        const uint4 ci = sh.codes[at][i][tid];
        const __half2 f = half_pow2(__shfl_sync(0xffffffffu, e_row, 4 * i + lane / 8) - e_ref);
        uint32_t w[4] = {ci.x, ci.y, ci.z, ci.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          __half2 lo, hi;
          e4m3x4_to_half(w[c], lo, hi);
          w[c] = half_to_e4m3x4(__hmul2(__hmul2(lo, f), f2[2 * c]), __hmul2(__hmul2(hi, f), f2[2 * c + 1]));
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        dst += 4 * cols;
      }
    } else {
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const uint4 ci = sh.codes[at][i][tid];
        const int e = __shfl_sync(0xffffffffu, e_row, 4 * i + lane / 8);
        const float s = e >= -127 ? pow2f(e) : 0.0f;
        uint32_t w[4] = {ci.x, ci.y, ci.z, ci.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float f[4];
          e4m3x4_to_float(w[c], f);
          w[c] = e4m3x4(f[0] * s * pow2f(-e_col[4 * c]), f[1] * s * pow2f(-e_col[4 * c + 1]),
                        f[2] * s * pow2f(-e_col[4 * c + 2]), f[3] * s * pow2f(-e_col[4 * c + 3]));
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        dst += 4 * cols;
      }
    }
    __syncwarp();  // every lane has read its words before the slot is filled again
    if (++at == kUseRing) at = 0;
#pragma unroll
    for (int k = 0; k < kUseRing - 1; ++k) live[k] = live[k + 1];
  }
  cp_async_wait<0>();
}

}  // namespace

cudaError_t save_rows_launch(const void* x, void* q, void* sf, int64_t groups, int64_t rows,
                             int64_t cols, bool pdl, cudaStream_t stream) {
  const int kpacks = (int)((cols + 511) / 512);
  const int64_t rows_pad = (rows + 3) / 4 * 4;
  const int64_t blocks = (groups * (rows_pad / 2) * kpacks + 7) / 8;
  return launch_op(save_rows_kernel, dim3((unsigned)blocks), 256, 0, pdl, stream,
                   (const __nv_bfloat16*)x, (uint8_t*)q, (uint32_t*)sf, groups, rows, rows_pad, cols, kpacks);
}

cudaError_t restore_rows_launch(const void* q, const void* sf, void* x, int dtype, int64_t groups,
                                int64_t rows, int64_t cols, bool pdl, cudaStream_t stream) {
  const int kpacks = (int)((cols + 511) / 512);
  const int64_t rows_pad = (rows + 3) / 4 * 4;
  const dim3 grid((unsigned)((groups * (rows_pad / 4) * kpacks + 7) / 8));
  const bool wide = ((uintptr_t)x & 31) == 0;
  if (dtype == DG_DTYPE_FP32)
    return launch_op(restore_rows_kernel<float>, grid, 256, 0, pdl, stream, (const uint8_t*)q,
                     (const uint32_t*)sf, (float*)x, groups, rows, rows_pad, cols, kpacks, wide);
  return launch_op(restore_rows_kernel<__nv_bfloat16>, grid, 256, 0, pdl, stream, (const uint8_t*)q,
                   (const uint32_t*)sf, (__nv_bfloat16*)x, groups, rows, rows_pad, cols, kpacks, wide);
}

cudaError_t use_cols_launch(const void* q, const void* sf, const int32_t* m_indices, void* qc,
                            void* sfc, int64_t rows, int64_t cols, int sms, bool pdl,
                            cudaStream_t stream) {
  const int rblocks = (int)((rows + 127) / 128), kblocks = (int)(cols / 128);
  const int64_t tiles = (int64_t)rblocks * kblocks;
  const dim3 grid((unsigned)std::min<int64_t>(tiles, (int64_t)kUseCtas * sms));
  cudaError_t e = set_smem(use_cols_kernel, sizeof(UseShared), sizeof(UseShared));
  if (e != cudaSuccess) return e;
  return launch_op(use_cols_kernel, grid, 128, sizeof(UseShared), pdl, stream, (const uint8_t*)q,
                   (const uint32_t*)sf, m_indices, (uint8_t*)qc, (uint32_t*)sfc, rows, (rows + 3) / 4 * 4, cols,
                   kblocks, rblocks);
}

}  // namespace dg
