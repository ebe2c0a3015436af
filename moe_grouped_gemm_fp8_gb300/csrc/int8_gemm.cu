// Product of 8-bit integers in tiles on the tensor cores: D = c + sa sb (a b^T).
//
// sm_103a's tcgen05 has no integer kind, but an 8-bit integer is a half exactly
// and so is a product of two in FP32: kind::f16, at its rate, gives what integer
// products would (sums past 2^24 round as FP32 sums do, far below the result's
// 16 bits).  Nothing is widened in memory: warps load the codes, turn them into
// halves in registers (1024 + 128 + c is a half whose low byte is c + 128; an
// addition takes the offset away: 5 instructions for 4 codes) and store them
// where the MMA reads them, in its 128-byte swizzle.
//
// One persistent CTA per SM, 16 warps: 0 issues the MMAs, 4-7 scale and store a
// tile's results from TMEM while the next tile's MMAs run (two accumulators),
// 8-15 load and widen.  Loads are two stages ahead in registers, so that the
// wait for a free stage does not put their latency into the chain.
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

constexpr int kIgThreads = 512;
constexpr int kIgProducers = 256;  // warps 8-15
constexpr int kIgStages = 4;
constexpr int kIgK = 64;  // columns of a stage: 128 bytes of halves
constexpr int kIgBand = 16;  // row blocks of a band of tiles

// FP32 D (bits 4-5 = 1), FP16 A and B (format 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int BN>
constexpr int ig_stage_bytes() { return (128 + BN) * 128; }
template <int BN>
constexpr size_t ig_smem() { return 1024 + (size_t)kIgStages * ig_stage_bytes<BN>() + 4 * 128 + 256; }

// Row block and column block of tile t: bands of kIgBand row blocks, in each
// the column blocks one after another, so that the CTAs at work share both.
__device__ __forceinline__ void ig_tile(int t, int mb_all, int nb_all, int& mb, int& nb) {
  const int band = t / (kIgBand * nb_all), first = band * kIgBand;
  const int height = min(kIgBand, mb_all - first), in = t - band * kIgBand * nb_all;
  nb = in / height;
  mb = first + in - nb * height;
}

// 16 codes at the 16-byte chunks 2 q and 2 q + 1 of a row of 128 bytes of halves.
__device__ __forceinline__ void ig_widen(uint32_t tile, int row, int q, const uint4& c) {
  uint32_t h[8];
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) DecodeInt8::four(w[i], h[2 * i], h[2 * i + 1]);
  const uint32_t line = tile + row * 128, x = row & 7;
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + (((2 * q) ^ x) << 4)), "r"(h[0]), "r"(h[1]),
               "r"(h[2]), "r"(h[3])
               : "memory");
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + (((2 * q + 1) ^ x) << 4)), "r"(h[4]), "r"(h[5]),
               "r"(h[6]), "r"(h[7])
               : "memory");
}

template <int BN>
__global__ void __launch_bounds__(kIgThreads, 1) int8_gemm_kernel(const Int8Args p) {
  constexpr int STAGES = kIgStages, STAGE = ig_stage_bytes<BN>();
  constexpr int NA = 2, NBP = BN / 64, NP = NA + NBP;  // 16-byte pieces of a producer thread
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const after = smem_raw + (base - smem_u32(smem_raw)) + STAGES * STAGE;
  float* const sb_row = reinterpret_cast<float*>(after);  // [4 warps][32]
  uint64_t* const bars = reinterpret_cast<uint64_t*>(after + 4 * 128);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + STAGES + s); };
  auto tfull = [&](int s) { return smem_u32(bars + 2 * STAGES + s); };
  auto tempty = [&](int s) { return smem_u32(bars + 2 * STAGES + 2 + s); };
  const uint32_t drain = smem_u32(bars + 2 * STAGES + 4);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kCols = 2 * BN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), kIgProducers / 32);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kCols);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();

  const int mb_all = (p.m + 127) / 128, nb_all = (p.n + BN - 1) / BN, tiles = mb_all * nb_all;
  const int kbs = (p.k + kIgK - 1) / kIgK;
  const uint64_t tmo = p.timeout_ns;

  if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0, pass = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++pass) {
        const uint32_t buf = pass & 1u;
        if (!wait_bounded(tempty(buf), ((pass >> 1) & 1u) ^ 1u, abort_flag, tmo, p.err, kSiteMmaTmemEmpty)) break;
        tc_fence_after();
        for (int kb = 0; kb < kbs; ++kb) {
          if (!wait_bounded(full(s), phase, abort_flag, tmo, p.err, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = smem_desc_kmajor_sw128(base + s * STAGE);
          const uint64_t bd = smem_desc_kmajor_sw128(base + s * STAGE + 16384);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma_f16(tmem + buf * BN, ad + 2 * j, bd + 2 * j, idesc_f16(128, BN), kb != 0 || j != 0);
          tc_commit(empty(s));
          if (++s == STAGES) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit(tfull(buf));
      }
      // the MMAs in flight end before the memory they use is given back
      tc_commit(drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0))
        if (global_timer_ns() - t0 > tmo) {
          record_error(p.err, DG_ERR_DEVICE_TIMEOUT, kSiteDrain);
          break;
        }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ load and widen
    const int pt = threadIdx.x - (kIgThreads - kIgProducers), row = pt >> 2, q = pt & 3;
    const int8_t* src[NP];
    uint32_t on = 0;  // bit i: piece i's row exists
    int lt = blockIdx.x, lk = 0;
    auto aim = [&]() {
      on = 0;
      if (lt >= tiles) return;
      int mb, nb;
      ig_tile(lt, mb_all, nb_all, mb, nb);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int rr = i < NA ? mb * 128 + i * 64 + row : nb * BN + (i - NA) * 64 + row;
        const bool in = rr < (i < NA ? p.m : p.n);
        on |= (uint32_t)in << i;
        src[i] = (i < NA ? p.a : p.b) + (int64_t)(in ? rr : 0) * (i < NA ? p.lda : p.ldb) + q * 16;
      }
    };
    auto load = [&](uint4 (&v)[NP]) {
      const int k = lk * kIgK;
      const bool in = k + q * 16 < p.k;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        v[i] = in && (on >> i & 1u) ? __ldg(reinterpret_cast<const uint4*>(src[i] + k)) : make_uint4(0, 0, 0, 0);
      if (++lk == kbs) {
        lk = 0;
        lt += gridDim.x;
        aim();
      }
    };
    aim();
    uint4 v[2][NP];
    load(v[0]);
    load(v[1]);
    const int mine = (int)blockIdx.x < tiles ? (tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    const int64_t stages = (int64_t)mine * kbs;
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t it = 0; it < stages && ok; it += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (it + h >= stages || !ok) break;
        if (!wait_bounded(empty(s), phase ^ 1u, abort_flag, tmo, p.err, kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        const uint32_t at = base + s * STAGE;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          ig_widen(i < NA ? at : at + 16384, (i < NA ? i : i - NA) * 64 + row, q, v[h][i]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(s));
        load(v[h]);
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scale and store
    const int quarter = warp & 3;
    float* const sbw = sb_row + quarter * 32;
    uint32_t pass = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++pass) {
      int mb, nb;
      ig_tile(t, mb_all, nb_all, mb, nb);
      const uint32_t buf = pass & 1u;
      const int m = mb * 128 + quarter * 32 + lane;
      const float sa = m < p.m ? __ldg(p.sa + m) : 0.0f;
      if (!wait_bounded(tfull(buf), (pass >> 1) & 1u, abort_flag, tmo, p.err, kSiteEpilogueTmemFull)) break;
      tc_fence_after();
      for (int ch = 0; ch < BN / 32; ++ch) {
        const int n0 = nb * BN + ch * 32;
        uint32_t acc[32];
        tc_ld_32x32b_x32(tmem + buf * BN + ch * 32 + ((uint32_t)(quarter * 32) << 16), acc);
        __syncwarp();  // the last chunk's scales are read
        sbw[lane] = n0 + lane < p.n ? __ldg(p.sb + n0 + lane) : 0.0f;
        __syncwarp();
        tc_wait_ld_regs(acc);
        if (ch == BN / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty(buf));
        }
        if (m >= p.m || n0 >= p.n) continue;
        const int64_t at = (int64_t)m * p.ldd + n0, from = (int64_t)m * p.ldc + n0;
        if (p.vector && n0 + 32 <= p.n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 cw = make_uint4(0, 0, 0, 0);
            if (p.c) cw = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.c) + from)[i];  // c may be d
            const uint32_t ci[4] = {cw.x, cw.y, cw.z, cw.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 s = *reinterpret_cast<const float2*>(sbw + i * 8 + j * 2);
              float2 cf = make_float2(0.0f, 0.0f);
              if (p.c)
                cf = p.fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&ci[j]))
                            : make_float2(bf16_lo(ci[j]), bf16_hi(ci[j]));
              const float x = fmaf(__uint_as_float(acc[i * 8 + j * 2]) * sa, s.x, cf.x);
              const float y = fmaf(__uint_as_float(acc[i * 8 + j * 2 + 1]) * sa, s.y, cf.y);
              if (p.fp16) {
                const __half2 v = __floats2half2_rn(x, y);
                o[j] = *reinterpret_cast<const uint32_t*>(&v);
              } else {
                o[j] = bf16x2_bits(x, y);
              }
            }
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.d) + at)[i] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (n0 + i < p.n) {
              float v = __uint_as_float(acc[i]) * sa;
              if (p.fp16) {
                v = fmaf(v, sbw[i], p.c ? __half2float(static_cast<const __half*>(p.c)[from + i]) : 0.0f);
                static_cast<__half*>(p.d)[at + i] = __float2half_rn(v);
              } else {
                v = fmaf(v, sbw[i], p.c ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.c)[from + i]) : 0.0f);
                static_cast<__nv_bfloat16*>(p.d)[at + i] = __float2bfloat16_rn(v);
              }
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <int BN>
cudaError_t ig_launch(const Int8Args& p, bool pdl, cudaStream_t stream) {
  cudaError_t e = set_smem(int8_gemm_kernel<BN>, ig_smem<BN>(), ig_smem<BN>());
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((p.m + 127) / 128) * ((p.n + BN - 1) / BN);
  return launch_op(int8_gemm_kernel<BN>, dim3((unsigned)std::min<int64_t>(tiles, p.sms)), kIgThreads, ig_smem<BN>(), pdl,
                   stream, p);
}

}  // namespace

cudaError_t int8_gemm_launch(Int8Args p, bool pdl, cudaStream_t stream) {
  cudaError_t e = error_word_address(&p.err);
  if (e != cudaSuccess) return e;
  const int64_t mb = (p.m + 127) / 128;
  if (mb * ((p.n + 255) / 256) >= p.sms) return ig_launch<256>(p, pdl, stream);
  if (mb * ((p.n + 127) / 128) >= p.sms) return ig_launch<128>(p, pdl, stream);
  return ig_launch<64>(p, pdl, stream);
}

}  // namespace dg
