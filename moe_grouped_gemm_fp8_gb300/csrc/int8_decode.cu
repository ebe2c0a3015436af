// Product of 8-bit integers too small for a tile an SM: D = c + sa sb (a b^T) with
// the operands' roles swapped.
//
// 128 rows of b (channels) take the MMA's 128 lanes and the tokens its columns, so
// that no lane is spent on tokens that do not exist; the columns are split over
// the CTAs of a cluster, whose partial sums meet in shared memory, each
// CTA adding some tokens' in the CTAs' order.  Bound by reading b once and by the
// depth of loads in flight: a CTA has 48 KB of b on its way in registers, and a
// start and an end of 7 us between them are all there is time for.  64 tokens, 4096 x
// 7168: 17.9 us in a graph, 1.75 TB/s (4.6 us at the copy's rate); by tiles of
// int8_gemm.cu 52, by int8_stream.cu's way 29.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "int8_gemm.h"
#include "int8_tile.cuh"

namespace dg {
namespace {

template <int TN>
struct IdPlan {
  static constexpr int kStage = (128 + TN) * 256, kFit = (200 * 1024) / kStage, kStages = kFit > 4 ? 4 : kFit;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 256;
  static constexpr uint32_t kCols = TN < 32 ? 32 : TN;  // of TMEM
  static_assert(TN * 128 * 4 <= kStages * kStage, "the partial sums take the stages' place");
};

template <int TN>
__global__ void __launch_bounds__(kIgThreads, 1) int8_decode_kernel(const Int8Args p, const int split) {
  using Plan = IdPlan<TN>;
  constexpr int STAGES = Plan::kStages, STAGE = Plan::kStage;
  constexpr int kAhead = TN <= 64 ? 3 : 2;  // stages whose loads are in flight in registers
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem_raw + (base - smem_u32(smem_raw)) + STAGES * STAGE);
  float* const part = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)));  // [token][128 channels]
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + STAGES + s); };
  const uint32_t done = smem_u32(bars + 2 * STAGES);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), strip = blockIdx.x / split, m0 = blockIdx.y * TN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), kIgWiden);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), Plan::kCols);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();

  const int all = (p.k + kIgK - 1) / kIgK;
  const int k0 = (int)((int64_t)all * rank / split), kbs = (int)((int64_t)all * (rank + 1) / split) - k0;
  const uint64_t tmo = p.timeout_ns;

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0;
      for (int kb = 0; kb < kbs; ++kb) {
        if (!wait_quick(full(s), phase, abort_flag, tmo, p.err, kSiteMmaFull)) break;
        fence_proxy_async_smem();
        tc_fence_after();
#pragma unroll
        for (int atom = 0; atom < 2; ++atom) {
          const uint64_t ad = smem_desc_kmajor_sw128(base + s * STAGE + atom * 16384);
          const uint64_t bd = smem_desc_kmajor_sw128(base + s * STAGE + 32768 + atom * (TN * 128));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma_f16<false>(tmem, ad + 2 * j, bd + 2 * j, idesc_f16(128, TN), kb != 0 || atom != 0 || j != 0);
        }
        tc_commit(empty(s));
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
      tc_commit(done);
    }
    __syncwarp();
  } else if (warp >= 8) {
    const int q = lane & 3, atom = lane >> 2 & 1, row = (warp - 8) * 4 + (lane >> 3);
    const int col = atom * 64 + q * 16;
    IgRows<128> w;
    IgRows<TN> t;
    w.aim(p.b, p.ldb, strip * 128, p.n, row, col);
    t.aim(p.a, p.lda, m0, p.m, row, col);
    int lk = k0;
    auto load = [&](uint4 (&vw)[IgRows<128>::kPieces], uint4 (&vt)[IgRows<TN>::kPieces]) {
      const int k = lk * kIgK;
      const bool in = lk < k0 + kbs && k + col < p.k;
      w.load(vw, p.ldb, k, in);
      t.load(vt, p.lda, k, in);
      ++lk;
    };
    uint4 vw[kAhead][IgRows<128>::kPieces], vt[kAhead][IgRows<TN>::kPieces];
#pragma unroll
    for (int h = 0; h < kAhead; ++h) load(vw[h], vt[h]);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = 0; kb < kbs && ok; kb += kAhead) {
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        if (kb + h >= kbs || !ok) break;
        if (!wait_quick(empty(s), phase ^ 1u, abort_flag, tmo, p.err, kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        w.store(vw[h], base + s * STAGE, row, atom, q);
        t.store(vt[h], base + s * STAGE + 32768, row, atom, q);
        __syncwarp();
        if (lane == 0) mbar_arrive(full(s));
        load(vw[h], vt[h]);
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
  }
  // Every thread waits for the last MMA: the stages' memory is the partial sums' from here on.
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(done, 0))
    if (global_timer_ns() - t0 > 2 * tmo + 1000000000ull) {
      record_error(p.err, DG_ERR_DEVICE_TIMEOUT, kSiteDrain);
      break;
    }
  __syncthreads();
  if (warp >= 4 && warp < 8) {
    tc_fence_after();
    const int quarter = warp & 3;
#pragma unroll
    for (int ch = 0; ch < (TN + 31) / 32; ++ch) {
      uint32_t acc[32];
      tc_ld_32x32b_x32(tmem + ch * 32 + ((uint32_t)(quarter * 32) << 16), acc);
      tc_wait_ld_regs(acc);
#pragma unroll
      for (int i = 0; i < (TN < 32 ? TN : 32); ++i) part[(ch * 32 + i) * 128 + quarter * 32 + lane] = __uint_as_float(acc[i]);
    }
    tc_fence_before();
  }
  cluster_sync_all();
  const int tokens = TN / split, first = rank * tokens;
  for (int i = threadIdx.x; i < tokens * 128; i += kIgThreads) {
    const int m = m0 + first + (i >> 7), n = strip * 128 + (i & 127);
    if (m >= p.m) break;
    if (n >= p.n) continue;
    const uint32_t at = smem_u32(part + (m - m0) * 128 + (i & 127));
    float v = 0.0f;
    for (int r = 0; r < split; ++r) v += __uint_as_float(ld_shared_cluster_u32(mapa_shared(at, (uint32_t)r)));
    v *= __ldg(p.sa + m);
    const float sb = __ldg(p.sb + n);
    const int64_t to = (int64_t)m * p.ldd + n, from = (int64_t)m * p.ldc + n;
    if (p.fp16)
      static_cast<__half*>(p.d)[to] =
          __float2half_rn(fmaf(v, sb, p.c ? __half2float(static_cast<const __half*>(p.c)[from]) : 0.0f));
    else
      static_cast<__nv_bfloat16*>(p.d)[to] =
          __float2bfloat16_rn(fmaf(v, sb, p.c ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.c)[from]) : 0.0f));
  }
  cluster_sync_all();  // the sums are read before their CTA ends
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, Plan::kCols);
  }
}

template <int TN>
cudaError_t id_launch(const Int8Args& p, int split, bool pdl, cudaStream_t stream) {
  using Plan = IdPlan<TN>;
  cudaError_t e = set_smem(int8_decode_kernel<TN>, Plan::kSmem, Plan::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.n + 127) / 128 * split), (unsigned)((p.m + TN - 1) / TN), 1);
  cfg.blockDim = dim3(kIgThreads, 1, 1);
  cfg.dynamicSmemBytes = Plan::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, int8_decode_kernel<TN>, p, split);
}

// Strips of 128 channels times blocks of 64 or 128 tokens.
int64_t id_units(const Int8Args& p) {
  return (int64_t)((p.n + 127) / 128) * (p.m <= 64 ? 1 : (p.m + 127) / 128);
}
}  // namespace

// Where two CTAs at least share each strip and block of tokens; without, the tiles
// of int8_gemm.cu are as quick or quicker (us in a graph, this kernel / the tiles: 24576 x
// 1536, 64 tokens 37.5 / 32.3, 96 48.6 / 32.6; with two CTAs: 7168 x 2048, 64 tokens
// 15.8 / 19.9; with four: 4096 x 7168, 96 tokens 26.2 / 52.0).
bool int8_decode_takes(const Int8Args& p) { return id_units(p) * 2 <= p.sms; }

cudaError_t int8_decode_launch(Int8Args p, bool pdl, cudaStream_t stream) {
  cudaError_t e = error_word_address(&p.err);
  if (e != cudaSuccess) return e;
  // as many CTAs as the device runs at once; clusters of 8 only up to half of it, so that all find room (17 of them: 64
  // tokens, 2112 x 7168, 21.7 us; with clusters of 4 16.1)
  const int64_t units = id_units(p), kbs = (p.k + kIgK - 1) / kIgK;
  int split = 1;
  while (split < 8 && units * split * 2 <= (split == 4 ? p.sms / 2 : p.sms) && 2 * split <= kbs) split *= 2;
  if (p.m <= 64) return id_launch<64>(p, split, pdl, stream);
  return id_launch<128>(p, split, pdl, stream);
}

}  // namespace dg
