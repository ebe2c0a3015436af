// Product of 8-bit integers in tiles on the tensor cores: D = c + sa sb (a b^T).
//
// sm_103a's tcgen05 has no integer kind, but an 8-bit integer is a half exactly
// and so is a product of two in FP32: kind::f16, at its rate, gives what integer
// products would while sums stay within 2^24, so always up to K = 1024.  Beyond, every 16
// columns the sum so far is cut to FP32's 24 bits, which is little next to the largest
// partial sum but not next to what is left where they cancel: of +-2^25.6 at
// K = 8192 results of up to 2^14.7 were off by 400 here, by 9 where warps share the columns.
// (The quantising of such a row itself leaves thousands.)
//
// Nothing is widened in memory: warps load the codes, turn them into
// halves in registers (1024 + 128 + c is a half whose low byte is c + 128; an
// addition takes the offset away: 5 instructions for 4 codes) and store them
// where the MMA reads them, in its 128-byte swizzle.
//
// What bounds it is the widening: every code is widened again in each tile that uses
// it (of 4096 x 4096 a's 19 times, b's 16).  So large products run on CTA pairs
// (cta_group::2): 256 x 256 tiles in which a CTA widens 128 rows of a and 128 of b, 64 KB
// a stage of 128 columns where a CTA alone would need 96 for half the products.  At 4096 x
// 4096 x 7168 the MMAs alone take 115 us, widening alone 119, both 202: they hardly
// overlap, although neither the tensor pipe (53%) nor shared memory (59%) is full; a
// first kernel that widens once is not tried.  Measured in a graph: 4096 x 4096 x 7168 202
// us (1.19 PFLOP/s, 63% of the measured BF16 burst), 4096 x 24576 x 1536 244 us (1.27).
// With little K the results take longer than the products: a warp stores 32 rows an
// instruction (4096 x 16384 x 128 80 us, with c 144, for 20 and 40 of bytes).  Codes brought raw into
// shared memory by TMA and widened from there were slower (253: they pass through
// it once more), loads three stages ahead too (234: registers spill).
//
// One persistent CTA per SM, 24 warps: 0 issues the MMAs (of a pair the first
// CTA's; the second's passes on that its stages are ready), 4-7 scale and store a
// tile's results from TMEM while the next tile's MMAs run (two accumulators),
// 8-23 load and widen.  Loads are two stages ahead
// in registers, so that the wait for a free stage does not put their latency
// into the chain.
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

constexpr int kIgBand = 16;  // row blocks of a band of tiles

// A tile: 128 (a pair: 256) rows of a by BN of b; of a pair each CTA widens half
// of both.
template <int BN, bool PAIR>
struct IgPlan {
  static constexpr int kRowsB = PAIR ? BN / 2 : BN;  // of b that a CTA widens
  static constexpr int kStage = (128 + kRowsB) * 256;
  // channel scales and a 32 x 33 tile of each storing warp, barriers
  static constexpr int kTail = 4 * (BN + 32 * 33) * 4 + 256;
  static constexpr int kFit = (232448 - 1024 - kTail) / kStage, kStages = kFit > 4 ? 4 : kFit;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kTail;
  static constexpr uint32_t kCols = 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;  // of TMEM
  static_assert(kStages >= 2 && kRowsB % 8 == 0, "");
};

// Row block and column block of tile t: bands of kIgBand row blocks, in each
// the column blocks one after another, so that the CTAs at work share both.
__device__ __forceinline__ void ig_tile(int t, int mb_all, int nb_all, int& mb, int& nb) {
  const int band = t / (kIgBand * nb_all), first = band * kIgBand;
  const int height = min(kIgBand, mb_all - first), in = t - band * kIgBand * nb_all;
  nb = in / height;
  mb = first + in - nb * height;
}

// 32 results of row m from column n0 on, all there and on 16 bytes.
__device__ __forceinline__ void ig_store(const Int8Args& p, const uint32_t (&acc)[32], float sa, const float* sbw, int m,
                                         int n0) {
  const int64_t at = (int64_t)m * p.ldd + n0, from = (int64_t)m * p.ldc + n0;
  uint4 all[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)  // c may be d
    all[i] = p.c ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.c) + from)[i] : make_uint4(0, 0, 0, 0);
  uint4 out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 cw = all[i];
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
    out[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  uint16_t* d = static_cast<uint16_t*>(p.d) + at;
  if (p.vector == 2) {
    st_global_32(d, out[0], out[1]);
    st_global_32(d + 16, out[2], out[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(d)[i] = out[i];
  }
}

// The same where rows are on no boundary or the columns end: by way of shared
// memory, so that a warp writes a row's 32 columns at once (a lane's own row, value
// by value, would touch 32 rows an instruction: 333 x 1001 x 1552 23 us against
// 17). c, which may be d, is added in shared memory, 16 rows at once, before any of
// them is stored (row by row each read waits for the store before it: 4096 x 16383 x
// 128 1280 us against 268; 8 at once 367, 32 at once 226, but their code then slows
// the aligned epilogue down, 80 to 88).
constexpr int kIgRowsAtOnce = 16;
__device__ __forceinline__ void ig_store_ragged(const Int8Args& p, const uint32_t (&acc)[32], float sa, const float* sbw,
                                                float* turn, int m0, int n0, int lane) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; ++i) turn[lane * 33 + i] = __uint_as_float(acc[i]) * sa;
  __syncwarp();
  const int n = n0 + lane;
  if (n >= p.n) return;
  float sb = sbw[lane];
  const int rows = min(32, p.m - m0);
  if (p.c) {
    const uint16_t* from = static_cast<const uint16_t*>(p.c) + (int64_t)m0 * p.ldc + n;
#pragma unroll 1
    for (int i0 = 0; i0 < rows; i0 += kIgRowsAtOnce) {
      uint16_t c[kIgRowsAtOnce];
#pragma unroll
      for (int i = 0; i < kIgRowsAtOnce; ++i) c[i] = from[min(i0 + i, rows - 1) * p.ldc];
#pragma unroll
      for (int i = 0; i < kIgRowsAtOnce; ++i) {
        const float was = p.fp16 ? __half2float(__ushort_as_half(c[i])) : __uint_as_float((uint32_t)c[i] << 16);
        float* v = turn + (i0 + i) * 33 + lane;  // of rows past the last as well, which nothing reads
        *v = fmaf(*v, sb, was);
      }
    }
    sb = 1.0f;
  }
#pragma unroll 8
  for (int i = 0; i < rows; ++i) {
    const int64_t at = (int64_t)(m0 + i) * p.ldd + n;
    const float v = fmaf(turn[i * 33 + lane], sb, 0.0f);
    if (p.fp16) static_cast<__half*>(p.d)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16_rn(v);
  }
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(kIgThreads, 1) int8_gemm_kernel(const Int8Args p) {
  using Plan = IgPlan<BN, PAIR>;
  constexpr int STAGES = Plan::kStages, STAGE = Plan::kStage, RB = Plan::kRowsB, kTileRows = PAIR ? 256 : 128;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const after = smem_raw + (base - smem_u32(smem_raw)) + STAGES * STAGE;
  float* const sb_row = reinterpret_cast<float*>(after);  // [4 warps][BN]
  uint64_t* const bars = reinterpret_cast<uint64_t*>(after + 4 * (BN + 32 * 33) * 4);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + STAGES + s); };
  auto tfull = [&](int s) { return smem_u32(bars + 2 * STAGES + s); };
  auto tempty = [&](int s) { return smem_u32(bars + 2 * STAGES + 2 + s); };
  const uint32_t drain = smem_u32(bars + 2 * STAGES + 4);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_ctarank() : 0, unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int units = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), kIgWiden + (PAIR && rank == 0 ? 1 : 0));  // and the second CTA's
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), PAIR ? 8 : 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), Plan::kCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), Plan::kCols);
      tmem_relinquish();
    }
    tc_fence_before();
  }
  griddep_wait();
  if constexpr (PAIR) cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();

  const int mb_all = (p.m + kTileRows - 1) / kTileRows, nb_all = (p.n + BN - 1) / BN, tiles = mb_all * nb_all;
  const int kbs = (p.k + kIgK - 1) / kIgK;
  const uint64_t tmo = p.timeout_ns;
  // an arrival that the MMAs' issuer waits for
  auto tell = [&](uint32_t bar) {
    if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(bar, 0));
    else mbar_arrive(bar);
  };
  auto commit = [&](uint32_t bar) {
    if constexpr (PAIR) tc_commit_pair(bar);
    else tc_commit(bar);
  };
  auto told = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    if constexpr (PAIR) return wait_quick<true>(bar, parity, abort_flag, tmo, p.err, site);
    else return wait_quick(bar, parity, abort_flag, tmo, p.err, site);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      if (rank == 0) {
        int s = 0;
        uint32_t phase = 0, pass = 0;
        bool ok = true;
        for (int t = unit; t < tiles && ok; t += units, ++pass) {
          const uint32_t buf = pass & 1u;
          if (!told(tempty(buf), ((pass >> 1) & 1u) ^ 1u, kSiteMmaTmemEmpty)) break;
          tc_fence_after();
          for (int kb = 0; kb < kbs; ++kb) {
            if (!told(full(s), phase, kSiteMmaFull)) {
              ok = false;
              break;
            }
            fence_proxy_async_smem();
            tc_fence_after();
#pragma unroll
            for (int atom = 0; atom < 2; ++atom) {
              const uint64_t ad = smem_desc_kmajor_sw128(base + s * STAGE + atom * 16384);
              const uint64_t bd = smem_desc_kmajor_sw128(base + s * STAGE + 32768 + atom * (RB * 128));
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_f16<PAIR>(tmem + buf * BN, ad + 2 * j, bd + 2 * j, idesc_f16(kTileRows, BN),
                                 kb != 0 || atom != 0 || j != 0);
            }
            commit(empty(s));
            if (++s == STAGES) {
              s = 0;
              phase ^= 1u;
            }
          }
          if (ok) commit(tfull(buf));
        }
        commit(drain);
      } else {
        // the second CTA's stages, for the first: one arrival across the cluster a stage, not one a warp (each waits
        // for the warp's own loads in flight)
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = unit; t < tiles && ok; t += units)
          for (int kb = 0; kb < kbs; ++kb) {
            if (!(ok = wait_quick(full(s), phase, abort_flag, tmo, p.err, kSiteMmaFull))) break;
            fence_proxy_async_smem();
            mbar_arrive_cluster(mapa_shared(full(s), 0));
            if (++s == STAGES) {
              s = 0;
              phase ^= 1u;
            }
          }
      }
      // the MMAs in flight end before the memory they use is given back
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0))
        if (global_timer_ns() - t0 > 2 * tmo + 1000000000ull) {
          record_error(p.err, DG_ERR_DEVICE_TIMEOUT, kSiteDrain);
          break;
        }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ load and widen
    const int q = lane & 3, atom = lane >> 2 & 1, row = (warp - 8) * 4 + (lane >> 3);
    const int col = atom * 64 + q * 16;
    IgRows<128> a;
    IgRows<RB> b;
    int lt = unit, lk = 0;
    auto aim = [&]() {
      if (lt >= tiles) {
        a.on = b.on = 0;
        return;
      }
      int mb, nb;
      ig_tile(lt, mb_all, nb_all, mb, nb);
      a.aim(p.a, p.lda, mb * kTileRows + rank * 128, p.m, row, col);
      b.aim(p.b, p.ldb, nb * BN + rank * RB, p.n, row, col);
    };
    auto load = [&](uint4 (&va)[IgRows<128>::kPieces], uint4 (&vb)[IgRows<RB>::kPieces]) {
      const int k = lk * kIgK;
      const bool in = k + col < p.k;
      a.load(va, p.lda, k, in);
      b.load(vb, p.ldb, k, in);
      if (++lk == kbs) {
        lk = 0;
        lt += units;
        aim();
      }
    };
    a.src = b.src = p.a;
    aim();
    uint4 va[kIgAhead][IgRows<128>::kPieces], vb[kIgAhead][IgRows<RB>::kPieces];
#pragma unroll
    for (int h = 0; h < kIgAhead; ++h) load(va[h], vb[h]);
    const int mine = unit < tiles ? (tiles - 1 - unit) / units + 1 : 0;
    const int stages = mine * kbs;
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = 0; it < stages && ok; it += kIgAhead) {
#pragma unroll
      for (int h = 0; h < kIgAhead; ++h) {
        if (it + h >= stages || !ok) break;
        if (!wait_quick(empty(s), phase ^ 1u, abort_flag, tmo, p.err, kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        a.store(va[h], base + s * STAGE, row, atom, q);
        b.store(vb[h], base + s * STAGE + 32768, row, atom, q);
        __syncwarp();
        if (lane == 0) mbar_arrive(full(s));
        load(va[h], vb[h]);
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scale and store
    const int quarter = warp & 3;
    float* const sbw = sb_row + quarter * BN;
    float* const turn = sb_row + 4 * BN + quarter * 32 * 33;
    uint32_t pass = 0;
    for (int t = unit; t < tiles; t += units, ++pass) {
      int mb, nb;
      ig_tile(t, mb_all, nb_all, mb, nb);
      const uint32_t buf = pass & 1u;
      const int m = mb * kTileRows + rank * 128 + quarter * 32 + lane;
      const float sa = m < p.m ? __ldg(p.sa + m) : 0.0f;
      __syncwarp();  // the last tile's scales are read
#pragma unroll
      for (int i = 0; i < BN; i += 32) sbw[i + lane] = nb * BN + i + lane < p.n ? __ldg(p.sb + nb * BN + i + lane) : 0.0f;
      __syncwarp();
      if (!wait_quick(tfull(buf), (pass >> 1) & 1u, abort_flag, tmo, p.err, kSiteEpilogueTmemFull)) break;
      tc_fence_after();
      for (int ch = 0; ch < BN / 32; ++ch) {
        const int n0 = nb * BN + ch * 32;
        uint32_t acc[32];
        tc_ld_32x32b_x32(tmem + buf * BN + ch * 32 + ((uint32_t)(quarter * 32) << 16), acc);
        tc_wait_ld_regs(acc);
        if (ch == BN / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) tell(tempty(buf));
        }
        if (p.vector && n0 + 32 <= p.n) {
          if (m < p.m) ig_store(p, acc, sa, sbw + ch * 32, m, n0);
        } else if (n0 < p.n && m - lane < p.m) {
          ig_store_ragged(p, acc, sa, sbw + ch * 32, turn, m - lane, n0, lane);
        }
      }
    }
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs are done with every role
  else __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, Plan::kCols);
    else tmem_dealloc(tmem, Plan::kCols);
  }
}

template <int BN, bool PAIR>
cudaError_t ig_launch(const Int8Args& p, bool pdl, cudaStream_t stream) {
  using Plan = IgPlan<BN, PAIR>;
  cudaError_t e = set_smem(int8_gemm_kernel<BN, PAIR>, Plan::kSmem, Plan::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((p.m + (PAIR ? 255 : 127)) / (PAIR ? 256 : 128)) * ((p.n + BN - 1) / BN);
  const int64_t units = std::min<int64_t>(tiles, PAIR ? p.sms / 2 : p.sms);
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(PAIR ? 2 * units : units), 1, 1);
  cfg.blockDim = dim3(kIgThreads, 1, 1);
  cfg.dynamicSmemBytes = Plan::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, int8_gemm_kernel<BN, PAIR>, p);
}

}  // namespace

cudaError_t int8_gemm_launch(Int8Args p, bool pdl, cudaStream_t stream) {
  cudaError_t e = error_word_address(&p.err);
  if (e != cudaSuccess) return e;
  // The tile whose waves take the least time.  A stage takes (us, measured at K = 7168 and 2048, one tile an SM): 128 x 64
  // 0.73, 128 x 128 0.82; of pairs 256 x 192 0.94, 256 x 224 0.96, 256 x 256 1.03.  (333 x 4096 x 7168: 78.6, 46.1, 53.1,
  // 53.5, 57.6 us; 2048 x 7168 x 2048: 135.5, 78.9, 61.5, 63.3, 54.6.)  What a tile's results take is not counted: below K of
  // about 700 they decide, and the choice there is not measured.
  struct {
    int bn, rows, slots, stage;
  } const tiles[] = {{64, 128, p.sms, 73},
                     {128, 128, p.sms, 82},
                     {192, 256, p.sms / 2, 94},
                     {224, 256, p.sms / 2, 96},
                     {256, 256, p.sms / 2, 103}};
  int best = 64;
  int64_t least = INT64_MAX;
  for (const auto& t : tiles) {
    if (t.slots < 1) continue;
    const int64_t all = (int64_t)((p.m + t.rows - 1) / t.rows) * ((p.n + t.bn - 1) / t.bn);
    const int64_t cost = (all + t.slots - 1) / t.slots * t.stage;
    if (cost < least) {
      least = cost;
      best = t.bn;
    }
  }
  switch (best) {
    case 64: return ig_launch<64, false>(p, pdl, stream);
    case 128: return ig_launch<128, false>(p, pdl, stream);
    case 192: return ig_launch<192, true>(p, pdl, stream);
    case 224: return ig_launch<224, true>(p, pdl, stream);
    default: return ig_launch<256, true>(p, pdl, stream);
  }
}

}  // namespace dg
