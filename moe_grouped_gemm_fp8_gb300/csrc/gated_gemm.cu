// Gated feed-forward product: both projections, the activation and the
// product in one kernel.
//
//   g = A Wg^T, u = A Wu^T (W = [Wg; Wu], E4M3 with the GEMMs' scales),
//   h = act(g) u, given as BF16 or as E4M3 codes with one power-of-two scale
//   per 1 x 128 row group, rounded once from FP32; optionally also [g | u] as
//   such codes, the 8-bit checkpoint of the backward pass.
//
// An output tile is 128 rows x 128 columns of h: its B tile is 128 rows of Wg
// and the matching 128 rows of Wu side by side, one 128 x 256 x 32 MMA per K
// step, so the tile's accumulator holds g in columns 0-127 and u in columns
// 128-255 and a row's group of 128 h columns lies inside it.  Neither g nor u
// reaches memory in more than 8 bits.
//
// Persistent CTAs of 12 warps in the GEMMs' roles (gemm_kernel.cuh): warp 0
// TMA producer, warp 1 MMA issuer, warp 2 scales, warps 4-11 epilogue.  Two
// accumulators of 256 columns would fill TMEM and leave no room for the
// scales, so there is one: the eight epilogue warps read it into registers
// (64 columns of g and the matching 64 of u each), hand it back, and work
// while the next tile's MMAs run.  The two warps that share 32 rows exchange
// their rows' maxima through shared memory.
//
// Bound by the tensor pipe for long A: 37k rows of 8 experts, K = 7168, F = 2048
// in 661 us (3.3 PFLOP/s, 0.85 of twice the BF16 burst); 4096 rows, E4M3 results
// and checkpoint, 91.9 us (2.6 PFLOP/s: 512 tiles take four rounds of 152 SMs).
// By reading W for short A: 16 experts of up to 256 rows 90.7 us (5.5 TB/s).
// 128 rows x 256 columns are the widest tile whose accumulator leaves TMEM room
// for the scales and whose rows' groups of 128 columns of h lie inside it; sharing
// W's tiles between two CTAs by multicast changed nothing (89.9 and 89.0 us), and
// sharing the last round's tiles, half of K each, cost what it saved.
#include "gemm_kernel.cuh"

#include "dg_ops.cuh"
#include "gated_gemm.h"

namespace dg {
namespace {

constexpr int kGateStages = 4;
using GateLayout = GemmLayout<256>;

struct GatePlan {
  static constexpr int kSfBase = 256;  // TMEM columns after the accumulator
  static_assert(kSfBase + kSfSlots * GateLayout::kSfCols <= 512, "TMEM over-subscribed");
  static constexpr int kXchBytes = 3 * 256 * 4;  // maxima of h, g, u: [128 rows][2 column halves]
  static constexpr size_t smem_bytes(int mode) {
    return (size_t)kGateStages * GateLayout::kStageBytes + (size_t)kSfSlots * GateLayout::kSfBufBytes + kXchBytes +
           1024 + 8 * (2 * kGateStages + 3 * kSfSlots + 3) + 32 +
           (mode == kMasked ? (size_t)4 * (2 * kMaxMaskedGroups + 1) : 0);
  }
};

// Both warps of a row quarter arrive with their wait's outcome and leave with
// the conjunction: neither goes on without the other after a timeout.
__device__ __forceinline__ bool pair_agree(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory");
}

__device__ __forceinline__ uint32_t abs_max64(const uint32_t (&r)[2][32]) {
  float m = 0.0f;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 32; i += 2) m = abs_max3(m, __uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1]));
  return __float_as_uint(m);
}

// 64 columns of one row, times inv, as E4M3 codes (16-byte aligned).
__device__ __forceinline__ void store_codes64(uint8_t* dst, const uint32_t (&r)[2][32], float inv) {
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 16 * p + 4 * i;
        w[i] = e4m3x4(__uint_as_float(r[c][k]) * inv, __uint_as_float(r[c][k + 1]) * inv,
                      __uint_as_float(r[c][k + 2]) * inv, __uint_as_float(r[c][k + 3]) * inv);
      }
      *reinterpret_cast<uint4*>(dst + 32 * c + 16 * p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int ACT>
__device__ __forceinline__ void gate_product(uint32_t (&g)[2][32], const uint32_t (&u)[2][32]) {
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      g[c][i] = __float_as_uint(gate_act<ACT>(__uint_as_float(g[c][i])) * __uint_as_float(u[c][i]));
}

template <int MODE>
__global__ void __launch_bounds__(kGemmThreadsEpi8, 1)
    fp8_gated_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                          const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfb,
                          const GatedArgs ga) {
  using L = GateLayout;
  using P = GatePlan;
  constexpr int STAGES = kGateStages;
  const GemmArgs& args = ga.base;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
  uint8_t* sfbuf = smem + STAGES * L::kStageBytes;
  uint32_t* xch = reinterpret_cast<uint32_t*>(sfbuf + kSfSlots * L::kSfBufBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(xch) + P::kXchBytes);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + STAGES + s); };
  auto sffull = [&](int p) { return smem_u32(bars + 2 * STAGES + p); };
  auto sfready = [&](int p) { return smem_u32(bars + 2 * STAGES + kSfSlots + p); };
  auto sfempty = [&](int p) { return smem_u32(bars + 2 * STAGES + 2 * kSfSlots + p); };
  constexpr int kB0 = 2 * STAGES + 3 * kSfSlots;
  const uint32_t tfull = smem_u32(bars + kB0), tempty = smem_u32(bars + kB0 + 1), drain = smem_u32(bars + kB0 + 2);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kB0 + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tile_start = reinterpret_cast<int*>(tmem_slot + 8);
  int* group_valid = tile_start + (kMaxMaskedGroups + 1);
  unsigned long long* const err = args.err;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int p = 0; p < kSfSlots; ++p) {
      mbar_init(sffull(p), 1);
      mbar_init(sfready(p), 1);
      mbar_init(sfempty(p), 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_sfa);
    tma_prefetch_desc(&tm_sfb);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  if (MODE == kMasked && warp == 2) {
    for (int g = lane; g < args.num_groups; g += 32) {
      const int v = __ldg(args.masked_m + g);
      const int c = v < 0 ? 0 : (v > args.m ? args.m : v);
      if (c != v) record_error(err, DG_ERR_DEVICE_BAD_INDEX, kSiteMaskedCount);
      group_valid[g] = c;
    }
    __syncwarp();
    if (lane == 0) {
      int acc = 0;
      for (int g = 0; g < args.num_groups; ++g) {
        tile_start[g] = acc;
        acc += (group_valid[g] + kBlockM - 1) / kBlockM * args.n_blocks;
      }
      tile_start[args.num_groups] = acc;
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();

  Scheduler<MODE> sched;
  sched.sk_ctl = nullptr;
  sched.args = &args;
  sched.tile_start = tile_start;
  sched.group_valid = group_valid;
  sched.pairs = nullptr;
  sched.cursor = 0;
  sched.kb_lo = 0;
  sched.kb_hi = args.k_blocks;
  sched.first = (int)blockIdx.x;
  sched.stride = (int)gridDim.x;
  sched.total = MODE == kMasked ? tile_start[args.num_groups] : args.m_blocks * args.n_blocks;
  const uint64_t tmo = args.timeout_ns;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRoles) : "memory");
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
          Tile tile;
          int kb0, kb1;
          const int st_it = sched.item(it, tile, kb0, kb1);
          if (st_it < 0) break;
          if (st_it == 0) continue;
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_one<kSuspendHintNs, true>(empty(stage), phase ^ 1u, abort_flag, tmo, err, kSiteProducerEmpty)) {
              ok = false;
              break;
            }
            const uint32_t sb = smem_u32(smem + stage * L::kStageBytes);
            const uint32_t fb = full(stage);
            mbar_arrive_expect_tx(fb, L::kTxAB);
            const bool drop = args.debug_drop_load && blockIdx.x == 0 && it == 0 && kb + 1 == args.debug_drop_load;
            if (!drop) {
              const int kx = kb * kBlockK, my = tile.mb * kBlockM, f0 = tile.nb * 128;
              DG_CHECK(err, kb >= 0 && kb < args.k_blocks && my >= 0 && my < args.m, kSiteCheckLoadA);
              DG_CHECK(err, f0 >= 0 && f0 < ga.f && tile.g >= 0 && tile.g < args.num_groups, kSiteCheckLoadB);
              if (MODE == kMasked) tma_load_3d(sb, &tm_a, fb, kx, my, tile.g);
              else tma_load_2d(sb, &tm_a, fb, kx, my);
              tma_load_3d(sb + L::kOffB, &tm_b, fb, kx, f0, tile.g);
              tma_load_3d(sb + L::kOffB + 128 * kBlockK, &tm_b, fb, kx, ga.f + f0, tile.g);
              issued |= 1u << stage;
              issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
            }
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        for (int s = 0; s < STAGES; ++s)
          if (issued & (1u << s))
            wait_drain<true>(full(s), (issued_parity >> s) & 1u, tmo, err, kSiteProducerDrain);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc0 = idesc_mxf8_e4m3(kBlockM, 256, 0, 0);
        int stage = 0;
        uint32_t phase = 0, pack = 0, acc_phase = 0;
        uint32_t sf_tmem = tmem_base + (uint32_t)P::kSfBase;
        bool ok = true;
        for (int it = 0; ok; ++it) {
          Tile tile;
          int kb0, kb1;
          const int st_it = sched.item(it, tile, kb0, kb1);
          if (st_it < 0) break;
          if (st_it == 0) continue;
          if (!wait_one<kSuspendHintNs, true>(tempty, acc_phase ^ 1u, abort_flag, tmo, err, kSiteMmaTmemEmpty)) break;
          tc_fence_after();
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_one<kSuspendHintNs, true>(full(stage), phase, abort_flag, tmo, err, kSiteMmaFull)) {
              ok = false;
              break;
            }
            const int slot = (int)(pack % kSfSlots);
            if (kb == kb0 || (kb & 3) == 0) {
              if (!wait_one<kSuspendHintNs, true>(sfready(slot), (pack / kSfSlots) & 1u, abort_flag, tmo, err,
                                                  kSiteMmaScaleReady)) {
                ok = false;
                break;
              }
              tc_fence_after();
              sf_tmem = tmem_base + (uint32_t)(P::kSfBase + slot * L::kSfCols);
            }
            const uint32_t sel = (uint32_t)(kb & 3);
            const uint32_t idesc = idesc0 | (sel << 4) | (sel << 29);
            const uint32_t st = smem_u32(smem + stage * L::kStageBytes);
            const uint64_t adesc = smem_desc_kmajor_sw128(st), bdesc = smem_desc_kmajor_sw128(st + L::kOffB);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc_mma_mxf8(tmem_base, adesc + 2u * j, bdesc + 2u * j, idesc, sf_tmem, sf_tmem + 4,
                          (kb != kb0 || j != 0) ? 1u : 0u);
            tc_commit(empty(stage));
            if ((kb & 3) == 3 || kb == kb1 - 1) {
              tc_commit(sfempty(slot));
              ++pack;
            }
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit(tfull);
          acc_phase ^= 1u;
        }
        tc_commit(drain);
        wait_drain<true>(drain, 0, tmo, err, kSiteDrain);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ scale warp
      PackCursor<Scheduler<MODE>> ld, lay;
      ld.init(sched);
      lay.init(sched);
      uint32_t n_loaded = 0, n_laid = 0;
      bool ok = true;
      while (!lay.done && ok) {
        while (!ld.done && n_loaded < n_laid + kSfLookahead) {
          const int slot = (int)(n_loaded % kSfSlots);
          int go = 1;
          if (lane == 0) {
            go = wait_one<kSuspendHintNs, true>(sfempty(slot), ((n_loaded / kSfSlots) & 1u) ^ 1u, abort_flag, tmo, err,
                                                kSiteScaleEmpty) ? 1 : 0;
            if (go) {
              const uint32_t buf = smem_u32(sfbuf + slot * L::kSfBufBytes);
              const uint32_t bar = sffull(slot);
              const int my = ld.tile.mb * kBlockM, f0 = ld.tile.nb * 128, kp = ld.kp;
              DG_CHECK(err, kp >= 0 && kp < (args.k_blocks + 3) / 4 && my >= 0 && my < args.m, kSiteCheckScale);
              mbar_arrive_expect_tx(bar, L::kTxSF);
              if (MODE == kMasked) tma_load_3d(buf + L::kRawA, &tm_sfa, bar, my, kp, ld.tile.g);
              else tma_load_2d(buf + L::kRawA, &tm_sfa, bar, my, kp);
              tma_load_3d(buf + L::kRawB, &tm_sfb, bar, f0, kp, ld.tile.g);
              tma_load_3d(buf + L::kRawB + 512, &tm_sfb, bar, ga.f + f0, kp, ld.tile.g);
            }
          }
          go = __shfl_sync(0xffffffffu, go, 0);
          if (!go) {
            ok = false;
            break;
          }
          ++n_loaded;
          ld.advance();
        }
        if (!ok) break;
        const int slot = (int)(n_laid % kSfSlots);
        if (!warp_wait<kSuspendHintNs, true>(sffull(slot), (n_laid / kSfSlots) & 1u, abort_flag, tmo, err,
                                             kSiteScaleFull)) {
          ok = false;
          break;
        }
        uint8_t* buf = sfbuf + slot * L::kSfBufBytes;
#pragma unroll
        for (int c = 0; c < 3; ++c) {  // A, Wg, Wu: 128 words each
          const uint32_t* raw = reinterpret_cast<const uint32_t*>(buf + L::kRawA + c * 512);
          const uint4 v = make_uint4(raw[lane], raw[32 + lane], raw[64 + lane], raw[96 + lane]);
          *reinterpret_cast<uint4*>(buf + L::kCpA + c * 512 + lane * 16) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const uint32_t sft = tmem_base + (uint32_t)(P::kSfBase + slot * L::kSfCols);
#pragma unroll
          for (int c = 0; c < 3; ++c)
            tc_cp_32x128b_warpx4(sft + 4 * c, smem_desc_sf_chunk(smem_u32(buf + L::kCpA + c * 512)));
          tc_commit(sfready(slot));
        }
        ++n_laid;
        lay.advance();
      }
      if (lane == 0) {
        for (uint32_t q = n_laid; q < n_loaded; ++q)
          wait_drain<true>(sffull((int)(q % kSfSlots)), (q / kSfSlots) & 1u, tmo, err, kSiteProducerDrain);
        if (n_laid > 0)
          wait_drain<true>(sfready((int)((n_laid - 1) % kSfSlots)), ((n_laid - 1) / kSfSlots) & 1u, tmo, err,
                           kSiteDrain);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi) : "memory");
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;
    const int pair_id = 1 + quarter;
    uint32_t* const mine = xch + (quarter * 32 + lane) * 2 + half;
    const uint32_t* const other = xch + (quarter * 32 + lane) * 2 + (half ^ 1);
    uint32_t acc_phase = 0;
    for (int it = 0;; ++it) {
      Tile tile;
      int tkb0, tkb1;
      const int st_it = sched.item(it, tile, tkb0, tkb1);
      if (st_it < 0) break;
      if (st_it == 0) continue;
      const bool arrived = warp_wait<kSuspendHintNs, true>(tfull, acc_phase, abort_flag, tmo, err,
                                                           kSiteEpilogueTmemFull);
      if (!pair_agree(pair_id, arrived)) break;
      acc_phase ^= 1u;
      tc_fence_after();
      uint32_t g[2][32], u[2][32];
      {
        const uint32_t t = tmem_base + (uint32_t)(half * 64) + ((uint32_t)(quarter * 32) << 16);
        tc_ld_32x32b_x32(t, g[0]);
        tc_ld_32x32b_x32(t + 32, g[1]);
        tc_ld_32x32b_x32(t + 128, u[0]);
        tc_ld_32x32b_x32(t + 160, u[1]);
        tc_wait_ld_regs(g[0]);
        tc_wait_ld_regs(g[1]);
        tc_wait_ld_regs(u[0]);
        tc_wait_ld_regs(u[1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty);

      const int row = tile.mb * kBlockM + quarter * 32 + lane;  // of its group (masked)
      const int col = tile.nb * 128 + half * 64;
      bool live = row < args.m;
      if (MODE == kContiguous) {
        const int id = __ldg(args.m_indices + row);
        if (id >= 0 && id != tile.g) record_error(err, DG_ERR_DEVICE_BAD_INDEX, kSiteContiguousIndex);
        live = id == tile.g;
      }
      if (MODE == kMasked) live = row < group_valid[tile.g];
      const int64_t orow = MODE == kMasked ? (int64_t)tile.g * args.m + row : row;
      DG_CHECK(err, col >= 0 && tile.nb >= 0 && tile.nb * 128 < ga.f && (!live || row < args.m), kSiteCheckStore);
      // scale words: [group][ceil(blocks / 4)][m_pad]; the dense form also
      // zeroes the words of the alignment padding
      const bool word = live || (MODE == kDense && row < ga.m_pad);
      auto store_scale = [&](uint32_t* sf, int blocks, int block, int e) {
        const int64_t kp = (blocks + 3) / 4;
        uint32_t* w = sf + ((MODE == kMasked ? tile.g * kp : 0) + (block >> 2)) * ga.m_pad + row;
        store_scale_byte(w, block, block == blocks - 1, live ? (uint32_t)(e + 127) : 0u);
      };

      if (ga.cq) {
        mine[256] = abs_max64(g);
        mine[512] = abs_max64(u);
        pair_sync(pair_id);
        const int eg = scale_exponent(__uint_as_float(max(mine[256], other[256])));
        const int eu = scale_exponent(__uint_as_float(max(mine[512], other[512])));
        if (live) {
          uint8_t* dst = ga.cq + orow * 2 * ga.f + col;
          store_codes64(dst, g, pow2f(-eg));
          store_codes64(dst + ga.f, u, pow2f(-eu));
        }
        if (word) {
          const int fb = ga.f / 128;
          if (half == 0) store_scale(ga.csf, 2 * fb, tile.nb, eg);
          else store_scale(ga.csf, 2 * fb, fb + tile.nb, eu);
        }
      }
      if (ga.activation == DG_ACT_SILU) gate_product<DG_ACT_SILU>(g, u);
      else gate_product<DG_ACT_GELU_TANH>(g, u);
      if (ga.hq) {
        mine[0] = abs_max64(g);
        pair_sync(pair_id);
        const int e = scale_exponent(__uint_as_float(max(mine[0], other[0])));
        if (live) store_codes64(ga.hq + orow * ga.f + col, g, pow2f(-e));
        if (word && half == 0) store_scale(ga.hsf, ga.f / 128, tile.nb, e);
      } else if (live) {
        __nv_bfloat16* dst = ga.h + orow * ga.ldh + col;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < 4; ++p)
            if (col + 32 * c + 8 * p < ga.f) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = bf16x2_bits(__uint_as_float(g[c][8 * p + 2 * i]), __uint_as_float(g[c][8 * p + 2 * i + 1]));
              *reinterpret_cast<uint4*>(dst + 32 * c + 8 * p) = make_uint4(w[0], w[1], w[2], w[3]);
            }
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int MODE>
struct GateTag {};

template <int MODE>
cudaError_t launch_mode(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sfa, const CUtensorMap& sfb,
                        const GatedArgs& args, int grid, cudaStream_t stream) {
  static_assert(GatePlan::smem_bytes(MODE) <= (size_t)kSmemLimit, "shared memory over the per-CTA limit");
  auto kern = fp8_gated_gemm_kernel<MODE>;
  const size_t smem = GatePlan::smem_bytes(MODE);
  cudaError_t e = set_smem_once<GateTag<MODE>>(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_op(kern, dim3((unsigned)grid), kGemmThreadsEpi8, smem, args.base.pdl != 0, stream, a, b, sfa, sfb,
                   args);
}

}  // namespace

cudaError_t gated_gemm_launch(int mode, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sfa,
                              const CUtensorMap& sfb, GatedArgs args, int grid, cudaStream_t stream) {
  unsigned long long* err = nullptr;
  cudaError_t e = error_word_address(&err);
  if (e != cudaSuccess) return e;
  args.base.err = err;
  switch (mode) {
    case kDense: return launch_mode<kDense>(a, b, sfa, sfb, args, grid, stream);
    case kContiguous: return launch_mode<kContiguous>(a, b, sfa, sfb, args, grid, stream);
    case kMasked: return launch_mode<kMasked>(a, b, sfa, sfb, args, grid, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dg
