// Gated feed-forward product for a few tokens (dense form), with the operand
// roles swapped: 128 rows of Wg and the matching 128 rows of Wu fill the lanes
// of two accumulators, TN tokens are their columns.  A lane of the epilogue
// then holds g and u of one column of h for its tokens, and a token's group of
// 128 columns is the CTA's 128 lanes.
//
// Bound by reading W once.  The K blocks of every strip of 128 columns are
// divided among the S CTAs of a cluster, so that the loads of short problems
// come from many SMs; each CTA then sends the others' token columns of its two
// partial sums through distributed shared memory, adds the S partials of its
// own in rank order (the same result whatever the timing) and finishes them.
// K = 7168, weights from HBM: F = 2048, 2 and 4 tokens 14.1 us (29 MB, 2.1 TB/s; a
// plain streaming read of as many bytes takes 7.1-7.4), F = 4096 15.2 us (3.9
// TB/s); the tiled kernel's 128-row tiles occupy 16 and 32 SMs there.
//
// Warp 0 loads by TMA, warp 1 lays the scales out and issues the MMAs, warps
// 2-5 are the epilogue (gemm_decode.cu's roles).  Every wait is bounded.
#include <atomic>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "gated_gemm.h"

namespace dg {
namespace {

constexpr int kGdThreads = 192;
constexpr int kGdMaxPacks = 8;  // scale words (4 K blocks each) a CTA loads: K ranges of <= 29 blocks
constexpr int kGdSmemBudget = 227 * 1024;
constexpr int gd_align1k(int x) { return (x + 1023) / 1024 * 1024; }

template <int TN, int S>
struct GdLayout {
  static_assert(TN == 32 || TN == 64, "token tile");
  static constexpr int kWTile = 128 * kBlockK;
  static constexpr int kStage = 2 * kWTile + TN * kBlockK;  // Wg, Wu, tokens
  static constexpr int kW = TN / S;                         // token columns each CTA finishes
  static_assert(kW % 4 == 0, "slices are sent 4 columns (16 bytes) at a time");
  // received partials: [sender slot][g, u][lane quarter][kW / 4][32 lanes][4 floats]
  static constexpr int kRecv = (S - 1) * 2 * 4 * kW * 32 * 4;
  static constexpr int kSfW = kGdMaxPacks * 512;            // per weight half, rearranged in place
  static constexpr int kSfA = gd_align1k(kGdMaxPacks * TN * 4);
  static constexpr int kCpA = kGdMaxPacks * 512;
  static constexpr int kXch = 3 * kW * 4 * 4;               // maxima: [g, u, h][kW][4 warps]
  static constexpr int kFixed = gd_align1k(kRecv) + 2 * kSfW + kSfA + kCpA + kXch + 512 + 1024;
  static constexpr int kStages = (kGdSmemBudget - kFixed) / kStage < 6 ? (kGdSmemBudget - kFixed) / kStage : 6;
  static_assert(kStages >= 2, "pipeline depth");
  static constexpr int kOffRecv = kStages * kStage;
  static constexpr int kOffSfG = kOffRecv + gd_align1k(kRecv);
  static constexpr int kOffSfU = kOffSfG + kSfW;
  static constexpr int kOffSfA = kOffSfU + kSfW;
  static constexpr int kOffCpA = kOffSfA + kSfA;
  static constexpr int kOffXch = kOffCpA + kCpA;
  static constexpr int kOffBar = kOffXch + kXch;
  static constexpr int kNumBars = 2 * kStages + 4;
  static constexpr int kOffCtl = kOffBar + 8 * kNumBars;
  static constexpr int kSmem = kOffCtl + 16 + 1024;
  static_assert(kSmem <= kGdSmemBudget, "shared memory");
  static constexpr uint32_t kSfBase = 2 * TN;               // accumulators of g and u, then 12 columns a pack
  static constexpr uint32_t kTmemCols = 2 * TN + 12 * kGdMaxPacks <= 256 ? 256u : 512u;
};

__device__ __forceinline__ void gd_cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void gd_cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes into a CTA of the cluster, counted on that CTA's mbarrier `bar`
// (both cluster addresses).
__device__ __forceinline__ void gd_send_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   addr),
               "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
               : "memory");
}

__device__ __forceinline__ bool gd_warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t tmo,
                                             unsigned long long* err, uint32_t site, bool cluster_scope = false) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0)
    ok = (cluster_scope ? wait_bounded_cluster(bar, parity, abort_flag, tmo, err, site)
                        : wait_bounded(bar, parity, abort_flag, tmo, err, site))
             ? 1
             : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Waits for a phase whatever the abort flag says (work in flight landing
// before exit), bounded in time.
__device__ __noinline__ void gd_drain(uint32_t bar, uint32_t parity, uint64_t tmo, unsigned long long* err,
                                      uint32_t site) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return;
    if ((it & 63u) == 0 && (global_timer_ns() - t0 > tmo || it >= (1u << 30))) {
      record_error(err, DG_ERR_DEVICE_TIMEOUT, site);
      return;
    }
  }
}

// The four epilogue warps' conjunction (all 128 threads take part whatever
// their waits gave, so none is left waiting for another).
__device__ __forceinline__ bool gd_agree(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// TMEM columns of the warp's 32 lanes into registers.
template <int N>
__device__ __forceinline__ void gd_load(uint32_t taddr, uint32_t (&v)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 32) tc_ld_32x32b_x32(taddr + (uint32_t)c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
}

template <int TN, int S>
__global__ void __launch_bounds__(kGdThreads, 1)
    fp8_gated_decode_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                            const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfb,
                            const GatedArgs ga) {
  using L = GdLayout<TN, S>;
  constexpr int STAGES = L::kStages;
  constexpr int W = L::kW;
  const GemmArgs& args = ga.base;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
  const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + STAGES + s); };
  const uint32_t sf_full = smem_u32(bars + 2 * STAGES);
  const uint32_t acc_full = smem_u32(bars + 2 * STAGES + 1);
  const uint32_t recv_full = smem_u32(bars + 2 * STAGES + 2);
  const uint32_t tmem_read = smem_u32(bars + 2 * STAGES + 3);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffCtl);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  unsigned long long* const err = args.err;
  const uint64_t tmo = args.timeout_ns;

  // this CTA's strip of 128 columns of h, its TN tokens and its K blocks [kb0, kb1)
  const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
  const int strip = (int)(blockIdx.x / S), f0 = strip * 128, t0 = (int)blockIdx.y * TN;
  const int kb0 = (int)(((int64_t)args.k_blocks * rank) / S);
  const int kb1 = (int)(((int64_t)args.k_blocks * (rank + 1)) / S);
  const int nkb = kb1 - kb0;  // >= 1: the host keeps S <= K blocks
  const int kp0 = kb0 >> 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(sf_full, 1);
    mbar_init(acc_full, 1);
    mbar_init(recv_full, 1);
    mbar_init(tmem_read, 4);
    mbar_arrive_expect_tx(recv_full, (uint32_t)L::kRecv);  // the others' partials (S = 1: completes now)
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_sfa);
    tma_prefetch_desc(&tm_sfb);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  __syncthreads();
  // Cluster barrier 1: every CTA's mbarriers exist before another CTA writes
  // into its memory.  Cluster barrier 2: a thread arrives once it writes no
  // other CTA's memory any more, and waits for it before its CTA exits.
  if constexpr (S > 1) gd_cluster_arrive();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();
  int issued = 0;  // stages armed (warp 0, lane 0)

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      // scale words, 8 packs from kp0 (packs past the end of K read as zero and are not used)
      mbar_arrive_expect_tx(sf_full, (uint32_t)(kGdMaxPacks * (256 + TN) * 4));
      DG_CHECK(err, f0 < ga.f && kp0 >= 0 && kp0 < (args.k_blocks + 3) / 4, kSiteCheckScale);
      tma_load_2d(smem_u32(smem + L::kOffSfG), &tm_sfb, sf_full, f0, kp0);
      tma_load_2d(smem_u32(smem + L::kOffSfU), &tm_sfb, sf_full, ga.f + f0, kp0);
      tma_load_2d(smem_u32(smem + L::kOffSfA), &tm_sfa, sf_full, t0, kp0);
      for (int i = 0; i < nkb; ++i) {
        const int s = i % STAGES;
        if (i >= STAGES && !wait_bounded(empty(s), (uint32_t)((i / STAGES) - 1) & 1u, abort_flag, tmo, err,
                                         kSiteProducerEmpty))
          break;
        const uint32_t st = smem_u32(smem + s * L::kStage);
        const int kx = (kb0 + i) * kBlockK;
        DG_CHECK(err, kb0 + i < args.k_blocks, kSiteCheckLoadB);
        mbar_arrive_expect_tx(full(s), (uint32_t)L::kStage);
        issued = i + 1;
        // test hook (dg_debug_set_drop_load): CTA 0 arms this stage and never fills it
        if (args.debug_drop_load && blockIdx.x == 0 && blockIdx.y == 0 && i + 1 == args.debug_drop_load) continue;
        tma_load_2d(st, &tm_b, full(s), kx, f0);
        tma_load_2d(st + L::kWTile, &tm_b, full(s), kx, ga.f + f0);
        tma_load_2d(st + 2 * L::kWTile, &tm_a, full(s), kx, t0);
      }
    }
    __syncwarp();
    if constexpr (S > 1) {
      gd_cluster_wait();
      gd_cluster_arrive();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales + MMA
    if (gd_warp_wait(sf_full, 0, abort_flag, tmo, err, kSiteScaleFull)) {
      // scale words -> the 32 x 16-byte chunks of tcgen05.cp (lane l: the words
      // of rows l, 32 + l, 64 + l, 96 + l); tokens past TN are 0.  Every lane
      // reads a pack's words before any lane writes its chunk.
      const int npk = ((kb1 - 1) >> 2) - kp0 + 1;
      uint32_t* const rg = reinterpret_cast<uint32_t*>(smem + L::kOffSfG);
      uint32_t* const ru = reinterpret_cast<uint32_t*>(smem + L::kOffSfU);
      const uint32_t* const ra = reinterpret_cast<const uint32_t*>(smem + L::kOffSfA);
      for (int p = 0; p < npk; ++p) {
        const int o = p * 128 + lane;
        const uint4 wg = make_uint4(rg[o], rg[o + 32], rg[o + 64], rg[o + 96]);
        const uint4 wu = make_uint4(ru[o], ru[o + 32], ru[o + 64], ru[o + 96]);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = 32 * j + lane < TN ? ra[p * TN + 32 * j + lane] : 0u;
        __syncwarp();
        *reinterpret_cast<uint4*>(smem + L::kOffSfG + p * 512 + lane * 16) = wg;
        *reinterpret_cast<uint4*>(smem + L::kOffSfU + p * 512 + lane * 16) = wu;
        *reinterpret_cast<uint4*>(smem + L::kOffCpA + p * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const uint32_t sf0 = tmem_base + L::kSfBase;
        DG_CHECK(err, args.debug_plant_check == 0 && npk >= 1 && npk <= kGdMaxPacks, kSiteCheckTmem);
        for (int p = 0; p < npk; ++p) {
          tc_cp_32x128b_warpx4(sf0 + 12 * p, smem_desc_sf_chunk(smem_u32(smem + L::kOffSfG + p * 512)));
          tc_cp_32x128b_warpx4(sf0 + 12 * p + 4, smem_desc_sf_chunk(smem_u32(smem + L::kOffSfU + p * 512)));
          tc_cp_32x128b_warpx4(sf0 + 12 * p + 8, smem_desc_sf_chunk(smem_u32(smem + L::kOffCpA + p * 512)));
        }
        constexpr uint32_t idesc0 = idesc_mxf8_e4m3(kBlockM, TN, 0, 0);
        for (int i = 0; i < nkb; ++i) {
          const int s = i % STAGES;
          if (!wait_bounded(full(s), (uint32_t)(i / STAGES) & 1u, abort_flag, tmo, err, kSiteMmaFull)) break;
          tc_fence_after();
          const int kb = kb0 + i;
          const uint32_t sel = (uint32_t)(kb & 3);
          const uint32_t idesc = idesc0 | (sel << 4) | (sel << 29);
          const uint32_t sft = sf0 + 12u * (uint32_t)((kb >> 2) - kp0);
          const uint32_t st = smem_u32(smem + s * L::kStage);
          const uint64_t wg = smem_desc_kmajor_sw128(st), wu = smem_desc_kmajor_sw128(st + L::kWTile);
          const uint64_t at = smem_desc_kmajor_sw128(st + 2 * L::kWTile);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t acc = (i != 0 || j != 0) ? 1u : 0u;
            tc_mma_mxf8(tmem_base, wg + 2u * j, at + 2u * j, idesc, sft, sft + 8, acc);
            tc_mma_mxf8(tmem_base + TN, wu + 2u * j, at + 2u * j, idesc, sft + 4, sft + 8, acc);
          }
          tc_commit(empty(s));
        }
        // every MMA (and scale copy) completes before TMEM can be freed
        tc_commit(acc_full);
        gd_drain(acc_full, 0, tmo, err, kSiteDrain);
      }
      __syncwarp();
    }
    // TMEM goes back as soon as the epilogue has read it
    if (lane == 0) gd_drain(tmem_read, 0, tmo, err, kSiteDrain);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
    if constexpr (S > 1) {
      gd_cluster_wait();
      gd_cluster_arrive();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                 // TMEM lane quarter of this warp
    const int col = f0 + q * 32 + lane;     // column of h of this lane
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    bool ok = gd_warp_wait(acc_full, 0, abort_flag, tmo, err, kSiteEpilogueTmemFull) && *abort_flag == 0;
    tc_fence_after();
    uint32_t v[2][TN];
    if (ok) {
      gd_load<TN>(taddr, v[0]);
      gd_load<TN>(taddr + TN, v[1]);
      tc_wait_ld();
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < TN; ++i) asm volatile("" : "+r"(v[k][i]));
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(tmem_read);
    // this CTA's token columns [rank * W, rank * W + W) of its own partials
    float f[2][W];
#pragma unroll
    for (int r = 0; r < S; ++r)
      if (r == (int)rank) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < W; ++j) f[k][j] = __uint_as_float(v[k][r * W + j]);
      }
    if constexpr (S > 1) {
      gd_cluster_wait();
      if (ok) {
#pragma unroll
        for (int o = 0; o < S; ++o) {
          if (o == (int)rank) continue;
          const int slot = (int)rank < o ? (int)rank : (int)rank - 1;
          const uint32_t rbar = mapa_shared(recv_full, (uint32_t)o);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t dst0 = mapa_shared(
                smem_u32(smem + L::kOffRecv) + (uint32_t)(((((slot * 2 + k) * 4 + q) * (W / 4)) * 32 + lane) * 16),
                (uint32_t)o);
#pragma unroll
            for (int j = 0; j < W / 4; ++j)
              gd_send_v4(dst0 + (uint32_t)(j * 512), v[k][o * W + 4 * j], v[k][o * W + 4 * j + 1],
                         v[k][o * W + 4 * j + 2], v[k][o * W + 4 * j + 3], rbar);
          }
        }
      }
      gd_cluster_arrive();  // barrier 2: no more writes to other CTAs
      if (ok) ok = gd_warp_wait(recv_full, 0, abort_flag, tmo, err, kSiteSplitFull, true);
      if (ok) {
        const uint8_t* recv = smem + L::kOffRecv;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float sum[W];
#pragma unroll
          for (int s = 0; s < S; ++s) {  // in rank order
            if (s == (int)rank) {
#pragma unroll
              for (int j = 0; j < W; ++j) sum[j] = s == 0 ? f[k][j] : sum[j] + f[k][j];
            } else {
              const int slot = s < (int)rank ? s : s - 1;
              const uint8_t* src = recv + ((((slot * 2 + k) * 4 + q) * (W / 4)) * 32 + lane) * 16;
#pragma unroll
              for (int j = 0; j < W / 4; ++j) {
                const float4 w = *reinterpret_cast<const float4*>(src + j * 512);
                sum[4 * j] = s == 0 ? w.x : sum[4 * j] + w.x;
                sum[4 * j + 1] = s == 0 ? w.y : sum[4 * j + 1] + w.y;
                sum[4 * j + 2] = s == 0 ? w.z : sum[4 * j + 2] + w.z;
                sum[4 * j + 3] = s == 0 ? w.w : sum[4 * j + 3] + w.w;
              }
            }
          }
#pragma unroll
          for (int j = 0; j < W; ++j) f[k][j] = sum[j];
        }
      }
    }
    // h, and with 8-bit results the maxima of its tokens' groups
    float h[W];
#pragma unroll
    for (int j = 0; j < W; ++j)
      h[j] = (ga.activation == DG_ACT_SILU ? gate_act<DG_ACT_SILU>(f[0][j]) : gate_act<DG_ACT_GELU_TANH>(f[0][j])) *
             f[1][j];
    const int tok0 = t0 + (int)rank * W;  // this CTA's first token
    uint32_t* const xch = reinterpret_cast<uint32_t*>(smem + L::kOffXch);
    if (ga.hq || ga.cq) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t mh = __reduce_max_sync(0xffffffffu, magnitude(h[j]));
        if (lane == 0) xch[(2 * W + j) * 4 + q] = mh;
        if (ga.cq) {
          const uint32_t mg = __reduce_max_sync(0xffffffffu, magnitude(f[0][j]));
          const uint32_t mu = __reduce_max_sync(0xffffffffu, magnitude(f[1][j]));
          if (lane == 0) {
            xch[j * 4 + q] = mg;
            xch[(W + j) * 4 + q] = mu;
          }
        }
      }
      ok = gd_agree(ok);
      if (ok) {
        auto byte_of = [&](int i) {
          const uint4 m = *reinterpret_cast<const uint4*>(xch + i * 4);
          return scale_byte(__uint_as_float(max(max(m.x, m.y), max(m.z, m.w))));
        };
        auto store = [&](const float (&x)[W], int base, uint8_t* codes, int64_t ld, uint32_t* sf, int block,
                         int blocks) {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const int t = tok0 + j;
            const uint32_t b = byte_of(base + j);
            if (t < args.m) codes[(int64_t)t * ld] = (uint8_t)(cvt_e4m3x2(x[j] * inverse_of_byte(b), 0.0f) & 0xFFu);
            if (q == 0 && lane == 0 && t < ga.m_pad)
              store_scale_byte(sf + (int64_t)(block >> 2) * ga.m_pad + t, block, block == blocks - 1,
                               t < args.m ? b : 0u);
          }
        };
        const int fb = ga.f / 128;
        if (ga.cq) {
          store(f[0], 0, ga.cq + col, 2 * (int64_t)ga.f, ga.csf, strip, 2 * fb);
          store(f[1], W, ga.cq + ga.f + col, 2 * (int64_t)ga.f, ga.csf, fb + strip, 2 * fb);
        }
        if (ga.hq) store(h, 2 * W, ga.hq + col, ga.f, ga.hsf, strip, fb);
      }
    }
    if (!ga.hq && ok && col < ga.f) {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (tok0 + j < args.m) ga.h[(int64_t)(tok0 + j) * ga.ldh + col] = __float2bfloat16_rn(h[j]);
    }
  }

  // ------------------------------------------------------------ teardown
  // After a wait gave up (the abort flag), loads still in flight land first.
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    gd_drain(sf_full, 0, tmo, err, kSiteProducerDrain);
    for (int i = issued - STAGES < 0 ? 0 : issued - STAGES; i < issued; ++i)
      gd_drain(full(i % STAGES), (uint32_t)(i / STAGES) & 1u, tmo, err, kSiteProducerDrain);
  }
  if constexpr (S > 1) {
    gd_cluster_wait();
    // after an abort the others' partials may still be landing: wait for them, briefly
    if (threadIdx.x == 0 && *abort_flag)
      gd_drain(recv_full, 0, tmo < 1000000u ? tmo : 1000000u, err, kSiteSplitFull);
  }
}

// Clusters of S CTAs that run at once on the current device: one CTA takes an
// SM's shared memory and a cluster's CTAs share a GPC, so this is less than
// SMs / S (measured at 16 strips of 56 K blocks: clusters of 8 in two waves
// 18.6 us, of 4 in one 13.6 us).
template <int TN, int S>
int gd_max_clusters() {
  auto kern = fp8_gated_decode_kernel<TN, S>;
  constexpr int smem = GdLayout<TN, S>::kSmem;
  if (set_smem(kern, smem, smem) != cudaSuccess) return 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, 1, 1);
  cfg.blockDim = dim3(kGdThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess ? n : 0;
}

template <int TN, int S>
cudaError_t gd_launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sfa, const CUtensorMap& sfb,
                      const GatedArgs& args, int strips, int token_blocks, cudaStream_t stream) {
  using L = GdLayout<TN, S>;
  auto kern = fp8_gated_decode_kernel<TN, S>;
  cudaError_t e = set_smem(kern, L::kSmem, L::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  unsigned n_attr = 0;
  if (S > 1) {
    attr[n_attr].id = cudaLaunchAttributeClusterDimension;
    attr[n_attr].val.clusterDim.x = S;
    attr[n_attr].val.clusterDim.y = 1;
    attr[n_attr].val.clusterDim.z = 1;
    ++n_attr;
  }
  if (args.base.pdl) {
    attr[n_attr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n_attr].val.programmaticStreamSerializationAllowed = 1;
    ++n_attr;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(strips * S), (unsigned)token_blocks, 1);
  cfg.blockDim = dim3(kGdThreads, 1, 1);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n_attr;
  return cudaLaunchKernelEx(&cfg, kern, a, b, sfa, sfb, args);
}

}  // namespace

int gated_decode_max_packs() { return kGdMaxPacks; }

int gated_decode_max_clusters(int tn, int split) {
  // per (device, tn, split) as count + 1 (0: not asked yet); racing callers store the same
  static std::atomic<int> cache[64][2][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int si = split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3;
  std::atomic<int>& slot = cache[dev][tn == 64][si];
  int c = slot.load(std::memory_order_relaxed);
  if (c == 0) {
    int n = 0;
    if (tn == 32) n = si == 0 ? gd_max_clusters<32, 1>() : si == 1 ? gd_max_clusters<32, 2>()
                                               : si == 2 ? gd_max_clusters<32, 4>() : gd_max_clusters<32, 8>();
    else n = si == 0 ? gd_max_clusters<64, 1>() : si == 1 ? gd_max_clusters<64, 2>()
                                      : si == 2 ? gd_max_clusters<64, 4>() : gd_max_clusters<64, 8>();
    c = n + 1;
    slot.store(c, std::memory_order_relaxed);
  }
  return c - 1;
}

cudaError_t gated_decode_launch(int tn, int split, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sfa,
                                const CUtensorMap& sfb, GatedArgs args, int strips, int token_blocks,
                                cudaStream_t stream) {
  unsigned long long* err = nullptr;
  cudaError_t e = error_word_address(&err);
  if (e != cudaSuccess) return e;
  args.base.err = err;
#define DG_GD_CASE(TN, S) \
  if (tn == TN && split == S) return gd_launch<TN, S>(a, b, sfa, sfb, args, strips, token_blocks, stream);
  DG_GD_CASE(32, 1) DG_GD_CASE(32, 2) DG_GD_CASE(32, 4) DG_GD_CASE(32, 8)
  DG_GD_CASE(64, 1) DG_GD_CASE(64, 2) DG_GD_CASE(64, 4) DG_GD_CASE(64, 8)
#undef DG_GD_CASE
  return cudaErrorInvalidValue;
}

}  // namespace dg
