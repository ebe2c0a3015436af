// Backward pass of the gated feed-forward product from its 8-bit checkpoint.
//
// With g, u the checkpoint's values and dh the gradient of h = act(g) u:
//   dg = dh u act'(g),  du = dh act(g),  h = act(g) u
// given as the E4M3 operands of the three gradient products: [dg | du] with
// one scale per 1 x 128 row group (for dX = [dg | du] W), [dg | du] and h
// with one scale per 128 rows of each column (for the weight gradients
// [dg | du]^T X and dY^T h).  Each is rounded once, from FP32.
//
// Rows past M and rows whose m_indices entry is negative count as zero,
// whatever their memory holds.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_device.cuh"
#include "dg_ops.cuh"

namespace dg {
namespace {

struct GatedBackwardArgs {
  const __nv_bfloat16* dh;   // [m, f], row stride lddh
  const uint8_t* gu;         // [m, 2f]
  const uint32_t* gu_sf;     // packed, [ceil(2f / 512), align(m, 4)]
  const int32_t* m_indices;  // nullable
  uint8_t* q;                // [m, 2f]
  uint32_t* sf;              // packed, as gu_sf
  uint8_t* qc;               // [align(m, 128), 2f]
  uint32_t* sfc;             // packed, [ceil(m / 512), 2f]
  uint8_t* hc;               // [align(m, 128), f]
  uint32_t* hsfc;            // packed, [ceil(m / 512), f]
  int64_t m, f, lddh;
  int fblocks, rblocks;
};

// Persistent CTAs of 16 warps, one a SM, over 128 x 128 tiles of h.  Warp w
// holds rows 8w .. 8w+7, lane l columns 4l .. 4l+3: a row group's maximum is
// one warp reduction, a column's 8 values in registers and one exchange
// through shared memory, and dg, du and h (96 values a thread) stay in
// registers from the arithmetic to the five stores.  The next tile is on its way
// into shared memory meanwhile; each thread copies and reads only its own
// pieces, so no barrier guards them, and rows that count as zero are filled
// with zeros instead of being read.
//
// HBM (4 bytes in and 5 out an element of h) leaves time for about 50
// instructions an element and it takes 42, with arithmetic in pairs and a warp's
// 16 row scales worked out by 16 lanes at once; 96 values a thread allow 16 warps
// an SM, whose issue slots are 57-61% busy.  37k x 2048 in 141 us (4.9 TB/s); with
// two tiles on their way 151, with the codes collected in shared memory and
// written by bulk copies 216, with eight columns of four rows a lane 164.
constexpr int kBackRing = 2;
constexpr int kBackThreads = 512;

struct BackStage {
  uint2 dh[8][kBackThreads];
  uint32_t g[8][kBackThreads];
  uint32_t u[8][kBackThreads];
};
struct BackShared {
  BackStage stage[kBackRing];
  float4 cmax[3][16][32];
  float4 cinv[3][32];
};

template <int ACT>
__global__ void __launch_bounds__(kBackThreads, 1) gated_backward_kernel(const GatedBackwardArgs p) {
  extern __shared__ uint4 smem[];
  BackShared& sh = *reinterpret_cast<BackShared*>(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t m_pad = (p.m + 3) / 4 * 4;
  const int tiles = p.fblocks * p.rblocks;
  const int64_t f2 = 2 * p.f;

  // What a fetch needs to know of its rows is loaded a round before it, and the
  // scale words it loads are decoded when their tile is worked on, so that no
  // load is waited for where it is issued.
  // Lanes 0-7: m_indices of the warp's row `lane` of tile t, negative where it counts as zero.
  auto row_index = [&](const TileWalk& w) {
    int index = -1;
    if (w.t < tiles && lane < 8) {
      const int64_t r = (int64_t)w.rb * 128 + warp * 8 + lane;
      if (r < p.m) index = p.m_indices ? __ldg(p.m_indices + r) : 0;
    }
    return index;
  };
  // word: in lanes 0-7 / 8-15 the scale word of g / u in the warp's row (lane % 8), 0 where it counts as zero.
  auto look = [&](const TileWalk& w, int index, uint32_t& live, uint32_t& word) {
    live = __ballot_sync(0xffffffffu, index >= 0);
    word = 0;
    if (lane < 16 && (live >> (lane & 7) & 1))
      word = __ldg(p.gu_sf + (int64_t)((lane < 8 ? w.cb : p.fblocks + w.cb) >> 2) * m_pad + (int64_t)w.rb * 128 +
                   warp * 8 + (lane & 7));
  };
  // Row i of the warp (dh and the checkpoint at d, c) into stage s; zeros where
  // it is not live.  The pointers stay inside the tensors all the same: they
  // walk over the warp's rows before m, and stop on the last one.
  auto fetch_row = [&](int i, int s, bool in, const __nv_bfloat16* d, const uint8_t* c) {
    BackStage& st = sh.stage[s];
    cp_async8_or_zero(&st.dh[i][tid], d, in);
    cp_async4_or_zero(&st.g[i][tid], c, in);
    cp_async4_or_zero(&st.u[i][tid], c + p.f, in);
  };
  struct Source {
    const __nv_bfloat16* d;
    const uint8_t* c;
    int left;  // rows of the warp before m
  };
  auto source = [&](const TileWalk& w) {
    const int64_t row0 = (int64_t)w.rb * 128 + warp * 8;
    const bool some = w.t < tiles && row0 < p.m;
    const int64_t r = some ? row0 : 0;
    const int64_t c = (some ? (int64_t)w.cb * 128 : 0) + lane * 4;
    return Source{p.dh + r * p.lddh + c, p.gu + r * f2 + c, some ? (int)min((int64_t)8, p.m - row0) : 0};
  };

  // live rows and scale words of the tiles in flight, oldest first
  uint32_t live[kBackRing], word[kBackRing];
  const int drb = gridDim.x / p.fblocks, dcb = gridDim.x % p.fblocks;
  TileWalk now, ahead;  // the tile worked on; the tile whose rows are looked up next
  now.init(blockIdx.x, p.fblocks);
  ahead = now;
#pragma unroll
  for (int s = 0; s < kBackRing - 1; ++s) {
    look(ahead, row_index(ahead), live[s], word[s]);
    Source src = source(ahead);
    for (int i = 0; i < 8; ++i) {
      fetch_row(i, s, live[s] >> i & 1, src.d, src.c);
      if (i + 1 < src.left) {
        src.d += p.lddh;
        src.c += f2;
      }
    }
    cp_async_commit();
    ahead.next(p.fblocks, drb, dcb);
  }
  int index = row_index(ahead);
  int at = 0;
  for (; now.t < tiles; now.next(p.fblocks, drb, dcb)) {
    look(ahead, index, live[kBackRing - 1], word[kBackRing - 1]);
    Source src = source(ahead);
    const int free_at = at == 0 ? kBackRing - 1 : at - 1;
    ahead.next(p.fblocks, drb, dcb);
    index = row_index(ahead);
    cp_async_wait<kBackRing - 2>();
    const int rb = now.rb, fb = now.cb;
    const int kmine = lane < 8 ? fb : p.fblocks + fb;
    const float scale = (live[0] >> (lane & 7) & 1) ? scale_of_byte((word[0] >> (8 * (kmine & 3))) & 0xFFu) : 0.0f;
    const int64_t row0 = (int64_t)rb * 128 + warp * 8;
    const int64_t col = (int64_t)fb * 128 + lane * 4;
    const BackStage& st = sh.stage[at];
    if (++at == kBackRing) at = 0;

    float2 dg[8][2], du[8][2], h[8][2];
    float mg[4] = {}, mu[4] = {}, mh[4] = {};
    float rowmax = 0.0f;  // lanes 0-7: of dg in the row (lane % 8); lanes 8-15: of du
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // a row of the next tile, copied row by row between the arithmetic
      fetch_row(i, free_at, live[kBackRing - 1] >> i & 1, src.d, src.c);
      if (i + 1 < src.left) {
        src.d += p.lddh;
        src.c += f2;
      }
      const float sg = __shfl_sync(0xffffffffu, scale, i), su = __shfl_sync(0xffffffffu, scale, 8 + i);
      const uint2 dv = st.dh[i][tid];
      float g[4], u[4];
      e4m3x4_to_float(st.g[i][tid], g);
      e4m3x4_to_float(st.u[i][tid], u);
      const float2 d[2] = {make_float2(bf16_lo(dv.x), bf16_hi(dv.x)), make_float2(bf16_lo(dv.y), bf16_hi(dv.y))};
      float rg = 0.0f, ru = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float2 a, da;
        gate_act_grad2<ACT>(mul2(make_float2(g[2 * c], g[2 * c + 1]), sg), a, da);
        const float2 uu = mul2(make_float2(u[2 * c], u[2 * c + 1]), su);
        dg[i][c] = mul2(mul2(d[c], uu), da);
        du[i][c] = mul2(d[c], a);
        h[i][c] = mul2(a, uu);
        rg = abs_max2(rg, dg[i][c]);
        ru = abs_max2(ru, du[i][c]);
      }
      rg = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rg)));
      ru = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(ru)));
      if (lane == i) rowmax = rg;
      if (lane == 8 + i) rowmax = ru;
    }
    cp_async_commit();
#pragma unroll
    for (int i = 0; i < 8; i += 2)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mg[2 * c] = abs_max3(mg[2 * c], dg[i][c].x, dg[i + 1][c].x);
        mg[2 * c + 1] = abs_max3(mg[2 * c + 1], dg[i][c].y, dg[i + 1][c].y);
        mu[2 * c] = abs_max3(mu[2 * c], du[i][c].x, du[i + 1][c].x);
        mu[2 * c + 1] = abs_max3(mu[2 * c + 1], du[i][c].y, du[i + 1][c].y);
        mh[2 * c] = abs_max3(mh[2 * c], h[i][c].x, h[i + 1][c].x);
        mh[2 * c + 1] = abs_max3(mh[2 * c + 1], h[i][c].y, h[i + 1][c].y);
      }
    sh.cmax[0][warp][lane] = make_float4(mg[0], mg[1], mg[2], mg[3]);
    sh.cmax[1][warp][lane] = make_float4(mu[0], mu[1], mu[2], mu[3]);
    sh.cmax[2][warp][lane] = make_float4(mh[0], mh[1], mh[2], mh[3]);

    __syncthreads();
    if (tid < 384) {
      const int k = tid / 128, c = tid % 128;
      const float* s = reinterpret_cast<const float*>(&sh.cmax[k][0][0]) + c;
      float a = 0.0f;
#pragma unroll
      for (int w = 0; w < 16; ++w) a = fmaxf(a, s[w * 128]);
      const uint32_t b = scale_byte(a);
      reinterpret_cast<float*>(sh.cinv[k])[c] = inverse_of_byte(b);
      const int64_t cc = (int64_t)fb * 128 + c;
      uint32_t* w = k == 2 ? p.hsfc + (int64_t)(rb >> 2) * p.f + cc
                           : p.sfc + (int64_t)(rb >> 2) * f2 + (k ? p.f : 0) + cc;
      store_scale_byte(w, rb, rb == p.rblocks - 1, b);
    }
    // the rows' scales and codes, while the columns' scales are worked out
    const uint32_t byte = scale_byte(rowmax);
    const float inv = inverse_of_byte(byte);
    if (lane < 16 && row0 + (lane & 7) < m_pad) {
      const int64_t r = row0 + (lane & 7);
      store_scale_byte(p.sf + (int64_t)(kmine >> 2) * m_pad + r, kmine, kmine == 2 * p.fblocks - 1, r < p.m ? byte : 0u);
    }
    uint8_t* qr = p.q + row0 * f2 + col;
    const int here = (int)min((int64_t)8, p.m - row0);  // rows of the warp inside m
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float ig = __shfl_sync(0xffffffffu, inv, i), iu = __shfl_sync(0xffffffffu, inv, 8 + i);
      if (i < here) {
        *reinterpret_cast<uint32_t*>(qr) = e4m3x4(mul2(dg[i][0], ig), mul2(dg[i][1], ig));
        *reinterpret_cast<uint32_t*>(qr + p.f) = e4m3x4(mul2(du[i][0], iu), mul2(du[i][1], iu));
      }
      qr += f2;
    }
    __syncthreads();
    const float4 ig = sh.cinv[0][lane], iu = sh.cinv[1][lane], ih = sh.cinv[2][lane];
    const float2 ig0 = make_float2(ig.x, ig.y), ig1 = make_float2(ig.z, ig.w);
    const float2 iu0 = make_float2(iu.x, iu.y), iu1 = make_float2(iu.z, iu.w);
    const float2 ih0 = make_float2(ih.x, ih.y), ih1 = make_float2(ih.z, ih.w);
    uint8_t* qc = p.qc + row0 * f2 + col;
    uint8_t* hc = p.hc + row0 * p.f + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      *reinterpret_cast<uint32_t*>(qc) = e4m3x4(mul2(dg[i][0], ig0), mul2(dg[i][1], ig1));
      *reinterpret_cast<uint32_t*>(qc + p.f) = e4m3x4(mul2(du[i][0], iu0), mul2(du[i][1], iu1));
      *reinterpret_cast<uint32_t*>(hc) = e4m3x4(mul2(h[i][0], ih0), mul2(h[i][1], ih1));
      qc += f2;
      hc += p.f;
    }
#pragma unroll
    for (int s = 0; s < kBackRing - 1; ++s) {
      live[s] = live[s + 1];
      word[s] = word[s + 1];
    }
  }
  cp_async_wait<0>();
}

}  // namespace

cudaError_t gated_backward_launch(const void* dh, int64_t lddh, const void* gu, const void* gu_sf,
                                  const int32_t* m_indices, void* q, void* sf, void* qc, void* sfc,
                                  void* hc, void* hsfc, int64_t m, int64_t f, int activation, int sms,
                                  bool pdl, cudaStream_t stream) {
  GatedBackwardArgs p;
  p.dh = (const __nv_bfloat16*)dh;
  p.gu = (const uint8_t*)gu;
  p.gu_sf = (const uint32_t*)gu_sf;
  p.m_indices = m_indices;
  p.q = (uint8_t*)q;
  p.sf = (uint32_t*)sf;
  p.qc = (uint8_t*)qc;
  p.sfc = (uint32_t*)sfc;
  p.hc = (uint8_t*)hc;
  p.hsfc = (uint32_t*)hsfc;
  p.m = m;
  p.f = f;
  p.lddh = lddh;
  p.fblocks = (int)(f / 128);
  p.rblocks = (int)((m + 127) / 128);
  const int tiles = p.fblocks * p.rblocks;
  const dim3 grid((unsigned)(tiles < sms ? tiles : sms));
  auto kern = activation == DG_ACT_SILU ? gated_backward_kernel<DG_ACT_SILU> : gated_backward_kernel<DG_ACT_GELU_TANH>;
  cudaError_t e = set_smem(kern, sizeof(BackShared), sizeof(BackShared));
  if (e != cudaSuccess) return e;
  return launch_op(kern, grid, kBackThreads, sizeof(BackShared), pdl, stream, p);
}

}  // namespace dg
