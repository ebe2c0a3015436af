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

// One CTA of 16 warps per 128 x 128 tile of h: warp w holds rows 8w .. 8w+7,
// lane l columns 4l .. 4l+3, so a row group's maximum is one warp reduction
// and a column's maximum is 8 values in registers and one exchange through
// shared memory.
template <int ACT>
__global__ void __launch_bounds__(512) gated_backward_kernel(const GatedBackwardArgs p) {
  __shared__ uint4 cmax[3][16][32];
  __shared__ float4 cinv[3][32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rb = blockIdx.x / p.fblocks, fb = blockIdx.x % p.fblocks;
  const int64_t row0 = (int64_t)rb * 128 + warp * 8;
  const int64_t col = (int64_t)fb * 128 + lane * 4;
  const int64_t m_pad = (p.m + 3) / 4 * 4;
  const int kg = fb, ku = p.fblocks + fb;  // column blocks of g and u in [g | u]
  float dg[8][4], du[8][4], h[8][4];
  uint32_t mg[4] = {}, mu[4] = {}, mh[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + i;
    uint2 dhv = make_uint2(0u, 0u);
    uint32_t gc = 0u, uc = 0u;
    float sg = 0.0f, su = 0.0f;
    if (r < p.m && (!p.m_indices || __ldg(p.m_indices + r) >= 0)) {
      dhv = ld_stream_u2(p.dh + r * p.lddh + col);
      gc = __ldg(reinterpret_cast<const uint32_t*>(p.gu + r * 2 * p.f + col));
      uc = __ldg(reinterpret_cast<const uint32_t*>(p.gu + r * 2 * p.f + p.f + col));
      sg = scale_of_byte((__ldg(p.gu_sf + (int64_t)(kg >> 2) * m_pad + r) >> (8 * (kg & 3))) & 0xFFu);
      su = scale_of_byte((__ldg(p.gu_sf + (int64_t)(ku >> 2) * m_pad + r) >> (8 * (ku & 3))) & 0xFFu);
    }
    const float d[4] = {bf16_lo(dhv.x), bf16_hi(dhv.x), bf16_lo(dhv.y), bf16_hi(dhv.y)};
    float g[4], u[4];
    e4m3x4_to_float(gc, g);
    e4m3x4_to_float(uc, u);
    uint32_t rg = 0, ru = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float a, da;
      gate_act_grad<ACT>(g[c] * sg, a, da);
      const float uu = u[c] * su;
      dg[i][c] = d[c] * uu * da;
      du[i][c] = d[c] * a;
      h[i][c] = a * uu;
      const uint32_t bg = abs_bits(dg[i][c]), bu = abs_bits(du[i][c]);
      rg = max(rg, bg);
      ru = max(ru, bu);
      mg[c] = max(mg[c], bg);
      mu[c] = max(mu[c], bu);
      mh[c] = max(mh[c], abs_bits(h[i][c]));
    }
    const int eg = scale_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, rg)));
    const int eu = scale_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, ru)));
    if (r < p.m) {
      const float ig = pow2f(-eg), iu = pow2f(-eu);
      uint8_t* qr = p.q + r * 2 * p.f + col;
      *reinterpret_cast<uint32_t*>(qr) = e4m3x4(dg[i][0] * ig, dg[i][1] * ig, dg[i][2] * ig, dg[i][3] * ig);
      *reinterpret_cast<uint32_t*>(qr + p.f) = e4m3x4(du[i][0] * iu, du[i][1] * iu, du[i][2] * iu, du[i][3] * iu);
    }
    if (lane == 0 && r < m_pad) {
      const bool in = r < p.m;
      store_scale_byte(p.sf + (int64_t)(kg >> 2) * m_pad + r, kg, false, in ? (uint32_t)(eg + 127) : 0u);
      store_scale_byte(p.sf + (int64_t)(ku >> 2) * m_pad + r, ku, ku == 2 * p.fblocks - 1,
                       in ? (uint32_t)(eu + 127) : 0u);
    }
  }
  cmax[0][warp][lane] = make_uint4(mg[0], mg[1], mg[2], mg[3]);
  cmax[1][warp][lane] = make_uint4(mu[0], mu[1], mu[2], mu[3]);
  cmax[2][warp][lane] = make_uint4(mh[0], mh[1], mh[2], mh[3]);
  __syncthreads();
  if (threadIdx.x < 384) {
    const int k = threadIdx.x / 128, c = threadIdx.x % 128;
    const uint32_t* s = reinterpret_cast<const uint32_t*>(&cmax[k][0][0]) + c;
    uint32_t a = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) a = max(a, s[w * 128]);
    const int e = scale_exponent(__uint_as_float(a));
    reinterpret_cast<float*>(cinv[k])[c] = pow2f(-e);
    const int64_t cc = (int64_t)fb * 128 + c;
    uint32_t* w = k == 2 ? p.hsfc + (int64_t)(rb >> 2) * p.f + cc
                         : p.sfc + (int64_t)(rb >> 2) * 2 * p.f + (k ? p.f : 0) + cc;
    store_scale_byte(w, rb, rb == p.rblocks - 1, (uint32_t)(e + 127));
  }
  __syncthreads();
  const float4 ig = cinv[0][lane], iu = cinv[1][lane], ih = cinv[2][lane];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + i;
    uint8_t* qr = p.qc + r * 2 * p.f + col;
    *reinterpret_cast<uint32_t*>(qr) = e4m3x4(dg[i][0] * ig.x, dg[i][1] * ig.y, dg[i][2] * ig.z, dg[i][3] * ig.w);
    *reinterpret_cast<uint32_t*>(qr + p.f) = e4m3x4(du[i][0] * iu.x, du[i][1] * iu.y, du[i][2] * iu.z, du[i][3] * iu.w);
    *reinterpret_cast<uint32_t*>(p.hc + r * p.f + col) =
        e4m3x4(h[i][0] * ih.x, h[i][1] * ih.y, h[i][2] * ih.z, h[i][3] * ih.w);
  }
}

}  // namespace

cudaError_t gated_backward_launch(const void* dh, int64_t lddh, const void* gu, const void* gu_sf,
                                  const int32_t* m_indices, void* q, void* sf, void* qc, void* sfc,
                                  void* hc, void* hsfc, int64_t m, int64_t f, int activation, bool pdl,
                                  cudaStream_t stream) {
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
  const dim3 grid((unsigned)(p.fblocks * p.rblocks));
  if (activation == DG_ACT_SILU)
    return launch_op(gated_backward_kernel<DG_ACT_SILU>, grid, 512, 0, pdl, stream, p);
  return launch_op(gated_backward_kernel<DG_ACT_GELU_TANH>, grid, 512, 0, pdl, stream, p);
}

}  // namespace dg
