// Gated feed-forward product for one to four tokens (dense form), without the
// tensor cores: a warp reads the rows of Wg and Wu of one column of h once and
// multiplies them with every token.
//
// Bound by reading W: a whole SM's warps have their loads in flight at once,
// with nothing in between but registers, where the tensor-core kernels pay for
// barriers, scale layouts, TMEM and the exchange of partial sums before the
// first and after the last byte.  A code costs about 2.5 instructions: it is
// decoded in pairs by way of halves (exact) and multiplied in FP32 pairs; the
// tokens wait in shared memory as FP32, their own scales multiplied in (exact),
// in the order the lanes read them.
//
// One token, K = 7168, F = 2048: 8.5-8.8 us (29 MB, 3.4 TB/s; a plain streaming
// read of as many bytes takes 7.1-7.4), F = 4096 13.8 us (4.2 TB/s).
//
// A group of 128 columns with one scale is 8 CTAs of 16 columns: for 8-bit
// results they form a cluster and tell one another their columns' maxima, which
// at F = 2048 costs 5 us (13.4-13.9; K = 1024 1-1.6 us).
#include <algorithm>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "gated_gemm.h"

namespace dg {
namespace {

constexpr int kGvWarps = 16;   // columns of h a CTA
constexpr int kGvCluster = 8;  // CTAs of a group of 128 columns
constexpr int kGvRing = 4;     // steps of 512 columns of W on their way into shared memory
constexpr int kGvRingBytes = kGvRing * 2 * kGvWarps * 32 * 16;
constexpr int kGvMaxSmem = 220 * 1024;  // dynamic shared memory of a CTA, at most

// Sixteen products of a lane: codes w with the tokens' values at xs.
template <int M>
__device__ __forceinline__ void gv_multiply(const uint4& w, const float4* xs, int64_t token, float scale,
                                            float (&acc)[M]) {
  float f[16];
  const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) e4m3x4_to_float(c[i], *reinterpret_cast<float(*)[4]>(&f[4 * i]));
#pragma unroll
  for (int t = 0; t < M; ++t) {
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = xs[t * token + i * 32];
      s = fma2(make_float2(f[4 * i], f[4 * i + 1]), make_float2(x.x, x.y), s);
      s = fma2(make_float2(f[4 * i + 2], f[4 * i + 3]), make_float2(x.z, x.w), s);
    }
    acc[t] = fmaf(s.x + s.y, scale, acc[t]);
  }
}

struct GemvArgs {
  GatedArgs g;
  const uint8_t* a;
  const uint32_t* sfa;
  const uint8_t* b;
  const uint32_t* sfb;
  int64_t lda, ldb;
  int32_t n_pad;  // align(2f, 4)
};

template <int M, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGvWarps, 2) fp8_gated_gemv_kernel(const GemvArgs p) {
  extern __shared__ float4 shared[];
  uint4* const ring = reinterpret_cast<uint4*>(shared);  // [kGvRing][Wg, Wu][threads]: each thread's own pieces
  float4* const xs = shared + kGvRingBytes / 16;         // [M][steps of 512 columns][4][32 lanes]
  __shared__ float vals[3][M][kGvWarps];              // g, u, h of the CTA's columns
  __shared__ uint32_t maxima[3][M][kGvCluster];       // of every CTA of the cluster
  // A CTA's shared memory may be written by the others of its cluster once it
  // runs: every thread says so here, and the maxima are sent only after all have.
  if constexpr (CLUSTER) cluster_arrive();
  const GatedArgs& ga = p.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int K = ga.base.k, m = ga.base.m;
  const int steps = (K + 511) / 512;
  const int col = blockIdx.x * kGvWarps + warp;  // of h
  const bool on = col < ga.f;
  const uint8_t* wg = p.b + (int64_t)(on ? col : 0) * p.ldb + lane * 16;
  const uint8_t* wu = wg + (int64_t)ga.f * p.ldb;
  griddep_wait();
  griddep_launch_dependents();

  // the first steps of W are on their way while the tokens are laid out
  auto slot = [&](int s, int which) { return ring + (s * 2 + which) * blockDim.x + threadIdx.x; };
  auto fetch = [&](int it) {
    if (it < steps) {
      const bool in = on && it * 512 + lane * 16 < K;
      cp_async16_or_zero(slot(it % kGvRing, 0), wg + (in ? it * 512 : 0), in);
      cp_async16_or_zero(slot(it % kGvRing, 1), wu + (in ? it * 512 : 0), in);
    }
    cp_async_commit();
  };
  for (int it = 0; it < kGvRing - 1; ++it) fetch(it);
  const int64_t token = (int64_t)steps * 128;  // float4s of one token
  for (int i = threadIdx.x; i < M * steps * 32; i += blockDim.x) {
    // 16 columns of a token
    const int t = i / (steps * 32), s = i % (steps * 32) / 32, l = i % 32;
    const int c = s * 512 + l * 16;
    float4* to = xs + t * token + s * 128 + l;
    uint4 q = make_uint4(0, 0, 0, 0);
    float scale = 0.0f;
    if (t < m && c < K) {
      q = __ldg(reinterpret_cast<const uint4*>(p.a + (int64_t)t * p.lda + c));
      scale = scale_of_byte((__ldg(p.sfa + (int64_t)s * ga.m_pad + t) >> (8 * (l / 8))) & 0xFFu);
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4];
      e4m3x4_to_float(w[j], f);
      to[j * 32] = make_float4(f[0] * scale, f[1] * scale, f[2] * scale, f[3] * scale);
    }
  }
  __syncthreads();

  float ag[M], au[M];
#pragma unroll
  for (int t = 0; t < M; ++t) ag[t] = au[t] = 0.0f;
  uint32_t sg = 0, su = 0;  // lane l: the scale words of step 32 n + l
  for (int it = 0; it < steps; ++it) {
    fetch(it + kGvRing - 1);  // into the slot read in the last step, by this thread alone
    if (it % 32 == 0) {
      const bool in = on && it + lane < steps;
      sg = in ? __ldg(p.sfb + (int64_t)(it + lane) * p.n_pad + col) : 0u;
      su = in ? __ldg(p.sfb + (int64_t)(it + lane) * p.n_pad + ga.f + col) : 0u;
    }
    cp_async_wait<kGvRing - 1>();
    const uint32_t bg = __shfl_sync(0xffffffffu, sg, it & 31), bu = __shfl_sync(0xffffffffu, su, it & 31);
    const float4* x = xs + (int64_t)it * 128 + lane;
    gv_multiply<M>(*slot(it % kGvRing, 0), x, token, scale_of_byte((bg >> (8 * (lane / 8))) & 0xFFu), ag);
    gv_multiply<M>(*slot(it % kGvRing, 1), x, token, scale_of_byte((bu >> (8 * (lane / 8))) & 0xFFu), au);
  }
#pragma unroll
  for (int t = 0; t < M; ++t) {
    const float v = warp_sum2(ag[t], au[t]);  // lanes 0-15: g, lanes 16-31: u
    const float g = __shfl_sync(0xffffffffu, v, 0), u = __shfl_sync(0xffffffffu, v, 16);
    const float h =
        (ga.activation == DG_ACT_SILU ? gate_act<DG_ACT_SILU>(g) : gate_act<DG_ACT_GELU_TANH>(g)) * u;
    if (lane == 0) {
      if (!CLUSTER || !ga.hq) {
        if (on && t < m) ga.h[(int64_t)t * ga.ldh + col] = __float2bfloat16_rn(h);
      }
      if (CLUSTER) {
        vals[0][t][warp] = g;
        vals[1][t][warp] = u;
        vals[2][t][warp] = h;
      }
    }
  }
  if constexpr (CLUSTER) {
    const uint32_t rank = cluster_ctarank();
    __syncthreads();
    cluster_wait();
    // warp w: the maximum of one of the 3 M rows of values, told to all 8 CTAs
    for (int i = warp; i < 3 * M; i += kGvWarps) {
      const float v = lane < kGvWarps ? vals[i / M][i % M][lane] : 0.0f;
      const uint32_t mx = __reduce_max_sync(0xffffffffu, magnitude(v));
      if (lane < kGvCluster)
        st_shared_cluster_u32(mapa_shared(smem_u32(&maxima[i / M][i % M][rank]), (uint32_t)lane), mx);
    }
    cluster_sync_all();  // the maxima have landed, and no CTA leaves before its own are told
    const int fb = ga.f / 128, group = blockIdx.x / kGvCluster;
    for (int i = threadIdx.x; i < 3 * M * kGvWarps; i += blockDim.x) {
      const int k = i / (M * kGvWarps), t = i / kGvWarps % M, w = i % kGvWarps;
      if (k == 2 ? !ga.hq : !ga.cq) continue;
      uint32_t mx = 0;
#pragma unroll
      for (int r = 0; r < kGvCluster; ++r) mx = max(mx, maxima[k][t][r]);
      const uint32_t e = scale_byte(__uint_as_float(mx));
      const int c = blockIdx.x * kGvWarps + w;
      const int blocks = k == 2 ? fb : 2 * fb, block = k == 1 ? fb + group : group;
      if (t < m) {
        uint8_t* q = k == 2 ? ga.hq + (int64_t)t * ga.f + c : ga.cq + (int64_t)t * 2 * ga.f + (k ? ga.f : 0) + c;
        *q = (uint8_t)(cvt_e4m3x2(vals[k][t][w] * inverse_of_byte(e), 0.0f) & 0xFFu);
      }
      if (w == 0 && rank == 0) {
        uint32_t* sf = (k == 2 ? ga.hsf : ga.csf) + (int64_t)(block >> 2) * ga.m_pad;
        // a token's scale, and with the last token the alignment padding's zeros
        if (t < m) store_scale_byte(sf + t, block, block == blocks - 1, e);
        if (t == M - 1)
          for (int r = m; r < ga.m_pad; ++r) store_scale_byte(sf + r, block, block == blocks - 1, 0u);
      }
    }
  }
}

template <int M>
cudaError_t gv_launch(const GemvArgs& p, size_t smem, cudaStream_t stream) {
  const bool cluster = p.g.hq || p.g.cq;
  auto kern = cluster ? fp8_gated_gemv_kernel<M, true> : fp8_gated_gemv_kernel<M, false>;
  cudaError_t e = set_smem(kern, smem, kGvMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (cluster) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = kGvCluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (p.g.base.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.g.f + kGvWarps - 1) / kGvWarps), 1, 1);
  cfg.blockDim = dim3(32 * kGvWarps, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

// Measured against the kernel with swapped operand roles (weights from HBM, us
// in a graph, this kernel / that one).  F = 2048, BF16: K = 7168, 1 token 8.7 /
// 13.7, 2 tokens 10.4 / 13.9, 4 tokens 17.0 / 14.1; K = 1024, 4 tokens 5.3 /
// 7.2; F = 4096, K = 7168: 1 token 13.8 / 14.9, 2 tokens 19.0 / 15.2.  With
// 8-bit results, F = 2048: K = 7168, 1 token 13.4 / 14.7, 2 tokens 21.4 / 14.9;
// K = 1024, 4 tokens 7.5 / 8.0; F = 4096, K = 7168, 1 token 14.9 / 16.0.  So: one token always; two where all CTAs run
// at once; three and four where they do and K is short, since each token adds
// its own products to every code.  Clusters of 8 need two CTAs an SM for that.
// The grid is as large as F asks, each CTA on whichever SM is free: under a limit
// of the SMs to use it is taken only where it has no more CTAs than those.
bool gated_gemv_takes(int64_t m, int64_t f, int64_t k, bool eight_bit, int sms, bool limited) {
  if (m < 1 || m > 4) return false;
  const int64_t tokens = m <= 2 ? m : 4;
  const int64_t smem = tokens * ((k + 511) / 512) * 2048 + kGvRingBytes;  // the tokens as FP32
  if (smem > kGvMaxSmem) return false;
  if (limited && (f + kGvWarps - 1) / kGvWarps > sms) return false;
  if (m == 1) return true;
  const int64_t per_sm = std::min<int64_t>(2, kGvMaxSmem / (smem + 2048));
  const bool once = (f + kGvWarps - 1) / kGvWarps <= per_sm * sms && (!eight_bit || per_sm == 2);
  return once && (m == 2 || k <= 2048);
}

cudaError_t gated_gemv_launch(const void* a, const void* sfa, const void* b, const void* sfb, int64_t lda, int64_t ldb,
                              const GatedArgs& args, cudaStream_t stream) {
  GemvArgs p;
  p.g = args;
  p.a = (const uint8_t*)a;
  p.sfa = (const uint32_t*)sfa;
  p.b = (const uint8_t*)b;
  p.sfb = (const uint32_t*)sfb;
  p.lda = lda;
  p.ldb = ldb;
  p.n_pad = (2 * args.f + 3) / 4 * 4;
  const int m = args.base.m;
  const size_t step = (size_t)((args.base.k + 511) / 512) * 2048;  // one token
  if (m == 1) return gv_launch<1>(p, kGvRingBytes + step, stream);
  if (m == 2) return gv_launch<2>(p, kGvRingBytes + 2 * step, stream);
  return gv_launch<4>(p, kGvRingBytes + 4 * step, stream);
}

}  // namespace dg
