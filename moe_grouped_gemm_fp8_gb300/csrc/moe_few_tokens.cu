// A whole mixture-of-experts layer for a few tokens in two kernels.
//
//   l = x r^T, the k best experts of each token and their weights w
//   g = x Wg^T, u = x Wu^T, h = act(g) u   (of each chosen expert)
//   y = c + sum over the chosen of w h Wd^T
//
// The first kernel computes the scores and brings x into the form that the
// products read.  The second is one cooperative launch: every CTA picks the
// experts for itself from the scores (the same way everywhere), then all share
// out the rows of the hit experts' Wg and Wu, meet at a barrier over the grid,
// and share out the rows of Wd.
//
// Bound by reading the hit experts' weights once.  Each goes through the tensor
// cores with all tokens of its expert at once (stream_mma.cuh).  x and h are
// carried as halves with a power of two per 128 columns: 11 bits (BF16 x
// exactly, but for values 2^29 below the largest of the 128), so that the only
// roundings are those and the result's own.
#include <algorithm>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "moe.h"
#include "stream_mma.cuh"

namespace dg {
namespace {

constexpr int kMoeWarps = 16;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMoeRing = 4;
constexpr int kMoeSplit = 4;  // warps that share the columns of 16 rows of Wg and Wu
constexpr int kMoeSlots = 1024;  // results of 16 rows of Wd waiting for their sum: (part, pair)
constexpr int kScoreThreads = 256;
constexpr int kScoreTokens = 8;  // tokens of a CTA of the first kernel

// ---------------------------------------------------------------- scores, and x as halves

// Adds p to hi + lo without loss (two-term sum).
__device__ __forceinline__ void add_exactly(float& hi, float& lo, float p) {
  const float t = hi + p;
  const float z = t - hi;
  lo += (hi - (t - z)) + (p - z);
  hi = t;
}

// The power of two that brings a maximum of magnitudes into [2^14, 2^15), and
// its inverse; 1 for 0.
__device__ __forceinline__ float half_scale(float amax, float& inverse) {
  int e = (int)(__float_as_uint(amax) >> 23) - 127 - 14;
  e = amax > 0.0f ? max(e, -112) : 0;
  inverse = pow2f(-e);
  return pow2f(e);
}
// |v|, 0 where v is infinite or no number: those stay what they are as halves
// and must not set the scale of the others.
__device__ __forceinline__ float finite_magnitude(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.0f;
}

// The row count of a padded batch; out of range: an error, and the nearest.
__device__ __forceinline__ int live_tokens(const MoeArgs& p) {
  if (!p.num_tokens) return p.tokens;
  const int n = __ldg(p.num_tokens);
  if (n < 0 || n > p.tokens) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.err, DG_ERR_DEVICE_BAD_INDEX, kSiteMoeTokens);
    return n < 0 ? 0 : p.tokens;
  }
  return n;
}

template <class R>
__device__ __forceinline__ void load8(const R* p, float (&f)[8]) {
  if constexpr (sizeof(R) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    f[0] = bf16_lo(a.x); f[1] = bf16_hi(a.x); f[2] = bf16_lo(a.y); f[3] = bf16_hi(a.y);
    f[4] = bf16_lo(a.z); f[5] = bf16_hi(a.z); f[6] = bf16_lo(a.w); f[7] = bf16_hi(a.w);
  }
}

// CTA (expert, 8 tokens): their scores; CTAs after those: a token's halves.
//
// The order of near scores decides which expert runs, so they are summed as if
// in 48 bits: BF16 products are exact in FP32 (with FP32 weights the product's
// rounding error is added too), and every sum keeps its rounding error.
template <class R>
__global__ void __launch_bounds__(kScoreThreads) moe_scores_kernel(const MoeArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int live = live_tokens(p);
  const int groups = (p.tokens + kScoreTokens - 1) / kScoreTokens;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int at = blockIdx.x;
  // the second kernel's counters
  for (int i = blockIdx.x * kScoreThreads + tid; i < p.counters; i += gridDim.x * kScoreThreads) p.counter[i] = 0;
  if (at >= p.experts * groups) {
    at -= p.experts * groups;
    if (at >= live) return;
    // 16 lanes take 128 columns of the token, 8 each
    const __nv_bfloat16* x = p.x + (int64_t)at * p.ldx;
    for (int c = tid * 8; c < (p.d + 511) / 512 * 512; c += kScoreThreads * 8) {
      float f[8] = {};
      const bool in = c < p.d;
      if (in) load8(x + c, f);
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_magnitude(f[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float inv;
      const float s = half_scale(m, inv);
      if (in) {
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i] * inv, f[2 * i + 1] * inv);
        *reinterpret_cast<uint4*>(p.xh + (int64_t)at * p.d + (c & ~127) + stream_half_at(c & 127)) =
            *reinterpret_cast<const uint4*>(h);
        if ((c & 127) == 0) p.xs[(int64_t)at * (p.d / 128) + c / 128] = s;
      }
    }
    return;
  }
  const int e = at % p.experts, t0 = at / p.experts * kScoreTokens;
  const int n = min(live - t0, kScoreTokens);
  if (n <= 0) return;
  const R* w = reinterpret_cast<const R*>(p.router) + (int64_t)e * p.d;
  const __nv_bfloat16* x = p.x + (int64_t)t0 * p.ldx;
  float hi[kScoreTokens], lo[kScoreTokens];
#pragma unroll
  for (int t = 0; t < kScoreTokens; ++t) hi[t] = lo[t] = 0.0f;
  for (int c = tid * 8; c < p.d; c += kScoreThreads * 8) {
    float wf[8];
    load8(w + c, wf);
#pragma unroll
    for (int t = 0; t < kScoreTokens; ++t) {
      if (t < n) {
        float xf[8];
        load8(x + (int64_t)t * p.ldx + c, xf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = wf[i] * xf[i];
          if constexpr (sizeof(R) == 4) lo[t] += fmaf(wf[i], xf[i], -v);
          add_exactly(hi[t], lo[t], v);
        }
      }
    }
  }
  __shared__ double sums[kScoreThreads / 32][kScoreTokens];
#pragma unroll
  for (int t = 0; t < kScoreTokens; ++t) {
    if (t < n) {
      double v = (double)hi[t] + (double)lo[t];
      // where a sum overflowed its error is no number
      if (!(fabsf(lo[t]) < INFINITY)) v = (double)hi[t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) sums[warp][t] = v;
    }
  }
  __syncthreads();
  if (tid < n) {
    double v = 0.0;
    for (int i = 0; i < kScoreThreads / 32; ++i) v += sums[i][tid];
    v += 0.0;  // -0 and 0 are one score
    const int64_t to = (int64_t)(t0 + tid) * p.experts + e;
    p.logits[to] = v;
    if (p.router_bias) p.select[to] = 1.0 / (1.0 + exp(-v)) + (double)__ldg(p.router_bias + e);
  }
}

// ---------------------------------------------------------------- the layer

struct MoeShared {
  int32_t pair_token[kMoeMaxTokens * kMoeMaxTopK];  // pairs in the order of their experts: the token
  int16_t pair_of[kMoeMaxTokens * kMoeMaxTopK];     // (token, j) -> its pair
  int16_t chosen[kMoeMaxTokens * kMoeMaxTopK];      // (token, j) -> expert
  float weight[kMoeMaxTokens * kMoeMaxTopK];        // (token, j)
  int16_t hit_expert[kMoeMaxExperts];               // hit experts, ascending
  int16_t hit_first[kMoeMaxExperts + 1];            // their first pairs
  int32_t scan[kMoeWarps];
  int32_t hits;
  int32_t last;  // abort flag of the barrier
};

// Order-preserving 64-bit integers of scores, 0 for what is no number.
__device__ __forceinline__ uint64_t score_key(double v) {
  if (!(v == v)) return 0;
  const int64_t b = __double_as_longlong(v);
  return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

// A warp picks the experts of token t and their weights.
__device__ void moe_pick(const MoeArgs& p, MoeShared& sh, int t, int lane) {
  const double* logits = p.logits + (int64_t)t * p.experts;
  const double* by = p.router_bias ? p.select + (int64_t)t * p.experts : logits;
  constexpr int kPer = kMoeMaxExperts / 32;
  uint64_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < p.experts ? score_key(__ldg(by + e)) : 0;
  }
  uint32_t taken = 0;  // bit i: expert i * 32 + lane is chosen, or is none
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i * 32 + lane >= p.experts) taken |= 1u << i;
  int mine = 0;  // lane j: the j-th choice
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = 0;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i)  // among equals the lowest stays
      if (!(taken >> i & 1u) && (key[i] >= best || at == 0x7fffffff)) {
        best = key[i];
        at = i * 32 + lane;
      }
    const bool any = at != 0x7fffffff;
    const uint32_t h = __reduce_max_sync(0xffffffffu, any ? (uint32_t)(best >> 32) : 0u);
    const bool c1 = any && (uint32_t)(best >> 32) == h;
    const uint32_t l = __reduce_max_sync(0xffffffffu, c1 ? (uint32_t)best : 0u);
    const bool c2 = c1 && (uint32_t)best == l;
    const int e = __reduce_min_sync(0xffffffffu, c2 ? at : 0x7fffffff);
    if ((e & 31) == lane) taken |= 1u << (e >> 5);
    if (lane == j) mine = e;
  }
  // weights: softmax over the chosen (renormalised) or over all, or the logistic function
  const bool on = lane < p.top_k;
  const double l = on ? __ldg(logits + mine) : -INFINITY;
  float w;
  if (p.score == DG_SCORE_SOFTMAX) {
    double m = l;
    if (!p.renormalize)
      for (int e = lane; e < p.experts; e += 32) m = fmax(m, __ldg(logits + e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    w = on ? expf((float)(l - m)) : 0.0f;
    float sum = w;
    if (!p.renormalize) {
      sum = 0.0f;
      for (int e = lane; e < p.experts; e += 32) sum += expf((float)(__ldg(logits + e) - m));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w /= sum;
  } else {
    w = on ? 1.0f / (1.0f + expf((float)-l)) : 0.0f;
    if (p.renormalize) {
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      w /= sum;
    }
  }
  w *= p.scale;
  if (on) {
    sh.chosen[t * p.top_k + lane] = (int16_t)mine;
    sh.weight[t * p.top_k + lane] = w;
    if (blockIdx.x == 0) {
      p.chosen_out[(int64_t)t * p.top_k + lane] = mine;
      p.weight_out[(int64_t)t * p.top_k + lane] = w;
    }
  }
}

// Pairs (token, j) in the order of (expert, token).
__device__ void moe_sort(const MoeArgs& p, MoeShared& sh, int live) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = live * p.top_k;
  int count = 0;
  if (tid < p.experts)
    for (int i = 0; i < pairs; ++i) count += sh.chosen[i] == tid;
  // prefix sums over the experts of (pairs, hit experts) in one word
  int v = count | (count > 0 ? 1 << 16 : 0);
  const int own = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) sh.scan[warp] = v;
  __syncthreads();
  int before = v - own;
  for (int i = 0; i < warp; ++i) before += sh.scan[i];
  if (count > 0) {
    const int hit = before >> 16;
    int at = before & 0xffff;
    sh.hit_expert[hit] = (int16_t)tid;
    sh.hit_first[hit] = (int16_t)at;
    for (int i = 0; i < pairs; ++i)
      if (sh.chosen[i] == tid) {
        sh.pair_token[at] = i / p.top_k;
        sh.pair_of[i] = (int16_t)at++;
      }
  }
  if (tid == kMoeThreads - 1) {
    sh.hits = (before + own) >> 16;
    sh.hit_first[(before + own) >> 16] = (int16_t)pairs;
  }
  __syncthreads();
}

// One stage of a warp's stream into its ring: rows row0 + 0..7 and row1 + 0..7
// of a matrix of cols columns, 128 columns at 128 chunk, and their scale words.
struct Rows {
  const uint8_t* a;    // the lane's first byte of row0 + r
  const uint8_t* b;    // and of row1 + r
  const uint32_t* sf;  // lanes 0..15: the row's first scale word
  int sf_ld;
  __device__ __forceinline__ void set(const uint8_t* w, const uint32_t* words, int rows, int cols, int row0, int row1,
                                      int lane) {
    const int r = lane >> 2, q = lane & 3;
    a = w + (int64_t)(row0 + r) * cols + q * 16;
    b = w + (int64_t)(row1 + r) * cols + q * 16;
    sf = words + (lane < 8 ? row0 + lane : row1 + (lane & 7));
    sf_ld = (rows + 3) / 4 * 4;
  }
  __device__ __forceinline__ void copy(uint32_t to, int chunk, int lane) const {
    const int64_t at = (int64_t)chunk * kStreamCols;
    cp_async16(to + lane * 16, a + at);
    cp_async16(to + 512 + lane * 16, b + at);
    cp_async16(to + 1024 + lane * 16, a + at + 64);
    cp_async16(to + 1536 + lane * 16, b + at + 64);
    if (lane < 16)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 2048 + lane * 4),
                   "l"(sf + (int64_t)(chunk >> 2) * sf_ld)
                   : "memory");
  }
};

// The tokens of a product: halves [row][cols] and their scales [row][cols / 128].
struct Tokens {
  const __half* h;
  const float* s;
  const int32_t* row;  // of token n (shared memory), or NULL: first + n
  int first, count, cols;
  __device__ __forceinline__ int at(int n) const { return row ? row[n] : first + n; }
};

// acc += a stage's 16 x 128 codes times the tokens' 128 columns.
template <int NB>
__device__ __forceinline__ void moe_stage(const uint8_t* stage, int chunk, const Tokens& t, int lane,
                                          float (&acc)[NB][4]) {
  const int r = lane >> 2, q = lane & 3;
  uint32_t a[8][4];
  stream_decode<DecodeE4m3>(stage, lane, a);
  const uint32_t* words = reinterpret_cast<const uint32_t*>(stage + 2048);
  const int shift = (chunk & 3) * 8;
  const float s0 = scale_of_byte(words[r] >> shift & 0xFFu), s1 = scale_of_byte(words[8 + r] >> shift & 0xFFu);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint4 b[4] = {};
    const int n = nb * 8 + r;
    if (n < t.count) {
      const uint4* src = reinterpret_cast<const uint4*>(t.h + (int64_t)t.at(n) * t.cols + chunk * kStreamCols) + q;
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = src[i * 4];
    }
    float d[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mma_f16(d, a[2 * i], b[i].x, b[i].y);
      mma_f16(d, a[2 * i + 1], b[i].z, b[i].w);
    }
    const int m = nb * 8 + 2 * q;
    const int chunks = t.cols / kStreamCols;
    const float x0 = m < t.count ? t.s[t.at(m) * chunks + chunk] : 0.0f;
    const float x1 = m + 1 < t.count ? t.s[t.at(m + 1) * chunks + chunk] : 0.0f;
    acc[nb][0] = fmaf(d[0], s0 * x0, acc[nb][0]);
    acc[nb][1] = fmaf(d[1], s0 * x1, acc[nb][1]);
    acc[nb][2] = fmaf(d[2], s1 * x0, acc[nb][2]);
    acc[nb][3] = fmaf(d[3], s1 * x1, acc[nb][3]);
  }
}

__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// h of an octet of columns for a hit expert's tokens, from the sums of g (acc 0,
// 1) and u (2, 3); the last of 16 octets brings their 128 columns into halves.
template <int NB>
__device__ __forceinline__ void moe_finish_up(const MoeArgs& p, int hit, int octet, int first, int count,
                                              const float (&acc)[NB][4], int lane) {
  const int r = lane >> 2, q = lane & 3;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = nb * 8 + 2 * q + i;
      const float g = acc[nb][i], u = acc[nb][2 + i];
      const float h = (p.activation == DG_ACT_SILU ? gate_act<DG_ACT_SILU>(g) : gate_act<DG_ACT_GELU_TANH>(g)) * u;
      if (n < count) p.h[(int64_t)(first + n) * p.f + octet * 8 + r] = h;
    }
  __threadfence();
  __syncwarp();
  const int block = octet >> 4, blocks = p.f / 128;
  int old = 0;
  if (lane == 0) old = (int)atomicAdd(p.counter + kMoeBarrierWords + hit * blocks + block, 1u);
  old = __shfl_sync(0xffffffffu, old, 0);
  if (old != 15) return;
  __threadfence();
  for (int n = 0; n < count; ++n) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p.h + (int64_t)(first + n) * p.f + block * 128) + lane);
    float m = fmaxf(fmaxf(finite_magnitude(v.x), finite_magnitude(v.y)), fmaxf(finite_magnitude(v.z), finite_magnitude(v.w)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    const float s = half_scale(m, inv);
    const __half2 a = __floats2half2_rn(v.x * inv, v.y * inv), b = __floats2half2_rn(v.z * inv, v.w * inv);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p.hh + (int64_t)(first + n) * p.f + block * 128 + stream_half_at(lane * 4)) = w;
    if (lane == 0) p.hs[(int64_t)(first + n) * blocks + block] = s;
  }
}

struct Work {
  const MoeArgs* p;
  MoeShared* sh;
  uint8_t* ring;     // the warp's
  float* exchange;   // kMoeSlots x 16
  int warp, lane;
};

// One unit of the first products: the sums of the warp's chunks, joined over the
// group's warps, and the group's first warp finishes them.
template <int NB, class Next>
__device__ __forceinline__ void moe_up_unit(const Work& w, int hit, int octet, int c0, int c1, int& stage, Next next) {
  const MoeArgs& p = *w.p;
  const int first = w.sh->hit_first[hit], count = w.sh->hit_first[hit + 1] - first;
  const Tokens t{p.xh, p.xs, w.sh->pair_token + first, 0, count, p.d};
  float acc[NB][4] = {};
  for (int c = c0; c < c1; ++c) {
    next();
    cp_async_wait<kMoeRing - 1>();
    __syncwarp();
    moe_stage<NB>(w.ring + stage * kStreamStageBytes, c, t, w.lane, acc);
    __syncwarp();
    stage = stage + 1 == kMoeRing ? 0 : stage + 1;
  }
  const int group = w.warp / kMoeSplit, rank = w.warp % kMoeSplit;
  float4* x = reinterpret_cast<float4*>(w.exchange) + (group * kMoeSplit * 8) * 32 + w.lane;
  if (rank)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) x[(rank * 8 + nb) * 32] = make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
  group_barrier(1 + group, 32 * kMoeSplit);
  if (rank == 0) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      for (int i = 1; i < kMoeSplit; ++i) {
        const float4 v = x[(i * 8 + nb) * 32];
        acc[nb][0] += v.x;
        acc[nb][1] += v.y;
        acc[nb][2] += v.z;
        acc[nb][3] += v.w;
      }
  }
  group_barrier(1 + group, 32 * kMoeSplit);  // read before it is written again
  if (rank == 0) moe_finish_up<NB>(p, hit, octet, first, count, acc, w.lane);
}

// One item of the second product: 16 rows of Wd of a hit expert, the warp's
// chunks, into the slots (part, pair).
template <int NB, class Next>
__device__ __forceinline__ void moe_down_item(const Work& w, int hit, int part, int c0, int c1, int& stage, Next next) {
  const MoeArgs& p = *w.p;
  const int first = w.sh->hit_first[hit], count = w.sh->hit_first[hit + 1] - first;
  const Tokens t{p.hh, p.hs, nullptr, first, count, p.f};
  float acc[NB][4] = {};
  for (int c = c0; c < c1; ++c) {
    next();
    cp_async_wait<kMoeRing - 1>();
    __syncwarp();
    moe_stage<NB>(w.ring + stage * kStreamStageBytes, c, t, w.lane, acc);
    __syncwarp();
    stage = stage + 1 == kMoeRing ? 0 : stage + 1;
  }
  const int r = w.lane >> 2, q = w.lane & 3;
  const int pairs = w.sh->hit_first[w.sh->hits];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = nb * 8 + 2 * q + i;
      if (n < count) {
        float* slot = w.exchange + (part * pairs + first + n) * 16;
        slot[r] = acc[nb][i];
        slot[8 + r] = acc[nb][2 + i];
      }
    }
}

#define MOE_BY_COUNT(count, call) \
  do {                            \
    if ((count) <= 8) call(1);    \
    else if ((count) <= 16) call(2); \
    else if ((count) <= 32) call(4); \
    else call(8);                 \
  } while (0)

__global__ void __launch_bounds__(kMoeThreads, 1) moe_layer_kernel(const MoeArgs p) {
  extern __shared__ uint8_t smem[];
  __shared__ MoeShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Work w{&p, &sh, smem + kMoeSlots * 64 + warp * (kMoeRing * kStreamStageBytes), reinterpret_cast<float*>(smem), warp, lane};
  const uint32_t ring = smem_u32(w.ring);
  griddep_wait();
  const int live = live_tokens(p);
  for (int t = warp; t < live; t += kMoeWarps) moe_pick(p, sh, t, lane);
  if (blockIdx.x == 0)  // rows past the last token: no expert
    for (int i = live * p.top_k + tid; i < p.tokens * p.top_k; i += kMoeThreads) {
      p.chosen_out[i] = -1;
      p.weight_out[i] = 0.0f;
    }
  if (tid == 0) sh.last = 0;
  __syncthreads();
  moe_sort(p, sh, live);
  const int hits = sh.hits;
  const int pairs = live * p.top_k;

  int put = 0, stage = 0;  // ring slots to fill and to read
  auto slot = [&]() {
    const uint32_t to = ring + put * kStreamStageBytes;
    put = put + 1 == kMoeRing ? 0 : put + 1;
    return to;
  };
  {
    // ---- g, u and h
    constexpr int kGroups = kMoeWarps / kMoeSplit;
    const int octets = p.f / 8, chunks = p.d / kStreamCols;
    const int units = hits * octets, step = gridDim.x * kGroups;
    const int rank = warp % kMoeSplit, c0 = chunks * rank / kMoeSplit, c1 = chunks * (rank + 1) / kMoeSplit;
    const int begin = blockIdx.x + gridDim.x * (warp / kMoeSplit);
    int ahead = c0 < c1 ? begin : units, ac = c0;
    Rows rows;
    auto aim = [&]() {
      if (ahead < units) {
        const int e = sh.hit_expert[ahead / octets], o = ahead % octets * 8;
        rows.set(p.up + (int64_t)e * 2 * p.f * p.d, p.up_sf + (int64_t)e * ((p.d + 511) / 512) * (2 * p.f), 2 * p.f, p.d,
                 o, p.f + o, lane);
      }
    };
    aim();
    auto next = [&]() {
      if (ahead < units) {
        rows.copy(slot(), ac, lane);
        if (++ac == c1) {
          ac = c0;
          ahead += step;
          aim();
        }
      }
      cp_async_commit();
    };
    for (int i = 0; i < kMoeRing - 1; ++i) next();
    for (int u = begin; u < units; u += step) {
      const int hit = u / octets, octet = u % octets;
      const int count = sh.hit_first[hit + 1] - sh.hit_first[hit];
#define MOE_CALL(NB) moe_up_unit<NB>(w, hit, octet, c0, c1, stage, next)
      MOE_BY_COUNT(count, MOE_CALL);
#undef MOE_CALL
    }
    cp_async_wait<0>();
    __syncwarp();
    put = stage = 0;
  }
  // ---- y
  const int tiles = p.d / 16, chunks = p.f / kStreamCols;
  int parts = 1;  // of a hit expert's columns, so that every warp has some
  while (parts < 16 && hits * parts < kMoeWarps && 2 * parts * pairs <= kMoeSlots && parts < chunks) parts *= 2;
  const int items = hits * parts;
  int at_tile = blockIdx.x, at_item = warp, ac = 0, ac1 = 0;
  Rows rows;
  auto aim = [&]() {
    while (at_tile < tiles) {
      for (; at_item < items; at_item += kMoeWarps) {
        const int part = at_item % parts;
        ac = chunks * part / parts;
        ac1 = chunks * (part + 1) / parts;
        if (ac < ac1) {
          const int e = sh.hit_expert[at_item / parts];
          rows.set(p.down + (int64_t)e * p.d * p.f, p.down_sf + (int64_t)e * ((p.f + 511) / 512) * p.d, p.d, p.f,
                   at_tile * 16, at_tile * 16 + 8, lane);
          return;
        }
      }
      at_item = warp;
      at_tile += gridDim.x;
      if (warp >= items) at_tile = tiles;
    }
  };
  aim();
  auto next = [&]() {
    if (at_tile < tiles) {
      rows.copy(slot(), ac, lane);
      if (++ac == ac1) {
        at_item += kMoeWarps;
        aim();
      }
    }
    cp_async_commit();
  };
  // Wd does not wait for h
  for (int i = 0; i < kMoeRing - 1; ++i) next();
  // barrier over the grid: all of h is there.  All CTAs run at once (cooperative launch).
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    atomicAdd(p.counter, 1u);
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1; ld_acquire_gpu(p.counter) < gridDim.x; ++it)
      if ((it & 63u) == 0 && (global_timer_ns() - t0 > p.timeout_ns || it >= (1u << 28))) {
        record_error(p.err, DG_ERR_DEVICE_TIMEOUT, kSiteMoeBarrier);
        sh.last = 1;
        break;
      }
    __threadfence();
  }
  __syncthreads();
  griddep_launch_dependents();
  const bool failed = sh.last != 0;
  for (int tile = blockIdx.x; tile < tiles && !failed; tile += gridDim.x) {
    for (int item = warp; item < items; item += kMoeWarps) {
      const int hit = item / parts, part = item % parts;
      const int count = sh.hit_first[hit + 1] - sh.hit_first[hit];
#define MOE_CALL(NB) \
  moe_down_item<NB>(w, hit, part, chunks * part / parts, chunks * (part + 1) / parts, stage, next)
      MOE_BY_COUNT(count, MOE_CALL);
#undef MOE_CALL
    }
    __syncthreads();
    for (int i = tid; i < live * 16; i += kMoeThreads) {
      const int t = i >> 4, row = i & 15;
      float v = 0.0f;
      for (int j = 0; j < p.top_k; ++j) {
        const int pair = sh.pair_of[t * p.top_k + j];
        float s = 0.0f;
        for (int k = 0; k < parts; ++k) s += w.exchange[(k * pairs + pair) * 16 + row];
        v = fmaf(sh.weight[t * p.top_k + j], s, v);
      }
      const int64_t col = (int64_t)tile * 16 + row;
      if (p.c) v += __bfloat162float(p.c[(int64_t)t * p.ldc + col]);
      p.y[(int64_t)t * p.ldy + col] = __float2bfloat16_rn(v);
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

constexpr size_t kMoeSmem = (size_t)kMoeSlots * 64 + (size_t)kMoeWarps * kMoeRing * kStreamStageBytes;

}  // namespace

uint64_t moe_few_tokens_layout(MoeArgs& a, void* workspace) {
  uint64_t at = 0;
  const uint64_t pairs = (uint64_t)a.tokens * a.top_k, t = a.tokens, d = a.d, f = a.f, e = a.experts;
  auto take = [&](uint64_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(workspace) + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const uint64_t hits = std::min<uint64_t>(e, pairs);
  a.counters = (int32_t)(kMoeBarrierWords + hits * (f / 128));
  a.counter = reinterpret_cast<uint32_t*>(take((uint64_t)a.counters * 4));
  a.logits = reinterpret_cast<double*>(take(t * e * 8));
  a.select = reinterpret_cast<double*>(take(t * e * 8));
  a.xh = reinterpret_cast<__half*>(take(t * d * 2));
  a.xs = reinterpret_cast<float*>(take(t * (d / 128) * 4));
  a.h = reinterpret_cast<float*>(take(pairs * f * 4));
  a.hh = reinterpret_cast<__half*>(take(pairs * f * 2));
  a.hs = reinterpret_cast<float*>(take(pairs * (f / 128) * 4));
  return at;
}

cudaError_t moe_few_tokens_launch(MoeArgs p, bool router_fp32, int sms, bool pdl, cudaStream_t stream) {
  cudaError_t e = error_word_address(&p.err);
  if (e != cudaSuccess) return e;
  const int groups = (p.tokens + kScoreTokens - 1) / kScoreTokens;
  const dim3 grid((unsigned)(p.experts * groups + p.tokens));
  e = router_fp32 ? launch_op(moe_scores_kernel<float>, grid, kScoreThreads, 0, pdl, stream, p)
                  : launch_op(moe_scores_kernel<__nv_bfloat16>, grid, kScoreThreads, 0, pdl, stream, p);
  if (e != cudaSuccess) return e;
  if ((e = set_smem(moe_layer_kernel, kMoeSmem, kMoeSmem)) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, 1, 1);
  cfg.blockDim = dim3(kMoeThreads, 1, 1);
  cfg.dynamicSmemBytes = kMoeSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_layer_kernel, p);
}

}  // namespace dg
