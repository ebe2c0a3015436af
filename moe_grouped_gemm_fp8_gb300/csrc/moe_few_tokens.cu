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
// Bound by reading the hit experts' weights once.  A producer warp keeps TMA
// copies of 32 KB of weights and of their expert's tokens in flight; 16 warps
// decode E4M3 to halves in registers (exact) and multiply by mma m16n8k16 with
// all tokens of the expert at once, 16 rows x 128 columns a warp and stage.
// tcgen05 would take the weights as they are in its block-scaled form, but each
// token's side as two (h: three) 8-bit pieces so as not to round it; for many tokens,
// where the multiplying warps bound this kernel, that is not tried.  Units of work
// are taken from a counter: SMs read at rates that differ by a quarter.
//
// Measured in a graph, D = 7168, F = 2048: one token, 8 of 32 experts, 85.5 us (352 MB,
// 4.1 TB/s; scores 6, choosing 3, first product 50, barrier 2, second product 23); 16
// tokens, 8 of 64 experts, 408 us (2.5 GB, 6.2 TB/s, 91% of the copy's rate); 64 tokens,
// 4 of 16 experts, 215 us (0.7 GB, 3.3 TB/s: the multiplying warps' instructions).
// 8 of 256 experts: 1 token 88 us, 16 (107 experts hit) 761 (1.09 of their bytes' time),
// 64 (221 hit) 1687 (1.17).
//
// x and h are carried as halves with a power of two per 128 columns: 11 bits
// (BF16 x exactly, but for values 2^29 below the largest of the 128; h with fewer
// bits below 2^-28 of it), so that the only roundings are those and the result's own:
// y is off by about 2^-12 of itself before it is rounded, an eighth of what BF16 rounds.
#include <algorithm>

#include "dg_device.cuh"
#include "dg_ops.cuh"
#include "moe.h"
#include "stream_mma.cuh"

namespace dg {
namespace {

constexpr int kMoeWarps = 16;     // that multiply
constexpr int kMoeFinishers = 3;  // that finish units; one more fetches
constexpr int kMoeThreads = 32 * (kMoeWarps + kMoeFinishers + 1);
constexpr int kMoeStages = 6;        // at most
constexpr int kMoeSmem = 210 * 1024;  // ring and exchange
constexpr int kScoreThreads = 256;
constexpr int kScoreTokens = 8;  // tokens of a CTA of the first kernel

// A token's 128 columns: 128 halves in the order in which the lanes read them,
// then their scale, and nothing up to a multiple of 16 bytes.  x lies by token,
// since its experts are not known yet: [token][columns / 128].  h lies by expert,
// so that a stage's tokens are one copy: [hit expert][columns / 128][its token], the
// pieces 320 bytes apart (8 lanes, two tokens, then read all banks).  Lane (r, q) of a
// warp holds, of weight rows r and r + 8, columns 32 q to 32 q + 31; product j
// (0..7) multiplies columns 32 q + 4 j + 0..3 of every q.  Of the halves, unit
// j / 2 comes first, then q, then 8 columns.
constexpr int kMoeChunkBytes = 272, kMoeHiddenBytes = 320;
__device__ __forceinline__ int moe_half_at(int k) { return ((k >> 3) & 3) * 32 + (k >> 5) * 8 + (k & 7); }

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

// exp(hi + lo), lo far below 1: hi alone costs a logit of -80 the 2^-19 of the result that it lacks.
__device__ __forceinline__ float exp_of(float hi, float lo) {
  const float e = expf(hi);
  return e > 0.0f ? fmaf(e, lo, e) : e;  // (next to an infinity lo is no number)
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

// Order-preserving 64-bit integers of scores, 0 for what is no number.
__device__ __forceinline__ uint64_t score_key(double v) {
  if (!(v == v)) return 0;
  const int64_t b = __double_as_longlong(v);
  return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

// Scores of expert e for tokens t0 .. t0 + n - 1 (n <= N), by a CTA.
//
// The order of near scores decides which expert runs, so they are summed as if
// in 48 bits: BF16 products are exact in FP32 (with FP32 weights the product's
// rounding error is added too), and every sum keeps its rounding error.
template <class R, int N>
__device__ __forceinline__ void moe_score(const MoeArgs& p, int e, int t0, int n) {
  constexpr int kDeep = N == 1 ? 4 : 1;  // steps whose loads are in flight at once
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const R* w = reinterpret_cast<const R*>(p.router) + (int64_t)e * p.d;
  const __nv_bfloat16* x = p.x + (int64_t)t0 * p.ldx;
  float hi[N] = {}, lo[N] = {};
  for (int c0 = tid * 8; c0 < p.d; c0 += kDeep * kScoreThreads * 8) {
    float wf[kDeep][8];
    uint4 xw[kDeep][N];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int c = c0 + k * kScoreThreads * 8;
      if (c < p.d) {
        load8(w + c, wf[k]);
#pragma unroll
        for (int t = 0; t < N; ++t)  // (tokens past the last: the last again, unused)
          xw[k][t] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)min(t, n - 1) * p.ldx + c));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) wf[k][i] = 0.0f;
#pragma unroll
        for (int t = 0; t < N; ++t) xw[k][t] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
#pragma unroll
      for (int t = 0; t < N; ++t) {
        const uint32_t xs[4] = {xw[k][t].x, xw[k][t].y, xw[k][t].z, xw[k][t].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xf = i & 1 ? bf16_hi(xs[i / 2]) : bf16_lo(xs[i / 2]);
          const float v = __fmul_rn(wf[k][i], xf);  // (not joined with the sum)
          if constexpr (sizeof(R) == 4) lo[t] += fmaf(wf[k][i], xf, -v);
          add_exactly(hi[t], lo[t], v);
        }
      }
  }
  // pairs (hi, lo) over the warp and the CTA: FP64 is slow here
  __shared__ float2 sums[kScoreThreads / 32][N];
#pragma unroll
  for (int t = 0; t < N; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h = __shfl_xor_sync(0xffffffffu, hi[t], o), l = __shfl_xor_sync(0xffffffffu, lo[t], o);
      add_exactly(hi[t], lo[t], h);
      lo[t] += l;
    }
    if (lane == 0) sums[warp][t] = make_float2(hi[t], lo[t]);
  }
  __syncthreads();
  if (tid < n) {
    double v = 0.0;
    for (int i = 0; i < kScoreThreads / 32; ++i) {
      const float2 f = sums[i][tid];
      v += (double)f.x;
      if (fabsf(f.y) < INFINITY) v += (double)f.y;  // where a sum overflowed its error is no number
    }
    v += 0.0;  // -0 and 0 are one score
    const int64_t to = (int64_t)(t0 + tid) * p.experts + e;
    const float h = (float)v;
    p.logits[to] = make_float2(h, fabsf(h) < INFINITY ? (float)(v - (double)h) : 0.0f);
    p.keys[to] = score_key(p.router_bias ? 1.0 / (1.0 + exp(-v)) + (double)__ldg(p.router_bias + e) : v);
  }
}

// CTA (expert, 8 tokens): their scores; CTAs after those: a token's halves.
template <class R>
__global__ void __launch_bounds__(kScoreThreads) moe_scores_kernel(const MoeArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int live = live_tokens(p);
  const int groups = (p.tokens + kScoreTokens - 1) / kScoreTokens;
  const int tid = threadIdx.x;
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
        uint8_t* to = p.xh + ((int64_t)at * (p.d / 128) + c / 128) * kMoeChunkBytes;
        *reinterpret_cast<uint4*>(to + 2 * moe_half_at(c & 127)) = *reinterpret_cast<const uint4*>(h);
        if ((c & 127) == 0) *reinterpret_cast<float*>(to + 256) = s;
      }
    }
    return;
  }
  const int e = at % p.experts, t0 = at / p.experts * kScoreTokens;
  const int n = min(live - t0, kScoreTokens);
  if (n <= 0) return;
  if (n > 4) moe_score<R, 8>(p, e, t0, n);
  else if (n > 1) moe_score<R, 4>(p, e, t0, n);
  else moe_score<R, 1>(p, e, t0, n);
}

// ---------------------------------------------------------------- routing

constexpr int kMoePairs = kMoeMaxTokens * kMoeMaxTopK;

// What a stage of the ring holds.
struct alignas(16) MoeStage {
  int16_t hit;    // hit expert, -1: no more
  uint8_t begin;  // the unit's first stage of a team
  uint8_t end;    // and its last
  int32_t chunk;  // the first 128 columns; past the last: nothing
  int32_t row;    // the unit's first row: column of h, or of y
  int16_t first;  // the expert's first pair
  uint8_t count;  // and their number
  uint8_t part;   // which share of the hit experts (y only)
};

struct MoeShared {
  uint64_t mask[kMoeMaxExperts];          // of an expert: its tokens
  int16_t chosen[kMoePairs];              // (token, j) -> expert
  float weight[kMoePairs];                // (token, j)
  uint8_t pair_token[kMoePairs];          // pairs in the order of (expert, token)
  uint8_t pair_slot[kMoePairs];           // and their j
  int16_t hit_expert[kMoeMaxExperts];     // hit experts, ascending
  int16_t hit_first[kMoeMaxExperts + 1];  // their first pairs
  int16_t first[kMoeMaxExperts];          // the same by expert
  uint64_t full[kMoeStages], empty[kMoeStages];  // of the ring's slots
  uint64_t summed[4], taken[4];                   // of the exchange's buffers
  MoeStage stage[kMoeStages], unit[4];
  int32_t scan[kMoeThreads / 32], most[kMoeThreads / 32];
  int32_t hits, most_tokens;
  int32_t abort;
  int32_t last;
};

// A warp picks the experts of token t and their weights, from 32 PER experts.
template <int PER>
__device__ void moe_pick(const MoeArgs& p, MoeShared& sh, int t, int lane) {
  const float2* logits = p.logits + (int64_t)t * p.experts;
  uint64_t key[PER];
  uint32_t taken = 0;  // bit i: expert i * 32 + lane is chosen, or is none
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < p.experts ? __ldg(reinterpret_cast<const unsigned long long*>(p.keys) + (int64_t)t * p.experts + e) : 0;
    if (e >= p.experts) taken |= 1u << i;
  }
  int mine = 0;  // lane j: the j-th choice
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = 0;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)  // among equals the lowest stays
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
  const float2 l = on ? __ldg(logits + mine) : make_float2(0.0f, 0.0f);
  float w;
  if (p.score == DG_SCORE_SOFTMAX) {
    // the first choice has the largest
    const float mh = __shfl_sync(0xffffffffu, l.x, 0), ml = __shfl_sync(0xffffffffu, l.y, 0);
    w = on ? expf((l.x - mh) + (l.y - ml)) : 0.0f;
    float sum = w;
    if (!p.renormalize) {
      sum = 0.0f;
      for (int e = lane; e < p.experts; e += 32) {
        const float2 o = __ldg(logits + e);
        sum += expf((o.x - mh) + (o.y - ml));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w /= sum;
  } else {
    // exp(min(l, 0)) / (1 + exp(-|l|)), which no l takes out of range; to be divided by their sum, all times
    // exp(-m), m the largest of the chosen l where that is below 0, so that the sum is 1/2 at least.
    float m = 0.0f;
    if (p.renormalize) {
      m = on ? l.x : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = fminf(m, 0.0f);
    }
    float2 low = l.x < 0.0f ? l : make_float2(0.0f, 0.0f);
    add_exactly(low.x, low.y, -m);
    w = on ? exp_of(low.x, low.y) / (1.0f + expf(-fabsf(l.x))) : 0.0f;
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
    atomicOr(reinterpret_cast<unsigned long long*>(&sh.mask[mine]), 1ull << t);
    sh.weight[t * p.top_k + lane] = w;
    if (blockIdx.x == 0) {
      p.chosen_out[(int64_t)t * p.top_k + lane] = mine;
      p.weight_out[(int64_t)t * p.top_k + lane] = w;
    }
  }
}

// The choices of all live tokens, then the pairs (token, j) in the order of
// (expert, token).
__device__ __forceinline__ void moe_route(const MoeArgs& p, MoeShared& sh, int live) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = live * p.top_k;
  for (int i = tid; i < p.experts; i += kMoeThreads) sh.mask[i] = 0;
  __syncthreads();
  for (int t = warp; t < live; t += kMoeThreads / 32) {
    if (p.experts <= 64) moe_pick<2>(p, sh, t, lane);
    else if (p.experts <= 256) moe_pick<8>(p, sh, t, lane);
    else moe_pick<kMoeMaxExperts / 32>(p, sh, t, lane);
  }
  if (blockIdx.x == 0)  // rows past the last token: no expert
    for (int i = pairs + tid; i < p.tokens * p.top_k; i += kMoeThreads) {
      p.chosen_out[i] = -1;
      p.weight_out[i] = 0.0f;
    }
  __syncthreads();
  // prefix sums over the experts of (pairs, hit experts) in one word
  const int count = tid < p.experts ? __popcll(sh.mask[tid]) : 0;
  int v = count | (count > 0 ? 1 << 16 : 0);
  const int own = v, most = __reduce_max_sync(0xffffffffu, count);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) {
    sh.scan[warp] = v;
    sh.most[warp] = most;
  }
  __syncthreads();
  if (tid < p.experts) {
    int before = v - own;
    for (int i = 0; i < warp; ++i) before += sh.scan[i];
    sh.first[tid] = (int16_t)(before & 0xffff);
    if (count > 0) {
      sh.hit_expert[before >> 16] = (int16_t)tid;
      sh.hit_first[before >> 16] = (int16_t)(before & 0xffff);
    }
  }
  if (tid == kMoeThreads - 1) {
    int all = 0, m = 0;
    for (int i = 0; i < kMoeThreads / 32; ++i) {
      all += sh.scan[i];
      m = max(m, sh.most[i]);
    }
    sh.hits = all >> 16;
    sh.hit_first[all >> 16] = (int16_t)pairs;
    sh.most_tokens = m;
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += kMoeThreads) {
    const int e = sh.chosen[i], t = i / p.top_k;
    const int at = sh.first[e] + __popcll(sh.mask[e] & ((1ull << t) - 1));
    sh.pair_token[at] = (uint8_t)t;
    sh.pair_slot[at] = (uint8_t)(i - t * p.top_k);
  }
  __syncthreads();
}

// ---------------------------------------------------------------- the layer

// How the stages of one of the two products lie: 2^LG tiles of 16 rows by
// 16 / 2^LG slices of 128 columns, a warp each ([slice][row][128 bytes], of Wg and
// Wu one after the other); then the rows' scale words; then the tokens.  More rows share a token's bytes, fewer make finer units: with 8
// tokens of one expert at least three stages of 32 rows fit, with 64 two of 128.
constexpr int up_lg(int max) { return max == 1 ? 1 : max <= 4 ? 2 : 3; }
constexpr int down_lg(int max) { return max == 1 ? 0 : max <= 4 ? 2 : 3; }
// GATHER: the tokens come four at a time by TMA gathers, packed.
template <bool UP, int LG, bool GATHER>
struct MoeShape {
  static constexpr int lg = LG, slices = kMoeWarps >> LG;
  // room of a token in a stage; from one 128 columns to the next, from one token to the next
  static constexpr int token_bytes = slices * (UP ? kMoeChunkBytes : kMoeHiddenBytes);
  static constexpr int kPlace = UP ? token_bytes + (GATHER ? 0 : (64 - token_bytes) & 127) : token_bytes;
  static __device__ __forceinline__ int slice_step(int count) { return UP ? kMoeChunkBytes : count * kMoeHiddenBytes; }
  static constexpr int token_step = UP ? kPlace : kMoeHiddenBytes;
  static __device__ __forceinline__ int stage_bytes(int most_tokens) {
    const int n = GATHER ? (most_tokens + 3) & ~3 : most_tokens;
    return (32768 + 512 + n * kPlace + 1023) & ~1023;
  }
};

// A copy takes the TMA unit about 90 cycles however small it is: where an expert can
// have many tokens, x comes four rows a copy (40 tokens to 16 experts: 288 us without,
// 266 with; 16 tokens to 64, mostly one to three each: 400 and 422).
constexpr bool moe_gathers(int max) { return max >= 4; }
// Teams of warps that take the stages by turns, a warp of two 16 rows and 256
// columns of each of its team's: fewer waits a byte than with all 16 warps on
// every stage (16 rows, 128 columns), and twice the independent products.  Each
// has its own slots (one whose team changed could be waited for a use too
// early), so the ring's are even: for many tokens, where three fit, one team.
constexpr int moe_teams(int max) { return max <= 2 ? 2 : 1; }
// Buffers of the exchange, and how the finishing warps share the work: units by
// turns where a unit is small, else each unit.
constexpr bool moe_turns(int max) { return max <= 2; }
constexpr int moe_buffers(int max) { return max == 1 ? 4 : max == 2 ? 3 : 1; }

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// The producer warp's side of a stage.
template <bool UP, bool GATHER, class Shape>
struct MoeFetch {
  static constexpr int lg = Shape::lg, slices = Shape::slices;
  const MoeArgs& p;
  const MoeShared& sh;
  const CUtensorMap* map;
  const CUtensorMap* map_x;  // GATHER
  int lane;
  // columns / 128 of the stage, and scale words
  __device__ __forceinline__ int slices_of(const MoeStage& st) const {
    return max(0, min(slices, (UP ? p.d : p.f) / 128 - st.chunk));
  }
  __device__ __forceinline__ int words_of(const MoeStage& st, int n) const { return ((st.chunk & 3) + n + 3) / 4; }
  __device__ __forceinline__ uint32_t bytes(const MoeStage& st) const {
    const int n = slices_of(st);
    if (n == 0) return 0;
    const int tokens = GATHER ? ((st.count + 3) & ~3) * Shape::token_bytes
                              : st.count * n * (UP ? kMoeChunkBytes : kMoeHiddenBytes);
    return (uint32_t)(32768 + (words_of(st, n) << lg) * 64 + tokens);
  }
  // 32 KB (slices past the last column come as zeros) and scale words
  __device__ __forceinline__ void weights(uint32_t to, uint32_t bar, const MoeStage& st) const {
    const int n = slices_of(st), cols = UP ? p.d : p.f, rows = UP ? 2 * p.f : p.d, e = sh.hit_expert[st.hit];
    if (n == 0) return;
    DG_CHECK(p.err, e >= 0 && e < p.experts && st.chunk >= 0 && st.chunk + n <= cols / 128 && st.row >= 0 &&
                        st.row + ((UP ? 8 : 16) << lg) <= (UP ? p.f : p.d),
             kSiteCheckLoadB);
    if (lane < (UP ? 2 : 1)) tma_load_3d(to + lane * 16384, map, bar, 0, e * rows + st.row + lane * p.f, st.chunk);
    constexpr int run = (UP ? 8 : 16) << lg;
    if (lane < (UP ? 2 : 1) * words_of(st, n)) {
      const int w = UP ? lane >> 1 : lane;
      const uint32_t* src = (UP ? p.up_sf : p.down_sf) +
                            ((int64_t)e * ((cols + 511) / 512) + (st.chunk >> 2) + w) * rows + st.row +
                            (UP && (lane & 1) ? p.f : 0);
      bulk_load(to + 32768 + lane * run * 4, src, (uint32_t)run * 4, bar);
    }
  }
  __device__ __forceinline__ void tokens(uint32_t to, uint32_t bar, const MoeStage& st) const {
    const int n = slices_of(st), chunks = (UP ? p.d : p.f) / 128;
    if (n == 0) return;
    DG_CHECK(p.err, st.first >= 0 && st.count >= 1 && st.first + st.count <= p.tokens * p.top_k &&
                        sh.pair_token[st.first + min(lane, st.count - 1)] < p.tokens,
             kSiteCheckLoadA);
    to += 32768 + 512;
    if constexpr (!UP) {
      if (lane == 0)
        bulk_load(to, p.hh + ((int64_t)st.first * chunks + (int64_t)st.chunk * st.count) * kMoeHiddenBytes,
                  (uint32_t)(n * st.count) * kMoeHiddenBytes, bar);
    } else if constexpr (GATHER) {
      // (the last four filled up with the last token)
      if (lane * 4 < st.count) {
        int row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = sh.pair_token[st.first + min(lane * 4 + i, st.count - 1)];
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(to + lane * 4 * Shape::token_bytes),
            "l"(reinterpret_cast<uint64_t>(map_x)), "r"(st.chunk * (kMoeChunkBytes / 8)), "r"(row[0]), "r"(row[1]),
            "r"(row[2]), "r"(row[3]), "r"(bar)
            : "memory");
      }
    } else {
      for (int t = lane; t < st.count; t += 32)
        bulk_load(to + t * Shape::kPlace,
                  p.xh + ((int64_t)sh.pair_token[st.first + t] * chunks + st.chunk) * kMoeChunkBytes,
                  (uint32_t)n * kMoeChunkBytes, bar);
    }
  }
};

// acc += a warp's 16 rows x 128 PER columns (slices from `slice` on) of a stage
// times its expert's tokens.
template <bool UP, class Shape, int PER, int MAX>
__device__ __forceinline__ void moe_multiply(const uint8_t* stage, int tile, int slice, int first_chunk, int chunks,
                                             int count, int lane, float (&acc)[MAX][4]) {
  constexpr int lg = Shape::lg;
  const int r = lane >> 2, q = lane & 3;
  // atoms of rows r and r + 8, in TMA's 128-byte swizzle: 16 bytes c of row r at c ^ r
  const uint8_t* low = stage + slice * (UP ? 1024 << lg : 2048 << lg) + tile * (UP ? 1024 : 2048) + r * 128;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(stage + 32768) + (UP ? tile * 8 + r : tile * 16 + r);
  // (columns of tokens that do not exist hold the last token's: nothing reads their sums)
  const int step = Shape::slice_step(count);
  const uint8_t* tokens = stage + 32768 + 512 + slice * step;
  const uint8_t* x = tokens + min(r, count - 1) * Shape::token_step + q * 16;
  const uint8_t* x0 = tokens + min(2 * q, count - 1) * Shape::token_step + 256;
  const uint8_t* x1 = tokens + min(2 * q + 1, count - 1) * Shape::token_step + 256;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int chunk = first_chunk + slice + i;
    if (i && chunk >= chunks) break;
    const uint8_t* lo = low + i * (UP ? 1024 << lg : 2048 << lg);
    const uint8_t* hi = lo + (UP ? 16384 : 1024);
    const uint32_t* word = words + ((chunk >> 2) - (first_chunk >> 2)) * (16 << lg);
    const int shift = (chunk & 3) * 8;
    const float s0 = scale_of_byte(word[0] >> shift & 0xFFu);
    const float s1 = scale_of_byte(word[UP ? 8 << lg : 8] >> shift & 0xFFu);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[4][4];
      const int c = ((2 * q + h) ^ r) * 16;
      const uint4 g = *reinterpret_cast<const uint4*>(lo + c), u = *reinterpret_cast<const uint4*>(hi + c);
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        DecodeE4m3::four(gw[j], a[j][0], a[j][2]);
        DecodeE4m3::four(uw[j], a[j][1], a[j][3]);
      }
#pragma unroll
      for (int nb = 0; nb < MAX; ++nb) {
        if (nb && nb * 8 >= count) break;
        const uint8_t* xb = (nb ? tokens + min(nb * 8 + r, count - 1) * Shape::token_step + q * 16 : x) +
                            i * step + h * 128;
        const uint4 b0 = *reinterpret_cast<const uint4*>(xb), b1 = *reinterpret_cast<const uint4*>(xb + 64);
        const int m = nb * 8 + 2 * q;
        const float t0 = *reinterpret_cast<const float*>(
            (nb ? tokens + min(m, count - 1) * Shape::token_step + 256 : x0) + i * step);
        const float t1 = *reinterpret_cast<const float*>(
            (nb ? tokens + min(m + 1, count - 1) * Shape::token_step + 256 : x1) + i * step);
        float d[4] = {};
        mma_f16(d, a[0], b0.x, b0.y);
        mma_f16(d, a[1], b0.z, b0.w);
        mma_f16(d, a[2], b1.x, b1.y);
        mma_f16(d, a[3], b1.z, b1.w);
        acc[nb][0] = fmaf(d[0], s0 * t0, acc[nb][0]);
        acc[nb][1] = fmaf(d[1], s0 * t1, acc[nb][1]);
        acc[nb][2] = fmaf(d[2], s1 * t0, acc[nb][2]);
        acc[nb][3] = fmaf(d[3], s1 * t1, acc[nb][3]);
      }
    }
  }
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A barrier of `threads` threads; whether `mine` holds for all of them.
__device__ __forceinline__ bool all_agree(int id, int threads, bool mine) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"((uint32_t)mine)
      : "memory");
  return all != 0;
}

__device__ __forceinline__ void add4(float4& v, const float4& o) {
  v.x += o.x;
  v.y += o.y;
  v.z += o.z;
  v.w += o.w;
}

// h of an octet of columns for a hit expert's tokens, from the slices' sums of g
// (x, y) and u (z, w), added in the slices' order.
template <class Shape>
__device__ __forceinline__ void moe_activate(const MoeArgs& p, const float4* sums, int blocks, int octet, int first,
                                             int count, int lane) {
  const int r = lane >> 2, q = lane & 3;
  for (int nb = 0; nb * 8 < count; ++nb) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < Shape::slices; ++i) {
      add4(v, sums[(i * blocks + nb) * 32]);
    }
    const float2 g = make_float2(v.x, v.y), u = make_float2(v.z, v.w);
    const float2 a = p.activation == DG_ACT_SILU
                         ? make_float2(gate_act<DG_ACT_SILU>(g.x), gate_act<DG_ACT_SILU>(g.y))
                         : make_float2(gate_act<DG_ACT_GELU_TANH>(g.x), gate_act<DG_ACT_GELU_TANH>(g.y));
    const int n = nb * 8 + 2 * q;
    float* h = p.h + (int64_t)(first + n) * p.f + octet * 8 + r;
    DG_CHECK(p.err, first + count <= p.tokens * p.top_k && octet * 8 + r < p.f, kSiteCheckStore);
    if (n < count) __stcg(h, a.x * u.x);
    if (n + 1 < count) __stcg(h + p.f, a.y * u.y);
  }
}

// The 128 columns of h of a block, for a hit expert's tokens, as halves.
__device__ __forceinline__ void moe_halves(const MoeArgs& p, int block, int first, int count, int lane) {
  const int blocks = p.f / 128;
  DG_CHECK(p.err, block < blocks && first + count <= p.tokens * p.top_k, kSiteCheckStore);
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
    uint8_t* to = p.hh + ((int64_t)first * blocks + (int64_t)block * count + n) * kMoeHiddenBytes;
    *reinterpret_cast<uint2*>(to + 2 * moe_half_at(lane * 4)) = w;
    if (lane == 0) *reinterpret_cast<float*>(to + 256) = s;
  }
}

// Four results of y: their sums over the experts, and c.
__device__ __forceinline__ void moe_store(const MoeArgs& p, int t, int64_t col, float4 v) {
  const float f[4] = {v.x, v.y, v.z, v.w};
  DG_CHECK(p.err, t < p.tokens && col + 4 <= p.d, kSiteCheckStore);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = p.c ? __bfloat162float(p.c[(int64_t)t * p.ldc + col + i]) : 0.0f;
    p.y[(int64_t)t * p.ldy + col + i] = __float2bfloat16_rn(f[i] + c);
  }
}

// The stages of a CTA's units, one after another.  Units come from a counter;
// the next one's number is asked for a unit ahead.  UP: (hit expert, rows), else
// (rows, share of the hit experts).
template <bool UP, int TEAMS>
struct MoeWalk {
  const MoeArgs& p;
  int hits, units, parts, rows, slices, chunks;
  uint32_t* claim;
  int lane;
  const MoeShared& sh;
  int u, claimed, hit, hit_end, chunk, row, part, count, stages;
  __device__ __forceinline__ void aim() {
    if (u >= units) return;
    claimed = 0;
    if (lane == 0) claimed = (int)atomicAdd(claim, 1u);
    chunk = count = 0;
    if (UP) {
      const int per = p.f / rows;
      hit = u / per;
      hit_end = hit + 1;
      row = (u - hit * per) * rows;
      part = 0;
    } else {
      const int tile = u / parts;
      part = u - tile * parts;
      hit = hits * part / parts;
      hit_end = hits * (part + 1) / parts;
      row = tile * rows;
    }
    // a multiple of the teams, so that each sees the unit's end
    stages = ((hit_end - hit) * ((chunks + slices - 1) / slices) + TEAMS - 1) / TEAMS * TEAMS;
  }
  __device__ __forceinline__ void begin() {
    u = blockIdx.x;
    aim();
  }
  __device__ __forceinline__ bool done() const { return u >= units; }
  __device__ __forceinline__ bool empty() const { return hit == hit_end; }
  __device__ __forceinline__ MoeStage stage() const {
    const int h = empty() ? hit - 1 : hit, first = sh.hit_first[h];
    return MoeStage{(int16_t)h, count < TEAMS, count + TEAMS >= stages, empty() ? chunks : chunk, row, (int16_t)first,
                    (uint8_t)(sh.hit_first[h + 1] - first), (uint8_t)part};
  }
  __device__ __forceinline__ void next() {
    if (++count == stages) {
      u = gridDim.x + __shfl_sync(0xffffffffu, claimed, 0);
      aim();
      return;
    }
    chunk += slices;
    if (chunk >= chunks) {
      chunk = 0;
      ++hit;
    }
  }
};

// MAX: blocks of 8 tokens an expert can have.
template <int MAX>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_layer_kernel(const __grid_constant__ MoeArgs p, const __grid_constant__ CUtensorMap map_up,
                     const __grid_constant__ CUtensorMap map_down, const __grid_constant__ CUtensorMap map_x) {
  using Up = MoeShape<true, up_lg(MAX), moe_gathers(MAX)>;
  using Down = MoeShape<false, down_lg(MAX), false>;
  // a finishing warp waits for its next unit, kMoeFinishers later: that buffer's last use must be one it has seen end
  static_assert(!moe_turns(MAX) || moe_buffers(MAX) >= kMoeFinishers, "a wait could pass a phase early");
  constexpr int kTeams = moe_teams(MAX);
  constexpr int kBuffers = moe_buffers(MAX), kUpRows = 8 << Up::lg, kDownRows = 16 << Down::lg;
  extern __shared__ uint8_t smem_raw[];
  __shared__ MoeShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - smem_u32(smem_raw));
  if (tid == 0) {
    for (int i = 0; i < kMoeStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), kMoeWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sh.summed[i]), kMoeWarps);
      mbar_init(smem_u32(&sh.taken[i]), moe_turns(MAX) ? 1 : kMoeFinishers);
    }
    sh.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_up);
    tma_prefetch_desc(&map_down);
    if (moe_gathers(MAX)) tma_prefetch_desc(&map_x);
  }
  griddep_wait();
  const int live = live_tokens(p);
  moe_route(p, sh, live);
  const int hits = sh.hits, most = sh.most_tokens, blocks = (most + 7) / 8;
  volatile int* const abort_flag = &sh.abort;

  // The exchange lies after the ring: sums of g and u ([tile][slice][8 tokens][lane]), then of y ([warp][token][16 rows]).
  const int up_buffer = kMoeWarps * blocks * 128, down_buffer = kMoeWarps * live * 16;
  const int exchange_bytes = kBuffers * 4 * max(up_buffer, down_buffer);
  float* const exchange = reinterpret_cast<float*>(smem + kMoeSmem - exchange_bytes);
  const int up_bytes = Up::stage_bytes(most), down_bytes = Down::stage_bytes(most);
  const int up_stages = min((kMoeSmem - exchange_bytes) / up_bytes, kMoeStages) / kTeams * kTeams;
  const int down_stages = min((kMoeSmem - exchange_bytes) / down_bytes, kMoeStages);
  const int tiles = p.d / kDownRows, up_chunks = p.d / 128, down_chunks = p.f / 128;
  // Shares of the hit experts, each a unit of its own, until there are two units an SM, of four stages at least.  (More
  // cost more in partial sums than finer units win: 16 shares where 4 do take 40 tokens' second product from 80 to
  // 125 us.)
  int parts = 1;
  while (2 * parts <= hits && parts < kMoeMaxParts && tiles * parts < 2 * (int)gridDim.x &&
         (int64_t)kDownRows * p.f * (hits / (2 * parts)) >= 4 * 32768)
    parts *= 2;

  uint32_t used = 0;  // bit s: parity of ring slot s's uses
  if (warp == kMoeWarps) {
    // ------------------------------------------------------------ fetch
    int s = 0;
    uint32_t armed = 0;  // bit s: slot s was filled
    bool ok = true;
    auto wait_free = [&]() {
      return wait_quick(smem_u32(&sh.empty[s]), (used >> s & 1u) ^ 1u, abort_flag, p.timeout_ns, p.err,
                          kSiteProducerEmpty);
    };
    // says what slot s will hold, and how many bytes that is
    auto arm = [&](const MoeStage& what, uint32_t bytes, int room = kMoeSmem) {
      DG_CHECK(p.err, bytes <= (uint32_t)room, kSiteCheckLoadA);
      if (lane == 0) {
        sh.stage[s] = what;
        mbar_arrive_expect_tx(smem_u32(&sh.full[s]), bytes);
      }
      __syncwarp();
      used ^= 1u << s;
      armed |= 1u << s;
    };
    const MoeStage none{-1, 0, 0, 0, 0, 0, 0, 0};
    {
      const MoeFetch<true, moe_gathers(MAX), Up> fetch{p, sh, &map_up, &map_x, lane};
      MoeWalk<true, kTeams> walk{p, hits, hits * (p.f / kUpRows), 1, kUpRows, Up::slices, up_chunks, p.counter + 2, lane, sh};
      int told = 0;
      for (walk.begin(); ok; s = s + 1 == up_stages ? 0 : s + 1) {
        if (!(ok = wait_free())) break;
        if (walk.done()) {
          arm(none, 0);  // to each team
          if (++told == kTeams) break;
          continue;
        }
        const MoeStage st = walk.stage();
        arm(st, fetch.bytes(st), up_bytes);
        fetch.weights(base + s * up_bytes, smem_u32(&sh.full[s]), st);
        fetch.tokens(base + s * up_bytes, smem_u32(&sh.full[s]), st);
        walk.next();
      }
    }
    // the second product's stages lie elsewhere in the ring: all of the first's are read before
    for (s = 0; s < up_stages && ok; ++s) ok = wait_free();
    s = 0;
    {
      const MoeFetch<false, false, Down> fetch{p, sh, &map_down, nullptr, lane};
      MoeWalk<false, 1> walk{p, hits, hits ? tiles * parts : 0, parts, kDownRows, Down::slices, down_chunks, p.counter + 3, lane, sh};
      walk.begin();
      // Wd does not wait for h
      int first = 0;
      for (; ok && first < down_stages && !walk.done(); ++first) {
        const MoeStage st = walk.stage();
        s = first;
        arm(st, fetch.bytes(st), down_bytes);
        fetch.weights(base + s * down_bytes, smem_u32(&sh.full[s]), st);
        walk.next();
      }
      // barrier over the grid: all of h is there.  All CTAs run at once (cooperative launch).
      if (lane == 0 && ok) {
        const uint64_t t0 = global_timer_ns();
        for (uint32_t it = 1; ld_acquire_gpu(p.counter) < gridDim.x; ++it)
          if ((it & 63u) == 0 && (*abort_flag || global_timer_ns() - t0 > p.timeout_ns || it >= (1u << 28))) {
            record_error(p.err, DG_ERR_DEVICE_TIMEOUT, kSiteMoeBarrier);
            sh.abort = 1;
            break;
          }
        __threadfence();
        asm volatile("fence.proxy.async;" ::: "memory");  // h was written by ordinary stores
      }
      __syncwarp();
      griddep_launch_dependents();
      for (int i = 0; i < first; ++i) {
        const MoeStage st = sh.stage[i];
        fetch.tokens(base + i * down_bytes, smem_u32(&sh.full[i]), st);
      }
      ok = ok && *abort_flag == 0;
      for (s = first == down_stages ? 0 : first; ok; s = s + 1 == down_stages ? 0 : s + 1) {
        if (!(ok = wait_free())) break;
        if (walk.done()) {
          arm(none, 0);
          break;
        }
        const MoeStage st = walk.stage();
        arm(st, fetch.bytes(st), down_bytes);
        fetch.weights(base + s * down_bytes, smem_u32(&sh.full[s]), st);
        fetch.tokens(base + s * down_bytes, smem_u32(&sh.full[s]), st);
        walk.next();
      }
    }
    // no copy is in flight when the CTA ends
    for (s = 0; s < kMoeStages; ++s)
      if (armed >> s & 1u) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(smem_u32(&sh.full[s]), (used >> s & 1u) ^ 1u) &&
               global_timer_ns() - t0 < p.timeout_ns + 1000000000ull) {
        }
      }
    return;
  }

  if (warp > kMoeWarps) {
    // ------------------------------------------------------------ finish units
    constexpr bool kTurns = moe_turns(MAX);
    constexpr int kTeam = kTurns ? 32 : 32 * kMoeFinishers;  // threads that share a unit
    const int finisher = warp - kMoeWarps - 1, member = kTurns ? 0 : finisher, thread = kTurns ? lane : member * 32 + lane;
    auto team_barrier = [&]() {
      if (kTurns) __syncwarp();
      else named_barrier(1, kTeam);
    };
    // The next unit that is this warp's; false where there is none (or a wait ran out).  A warp looks at its own units
    // alone: their buffers stay until it gives them back.
    constexpr int kStep = kTurns ? kMoeFinishers : 1;
    int n = kTurns ? finisher : 0;
    MoeStage st;
    bool ok = true;
    auto take = [&]() {
      ok = wait_quick(smem_u32(&sh.summed[n % kBuffers]), (n / kBuffers) & 1, abort_flag, p.timeout_ns, p.err,
                        kSiteMoeSums);
      // (warps that share units meet at barriers: all go on, or none)
      if (!kTurns) ok = all_agree(1, kTeam, ok);
      if (ok) st = sh.unit[n % kBuffers];
      return ok && st.hit >= 0;
    };
    auto give = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.taken[n % kBuffers]));
      n += kStep;
    };
    while (take()) {
      const int first = st.first, count = st.count;
      const float4* sums = reinterpret_cast<const float4*>(exchange + n % kBuffers * up_buffer) + lane;
      int octets = 0;
      for (int tile = member; tile < 1 << Up::lg; tile += kTeam / 32, ++octets)
        moe_activate<Up>(p, sums + tile * Up::slices * blocks * 32, blocks, st.row / 8 + tile, first, count, lane);
      give();
      // the last of 16 octets brings their 128 columns into halves
      __threadfence();
      __syncwarp();
      const int block = st.row / 128;
      int old = 0;
      if (lane == 0)
        old = (int)atomicAdd(p.counter + kMoeBarrierWords + st.hit * down_chunks + block, (uint32_t)octets);
      old = __shfl_sync(0xffffffffu, old, 0);
      if (old + octets == 16) {
        __threadfence();
        moe_halves(p, block, first, count, lane);
      }
    }
    if (ok) {
      give();
      // the units of the second product are counted from st.row on
      n = st.row + (kTurns ? (finisher + kMoeFinishers - st.row % kMoeFinishers) % kMoeFinishers : 0);
    }
    __threadfence();
    named_barrier(2, 32 * kMoeFinishers);
    if (tid == 32 * (kMoeWarps + 1)) {
      __threadfence();
      atomicAdd(p.counter, 1u);
    }
    const int64_t share = (int64_t)p.tokens * p.d;
    while (ok && take()) {
      // 4 neighbouring rows of a token a thread
      const float* sums = exchange + n % kBuffers * down_buffer;
      const int items = live * (kDownRows / 4);
      for (int i = thread; i < items; i += kTeam) {
        const int row = i % (kDownRows / 4) * 4, t = i / (kDownRows / 4);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < Down::slices; ++k)  // warps k << lg + tile
          add4(v, *reinterpret_cast<const float4*>(sums + (((k << Down::lg) + (row >> 4)) * live + t) * 16 + (row & 15)));
        if (parts == 1) moe_store(p, t, st.row + row, v);
        else __stcg(reinterpret_cast<float4*>(p.part + st.part * share + (int64_t)t * p.d + st.row + row), v);
      }
      give();
      if (parts > 1) {
        // the last of the shares adds them, in their order
        __threadfence();
        team_barrier();
        int last = 0;
        if (thread == 0) {
          last = atomicAdd(p.counter + p.tile_counter + st.row / kDownRows, 1u) == (uint32_t)parts - 1;
          if (!kTurns) sh.last = last;
        }
        team_barrier();
        last = kTurns ? __shfl_sync(0xffffffffu, last, 0) : sh.last;
        if (last) {
          __threadfence();
          for (int i = thread; i < items; i += kTeam) {
            const int row = i % (kDownRows / 4) * 4, t = i / (kDownRows / 4);
            const float* from = p.part + (int64_t)t * p.d + st.row + row;
            float4 all[kMoeMaxParts];
#pragma unroll
            for (int k = 0; k < kMoeMaxParts; ++k)
              all[k] = k < parts ? __ldcg(reinterpret_cast<const float4*>(from + k * share)) : make_float4(0, 0, 0, 0);
#pragma unroll
            for (int k = 1; k < kMoeMaxParts; ++k) add4(all[0], all[k]);
            moe_store(p, t, st.row + row, all[0]);
          }
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- multiply
  const int team = warp / (kMoeWarps / kTeams), member = warp % (kMoeWarps / kTeams);
  int s = team, n = 0;  // ring slot; units so far
  MoeStage st;
  bool ok = true;
  // the team's next stage, or false where there is none (or a wait ran out)
  auto take = [&]() {
    ok = wait_quick(smem_u32(&sh.full[s]), used >> s & 1u, abort_flag, p.timeout_ns, p.err, kSiteMmaFull);
    if (ok) st = sh.stage[s];
    return ok && st.hit >= 0;
  };
  auto give = [&](int stages, int step) {
    __syncwarp();
    if (lane == 0) mbar_arrive_n(smem_u32(&sh.empty[s]), (uint32_t)step);
    used ^= 1u << s;
    s = s + step >= stages ? s + step - stages : s + step;
  };
  // a buffer of the exchange is free / holds unit `now`'s sums
  auto wait_taken = [&]() {
    ok = wait_quick(smem_u32(&sh.taken[n % kBuffers]), ((n / kBuffers) & 1) ^ 1, abort_flag, p.timeout_ns, p.err,
                      kSiteMoeSums);
  };
  auto hand_over = [&](const MoeStage& now) {
    if (tid == 0) sh.unit[n % kBuffers] = now;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.summed[n % kBuffers]));
    ++n;
  };
  // tells each finishing warp that a product has no more units, and where the next one's count begins
  auto finish = [&]() {
    constexpr int kTold = moe_turns(MAX) ? kMoeFinishers : 1;
    const int next = n + kTold;
    for (int i = 0; i < kTold && ok; ++i) {
      wait_taken();
      if (ok) hand_over(MoeStage{-1, 0, 0, 0, next, 0, 0, 0});
    }
  };
  float acc[MAX][4];
  auto clear = [&]() {
#pragma unroll
    for (int nb = 0; nb < MAX; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nb][i] = 0.0f;
  };
  {
    const int tile = member & ((1 << Up::lg) - 1), slice = member >> Up::lg;
    while (take()) {
      if (st.begin) clear();
      if (st.chunk + kTeams * slice < up_chunks)
        moe_multiply<true, Up, kTeams, MAX>(smem + s * up_bytes, tile, kTeams * slice, st.chunk, up_chunks, st.count,
                                            lane, acc);
      const MoeStage now = st;
      give(up_stages, kTeams);
      if (!now.end) continue;
      wait_taken();
      if (!ok) break;
      float4* sums = reinterpret_cast<float4*>(exchange + n % kBuffers * up_buffer) +
                     (tile * Up::slices + team * (Up::slices / kTeams) + slice) * blocks * 32 + lane;
#pragma unroll
      for (int nb = 0; nb < MAX; ++nb)
        if (nb * 8 < now.count) sums[nb * 32] = make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
      hand_over(now);
    }
    if (ok) {
      give(up_stages, kTeams);
      finish();
    }
    // the other team's slots have been used as often as this one's
    if (kTeams == 2) used = team == 0 ? used | used << 1 : used | used >> 1;
    s = 0;
  }
  // (in the second product, where each expert's sums are taken out one by one, all warps take every stage)
  const int tile = warp & ((1 << Down::lg) - 1), slice = warp >> Down::lg, r = lane >> 2, q = lane & 3;
  bool fresh = true;  // nothing of this unit is in the exchange
  while (ok && take()) {
    if (st.chunk == 0) clear();
    if (st.chunk + slice < down_chunks)
      moe_multiply<false, Down, 1, MAX>(smem + s * down_bytes, tile, slice, st.chunk, down_chunks, st.count, lane, acc);
    const MoeStage now = st;
    give(down_stages, 1);
    if (now.chunk + Down::slices < down_chunks) continue;
    float* const mine = exchange + n % kBuffers * down_buffer + warp * live * 16;  // [token][16 rows]
    if (fresh) {
      wait_taken();
      if (!ok) break;
      for (int i = lane; i < live * 16; i += 32) mine[i] = 0.0f;
      __syncwarp();
    }
    // an expert's sums, with the weight of each of its tokens
#pragma unroll
    for (int nb = 0; nb < MAX; ++nb) {
      if (nb * 8 >= now.count) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = nb * 8 + 2 * q + i;
        if (m < now.count) {
          const int t = sh.pair_token[now.first + m];
          const float w = sh.weight[t * p.top_k + sh.pair_slot[now.first + m]];
          float* y = mine + t * 16 + r;
          y[0] = fmaf(w, acc[nb][i], y[0]);
          y[8] = fmaf(w, acc[nb][2 + i], y[8]);
        }
      }
    }
    __syncwarp();
    fresh = now.end != 0;
    if (fresh) hand_over(now);
  }
  if (ok) finish();
}

template <int MAX>
cudaError_t moe_layer_launch(const MoeArgs& p, const void* up, const void* down, MoeEncode encode, int sms,
                             cudaStream_t stream) {
  constexpr size_t smem = kMoeSmem + 1024;
  CUtensorMap map_up, map_down, map_x = {};
  if (!encode(&map_up, up, p.d, (uint64_t)p.experts * 2 * p.f, 8 << up_lg(MAX), kMoeWarps >> up_lg(MAX)) ||
      !encode(&map_down, down, p.f, (uint64_t)p.experts * p.d, 16 << down_lg(MAX), kMoeWarps >> down_lg(MAX)))
    return cudaErrorInvalidValue;
  // x as words of 8 bytes [tokens][d / 128 * 34], a row's slices a box (box_rows 0: not weights)
  if (moe_gathers(MAX) && !encode(&map_x, p.xh, (uint64_t)(p.d / 128) * (kMoeChunkBytes / 8), p.tokens, 0,
                                  (kMoeWarps >> up_lg(MAX)) * (kMoeChunkBytes / 8)))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem(moe_layer_kernel<MAX>, smem, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // sets itself up while the scores are computed
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, 1, 1);
  cfg.blockDim = dim3(kMoeThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_layer_kernel<MAX>, p, map_up, map_down, map_x);
}

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
  a.tile_counter = (int32_t)(kMoeBarrierWords + hits * (f / 128));
  a.counters = (int32_t)(a.tile_counter + d / 16);
  a.counter = reinterpret_cast<uint32_t*>(take((uint64_t)a.counters * 4));
  a.logits = reinterpret_cast<float2*>(take(t * e * 8));
  a.keys = reinterpret_cast<uint64_t*>(take(t * e * 8));
  a.xh = take(t * (d / 128) * kMoeChunkBytes);
  a.h = reinterpret_cast<float*>(take(pairs * f * 4));
  a.hh = take(pairs * (f / 128) * kMoeHiddenBytes);
  a.part = reinterpret_cast<float*>(take(kMoeMaxParts * t * d * 4));
  return at;
}

cudaError_t moe_few_tokens_launch(MoeArgs p, const void* up, const void* down, MoeEncode encode, bool router_fp32,
                                  int sms, bool pdl, cudaStream_t stream) {
  cudaError_t e = error_word_address(&p.err);
  if (e != cudaSuccess) return e;
  const int groups = (p.tokens + kScoreTokens - 1) / kScoreTokens;
  const dim3 grid((unsigned)(p.experts * groups + p.tokens));
  e = router_fp32 ? launch_op(moe_scores_kernel<float>, grid, kScoreThreads, 0, pdl, stream, p)
                  : launch_op(moe_scores_kernel<__nv_bfloat16>, grid, kScoreThreads, 0, pdl, stream, p);
  if (e != cudaSuccess) return e;
  // (an expert has at most all tokens)
  if (p.tokens <= 8) return moe_layer_launch<1>(p, up, down, encode, sms, stream);
  if (p.tokens <= 16) return moe_layer_launch<2>(p, up, down, encode, sms, stream);
  if (p.tokens <= 32) return moe_layer_launch<4>(p, up, down, encode, sms, stream);
  return moe_layer_launch<8>(p, up, down, encode, sms, stream);
}

}  // namespace dg
