// Arguments and launch of the mixture-of-experts layer for a few tokens.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dg_internal.h"

namespace dg {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeBarrierWords = 32;  // the grid barrier's counter, on a line of its own

struct MoeArgs {
  const __nv_bfloat16* x;      // [tokens, d], row stride ldx
  const void* router;          // FP32 or BF16 [experts, d]
  const float* router_bias;    // nullable, [experts]
  const uint8_t* up;           // E4M3 [experts, 2f, d] and packed scales
  const uint32_t* up_sf;
  const uint8_t* down;         // E4M3 [experts, d, f] and packed scales
  const uint32_t* down_sf;
  const __nv_bfloat16* c;      // nullable, [tokens, d], row stride ldc
  const int32_t* num_tokens;   // nullable, on the device
  __nv_bfloat16* y;            // [tokens, d], row stride ldy
  int32_t* chosen_out;         // [tokens, top_k]
  float* weight_out;
  int64_t ldx, ldc, ldy;
  int32_t tokens, d, f, experts, top_k;
  int32_t score, renormalize, activation;
  float scale;
  uint64_t timeout_ns;
  unsigned long long* err;
  // the workspace (moe_few_tokens_layout)
  uint32_t* counter;           // grid barrier, then octets done of each (hit expert, 128 columns of h)
  int32_t counters;
  double* logits;              // [tokens, experts]
  double* select;              // [tokens, experts]: scores with the bias, where there is one
  __half* xh;                  // [tokens, d] in the streams' order, and a scale per 128
  float* xs;
  float* h;                    // [tokens * top_k, f], pairs in the order of their experts
  __half* hh;                  // the same as halves in the streams' order, and a scale per 128
  float* hs;
};

// Sets the workspace's pointers; the bytes it takes.
uint64_t moe_few_tokens_layout(MoeArgs& a, void* workspace);
cudaError_t moe_few_tokens_launch(MoeArgs p, bool router_fp32, int sms, bool pdl, cudaStream_t stream);

}  // namespace dg
