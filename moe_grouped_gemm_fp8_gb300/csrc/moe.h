// Arguments and launch of the mixture-of-experts layer for a few tokens.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_internal.h"

namespace dg {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxParts = 8;        // shares of the hit experts in the second product
constexpr int kMoeBarrierWords = 32;  // the grid barrier's counter and those of the units

// Encodes weights of `rows` rows and `cols` columns as bytes [cols / 128][rows][128]
// in boxes of slices x box_rows x 128, 128-byte swizzle; with box_rows 0, words of 8
// bytes [rows][cols] in boxes of one row x slices.
using MoeEncode = bool (*)(CUtensorMap* to, const void* base, uint64_t cols, uint64_t rows,
                           uint32_t box_rows, uint32_t slices);

struct MoeArgs {
  const __nv_bfloat16* x;      // [tokens, d], row stride ldx
  const void* router;          // FP32 or BF16 [experts, d]
  const float* router_bias;    // nullable, [experts]
  const uint32_t* up_sf;       // packed scales of the weights
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
  uint32_t* counter;           // grid barrier, units taken; octets done of each (hit expert, 128 columns of h);
                               // from tile_counter: shares done of each rows of y
  int32_t counters, tile_counter;
  float2* logits;              // [tokens, experts], an FP32 and what it lacks
  uint64_t* keys;              // [tokens, experts]: ordered as what the choice goes by
  uint8_t* xh;                 // [tokens, d / 128] chunks as the products read them
  float* h;                    // [tokens * top_k, f], pairs in the order of their experts
  uint8_t* hh;                 // by hit expert [f / 128][its tokens] chunks
  float* part;                 // [shares, tokens, d]
};

// Sets the workspace's pointers; the bytes it takes.
uint64_t moe_few_tokens_layout(MoeArgs& a, void* workspace);
// up: E4M3 [experts, 2f, d]; down: E4M3 [experts, d, f]
cudaError_t moe_few_tokens_launch(MoeArgs p, const void* up, const void* down, MoeEncode encode, bool router_fp32,
                                  int sms, bool pdl, cudaStream_t stream);

}  // namespace dg
