// Arguments and launches of the gated feed-forward product's kernels.
#pragma once

#include "dg_internal.h"

namespace dg {

struct GatedArgs {
  GemmArgs base;           // m, k, groups, blocks (n_blocks: of 128 columns of h), timeouts
  __nv_bfloat16* h;        // BF16 result [.., m, f], row stride ldh; or:
  uint8_t* hq;             // E4M3 result [.., m, f] and its packed scales
  uint32_t* hsf;
  uint8_t* cq;             // nullable: E4M3 [.., m, 2f] of [g | u] and its packed scales
  uint32_t* csf;
  int64_t ldh;
  int32_t f;
  int32_t m_pad;           // align(m, 4): rows of a scale word's line
  int32_t activation;      // dg_activation
};

// gated_gemm.cu; mode kDense, kContiguous or kMasked
cudaError_t gated_gemm_launch(int mode, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sfa,
                              const CUtensorMap& sfb, GatedArgs args, int grid, cudaStream_t stream);


// gated_decode.cu; tn = tokens per CTA (32 or 64), split = CTAs per cluster (1,
// 2, 4 or 8); each CTA's K range spans at most gated_decode_max_packs() scale
// words of 4 K blocks
cudaError_t gated_decode_launch(int tn, int split, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& sfa,
                                const CUtensorMap& sfb, GatedArgs args, int strips, int token_blocks,
                                cudaStream_t stream);
int gated_decode_max_packs();
int gated_decode_max_clusters(int tn, int split);  // that run at once on the current device


// gated_gemv.cu: one to four tokens without the tensor cores
// sms: SMs it may use; limited: fewer than the device has
bool gated_gemv_takes(int64_t m, int64_t f, int64_t k, bool eight_bit, int sms, bool limited);
cudaError_t gated_gemv_launch(const void* a, const void* sfa, const void* b, const void* sfb, int64_t lda, int64_t ldb,
                              const GatedArgs& args, cudaStream_t stream);

}  // namespace dg
