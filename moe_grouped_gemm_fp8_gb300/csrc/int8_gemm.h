// Arguments and launches of the product of 8-bit integers.
#pragma once

#include <cuda_runtime.h>

#include "dg_internal.h"

namespace dg {

struct Int8Args {
  const int8_t* a;   // [m, k], row stride lda
  const float* sa;   // [m]
  const int8_t* b;   // [n, k], row stride ldb
  const float* sb;   // [n]
  const void* c;     // nullable, [m, n] of the result's type, row stride ldc
  void* d;           // [m, n] BF16 or FP16, row stride ldd
  int64_t lda, ldb, ldc, ldd;
  int32_t m, n, k;
  int32_t fp16;      // the result's type: FP16, else BF16
  int32_t vector;    // rows of d and c may be accessed 16 bytes at a time; 2: rows of d are on 32
  int32_t sms;
  uint64_t timeout_ns;
  unsigned long long* err;
};

// int8_stream.cu: a few rows of a, without widening them in memory
bool int8_stream_takes(const Int8Args& p);
cudaError_t int8_stream_launch(const Int8Args& p, bool pdl, cudaStream_t stream);
// int8_decode.cu: operand roles swapped, columns split over clusters
bool int8_decode_takes(const Int8Args& p);
cudaError_t int8_decode_launch(Int8Args p, bool pdl, cudaStream_t stream);
// int8_gemm.cu: tiles on the tensor cores
cudaError_t int8_gemm_launch(Int8Args p, bool pdl, cudaStream_t stream);

// int8_quant.cu
cudaError_t quantize_int8_launch(const void* x, int dtype, int8_t* q, float* scales, int64_t rows, int64_t cols,
                                 int64_t ldx, int sms, bool pdl, cudaStream_t stream);

}  // namespace dg
