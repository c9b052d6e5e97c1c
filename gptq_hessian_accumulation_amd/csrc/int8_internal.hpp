// Internal interface of the 8-bit integer operators: rows held as codes with
// scales, and the product of two such matrices.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hess {

// Rows of d values of a type as int8 codes.  block 0: one float scale a row;
// block 32: one exponent byte for 32 columns (groups a row).
struct Int8Rows {
  const void* x;  // quantize: the values; dequantize: the output
  int64_t ldx;
  int8_t* codes;
  int64_t ldc;
  void* scale;    // n floats, or n x groups bytes
  int64_t n, d;
  int64_t pad;    // columns written: d, or more (zeros past d)
};
hipError_t launch_int8_quantize(const Int8Rows& r, int block, int dtype, hipStream_t stream);
hipError_t launch_int8_dequantize(const Int8Rows& r, int block, int dtype, hipStream_t stream);

// y[t][o] = (sum_k a[t][k] b[o][k]) sa[t] sb[o].
struct Int8Gemm {
  const int8_t* a;  // M x K
  int64_t lda;
  const float* sa;
  const int8_t* b;  // N x K
  int64_t ldb;
  const float* sb;
  void* y;
  int64_t ldy;
  int64_t M, N, K;
};

// Operands of any alignment, no workspace.
hipError_t launch_int8_few(const Int8Gemm& g, int dtype, hipStream_t stream);

}  // namespace hess
