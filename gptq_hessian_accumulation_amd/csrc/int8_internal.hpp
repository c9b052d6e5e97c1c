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
struct PackCodes;
// block 0, and in the same launch the copy of one matrix of codes (count 0 or 1).
hipError_t launch_int8_quantize_and_pack(const Int8Rows& r, int dtype, const PackCodes& p, hipStream_t stream);
// What a backward pass needs of a linear layer, in one launch: up to two sets of
// rows with a scale each as values of dtype (rows.x null: not wanted), and dy
// copied to rows of dy_pad values (src null: not wanted).
struct GradOperands {
  Int8Rows rows[2];
  const void* src;
  void* dst;
  int64_t ld, n, cols, pad;
};
hipError_t launch_int8_grad_operands(const GradOperands& g, int dtype, hipStream_t stream);
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
  const void* x;    // one row: the values that a would hold
  int64_t ldx;
  int* ws;          // partial tiles of the split items
  // schedule: tiles 0 .. full - 1 are done whole; each of the others is cut into
  // `parts` ranges of part_len K-iterations, whose partial sums go to workspace
  // slot part * (ntiles - full) + (tile - full)
  int tm, tn, ntiles, full, parts, part_len, niter;
};

// Operands of any alignment, no workspace.
hipError_t launch_int8_few(const Int8Gemm& g, int dtype, hipStream_t stream);
// One row of values x of dtype (M = 1, K <= kInt8One; a and sa not read).
hipError_t launch_int8_one(const Int8Gemm& g, int dtype, hipStream_t stream);
constexpr int64_t kInt8One = 8192;

// Chooses the tile's edge (returned) and fills the schedule.
int int8_schedule(Int8Gemm& g);
// By tiles: every row of a and b 16-byte aligned, a's codes zero from K to the
// next multiple of 16.
hipError_t launch_int8_tile(const Int8Gemm& g, int edge, int dtype, hipStream_t stream);

// Whether a product of n rows of a, d long, takes the kernel without tiles, whose
// workgroups take all of K: 33 to 64 rows only up to 8191 columns.  64 rows, without
// and with tiles, us: 4096 x 2048 8.0 / 12.4, 6144 x 2560 13.7 / 13.8, 4096 x 8192
// 16.7 / 14.3, 8192 x 1024 13.0 / 14.3, 8192 x 2560 17.2 / 15.0, 8192 x 8192 28.6 /
// 24.0, 8192 x 16384 38.1 / 41.7, 16384 x 2048 23.8 / 17.3, 16384 x 8192 55.4 / 41.1;
// 32 rows, 16384 x 8192 35.7 / 41.1.  (The first number of a product is d, the second
// f.  The rule goes by d alone, and three of these take the slower way, by 9 to 17%:
// 4096 x 8192, 8192 x 1024 and 8192 x 16384.)
inline bool int8_few(int64_t n, int64_t d) { return n <= 32 || (n <= 64 && d < 8192); }

// Copies up to two matrices of rows[m] x cols bytes (row stride ld[m]) to rows of
// pad >= cols (a multiple of 16) bytes, zeros past cols.
struct PackCodes {
  const int8_t* src[2];
  int8_t* dst[2];
  int64_t ld[2], rows[2];
  int count;
  int64_t cols, pad;
};
hipError_t launch_pack_codes(const PackCodes& p, hipStream_t stream);

}  // namespace hess
