// Internal interface of the gated feed-forward block: the three products it
// consists of, their tile schedule, and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8_internal.hpp"

namespace hess {

enum FfnMode {
  kFfnFwd = 0,  // h = act(x Wg^T) * (x Wu^T)          M = n, N = f (half a tile's columns each), K = d
  kFfnDx = 1,   // dx = dg Wg + du Wu                   M = n, N = d, K = f, two segments (or one: dy W)
  kFfnDw = 2,   // [dWg; dWu] = [dg du]^T x             M = 2 fp, N = d, K = n
};

// One product.  The pre-activation pair g, u and its gradient dg, du are kept
// as one n x 2 fp matrix (fp = f rounded up to 8, columns f .. fp - 1 zero):
// g or dg in the first fp columns, u or du in the last.
struct FfnGemm {
  const void* a;   // fwd: x (n x d); dx and dw: the n x 2 fp gradient pair
  int64_t lda;
  const void* b0;  // fwd and dx: Wg (f x d); dw: x (n x d)
  int64_t ldb0;
  const void* b1;  // fwd and dx: Wu
  int64_t ldb1;
  void* o0;        // fwd: h; dx: dx; dw: dWg
  int64_t ldo0;
  void* o1;        // fwd: the pre-activation pair, row stride 2 fp, or null; dw: dWu
  int64_t ldo1;
  float* ws;       // partial tiles of the split items
  int64_t M, N, K;
  int64_t f, fp;
  int act;
  int pre32;       // fwd: o1 is float32 whatever the type
  int pre8;        // fwd: o1 is the pair as int8 codes in blocks of 32 (see pair8_cols)
  int segs;        // dx: segments of K
  // schedule: tiles 0 .. full - 1 of the blocked order are done whole; each of
  // the others is cut into `parts` ranges of part_len K-iterations, whose
  // partial sums go to workspace slot part * (ntiles - full) + (tile - full)
  int tm, tn, ntiles, full, parts, part_len, niter;
};

// Chooses the tile's edge (returned) and fills the schedule.
int ffn_schedule(FfnGemm& g, int mode, int dtype);

// A schedule in place of the estimate's, process-wide: tiles of this edge (0:
// the estimate's own choice), the first `whole` of them done whole and the
// others in `parts` ranges of K.
struct FfnForced {
  int edge, whole, parts;
};
void ffn_force_schedule(FfnForced f);
FfnForced ffn_forced();

// One product by tiles.  Every operand row 16-byte aligned; where an operand's
// rows run along K, K is a whole number of 16-byte pieces.
hipError_t launch_ffn_gemm(const FfnGemm& g, int mode, int edge, int dtype, hipStream_t stream);

// The forward product of at most kFfnFew tokens: operands of any alignment, no
// workspace.
constexpr int64_t kFfnFew = 64;

// Whether up to kFfnFew tokens take that kernel also where tiles could read the
// operands in place.  Every workgroup reads all of x, padded to 16, 32 or 64
// tokens, so tiles, which split K over workgroups, gain as x grows; past 32
// tokens a second round of workgroups (one for 16 features, 256 CUs) costs
// more than they do.  Few tokens against tiles, us, weights not in any cache:
//   bf16, 16 tokens   2560 x 2816 11.0 / 15.8   4096 x 11264 40.7 / 51.5
//         32 tokens   2560 x 2816 15.2 / 16.5   4096 x 11264 50.2 / 54.1   8192 x 2816 40.3 / 30.8
//         64 tokens   1024 x 2816  9.1 / 12.2   2560 x 2816 18.5 / 19.0    4096 x 2816 25.6 / 20.6
//                     2560 x 5632 32.3 / 30.1   4096 x 11264 69.9 / 60.0
//   float32, 32 tokens  2560 x 2816 25.0 / 28.4   4096 x 2816 34.5 / 36.5   4096 x 11264 118 / 111
//            64 tokens  1024 x 2816 19.7 / 19.4   2560 x 2816 41.9 / 30.7   4096 x 11264 152 / 116
// The limit's worst case is near 32 bf16 tokens at 4096 x 1024: 20.6 / 16.7.
inline bool ffn_prefers_few(int64_t n, int64_t d, int64_t f, int64_t esize) {
  if (n <= 16) return true;
  if (n <= 32) return 32 * d * esize <= 320 * 1024;
  return n <= kFfnFew && f <= 4096 && 64 * d * esize <= 320 * 1024;
}
hipError_t launch_ffn_few(const FfnGemm& g, int dtype, hipStream_t stream);

// Copies up to three matrices of rows[m] x cols 16-bit values (row stride
// ld[m]) to rows of pad >= cols (a multiple of 8) values, zeros past cols.
struct PackRows {
  const void* src[3];
  void* dst[3];
  int64_t ld[3], rows[3];
  int count, cols, pad;
};
hipError_t launch_pack_rows16(const PackRows& p, hipStream_t stream);

// The pair in 8 bits: rows of pair8_cols(f) bytes, fq = f rounded up to 32: the
// codes of g in the first fq, those of u in the next, then an exponent byte for
// each block of 32 of g and of u.
inline int64_t pair8_cols(int64_t f) {
  const int64_t fq = (f + 31) / 32 * 32;
  return (2 * fq + fq / 16 + 15) / 16 * 16;
}

// In what type the pair is kept.
enum PairType { kPairSame = 0, kPairF32 = 1, kPairI8 = 2 };

// dg = dh u act'(g), du = dh act(g) into the n x 2 fp pair dgu (columns past f zero).
// The pair in 8 bits: x8, where its x is not null, is restored in the same launch
// (blocks of 32).
hipError_t launch_ffn_dgu(const void* dh, int64_t lddh, const void* preact, PairType pair, void* dgu, int64_t n,
                          int64_t f, int64_t fp, int act, int dtype, const Int8Rows& x8, hipStream_t stream);

// Zeros rows x cols elements of esize bytes at p (row stride ld elements).
hipError_t launch_zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int esize, hipStream_t stream);

}  // namespace hess
