// C ABI of the gated feed-forward block and the top-logit distillation loss
// (declared in include/hess.h): argument checks, workspace layout, dispatch.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../../include/hess.h"
#include "distill_internal.hpp"
#include "ffn_internal.hpp"
#include "hess_internal.hpp"
#include "ops_checks.hpp"

using namespace hess;

namespace {

constexpr int64_t kMaxVocab = (int64_t)1 << 28;
constexpr int kMaxTop = 1024;

// The tiles take 16-byte pieces of the rows of x and the weights: widths that
// are no whole number of them are copied to padded rows in the workspace.
int64_t piece(int dtype) { return 16 / elem_bytes(dtype); }
bool packed(int64_t d, int dtype) { return d % piece(dtype) != 0; }
int64_t pack_bytes(int64_t rows, int64_t d, int dtype) { return up(rows * up(d, piece(dtype)) * elem_bytes(dtype), 256); }

// Workspace: forward: packed x, gate, up | partial tiles; backward: the
// gradient pair | packed x, gate, up | x restored from 8 bits | partial tiles.
struct FfnWork {
  int64_t pack, x8, slots, total;
};
FfnGemm two_segments(FfnGemm g) {
  g.segs = 2;
  return g;
}
FfnWork ffn_work(int64_t n, int64_t d, int64_t f, int dtype, bool backward, bool pre8 = false, bool x8 = false) {
  FfnWork w{};
  // (a pair in 8 bits comes from tiles, whose workgroups hold whole blocks of it)
  if (!backward && !pre8 && n <= kFfnFew && (packed(d, dtype) || ffn_prefers_few(n, d, f, elem_bytes(dtype)))) return w;
  w.pack = backward ? up(n * 2 * up(f, 8) * elem_bytes(dtype), 256) : 0;
  w.x8 = w.pack + (packed(d, dtype) ? pack_bytes(n, d, dtype) + 2 * pack_bytes(f, d, dtype) : 0);
  w.slots = w.x8 + (x8 ? pack_bytes(n, d, dtype) : 0);
  w.total = w.slots + (backward ? std::max(slot_bytes(two_segments(shape(n, d, f)), kFfnDx, dtype),
                                           slot_bytes(shape(2 * up(f, 8), d, n), kFfnDw, dtype))
                                : slot_bytes(shape(n, f, d), kFfnFwd, dtype));
  return w;
}

// The pair's type from the bits added to act, which are taken off (both: none).
PairType pair_type(int& act) {
  const int bits = act < 0 ? 0 : act & (HESS_PREACT_F32 | HESS_PREACT_I8);
  if (bits == (HESS_PREACT_F32 | HESS_PREACT_I8)) return kPairSame;
  act &= ~bits;
  return bits == HESS_PREACT_F32 ? kPairF32 : bits == HESS_PREACT_I8 ? kPairI8 : kPairSame;
}
Mat pair_mat(const void* p, PairType pair, int64_t n, int64_t f) {
  if (pair == kPairI8) return {"preact", p, pair8_cols(f), n, pair8_cols(f), 1};
  return {"preact", p, 2 * up(f, 8), n, 2 * up(f, 8), pair == kPairF32 ? 4 : 0};
}

// x, gate and up as the tiles take them: where they are, or copied to padded
// rows.
struct FfnOperands {
  const void *x, *wg, *wu;
  int64_t ldx, ldg, ldu, d;
};
// Whether rows of x, gate and up start where the tiles can read them.
bool rows_in_place(const FfnOperands& o, int64_t n, int64_t f, int dtype) {
  const int64_t step = piece(dtype);
  return aligned(o.x, 16) && aligned(o.wg, 16) && aligned(o.wu, 16) && (n <= 1 || o.ldx % step == 0) &&
         (f <= 1 || (o.ldg % step == 0 && o.ldu % step == 0));
}
int place_operands(FfnOperands& o, char* pack, int64_t n, int64_t f, int dtype, bool want_x, bool want_w,
                   hipStream_t s) {
  const int64_t step = piece(dtype);
  if (!packed(o.d, dtype)) {
    if (!rows_in_place(o, n, f, dtype))
      return fail(HESS_EALIGN, "rows of x, w_gate and w_up must be 16-byte aligned where a row is a multiple of 16 bytes");
    return HESS_OK;
  }
  const int64_t pad = up(o.d, step), half = elem_bytes(dtype) / 2;  // a float32 moves as two 16-bit halves
  char* pg = pack + pack_bytes(n, o.d, dtype);
  char* pu = pg + pack_bytes(f, o.d, dtype);
  PackRows p{};
  p.cols = (int)(o.d * half);
  p.pad = (int)(pad * half);
  auto add = [&](const void* src, int64_t ld, int64_t rows, void* dst) {
    p.src[p.count] = src;
    p.dst[p.count] = dst;
    p.ld[p.count] = ld * half;
    p.rows[p.count++] = rows;
  };
  if (want_x) add(o.x, o.ldx, n, pack);
  if (want_w) add(o.wg, o.ldg, f, pg);
  if (want_w) add(o.wu, o.ldu, f, pu);
  if (p.count > 0) {
    const hipError_t e = launch_pack_rows16(p, s);
    if (e != hipSuccess) return hip_fail(e, "operand copy launch");
  }
  o = FfnOperands{pack, pg, pu, pad, pad, pad, pad};
  return HESS_OK;
}

// The backward pass; x8: x is its codes (with row stride ldx) in blocks of 32.
int ffn_backward(const void* dh, int64_t lddh, const void* x, int64_t ldx, const Int8Rows* x8, const void* w_gate,
                 int64_t ldg, const void* w_up, int64_t ldu, const void* preact, int dtype, int act, int64_t n,
                            int64_t d, int64_t f, void* dx, int64_t lddx, void* dw_gate, int64_t lddg, void* dw_up,
                            int64_t lddu, void* work, int64_t work_bytes, hess_stream_t stream) {
  if (int rc = check_ffn_sizes(n, d, f, dtype)) return rc;
  const PairType pair = pair_type(act);
  if (act < HESS_SILU || act > HESS_GELU_TANH) return fail(HESS_EINVAL, "unknown activation %d", act);
  if (!dw_gate != !dw_up) return fail(HESS_EINVAL, "dw_gate and dw_up: both or neither");
  const int64_t es = elem_bytes(dtype), fp = up(f, 8);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t exps = x8 ? n * ((d + 31) / 32) : 0;
  const Mat ins[6] = {{"dh", dh, lddh, n, f},
                      {"x", x, ldx, n, d, x8 ? 1 : 0},
                      {"w_gate", w_gate, ldg, f, d},
                      {"w_up", w_up, ldu, f, d},
                      pair_mat(preact, pair, n, f),
                      {"x_exponents", x8 ? x8->scale : nullptr, exps, 1, exps, 1}};
  const Mat outs[3] = {{"dx", dx, lddx, n, d}, {"dw_gate", dw_gate, lddg, f, d}, {"dw_up", dw_up, lddu, f, d}};
  for (const Mat& m : ins) {
    if (n == 0 && m.rows == 0) continue;
    if (&m == &ins[1] && !x && !dw_gate) continue;  // dx alone does not read it
    if (&m == &ins[5]) {
      if (n > 0 && x8 && dw_gate && !m.p) return fail(HESS_EINVAL, "null x_exponents");
      continue;
    }
    if (int rc = check_mat(m, m.own ? 1 : es)) return rc;
  }
  for (const Mat& m : outs)
    if (m.p && m.rows > 0)
      if (int rc = check_mat(m, es)) return rc;
  if (!aligned(preact, 16)) return fail(HESS_EALIGN, "preact not 16-byte aligned");
  const FfnWork room = n > 0 ? ffn_work(n, d, f, dtype, true, false, x8 != nullptr) : FfnWork{};
  if (int rc = check_work(work, work_bytes, room.total)) return rc;
  if (int rc = check_outputs(outs, 3, ins, 6, es, work, room.total)) return rc;
  hipError_t e = hipSuccess;
  if (n == 0) {
    if (dw_gate) {
      e = launch_zero_rows(dw_gate, lddg, f, d, (int)es, s);
      if (e == hipSuccess) e = launch_zero_rows(dw_up, lddu, f, d, (int)es, s);
    }
    return e == hipSuccess ? HESS_OK : hip_fail(e, "gradient clear launch");
  }
  if (!dx && !dw_gate) return HESS_OK;

  char* dgu = static_cast<char*>(work);
  float* slots = reinterpret_cast<float*>(dgu + room.slots);
  // x in 8 bits is restored to rows that the tiles read where they are
  const int64_t dp = up(d, piece(dtype));
  Int8Rows restored{};
  if (x8 && dw_gate) restored = {dgu + room.x8, dp, x8->codes, ldx, x8->scale, n, d, dp};
  FfnOperands o{x8 ? dgu + room.x8 : x, w_gate, w_up, x8 ? dp : ldx, ldg, ldu, d};
  if (int rc = place_operands(o, dgu + room.pack, n, f, dtype, dw_gate && !x8, dx != nullptr, s)) return rc;
  if (x8) o.x = dgu + room.x8, o.ldx = dp;
  e = launch_ffn_dgu(dh, lddh, preact, pair, dgu, n, f, fp, act, dtype, restored, s);
  if (e != hipSuccess) return hip_fail(e, "gate gradient launch");
  if (dx) {
    FfnGemm g = shape(n, d, f);
    g.segs = 2;
    g.a = dgu;
    g.lda = 2 * fp;
    g.b0 = o.wg;
    g.ldb0 = o.ldg;
    g.b1 = o.wu;
    g.ldb1 = o.ldu;
    g.o0 = dx;
    g.ldo0 = lddx;
    g.ws = slots;
    g.f = f;
    g.fp = fp;
    if (int rc = run_product(g, kFfnDx, dtype, room.total - room.slots, s, "input gradient launch")) return rc;
  }
  if (dw_gate) {
    FfnGemm g = shape(2 * fp, d, n);
    g.a = dgu;
    g.lda = 2 * fp;
    g.b0 = o.x;
    g.ldb0 = o.ldx;
    g.o0 = dw_gate;
    g.ldo0 = lddg;
    g.o1 = dw_up;
    g.ldo1 = lddu;
    g.ws = slots;
    g.f = f;
    g.fp = fp;
    if (int rc = run_product(g, kFfnDw, dtype, room.total - room.slots, s, "weight gradient launch")) return rc;
  }
  return HESS_OK;
}

}  // namespace

extern "C" {

int hess_set_ffn_schedule(int edge, int whole, int parts) {
  if (edge != 0 && edge != 64 && edge != 128 && edge != 256)
    return fail(HESS_EINVAL, "tile edge must be 0, 64, 128 or 256");
  if (whole < 0 || parts < 1 || parts > 64) return fail(HESS_EINVAL, "whole < 0, or parts outside [1, 64]");
  ffn_force_schedule({edge, whole, parts});
  return HESS_OK;
}

int64_t hess_gated_ffn_preact_cols(int64_t f) {
  if (f < 1 || f > kMaxWidth) {
    fail(HESS_EINVAL, "f = %lld outside [1, 2^17]", (long long)f);
    return -1;
  }
  return 2 * up(f, 8);
}

int64_t hess_gated_ffn_workspace(int64_t n, int64_t d, int64_t f, int dtype, int backward) {
  if (check_ffn_sizes(n, d, f, dtype) != HESS_OK) return -1;
  if (n == 0) return 0;
  const int64_t need = ffn_work(n, d, f, dtype, backward != 0, false, backward == 3).total;
  return backward == 2 ? std::max(need, ffn_work(n, d, f, dtype, false, true).total) : need;
}

int64_t hess_gated_ffn_i8_workspace(int64_t n, int64_t d, int64_t f, int dtype) {
  if (check_ffn_sizes(n, d, f, dtype) != HESS_OK) return -1;
  return n == 0 ? 0 : ffn_work(n, d, f, dtype, false, true).total;
}

int64_t hess_gated_ffn_preact_i8_cols(int64_t f) {
  if (f < 1 || f > kMaxWidth) {
    fail(HESS_EINVAL, "f = %lld outside [1, 2^17]", (long long)f);
    return -1;
  }
  return pair8_cols(f);
}

int hess_gated_ffn_forward(const void* x, int64_t ldx, const void* w_gate, int64_t ldg, const void* w_up, int64_t ldu,
                           int dtype, int act, int64_t n, int64_t d, int64_t f, void* h, int64_t ldh, void* preact,
                           void* work, int64_t work_bytes, hess_stream_t stream) {
  if (int rc = check_ffn_sizes(n, d, f, dtype)) return rc;
  const PairType pair = pair_type(act);
  if (act < HESS_SILU || act > HESS_GELU_TANH) return fail(HESS_EINVAL, "unknown activation %d", act);
  if (n == 0) return HESS_OK;
  const int64_t es = elem_bytes(dtype), fp = up(f, 8);
  const Mat ins[3] = {{"x", x, ldx, n, d}, {"w_gate", w_gate, ldg, f, d}, {"w_up", w_up, ldu, f, d}};
  const Mat outs[2] = {{"h", h, ldh, n, f}, pair_mat(preact, pair, n, f)};
  const bool pre8 = preact && pair == kPairI8;
  for (const Mat& m : ins)
    if (int rc = check_mat(m, es)) return rc;
  if (int rc = check_mat(outs[0], es)) return rc;
  if (!aligned(preact, 16)) return fail(HESS_EALIGN, "preact not 16-byte aligned");
  FfnOperands o{x, w_gate, w_up, ldx, ldg, ldu, d};
  // few tokens whose rows the tiles cannot read where they are: no copies
  const bool few = !pre8 && n <= kFfnFew && (packed(d, dtype) || ffn_prefers_few(n, d, f, es) || !rows_in_place(o, n, f, dtype));
  const FfnWork room = few ? FfnWork{} : ffn_work(n, d, f, dtype, false, pre8);
  if (int rc = check_work(work, work_bytes, room.total)) return rc;
  if (int rc = check_outputs(outs, 2, ins, 3, es, work, room.total)) return rc;

  hipStream_t s = static_cast<hipStream_t>(stream);
  char* base = static_cast<char*>(work);
  if (!few)
    if (int rc = place_operands(o, base, n, f, dtype, true, true, s)) return rc;
  FfnGemm g = shape(n, f, o.d);
  g.a = o.x;
  g.lda = o.ldx;
  g.b0 = o.wg;
  g.ldb0 = o.ldg;
  g.b1 = o.wu;
  g.ldb1 = o.ldu;
  g.o0 = h;
  g.ldo0 = ldh;
  g.o1 = preact;
  g.ldo1 = pre8 ? pair8_cols(f) : 2 * fp;
  g.ws = few ? nullptr : reinterpret_cast<float*>(base + room.slots);
  g.f = f;
  g.fp = fp;
  g.act = act;
  g.pre32 = pair == kPairF32;
  g.pre8 = pre8;
  if (!few) return run_product(g, kFfnFwd, dtype, room.total - room.slots, s, "gated feed-forward launch");
  const hipError_t e = launch_ffn_few(g, dtype, s);
  return e == hipSuccess ? HESS_OK : hip_fail(e, "gated feed-forward launch");
}

int hess_gated_ffn_backward(const void* dh, int64_t lddh, const void* x, int64_t ldx, const void* w_gate, int64_t ldg,
                            const void* w_up, int64_t ldu, const void* preact, int dtype, int act, int64_t n,
                            int64_t d, int64_t f, void* dx, int64_t lddx, void* dw_gate, int64_t lddg, void* dw_up,
                            int64_t lddu, void* work, int64_t work_bytes, hess_stream_t stream) {
  return ffn_backward(dh, lddh, x, ldx, nullptr, w_gate, ldg, w_up, ldu, preact, dtype, act, n, d, f, dx, lddx, dw_gate,
                      lddg, dw_up, lddu, work, work_bytes, stream);
}

int hess_gated_ffn_backward_x8(const void* dh, int64_t lddh, const int8_t* x_codes, int64_t ldc,
                               const uint8_t* x_exponents, const void* w_gate, int64_t ldg, const void* w_up,
                               int64_t ldu, const void* preact, int dtype, int act, int64_t n, int64_t d, int64_t f,
                               void* dx, int64_t lddx, void* dw_gate, int64_t lddg, void* dw_up, int64_t lddu,
                               void* work, int64_t work_bytes, hess_stream_t stream) {
  Int8Rows x8{};
  x8.codes = const_cast<int8_t*>(x_codes);
  x8.scale = const_cast<uint8_t*>(x_exponents);
  return ffn_backward(dh, lddh, x_codes, ldc, &x8, w_gate, ldg, w_up, ldu, preact, dtype, act, n, d, f, dx, lddx, dw_gate,
                      lddg, dw_up, lddu, work, work_bytes, stream);
}

int64_t hess_distill_topk_workspace(int64_t n, int64_t vocab, int dtype) {
  if (!dtype_ok(dtype) || n < 0 || n > kMaxRows || vocab < 1 || vocab > kMaxVocab) {
    fail(HESS_EINVAL, "bad dtype, or n = %lld outside [0, 2^24], or vocab = %lld outside [1, 2^28]", (long long)n,
         (long long)vocab);
    return -1;
  }
  return distill_workspace(n, vocab, dtype);
}

}  // extern "C"

namespace {

int check_distill(const DistillParams& P, int dtype, int values_dtype) {
  if (!dtype_ok(dtype) || !dtype_ok(values_dtype))
    return fail(HESS_EINVAL, "unknown dtype %d or values_dtype %d", dtype, values_dtype);
  if (P.n < 0 || P.n > kMaxRows) return fail(HESS_EINVAL, "n = %lld outside [0, 2^24]", (long long)P.n);
  if (P.vocab < 1 || P.vocab > kMaxVocab)
    return fail(HESS_EINVAL, "vocab = %lld outside [1, 2^28]", (long long)P.vocab);
  if (P.k < 1 || P.k > kMaxTop) return fail(HESS_EINVAL, "k = %d outside [1, %d]", P.k, kMaxTop);
  // (the reciprocal of a subnormal one passes float32's range)
  if (!(P.temperature >= FLT_MIN) || !std::isfinite(P.temperature))
    return fail(HESS_EINVAL, "temperature %g not positive and finite, or below 2^-126", (double)P.temperature);
  if (P.n == 0) return HESS_OK;
  if (!P.z || !P.ids || !P.values) return fail(HESS_EINVAL, "null logits, ids or values");
  const int64_t es = elem_bytes(dtype);
  const int64_t widest = (int64_t)1 << 30;
  if (P.ldz < P.vocab || P.ldz > widest || P.ldi < P.k || P.ldi > widest || P.ldv < P.k || P.ldv > widest)
    return fail(HESS_EINVAL, "a row stride is below its row length or above 2^30");
  if (!aligned(P.z, es) || !aligned(P.ids, P.ids64 ? 8 : 4) || !aligned(P.values, elem_bytes(values_dtype)))
    return fail(HESS_EALIGN, "logits, ids or values not aligned to the element size");
  if (!aligned(P.weight, 4)) return fail(HESS_EALIGN, "weight not float-aligned");
  if (P.dz) {
    if (P.lddz < P.vocab || P.lddz > widest) return fail(HESS_EINVAL, "row stride of dlogits below vocab or above 2^30");
    if (!aligned(P.dz, es)) return fail(HESS_EALIGN, "dlogits not aligned to its element size");
  }
  return HESS_OK;
}

struct Span {
  const char* name;
  const void* p;
  int64_t bytes;
};

// The outputs must not meet the inputs or one another; dlogits may be logits.
// extra: further outputs (and the workspace), or with extra_in further inputs.
int check_distill_overlap(const DistillParams& P, int dtype, int values_dtype, const Span* extra, int nextra,
                          bool extra_in) {
  const int64_t es = elem_bytes(dtype);
  auto rows = [&](int64_t ld, int64_t cols, int64_t e) { return ((P.n - 1) * ld + cols) * e; };
  const Span ins[4] = {{"logits", P.z, rows(P.ldz, P.vocab, es)},
                       {"ids", P.ids, rows(P.ldi, P.k, P.ids64 ? 8 : 4)},
                       {"values", P.values, rows(P.ldv, P.k, elem_bytes(values_dtype))},
                       {"weight", P.weight, P.weight ? P.n * 4 : 0}};
  const Span dz{"dlogits", P.dz, P.dz ? rows(P.lddz, P.vocab, es) : 0};
  auto meet = [](const Span& a, const Span& b) {
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && overlaps(a.p, a.bytes, b.p, b.bytes);
  };
  for (int i = 0; i < 4; ++i) {
    if (meet(dz, ins[i]) && !(i == 0 && P.dz == P.z && P.lddz == P.ldz))
      return fail(HESS_EINVAL, "dlogits overlaps %s", ins[i].name);
    for (int j = 0; j < nextra && !extra_in; ++j)
      if (meet(extra[j], ins[i])) return fail(HESS_EINVAL, "%s overlaps %s", extra[j].name, ins[i].name);
  }
  for (int j = 0; j < nextra; ++j) {
    if (meet(dz, extra[j])) return fail(HESS_EINVAL, "dlogits overlaps %s", extra[j].name);
    for (int i = j + 1; i < nextra && !extra_in; ++i)
      if (meet(extra[i], extra[j])) return fail(HESS_EINVAL, "%s overlaps %s", extra[i].name, extra[j].name);
  }
  return HESS_OK;
}

}  // namespace

extern "C" {

int hess_distill_topk(const void* logits, int64_t ldz, int dtype, int64_t n, int64_t vocab, const void* ids, int ids64,
                      int64_t ldi, const void* values, int values_dtype, int64_t ldv, int k, const float* weight,
                      float temperature, float* loss, float* stats, void* dlogits, int64_t lddz, void* work,
                      int64_t work_bytes, hess_stream_t stream) {
  DistillParams P{};
  P.z = logits, P.ldz = ldz, P.n = n, P.vocab = vocab;
  P.ids = ids, P.ids64 = ids64 != 0, P.ldi = ldi;
  P.values = values, P.values_dtype = values_dtype, P.ldv = ldv, P.k = k;
  P.weight = weight, P.temperature = temperature;
  P.loss = loss, P.stats = stats, P.dz = dlogits, P.lddz = lddz;
  if (int rc = check_distill(P, dtype, values_dtype)) return rc;
  if (n == 0) return HESS_OK;
  if (!loss) return fail(HESS_EINVAL, "null loss");
  if (!aligned(loss, 4) || !aligned(stats, 4)) return fail(HESS_EALIGN, "loss or stats not aligned");
  const int64_t need = distill_workspace(n, vocab, dtype);
  if (int rc = check_work(work, work_bytes, need)) return rc;
  const Span extra[3] = {{"loss", loss, n * 4}, {"stats", stats, stats ? n * 8 : 0}, {"the workspace", work, need}};
  if (int rc = check_distill_overlap(P, dtype, values_dtype, extra, 3, false)) return rc;
  P.work = work;
  const hipError_t e = launch_distill(P, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? HESS_OK : hip_fail(e, "distillation loss launch");
}

int hess_distill_topk_backward(const float* dloss, const void* logits, int64_t ldz, int dtype, int64_t n,
                               int64_t vocab, const void* ids, int ids64, int64_t ldi, const void* values,
                               int values_dtype, int64_t ldv, int k, const float* weight, float temperature,
                               const float* stats, void* dlogits, int64_t lddz, hess_stream_t stream) {
  DistillParams P{};
  P.z = logits, P.ldz = ldz, P.n = n, P.vocab = vocab;
  P.ids = ids, P.ids64 = ids64 != 0, P.ldi = ldi;
  P.values = values, P.values_dtype = values_dtype, P.ldv = ldv, P.k = k;
  P.weight = weight, P.temperature = temperature;
  P.dloss = dloss, P.stats = const_cast<float*>(stats), P.dz = dlogits, P.lddz = lddz;
  if (int rc = check_distill(P, dtype, values_dtype)) return rc;
  if (n == 0) return HESS_OK;
  if (!dloss || !stats || !dlogits) return fail(HESS_EINVAL, "null dloss, stats or dlogits");
  if (!aligned(dloss, 4) || !aligned(stats, 4)) return fail(HESS_EALIGN, "dloss or stats not aligned");
  const Span extra[2] = {{"dloss", dloss, n * 4}, {"stats", stats, n * 8}};
  if (int rc = check_distill_overlap(P, dtype, values_dtype, extra, 2, true)) return rc;
  const hipError_t e = launch_distill_backward(P, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? HESS_OK : hip_fail(e, "distillation gradient launch");
}

}  // extern "C"
