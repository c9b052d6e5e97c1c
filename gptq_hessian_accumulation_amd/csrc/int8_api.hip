// C ABI of the 8-bit integer operators (declared in include/hess.h): argument
// checks, workspace layout, dispatch.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/hess.h"
#include "ffn_internal.hpp"
#include "hess_internal.hpp"
#include "int8_internal.hpp"
#include "ops_checks.hpp"

using namespace hess;

namespace {

int check_codes(const char* name, const void* p, int64_t ld, int64_t cols) { return check_mat({name, p, ld, 0, cols}, 1); }

int check_scale(const char* name, const void* p) {
  if (!p) return fail(HESS_EINVAL, "null %s", name);
  if (!aligned(p, 4)) return fail(HESS_EALIGN, "%s not float-aligned", name);
  return HESS_OK;
}

// Checks of a set of rows held as codes; bytes of its scales.
int check_rows(int64_t n, int64_t d, int block, int dtype, const void* x, int64_t ldx, const void* codes, int64_t ldc,
               const void* scale, const char* values) {
  if (int rc = check_ffn_sizes(n, d, 1, dtype)) return rc;
  if (block != 0 && block != 32) return fail(HESS_EINVAL, "block %d is neither 0 nor 32", block);
  if (n == 0) return HESS_OK;
  if (int rc = check_mat({values, x, ldx, n, d}, elem_bytes(dtype))) return rc;
  if (int rc = check_codes("codes", codes, ldc, d)) return rc;
  if (block == 0) return check_scale("scale", scale);
  return scale ? HESS_OK : fail(HESS_EINVAL, "null scale");
}
int64_t scale_bytes(int64_t n, int64_t d, int block) { return block == 0 ? 4 * n : n * ((d + 31) / 32); }

int check_product(int64_t n, int64_t d, int64_t f, int dtype) {
  if (int rc = check_ffn_sizes(n, d, f, dtype)) return rc;
  // (int32 sums of products of up to 2^14)
  return d < kMaxWidth ? HESS_OK : fail(HESS_EINVAL, "d = %lld: sums of 2^17 products pass 32 bits", (long long)d);
}

// Codes as the product's tiles take them: rows of a multiple of 16 bytes.
int64_t code_stride(int64_t d) { return up(d, 16); }

Int8Gemm product(int64_t n, int64_t d, int64_t f) {
  Int8Gemm g{};
  g.M = n, g.N = f, g.K = d;
  return g;
}

// Workspace of a product: a, b with padded rows | partial tiles; before them for
// a linear layer the codes and scales of x.  Room for copied rows is there
// where d is no multiple of 16: of a only if it is copied (a linear layer's codes
// of x have padded rows as they are), of b in any case, since sizes do not tell
// whether its rows can be read where they are.
struct ProductWork {
  int64_t a, b, slots, total;
};
int64_t int8_slots(Int8Gemm g) {
  const int edge = int8_schedule(g);
  return (int64_t)(g.ntiles - g.full) * g.parts * edge * edge * 4;
}
ProductWork product_work(int64_t n, int64_t d, int64_t f, bool copy_a) {
  ProductWork w{};
  if (int8_few(n, d)) return w;
  const bool copy = d % 16 != 0;
  w.b = copy && copy_a ? up(n * code_stride(d), 256) : 0;
  w.slots = w.b + (copy ? up(f * code_stride(d), 256) : 0);
  w.total = w.slots + int8_slots(product(n, d, f));
  return w;
}
struct LinearWork {
  int64_t scale, product, total;
};
LinearWork linear_work(int64_t n, int64_t d, int64_t f, bool given) {
  LinearWork w{};
  if (n == 1 && d <= kInt8One) return w;  // quantized by the product itself, or into x_codes
  if (!given) {
    w.scale = up(n * code_stride(d), 256);
    w.product = w.scale + up(4 * n, 256);
  }
  w.total = w.product + product_work(n, d, f, false).total;
  return w;
}

bool rows_of_16(const void* p, int64_t ld, int64_t rows) { return aligned(p, 16) && (rows <= 1 || ld % 16 == 0); }

// Puts codes with padded rows in the workspace in place of m's.
void copied(PackCodes& p, const int8_t*& m, int64_t& ld, int64_t rows, int64_t d, char* dst) {
  p.cols = d, p.pad = code_stride(d);
  p.src[p.count] = m, p.ld[p.count] = ld, p.rows[p.count] = rows;
  p.dst[p.count++] = reinterpret_cast<int8_t*>(dst);
  m = reinterpret_cast<int8_t*>(dst), ld = p.pad;
}
// Whether the tiles cannot take b's rows where they are (d no multiple of 16).
bool untidy(const Int8Gemm& g) {
  return !int8_few(g.M, g.K) && g.K % 16 != 0 && !(rows_of_16(g.b, g.ldb, g.N) && g.ldb >= code_stride(g.K));
}
// The codes of b that a product reads: tiles that take its rows where they are
// read whole 16-byte pieces, those behind the last row's codes among them.
Mat codes_read(const char* name, const Int8Gemm& g) {
  return {name, g.b, g.ldb, g.N, int8_few(g.M, g.K) || untidy(g) ? g.K : code_stride(g.K), 1};
}

// One product; its operands are as the kernel for its size takes them.
int run_int8(Int8Gemm g, char* work, const ProductWork& room, int dtype, hipStream_t s) {
  if (int8_few(g.M, g.K)) {
    const hipError_t e = launch_int8_few(g, dtype, s);
    return e == hipSuccess ? HESS_OK : hip_fail(e, "8-bit product launch");
  }
  const int edge = int8_schedule(g);
  if ((int64_t)(g.ntiles - g.full) * g.parts * edge * edge * 4 > room.total - room.slots)
    return fail(HESS_EINVAL, "schedule changed during the call");
  g.ws = reinterpret_cast<int*>(work + room.slots);
  const hipError_t e = launch_int8_tile(g, edge, dtype, s);
  return e == hipSuccess ? HESS_OK : hip_fail(e, "8-bit product launch");
}

// Backward workspace: dy with padded rows | weights | x, both in the
// gradients' type | partial tiles.
struct LinearGradWork {
  int64_t w, x, slots, total;
};
int64_t piece(int dtype) { return 16 / elem_bytes(dtype); }
LinearGradWork grad_work(int64_t n, int64_t d, int64_t f, int dtype, bool want_x, bool want_w) {
  const int64_t es = elem_bytes(dtype), dp = up(d, piece(dtype)), fp = up(f, piece(dtype));
  LinearGradWork r{};
  r.w = f == fp ? 0 : up(n * fp * es, 256);
  r.x = r.w + (want_x ? up(f * dp * es, 256) : 0);
  r.slots = r.x + (want_w ? up(n * dp * es, 256) : 0);
  FfnGemm gx = shape(n, d, f), gw = shape(fp, d, n);
  gx.segs = 1;
  r.total = r.slots + std::max(want_x ? slot_bytes(gx, kFfnDx, dtype) : 0, want_w ? slot_bytes(gw, kFfnDw, dtype) : 0);
  return r;
}

}  // namespace

extern "C" {

int hess_int8_quantize(const void* x, int64_t ldx, int dtype, int64_t n, int64_t d, int block, int8_t* codes,
                       int64_t ldc, int64_t pad, void* scale, hess_stream_t stream) {
  if (int rc = check_rows(n, d, block, dtype, x, ldx, codes, ldc, scale, "x")) return rc;
  if (n == 0) return HESS_OK;
  if (pad < d || pad > ldc) return fail(HESS_EINVAL, "pad = %lld outside [d, ldc]", (long long)pad);
  const Mat in{"x", x, ldx, n, d};
  const Mat outs[2] = {{"codes", codes, ldc, n, pad, 1}, {"scale", scale, scale_bytes(n, d, block), 1, scale_bytes(n, d, block), 1}};
  if (int rc = check_outputs(outs, 2, &in, 1, elem_bytes(dtype), nullptr, 0)) return rc;
  const Int8Rows r{x, ldx, codes, ldc, scale, n, d, pad};
  const hipError_t e = launch_int8_quantize(r, block, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? HESS_OK : hip_fail(e, "quantize launch");
}

int hess_int8_dequantize(const int8_t* codes, int64_t ldc, const void* scale, int64_t n, int64_t d, int block,
                         void* x, int64_t ldx, int dtype, hess_stream_t stream) {
  if (int rc = check_rows(n, d, block, dtype, x, ldx, codes, ldc, scale, "x")) return rc;
  if (n == 0) return HESS_OK;
  const Mat out{"x", x, ldx, n, d};
  const Mat ins[2] = {{"codes", codes, ldc, n, d, 1}, {"scale", scale, scale_bytes(n, d, block), 1, scale_bytes(n, d, block), 1}};
  if (int rc = check_outputs(&out, 1, ins, 2, elem_bytes(dtype), nullptr, 0)) return rc;
  const Int8Rows r{x, ldx, const_cast<int8_t*>(codes), ldc, const_cast<void*>(scale), n, d, d};
  const hipError_t e = launch_int8_dequantize(r, block, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? HESS_OK : hip_fail(e, "dequantize launch");
}

int64_t hess_int8_matmul_workspace(int64_t n, int64_t d, int64_t f) {
  if (check_product(n, d, f, HESS_BF16) != HESS_OK) return -1;
  return n == 0 ? 0 : product_work(n, d, f, true).total;
}

int hess_int8_matmul(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* b, int64_t ldb,
                     const float* b_scale, int64_t n, int64_t d, int64_t f, void* y, int64_t ldy, int dtype, void* work,
                     int64_t work_bytes, hess_stream_t stream) {
  if (int rc = check_product(n, d, f, dtype)) return rc;
  if (n == 0) return HESS_OK;
  if (int rc = check_codes("a", a, lda, d)) return rc;
  if (int rc = check_codes("b", b, ldb, d)) return rc;
  if (int rc = check_scale("a_scale", a_scale)) return rc;
  if (int rc = check_scale("b_scale", b_scale)) return rc;
  const int64_t es = elem_bytes(dtype);
  const Mat out{"y", y, ldy, n, f};
  if (int rc = check_mat(out, es)) return rc;
  Int8Gemm g = product(n, d, f);
  g.a = a, g.lda = lda, g.sa = a_scale;
  g.b = b, g.ldb = ldb, g.sb = b_scale;
  g.y = y, g.ldy = ldy;
  const Mat ins[4] = {{"a", a, lda, n, d, 1}, codes_read("b", g), {"a_scale", a_scale, n, 1, n, 4}, {"b_scale", b_scale, f, 1, f, 4}};
  const ProductWork room = product_work(n, d, f, true);
  if (int rc = check_work(work, work_bytes, room.total)) return rc;
  if (int rc = check_outputs(&out, 1, ins, 4, es, work, room.total)) return rc;
  char* base = static_cast<char*>(work);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!int8_few(n, d) && d % 16 == 0 && (!rows_of_16(a, lda, n) || !rows_of_16(b, ldb, f)))
    return fail(HESS_EALIGN, "rows of codes must be 16-byte aligned where d is a multiple of 16");
  if (!int8_few(n, d) && d % 16 != 0) {
    PackCodes p{};
    const bool copy_b = untidy(g);
    copied(p, g.a, g.lda, n, d, base + room.a);
    if (copy_b) copied(p, g.b, g.ldb, f, d, base + room.b);
    const hipError_t e = launch_pack_codes(p, s);
    if (e != hipSuccess) return hip_fail(e, "operand copy launch");
  }
  return run_int8(g, base, room, dtype, s);
}

int64_t hess_int8_linear_workspace(int64_t n, int64_t d, int64_t f, int dtype, int pass) {
  if (check_product(n, d, f, dtype) != HESS_OK) return -1;
  if (pass < 0 || pass > 4) {
    fail(HESS_EINVAL, "pass %d outside [0, 4]", pass);
    return -1;
  }
  if (n == 0) return 0;
  return pass == 0 || pass == 4 ? linear_work(n, d, f, pass == 4).total : grad_work(n, d, f, dtype, pass & 1, pass & 2).total;
}

int hess_int8_linear_forward(const void* x, int64_t ldx, int dtype, const int8_t* w, int64_t ldw, const float* w_scale,
                             int64_t n, int64_t d, int64_t f, void* y, int64_t ldy, int8_t* x_codes, int64_t ldc,
                             float* x_scale, void* work, int64_t work_bytes, hess_stream_t stream) {
  if (int rc = check_product(n, d, f, dtype)) return rc;
  if (!x_codes != !x_scale) return fail(HESS_EINVAL, "x_codes and x_scale: both or neither");
  if (n == 0) return HESS_OK;
  const int64_t es = elem_bytes(dtype);
  Int8Gemm g = product(n, d, f);
  g.b = w, g.ldb = ldw, g.sb = w_scale;
  g.y = y, g.ldy = ldy;
  const Mat ins[3] = {{"x", x, ldx, n, d}, codes_read("w", g), {"w_scale", w_scale, f, 1, f, 4}};
  if (int rc = check_mat(ins[0], es)) return rc;
  if (int rc = check_codes("w", w, ldw, d)) return rc;
  if (int rc = check_scale("w_scale", w_scale)) return rc;
  const Mat outs[3] = {{"y", y, ldy, n, f}, {"x_codes", x_codes, ldc, n, code_stride(d), 1}, {"x_scale", x_scale, n, 1, n, 4}};
  if (int rc = check_mat(outs[0], es)) return rc;
  if (x_codes) {
    if (int rc = check_codes("x_codes", x_codes, ldc, code_stride(d))) return rc;
    if (!aligned(x_codes, 16) || ldc % 16 != 0) return fail(HESS_EALIGN, "rows of x_codes not 16-byte aligned");
    if (int rc = check_scale("x_scale", x_scale)) return rc;
  }
  const LinearWork room = linear_work(n, d, f, x_codes != nullptr);
  if (int rc = check_work(work, work_bytes, room.total)) return rc;
  if (int rc = check_outputs(outs, 3, ins, 3, es, work, room.total)) return rc;
  if (!int8_few(n, d) && d % 16 == 0 && !rows_of_16(w, ldw, f))
    return fail(HESS_EALIGN, "rows of w must be 16-byte aligned where d is a multiple of 16");
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* base = static_cast<char*>(work);
  if (n == 1 && d <= kInt8One && !x_codes) {
    g.x = x, g.ldx = ldx;
    const hipError_t e = launch_int8_one(g, dtype, s);
    return e == hipSuccess ? HESS_OK : hip_fail(e, "8-bit product launch");
  }
  if (!x_codes) {
    x_codes = reinterpret_cast<int8_t*>(base);
    ldc = code_stride(d);
    x_scale = reinterpret_cast<float*>(base + room.scale);
  }
  const ProductWork rest = product_work(n, d, f, false);
  const Int8Rows r{x, ldx, x_codes, ldc, x_scale, n, d, code_stride(d)};
  PackCodes p{};
  if (untidy(g)) copied(p, g.b, g.ldb, f, d, base + room.product + rest.b);
  const hipError_t e = launch_int8_quantize_and_pack(r, dtype, p, s);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  g.a = x_codes, g.lda = ldc, g.sa = x_scale;
  return run_int8(g, base + room.product, rest, dtype, s);
}

int hess_int8_linear_backward(const void* dy, int64_t lddy, int dtype, const int8_t* x_codes, int64_t ldc,
                              const float* x_scale, const int8_t* w, int64_t ldw, const float* w_scale, int64_t n,
                              int64_t d, int64_t f, void* dx, int64_t lddx, void* dw, int64_t lddw, void* work,
                              int64_t work_bytes, hess_stream_t stream) {
  if (int rc = check_product(n, d, f, dtype)) return rc;
  const int64_t es = elem_bytes(dtype), dp = up(d, piece(dtype)), fp = up(f, piece(dtype));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Mat outs[2] = {{"dx", dx, lddx, n, d}, {"dw", dw, lddw, f, d}};
  for (const Mat& m : outs)
    if (m.p && m.rows > 0)
      if (int rc = check_mat(m, es)) return rc;
  if (n == 0) {
    if (!dw) return HESS_OK;
    const hipError_t e = launch_zero_rows(dw, lddw, f, d, (int)es, s);
    return e == hipSuccess ? HESS_OK : hip_fail(e, "gradient clear launch");
  }
  if (!dx && !dw) return HESS_OK;
  const Mat ins[5] = {{"dy", dy, lddy, n, f},
                      {"x_codes", dw ? x_codes : nullptr, ldc, n, d, 1},
                      {"x_scale", dw ? x_scale : nullptr, n, 1, n, 4},
                      {"w", dx ? w : nullptr, ldw, f, d, 1},
                      {"w_scale", dx ? w_scale : nullptr, f, 1, f, 4}};
  if (int rc = check_mat(ins[0], es)) return rc;
  if (f == fp && (!aligned(dy, 16) || (n > 1 && lddy % piece(dtype) != 0)))
    return fail(HESS_EALIGN, "rows of dy must be 16-byte aligned where a row is a multiple of 16 bytes");
  if (dw) {
    if (int rc = check_codes("x_codes", x_codes, ldc, d)) return rc;
    if (int rc = check_scale("x_scale", x_scale)) return rc;
  }
  if (dx) {
    if (int rc = check_codes("w", w, ldw, d)) return rc;
    if (int rc = check_scale("w_scale", w_scale)) return rc;
  }
  const LinearGradWork room = grad_work(n, d, f, dtype, dx != nullptr, dw != nullptr);
  if (int rc = check_work(work, work_bytes, room.total)) return rc;
  if (int rc = check_outputs(outs, 2, ins, 5, es, work, room.total)) return rc;

  char* base = static_cast<char*>(work);
  GradOperands o{};
  if (dx) o.rows[0] = {base + room.w, dp, const_cast<int8_t*>(w), ldw, const_cast<float*>(w_scale), f, d, dp};
  if (dw) o.rows[1] = {base + room.x, dp, const_cast<int8_t*>(x_codes), ldc, const_cast<float*>(x_scale), n, d, dp};
  if (f != fp) {
    o.src = dy, o.dst = base, o.ld = lddy, o.n = n, o.cols = f, o.pad = fp;
    dy = base;
    lddy = fp;
  }
  const hipError_t e = launch_int8_grad_operands(o, dtype, s);
  if (e != hipSuccess) return hip_fail(e, "operand launch");
  float* slots = reinterpret_cast<float*>(base + room.slots);
  if (dx) {
    FfnGemm g = shape(n, d, f);
    g.segs = 1;
    g.a = dy, g.lda = lddy;
    g.b0 = base + room.w, g.ldb0 = dp;
    g.b1 = g.b0, g.ldb1 = dp;
    g.o0 = dx, g.ldo0 = lddx;
    g.ws = slots;
    g.f = f, g.fp = fp;
    if (int rc = run_product(g, kFfnDx, dtype, room.total - room.slots, s, "input gradient launch")) return rc;
  }
  if (dw) {
    FfnGemm g = shape(fp, d, n);
    g.a = dy, g.lda = lddy;
    g.b0 = base + room.x, g.ldb0 = dp;
    g.o0 = dw, g.ldo0 = lddw;
    g.ws = slots;
    g.f = f, g.fp = fp;
    if (int rc = run_product(g, kFfnDw, dtype, room.total - room.slots, s, "weight gradient launch")) return rc;
  }
  return HESS_OK;
}

}  // extern "C"
