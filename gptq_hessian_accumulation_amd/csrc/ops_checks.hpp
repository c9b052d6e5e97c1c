// Argument checks and product launches shared by the C entry points of the
// operators on activations (feed-forward block, loss, 8-bit integers).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/hess.h"
#include "ffn_internal.hpp"
#include "hess_internal.hpp"

namespace hess {

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxWidth = (int64_t)1 << 17;
constexpr int64_t kMaxStride = (int64_t)1 << 20;

inline bool dtype_ok(int t) { return t == HESS_BF16 || t == HESS_F32 || t == HESS_F16; }
inline int64_t elem_bytes(int t) { return t == HESS_F32 ? 4 : 2; }
inline int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)a == 0; }

// A matrix argument: rows x cols at p with row stride ld elements.
struct Mat {
  const char* name;
  const void* p;
  int64_t ld, rows, cols;
  int64_t own = 0;  // bytes of an element, where it is not the call's type
  int64_t bytes(int64_t es) const { return rows > 0 ? ((rows - 1) * ld + cols) * (own ? own : es) : 0; }
};

inline int check_mat(const Mat& m, int64_t es) {
  if (!m.p) return fail(HESS_EINVAL, "null %s", m.name);
  if (m.ld < m.cols || m.ld > kMaxStride)
    return fail(HESS_EINVAL, "row stride %lld of %s outside [%lld, %lld]", (long long)m.ld, m.name, (long long)m.cols,
                (long long)kMaxStride);
  if (!aligned(m.p, es)) return fail(HESS_EALIGN, "%s not aligned to its element size", m.name);
  return HESS_OK;
}

// No output may meet another output or an input.
inline int check_outputs(const Mat* outs, int no, const Mat* ins, int ni, int64_t es, const void* work, int64_t wbytes) {
  for (int a = 0; a < no; ++a) {
    if (!outs[a].p) continue;
    for (int b = 0; b < ni; ++b)
      if (ins[b].p && overlaps(outs[a].p, outs[a].bytes(es), ins[b].p, ins[b].bytes(es)))
        return fail(HESS_EINVAL, "%s overlaps %s", outs[a].name, ins[b].name);
    for (int b = a + 1; b < no; ++b)
      if (outs[b].p && overlaps(outs[a].p, outs[a].bytes(es), outs[b].p, outs[b].bytes(es)))
        return fail(HESS_EINVAL, "%s overlaps %s", outs[a].name, outs[b].name);
    if (wbytes > 0 && overlaps(outs[a].p, outs[a].bytes(es), work, wbytes))
      return fail(HESS_EINVAL, "%s overlaps the workspace", outs[a].name);
  }
  for (int b = 0; b < ni; ++b)
    if (wbytes > 0 && ins[b].p && overlaps(ins[b].p, ins[b].bytes(es), work, wbytes))
      return fail(HESS_EINVAL, "%s overlaps the workspace", ins[b].name);
  return HESS_OK;
}

inline int check_ffn_sizes(int64_t n, int64_t d, int64_t f, int dtype) {
  if (!dtype_ok(dtype)) return fail(HESS_EINVAL, "unknown dtype %d", dtype);
  if (n < 0 || n > kMaxRows) return fail(HESS_EINVAL, "n = %lld outside [0, 2^24]", (long long)n);
  if (d < 1 || d > kMaxWidth || f < 1 || f > kMaxWidth)
    return fail(HESS_EINVAL, "d = %lld, f = %lld outside [1, 2^17]", (long long)d, (long long)f);
  return HESS_OK;
}

inline int check_work(const void* work, int64_t have, int64_t need) {
  if (need == 0) return HESS_OK;
  if (!work) return fail(HESS_EINVAL, "null workspace");
  if (!aligned(work, 16)) return fail(HESS_EALIGN, "workspace not 16-byte aligned");
  if (have < need)
    return fail(HESS_EINVAL, "workspace of %lld bytes, %lld needed", (long long)have, (long long)need);
  return HESS_OK;
}

inline FfnGemm shape(int64_t M, int64_t N, int64_t K) {
  FfnGemm g{};
  g.M = M;
  g.N = N;
  g.K = K;
  return g;
}

// Bytes of partial tiles a product needs.
inline int64_t slot_bytes(FfnGemm g, int mode, int dtype) {
  const int edge = ffn_schedule(g, mode, dtype);
  return (int64_t)(g.ntiles - g.full) * g.parts * edge * edge * 4;
}

// One product by tiles, its partial sums in `room` bytes at g.ws.  (The schedule
// is the one the room was taken for, unless hess_set_ffn_schedule ran between.)
inline int run_product(FfnGemm& g, int mode, int dtype, int64_t room, hipStream_t s, const char* what) {
  const int edge = ffn_schedule(g, mode, dtype);
  if ((int64_t)(g.ntiles - g.full) * g.parts * edge * edge * 4 > room)
    return fail(HESS_EINVAL, "schedule changed during the call");
  const hipError_t e = launch_ffn_gemm(g, mode, edge, dtype, s);
  return e == hipSuccess ? HESS_OK : hip_fail(e, what);
}

}  // namespace hess
