// The product of int8 rows, both operands straight from memory into
// v_mfma_i32_16x16x64_i8 (any alignment, no LDS for them, no workspace).
//
// Sums are int32 and exact: |a b| <= 2^14 and K < 2^17.  The output takes the
// sum as a float32 (2^-24), times the two scales, rounded once to its type.

#include <type_traits>

#include "int8_device.hpp"
#include "int8_internal.hpp"

namespace hess {

namespace {

__device__ __forceinline__ i32x4 mma_i8(const u32x4& a, const u32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// The first `left` of 16 codes at p, zeros after them.
__device__ __forceinline__ u32x4 load_part(const int8_t* p, int64_t left) {
  u32x4 o{};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < left) o[e / 4] |= (uint32_t)(uint8_t)p[e] << (8 * (e % 4));
  return o;
}

// 16 features and 16 MB tokens a workgroup, whose W waves split K, U pieces of
// 64 codes in flight each.  Rows past the matrix read its last row instead;
// their sums are not stored.
template <int DT, int MB, int W, int U> __global__ void __launch_bounds__(64 * W) int8_few(Int8Gemm P) {
  typedef typename Elem<DT>::type T;
  __shared__ i32x4 part[W][MB][64];
  const int lane = threadIdx.x & 63, r = lane & 15, at = (lane >> 4) * 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t f0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (16 * MB);
  const int8_t* b = P.b + min(f0 + r, P.N - 1) * P.ldb + at;
  const int8_t* a[MB];
#pragma unroll
  for (int q = 0; q < MB; ++q) a[q] = P.a + min(t0 + 16 * q + r, P.M - 1) * P.lda + at;
  i32x4 acc[MB];
#pragma unroll
  for (int q = 0; q < MB; ++q) acc[q] = i32x4{};
  const int units = (int)(P.K / 64);
  const int per = (units + W - 1) / W;
  int u = min(units, wave * per);
  const int u1 = min(units, u + per);
  auto go = [&](auto count) {
    constexpr int C = decltype(count)::value;
    u32x4 vb[C], va[C][MB];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      vb[i] = *reinterpret_cast<const u32x4_at1*>(b + (int64_t)(u + i) * 64);
#pragma unroll
      for (int q = 0; q < MB; ++q) va[i][q] = *reinterpret_cast<const u32x4_at1*>(a[q] + (int64_t)(u + i) * 64);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads on their way before the first is waited for
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int q = 0; q < MB; ++q) acc[q] = mma_i8(vb[i], va[i][q], acc[q]);
    u += C;
  };
  while (u + U <= u1) go(std::integral_constant<int, U>());
  while (u < u1) go(std::integral_constant<int, 1>());
  if (wave == W - 1 && (int64_t)units * 64 < P.K) {
    const int64_t left = P.K - (int64_t)units * 64 - at;
    const u32x4 vb = load_part(b + (int64_t)units * 64, left);
#pragma unroll
    for (int q = 0; q < MB; ++q) acc[q] = mma_i8(vb, load_part(a[q] + (int64_t)units * 64, left), acc[q]);
  }
#pragma unroll
  for (int q = 0; q < MB; ++q) part[wave][q][lane] = acc[q];
  __syncthreads();
  // block q: lane l holds token 16 q + l % 16, features 4 (l / 16) .. + 3
  for (int id = threadIdx.x; id < MB * 64; id += 64 * W) {
    const int l = id & 63, q = id >> 6;
    i32x4 s = part[0][q][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][q][l];
    const int64_t row = t0 + 16 * q + (l & 15), c = f0 + 4 * (l >> 4);
    if (row >= P.M) continue;
    const float sa = P.sa[row];
    T* y = static_cast<T*>(P.y) + row * P.ldy + c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < P.N) y[j] = from_f32<T>(scale_sum(s[j], P.sb[c + j], sa));
  }
}

template <int DT> void launch_type(const Int8Gemm& g, hipStream_t stream) {
  // (a grid has at most 65,535 rows)
  for (int64_t r0 = 0; r0 < g.M; r0 += 32768 * 16) {
    Int8Gemm p = g;
    p.M = g.M - r0 < 32768 * 16 ? g.M - r0 : 32768 * 16;
    p.a = g.a + r0 * g.lda;
    p.sa = g.sa + r0;
    p.y = static_cast<char*>(g.y) + r0 * g.ldy * Elem<DT>::size;
    int8_few<DT, 1, 4, 4><<<dim3((unsigned)((p.N + 15) / 16), (unsigned)((p.M + 15) / 16)), 256, 0, stream>>>(p);
  }
}

}  // namespace

hipError_t launch_int8_few(const Int8Gemm& g, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) launch_type<kInBF16>(g, stream);
  else if (dtype == kInF16) launch_type<kInF16>(g, stream);
  else launch_type<kInF32>(g, stream);
  return hipGetLastError();
}

}  // namespace hess
