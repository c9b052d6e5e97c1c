// The gated feed-forward block, forward, for few tokens (a decoding step).
//
// Bound by the weights' bytes.  A workgroup takes 16 or 32 features of both
// projections and the whole of K: its waves split K, each lane loads 16 bytes
// of one weight row straight into the matrix instruction's operand (no LDS,
// any alignment; 64 consecutive bytes a row and instruction), x comes from L2
// the same way, and the waves' sums meet in LDS before the activation.  One
// launch, no workspace, every weight byte read once.  One bf16 token at 4096 x
// 11264: 32.9 us, 5.6 TB/s, where the last-level cache holds some of the
// weights, and 35.2 us, 5.2 TB/s, where it holds none (a large read reaches
// 5.6); 24 fp16 tokens at 2560 x 9728: 31 us, 3.2 TB/s,
// where x, read again for every 32 features, costs about as much as a third of
// the weights.
//
// Rows of x past n and features past f read the last row instead; their sums
// are not stored.

#include <type_traits>

#include "ffn_device.hpp"
#include "hess_device.hpp"

namespace hess {

namespace {

typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));

template <class T> __device__ __forceinline__ u32x4 load16(const T* p) {
  if constexpr (sizeof(T) == 2) return *reinterpret_cast<const u32x4_at2*>(p);
  else return *reinterpret_cast<const u32x4_at4*>(p);
}
// The first `left` elements at p, zeros after them (left: what is left of a row
// at a lane's chunk, so any number below 64 / sizeof(T), zero and less too).
template <class T> __device__ __forceinline__ u32x4 load_part(const T* p, int left) {
  constexpr int N = 16 / sizeof(T);
  typedef T TN __attribute__((ext_vector_type(16 / sizeof(T))));
  TN t;
#pragma unroll
  for (int e = 0; e < N; ++e) t[e] = e < left ? p[e] : (T)0.0f;
  return __builtin_bit_cast(u32x4, t);
}

// MB blocks of 16 tokens, FB of 16 features, W waves, U pieces in flight.
template <int DT, int MB, int FB, int W, int U> __global__ void __launch_bounds__(64 * W) ffn_few(FfnGemm P) {
  typedef typename Elem<DT>::type T;
  constexpr int kPiece = 16 / sizeof(T), kUnit = 4 * kPiece;
  __shared__ f32x4 part[W][2 * FB * MB][64];
  const int lane = threadIdx.x & 63, r = lane & 15, at = (lane >> 4) * kPiece;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t f0 = (int64_t)blockIdx.x * (16 * FB);
  const T *b[2 * FB], *a[MB];
#pragma unroll
  for (int q = 0; q < FB; ++q) {
    const int64_t feat = min(f0 + 16 * q + r, P.N - 1);
    b[q] = static_cast<const T*>(P.b0) + feat * P.ldb0 + at;
    b[FB + q] = static_cast<const T*>(P.b1) + feat * P.ldb1 + at;
  }
#pragma unroll
  for (int q = 0; q < MB; ++q) a[q] = static_cast<const T*>(P.a) + min((int64_t)(16 * q + r), P.M - 1) * P.lda + at;

  f32x4 acc[2 * FB][MB];
#pragma unroll
  for (int p = 0; p < 2 * FB; ++p)
#pragma unroll
    for (int q = 0; q < MB; ++q) acc[p][q] = f32x4{};
  const int units = (int)(P.K / kUnit);
  const int per = (units + W - 1) / W;
  int u = min(units, wave * per);
  const int u1 = min(units, u + per);
  auto go = [&](auto count) {
    constexpr int C = decltype(count)::value;
    u32x4 vb[C][2 * FB], va[C][MB];
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int p = 0; p < 2 * FB; ++p) vb[i][p] = load16(b[p] + (u + i) * kUnit);
#pragma unroll
      for (int q = 0; q < MB; ++q) va[i][q] = load16(a[q] + (u + i) * kUnit);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads on their way before the first is waited for
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int p = 0; p < 2 * FB; ++p)
#pragma unroll
        for (int q = 0; q < MB; ++q) acc[p][q] = mma16<DT>(vb[i][p], va[i][q], acc[p][q]);
    u += C;
  };
  while (u + U <= u1) go(std::integral_constant<int, U>());
  while (u < u1) go(std::integral_constant<int, 1>());
  if (wave == W - 1 && (int64_t)units * kUnit < P.K) {
    // the last, shorter unit
    const int left = (int)(P.K - (int64_t)units * kUnit) - at;
    u32x4 va[MB];
#pragma unroll
    for (int q = 0; q < MB; ++q) va[q] = load_part(a[q] + (int64_t)units * kUnit, left);
#pragma unroll
    for (int p = 0; p < 2 * FB; ++p) {
      const u32x4 vb = load_part(b[p] + (int64_t)units * kUnit, left);
#pragma unroll
      for (int q = 0; q < MB; ++q) acc[p][q] = mma16<DT>(vb, va[q], acc[p][q]);
    }
  }
#pragma unroll
  for (int p = 0; p < 2 * FB; ++p)
#pragma unroll
    for (int q = 0; q < MB; ++q) part[wave][p * MB + q][lane] = acc[p][q];
  __syncthreads();
  // block (p, q): lane l holds token 16 q + l % 16, features 16 p + 4 (l / 16) .. + 3
  for (int id = threadIdx.x; id < FB * MB * 64; id += 64 * W) {
    const int l = id & 63, blk = id >> 6, p = blk / MB, q = blk % MB;
    f32x4 g = part[0][p * MB + q][l], v = part[0][(FB + p) * MB + q][l];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const f32x4 x = part[w][p * MB + q][l], y = part[w][(FB + p) * MB + q][l];
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] += x[j], v[j] += y[j];
    }
    const int64_t c = f0 + 16 * p + 4 * (l >> 4);
    float gg[4], uu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) gg[j] = g[j], uu[j] = v[j];
    put_fwd<DT>(P, 16 * q + (l & 15), c, gg, uu);
  }
}

template <int DT, int MB, int FB, int U> void launch_few(const FfnGemm& g, hipStream_t stream) {
  ffn_few<DT, MB, FB, 4, U><<<(unsigned)((g.N + 16 * FB - 1) / (16 * FB)), 256, 0, stream>>>(g);
}

// 16 features a workgroup leave no second round of workgroups up to 4096
// features; past that, 32 read x half as often.  32 tokens, 16 against 32
// features, us: bf16 2560 x 4096 15.8 / 19.3, 2560 x 4160 23.1 / 18.6, 2560 x
// 8192 26.2 / 21.2, 4096 x 11264 53.7 / 50.2; float32 2560 x 4096 26.5 / 40.6,
// 2560 x 5632 50.7 / 41.2, 4096 x 11264 120 / 118.  One block of tokens gains
// nothing (16 tokens, 4096 x 11264 40.7 / 45.5), nor do four (64 tokens, 64
// features: 2560 x 8192 33.9 / 44.6, 4096 x 11264 69.9 / 64.7).
template <int DT> void launch_type(const FfnGemm& g, hipStream_t stream) {
  if (g.M <= 16) launch_few<DT, 1, 1, 4>(g, stream);
  else if (g.M <= 32 && g.N > 4096) launch_few<DT, 2, 2, 2>(g, stream);
  else if (g.M <= 32) launch_few<DT, 2, 1, 4>(g, stream);
  else launch_few<DT, 4, 1, 2>(g, stream);
}

}  // namespace

hipError_t launch_ffn_few(const FfnGemm& g, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) launch_type<kInBF16>(g, stream);
  else if (dtype == kInF16) launch_type<kInF16>(g, stream);
  else launch_type<kInF32>(g, stream);
  return hipGetLastError();
}

}  // namespace hess
