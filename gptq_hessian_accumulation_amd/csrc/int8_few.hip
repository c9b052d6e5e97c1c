// The product of few int8 rows, both operands straight from memory into
// v_mfma_i32_16x16x64_i8 (any alignment, no LDS for them, no workspace): a decoding
// step, bound by the weights' bytes.  A workgroup takes all of K, its waves a share
// each, and their sums meet in LDS.  One row: 4096 x 11264 11.0 to 11.6 us with its
// quantization where the weights come from memory (46 MB: 4.1 TB/s), 9.3 to 9.6 where
// the last-level cache has them; 10.9 to 11.2 without it, where a launch that
// quantizes the row first adds 3.2.  24 rows at 2560 x 9728: 8.5 to 9.6 us.
//
// Sums are int32 and exact: |a b| <= 2^14 and K < 2^17.  The output takes the
// sum as a float32 (2^-24), times the two scales, rounded once to its type.

#include <type_traits>

#include "ffn_device.hpp"
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

// 16 FB features and 16 MB tokens a workgroup, whose W waves split K, U pieces of
// 64 codes in flight each.  Rows past the matrix read its last row instead;
// their sums are not stored.
template <int DT, int MB, int FB, int W, int U> __global__ void __launch_bounds__(64 * W) int8_few(Int8Gemm P) {
  typedef typename Elem<DT>::type T;
  __shared__ i32x4 part[W][FB * MB][64];
  const int lane = threadIdx.x & 63, r = lane & 15, at = (lane >> 4) * 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t f0 = (int64_t)blockIdx.x * (16 * FB), t0 = (int64_t)blockIdx.y * (16 * MB);
  const int8_t *b[FB], *a[MB];
#pragma unroll
  for (int q = 0; q < FB; ++q) b[q] = P.b + min(f0 + 16 * q + r, P.N - 1) * P.ldb + at;
#pragma unroll
  for (int q = 0; q < MB; ++q) a[q] = P.a + min(t0 + 16 * q + r, P.M - 1) * P.lda + at;
  i32x4 acc[FB][MB];
#pragma unroll
  for (int p = 0; p < FB; ++p)
#pragma unroll
    for (int q = 0; q < MB; ++q) acc[p][q] = i32x4{};
  const int units = (int)(P.K / 64);
  const int per = (units + W - 1) / W;
  int u = min(units, wave * per);
  const int u1 = min(units, u + per);
  auto go = [&](auto count) {
    constexpr int C = decltype(count)::value;
    u32x4 vb[C][FB], va[C][MB];
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int p = 0; p < FB; ++p) vb[i][p] = *reinterpret_cast<const u32x4_at1*>(b[p] + (u + i) * 64);
#pragma unroll
      for (int q = 0; q < MB; ++q) va[i][q] = *reinterpret_cast<const u32x4_at1*>(a[q] + (u + i) * 64);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads on their way before the first is waited for
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int p = 0; p < FB; ++p)
#pragma unroll
        for (int q = 0; q < MB; ++q) acc[p][q] = mma_i8(vb[i][p], va[i][q], acc[p][q]);
    u += C;
  };
  while (u + U <= u1) go(std::integral_constant<int, U>());
  while (u < u1) go(std::integral_constant<int, 1>());
  if (wave == W - 1 && units * 64 < P.K) {
    const int64_t left = P.K - units * 64 - at;
    u32x4 va[MB];
#pragma unroll
    for (int q = 0; q < MB; ++q) va[q] = load_part(a[q] + units * 64, left);
#pragma unroll
    for (int p = 0; p < FB; ++p) {
      const u32x4 vb = load_part(b[p] + units * 64, left);
#pragma unroll
      for (int q = 0; q < MB; ++q) acc[p][q] = mma_i8(vb, va[q], acc[p][q]);
    }
  }
#pragma unroll
  for (int p = 0; p < FB; ++p)
#pragma unroll
    for (int q = 0; q < MB; ++q) part[wave][p * MB + q][lane] = acc[p][q];
  __syncthreads();
  // block (p, q): lane l holds token 16 q + l % 16, features 16 p + 4 (l / 16) .. + 3
  for (int id = threadIdx.x; id < FB * MB * 64; id += 64 * W) {
    const int l = id & 63, blk = id >> 6, p = blk / MB, q = blk % MB;
    i32x4 s = part[0][blk][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][blk][l];
    const int64_t row = t0 + 16 * q + (l & 15), c = f0 + 16 * p + 4 * (l >> 4);
    if (row >= P.M || c >= P.N) continue;
    const float sa = P.sa[row];
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = c + j < P.N ? scale_sum(s[j], P.sb[c + j], sa) : 0.0f;
    store_n(static_cast<T*>(P.y) + row * P.ldy + c, v, (int)min((int64_t)4, P.N - c));
  }
}

// The workgroup's waves meet with their LDS writes done; loads from memory stay in
// flight (__syncthreads would wait for them).
__device__ __forceinline__ void meet_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// One row of values: every workgroup quantizes it for itself into LDS (one
// launch, and no codes in memory).  The row's loads go first and the first
// weights' right behind them, so that these arrive while the largest magnitude
// is found.  X pieces of 8 values a thread.
template <int DT, int W, int U, int X> __global__ void __launch_bounds__(64 * W) int8_one(Int8Gemm P) {
  typedef typename Elem<DT>::type T;
  constexpr int kLen = X * W * 512;
  __shared__ __attribute__((aligned(16))) char codes[kLen];
  __shared__ i32x4 part[W][64];
  __shared__ uint32_t tops[W];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, at = (lane >> 4) * 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t f0 = (int64_t)blockIdx.x * 16;
  const int K = (int)P.K;
  const T* x = static_cast<const T*>(P.x);
  float v[X][8];
#pragma unroll
  for (int i = 0; i < X; ++i) {
    const int c = (i * 64 * W + tid) * 8;
    if (c < K) load8(x + c, K - c, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
  }
  const int8_t* b = P.b + min(f0 + r, P.N - 1) * P.ldb + at;
  const int units = K / 64, per = (units + W - 1) / W;
  int u = min(units, wave * per);
  const int u1 = min(units, u + per);
  // (pieces past the wave's share read the last whole one of the row again: their
  // products are dropped)
  u32x4 vb[U];
  const int last = max(units - 1, 0);
  if (units > 0)
#pragma unroll
    for (int i = 0; i < U; ++i) vb[i] = *reinterpret_cast<const u32x4_at1*>(b + min(u + i, last) * 64);
  __builtin_amdgcn_sched_barrier(0);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < X; ++i) top = max(top, top_of(v[i]));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if (lane == 0) tops[wave] = top;
  meet_lds();
#pragma unroll
  for (int w = 0; w < W; ++w) top = max(top, tops[w]);
  const RowCode<T> code(top);
#pragma unroll
  for (int i = 0; i < X; ++i) {
    int k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = code(v[i][j]);
    *reinterpret_cast<uint2*>(codes + (i * 64 * W + tid) * 8) =
        uint2{pack4(k[0], k[1], k[2], k[3]), pack4(k[4], k[5], k[6], k[7])};
  }
  meet_lds();
  const char* a = codes + at;
  auto code16 = [&](int unit) { return *reinterpret_cast<const u32x4*>(a + unit * 64); };
  i32x4 acc{};
  if (units > 0) {
    const int mine = u1 - u;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const u32x4 q = i < mine ? code16(u + i) : u32x4{};
      acc = mma_i8(vb[i], q, acc);
    }
    u += min(U, mine);
  }
  auto go = [&](auto count) {
    constexpr int C = decltype(count)::value;
    u32x4 w[C];
#pragma unroll
    for (int i = 0; i < C; ++i) w[i] = *reinterpret_cast<const u32x4_at1*>(b + (u + i) * 64);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < C; ++i) acc = mma_i8(w[i], code16(u + i), acc);
    u += C;
  };
  while (u + 4 <= u1) go(std::integral_constant<int, 4>());
  while (u < u1) go(std::integral_constant<int, 1>());
  if (wave == W - 1 && units * 64 < K) acc = mma_i8(load_part(b + units * 64, K - units * 64 - at), code16(units), acc);
  part[wave][lane] = acc;
  __syncthreads();
  // every lane of a 16-lane row holds the same sums: features 4 (l / 16) .. + 3
  if (tid < 64 && r == 0) {
    i32x4 s = part[0][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][lane];
    const int64_t c = f0 + 4 * (lane >> 4);
    if (c >= P.N) return;
    const float sa = row_scale(top);
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = c + j < P.N ? scale_sum(s[j], P.sb[c + j], sa) : 0.0f;
    store_n(static_cast<T*>(P.y) + c, o, (int)min((int64_t)4, P.N - c));
  }
}

template <int DT, int MB, int FB, int W, int U> void launch_few(const Int8Gemm& g, hipStream_t stream) {
  const unsigned gx = (unsigned)((g.N + 16 * FB - 1) / (16 * FB)), gy = (unsigned)((g.M + 16 * MB - 1) / (16 * MB));
  int8_few<DT, MB, FB, W, U><<<dim3(gx, gy), 64 * W, 0, stream>>>(g);
}

// As few features a workgroup as leave at most one workgroup for each of the 256
// CUs: more read the codes of a less often, fewer fill the card.  Up to 32 tokens
// two blocks of them, up to 64 four, or twice two where that still leaves one
// workgroup a CU.  us, weights in the last-level cache, for blocks of (16 tokens,
// 16 features):
//   24 tokens  4096 x 4096    (2, 1)  8.5  (2, 2) 11.1  (2, 3) 12.1
//              4096 x 6144    (2, 1) 12.3  (2, 2) 11.0  (2, 3) 11.8  (2, 4) 13.6  (20 tokens)
//              2560 x 9728    (2, 1) 12.9  (2, 2) 12.4  (2, 3)  9.6  (2, 4) 10.6
//   32 tokens  4096 x 11264   (2, 1) 20.2  (2, 2) 18.5  (2, 3) 13.5  (2, 4) 15.2
//   64 tokens  2560 x 2560    (2, 1) 10.0  (2, 2)  7.9  (2, 3)  9.7  (4, 3) 11.9
//              4096 x 6144    (2, 2) 18.3  (2, 3) 13.3  (4, 3) 17.3  (4, 4) 18.9
//              4096 x 11264   (2, 3) 22.6  (2, 4) 25.3  (4, 3) 18.0  (4, 4) 19.6
// Up to 16 tokens one block of 16 features is best or within 7% (4096 x 11264:
// 14.4 against 13.4 for (2, 4)).
template <int DT> void launch_type(const Int8Gemm& g, hipStream_t stream) {
  const int64_t wide = 256 * 16;  // features of one block a CU
  if (g.M <= 16) {
    launch_few<DT, 1, 1, 4, 4>(g, stream);
  } else if (g.M <= 32 || 2 * g.N <= 3 * wide) {
    const int64_t blocks = g.M <= 32 ? g.N : 2 * g.N;
    if (blocks <= wide) launch_few<DT, 2, 1, 4, 4>(g, stream);
    else if (blocks <= 2 * wide) launch_few<DT, 2, 2, 4, 4>(g, stream);
    else if (blocks <= 3 * wide) launch_few<DT, 2, 3, 8, 2>(g, stream);
    else launch_few<DT, 2, 4, 8, 2>(g, stream);
  } else if (g.N <= 3 * wide) {
    launch_few<DT, 4, 3, 8, 2>(g, stream);
  } else {
    launch_few<DT, 4, 4, 8, 2>(g, stream);
  }
}

template <int DT, int W, int U, int X> void launch_one(const Int8Gemm& g, hipStream_t stream) {
  int8_one<DT, W, U, X><<<(unsigned)((g.N + 15) / 16), 64 * W, 0, stream>>>(g);
}

// us for (waves, units in flight): long rows whose workgroups leave CUs free split
// K over more waves: 4096 x 4096 (16, 4) 6.2, (8, 4) 7.5, (4, 4) 7.6; 8192 x 2816
// (16, 4) 8.0, (8, 4) 9.3; but 1001 x 2731 (16, 4) 8.6, (4, 4) 6.2.  Otherwise four
// waves, with eight units in flight for shares of more than ten: 4096 x 11264
// (4, 8) 11.0, (4, 4) 11.4; 2560 x 9728 (4, 8) 9.0, (4, 4) 8.6.
template <int DT> void launch_one_type(const Int8Gemm& g, hipStream_t stream) {
  if (g.N <= 4096 && g.K > 2048) launch_one<DT, 16, 4, 1>(g, stream);
  else if (g.K > 4096) launch_one<DT, 8, 4, 2>(g, stream);
  else if (g.K / 64 > 4 * 10) launch_one<DT, 4, 8, 2>(g, stream);
  else launch_one<DT, 4, 4, 2>(g, stream);
}

}  // namespace

hipError_t launch_int8_few(const Int8Gemm& g, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) launch_type<kInBF16>(g, stream);
  else if (dtype == kInF16) launch_type<kInF16>(g, stream);
  else launch_type<kInF32>(g, stream);
  return hipGetLastError();
}

hipError_t launch_int8_one(const Int8Gemm& g, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) launch_one_type<kInBF16>(g, stream);
  else if (dtype == kInF16) launch_one_type<kInF16>(g, stream);
  else launch_one_type<kInF32>(g, stream);
  return hipGetLastError();
}

}  // namespace hess
