// Device code shared by the products of the gated feed-forward block: the
// activations, the outputs' stores, and the order of the tiles.
#pragma once

#include "elem.hpp"
#include "ffn_internal.hpp"
#include "hess_device.hpp"
#include "../../include/hess.h"

namespace hess {

// act(g) and act'(g) in float32.  tanh goes through the sigmoid
// (0.5 (1 + tanh s) = sigmoid(2 s)) and the sigmoid through exp(-|v|), so the
// left tails keep their relative accuracy down to the smallest numbers.
// Exact: float32 outputs, where the exponential's last bits count; otherwise
// the hardware exponential of a rounded argument.
template <bool Exact> __device__ __forceinline__ float sigmoidf(float v) {
  const float e = Exact ? expf(-fabsf(v)) : __expf(-fabsf(v));
  const float top = v >= 0.0f ? 1.0f : e;
  if constexpr (Exact) return top / (1.0f + e);
  else return top * __builtin_amdgcn_rcpf(1.0f + e);
}

// 0.5 erfcx(z) / t by powers of t, and what the float constant -0.72134751
// leaves of -log2(e) / 2.
constexpr float kErfcx[9] = {0.0846030036f, 0.0852006927f, 0.075317605f,  0.102853764f, -0.0361971718f,
                             0.257281024f,  -0.241219981f, 0.2353499f, -0.0631888159f};
constexpr float kLog2eHalfLow = -9.62981495e-09f;

// The normal distribution function, and exp(-g^2 / 2).  For g <= 0 it is
// exp(-z^2) erfcx(z) / 2 with z = |g| / sqrt 2, and erfcx(z) a polynomial in
// t = 1 / (1 + 0.3 z) times t, fitted here for the least relative error on
// 0 <= z <= 14 (4e-8).  The exponent -g^2 log2(e) / 2 is formed in two parts,
// so that the far tail is as accurate as the middle.  In float32 g times it is
// off by up to 5.4e-7 (measured at 6 million g in [-13, 13]: 4.2e-7 below -3,
// 5.0e-7 to -0.1, 5.4e-7 around 0, 1.3e-7 above 1).  |g| past 20 counts as 20,
// where the tail is below float32's range.
__device__ __forceinline__ float normal_cdf(float g, float& e) {
  const float s = fminf(fabsf(g), 20.0f);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f * 0.70710678118654752f, s, 1.0f));
  const float hi = s * s, x = hi * -0.72134751f;
  float lo = fmaf(hi, -0.72134751f, -x);
  lo = fmaf(hi, kLog2eHalfLow, lo);
  lo = fmaf(fmaf(s, s, -hi), -0.72134751f, lo);
  const float p = __builtin_amdgcn_exp2f(x);
  e = fmaf(p, lo * 0.69314718f, p);
  float q = kErfcx[8];
#pragma unroll
  for (int k = 7; k >= 0; --k) q = fmaf(q, t, kErfcx[k]);
  const float tail = e * t * q;
  return g > 0.0f ? 1.0f - tail : tail;
}

template <bool Exact> __device__ __forceinline__ float act_value(float g, int act) {
  if (act == HESS_SILU) return g * sigmoidf<Exact>(g);
  if (act == HESS_GELU) {
    float e;
    return g * normal_cdf(g, e);
  }
  return g * sigmoidf<Exact>(1.5957691216057308f * (g + 0.044715f * g * g * g));
}

template <bool Exact> __device__ __forceinline__ void act_both(float g, int act, float& a, float& da) {
  if (act == HESS_SILU) {
    const float s = sigmoidf<Exact>(g);
    a = g * s;
    da = s * (1.0f + g * (1.0f - s));
  } else if (act == HESS_GELU) {
    float e;
    const float c = normal_cdf(g, e);
    a = g * c;
    da = fmaf(g * 0.39894228040143268f, e, c);
  } else {
    const float s = sigmoidf<Exact>(1.5957691216057308f * (g + 0.044715f * g * g * g));
    a = g * s;
    // (the cap keeps 0 times infinity out of the far ends)
    da = s + g * s * (1.0f - s) * 1.5957691216057308f * fminf(1.0f + 0.134145f * g * g, 1e30f);
  }
}

// acc += A B over 64 bytes of K, of which each 16-lane row holds a 16-byte
// chunk (in float32 each instruction takes one value of every chunk).
template <int DT> __device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, f32x4 acc) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  if constexpr (DT == kInBF16) {
    return mfma16x16x32(a, b, acc);
  } else if constexpr (DT == kInF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0,
                                                  0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[j]), __uint_as_float(b[j]), acc, 0, 0, 0);
    return acc;
  }
}

// N consecutive outputs of one row (one store of any alignment); `left` of
// them lie inside the matrix.
template <class T, int N> __device__ __forceinline__ void store_n(T* p, const float (&v)[N], int left) {
  typedef T TN __attribute__((ext_vector_type(N)));
  typedef TN TU __attribute__((aligned(sizeof(T))));
  if (left >= N) {
    TN o;
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = from_f32<T>(v[j]);
    *reinterpret_cast<TU*>(p) = o;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < left) p[j] = from_f32<T>(v[j]);
  }
}

// Outputs of row r, columns c .. c + N - 1 (dx, dw).
template <int DT, int Mode, int N>
__device__ __forceinline__ void put(const FfnGemm& P, int64_t r, int64_t c, const float (&v)[N]) {
  typedef typename Elem<DT>::type T;
  if (r >= P.M || c >= P.N) return;
  const int left = (int)min((int64_t)N, P.N - c);
  if constexpr (Mode == kFfnDx) {
    store_n(static_cast<T*>(P.o0) + r * P.ldo0 + c, v, left);
  } else {
    if (r < P.fp) {
      if (r < P.f) store_n(static_cast<T*>(P.o0) + r * P.ldo0 + c, v, left);
    } else if (r - P.fp < P.f) {
      store_n(static_cast<T*>(P.o1) + (r - P.fp) * P.ldo1 + c, v, left);
    }
  }
}

// The pre-activations of row r, features c .. c + N - 1.
template <class T, int N>
__device__ __forceinline__ void put_preact(const FfnGemm& P, int64_t r, int64_t c, const float (&g)[N],
                                           const float (&u)[N]) {
  const int64_t at = r * 2 * P.fp + c;
  if (sizeof(T) == 4 || P.pre32) {
    float* q = static_cast<float*>(P.o1) + at;
    store_n(q, g, N);
    store_n(q + P.fp, u, N);
  } else {
    T* q = static_cast<T*>(P.o1) + at;
    store_n(q, g, N);
    store_n(q + P.fp, u, N);
  }
}

// Outputs of row r, features c .. c + N - 1 of the forward pass.
template <int DT, int N>
__device__ __forceinline__ void put_fwd(const FfnGemm& P, int64_t r, int64_t c, const float (&g)[N],
                                        const float (&u)[N]) {
  typedef typename Elem<DT>::type T;
  if (r >= P.M || c >= P.fp) return;
  float h[N];
#pragma unroll
  for (int j = 0; j < N; ++j) h[j] = act_value<DT == kInF32>(g[j], P.act) * u[j];
  if (c < P.N) store_n(static_cast<T*>(P.o0) + r * P.ldo0 + c, h, (int)min((int64_t)N, P.N - c));
  if (!P.o1) return;
  // columns f .. fp - 1 are zeros: absent weight rows read as zeros, but times
  // an infinite x they are none
  float gz[N], uz[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    gz[j] = c + j < P.N ? g[j] : 0.0f;
    uz[j] = c + j < P.N ? u[j] : 0.0f;
  }
  put_preact<T>(P, r, c, gz, uz);
}

// Tile t of the blocked order: groups of 8 (dW: 4) tile rows, column by column
// inside a group, so that consecutive tiles (one XCD's, see item_of_block)
// share few operand panels.  At 8192 x 4096 x 11264, bf16: dW 1316 us with 4,
// 1363 with 8, 1324 with 2; forward at 16384 tokens 2353 us with 8, 2380 with
// 4, 2425 with 16.
template <int Mode> __device__ __forceinline__ void tile_coords(const FfnGemm& P, int t, int& I, int& J) {
  constexpr int kGroupM = Mode == kFfnDw ? 4 : 8;
  const int per = kGroupM * P.tn;
  const int grp = t / per;
  const int rows = min(kGroupM, P.tm - grp * kGroupM);
  const int in = t - grp * per;
  J = in / rows;
  I = grp * kGroupM + in - J * rows;
}

// Workgroup b of n runs on XCD b % 8: give each XCD a consecutive run of items.
__device__ __forceinline__ int item_of_block(int b, int n) {
  const int q = n >> 3, r = n & 7, x = b & 7;
  return x * q + min(x, r) + (b >> 3);
}

}  // namespace hess
