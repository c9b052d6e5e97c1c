// Device code shared by the 8-bit integer operators and the 8-bit activation
// checkpoints: blocks of 32 columns with a power-of-two step.
#pragma once

#include "elem.hpp"
#include "hess_device.hpp"
#include "int8_internal.hpp"

namespace hess {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
typedef uint2 uint2_at1 __attribute__((aligned(1)));

constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The exponent byte b of a block whose largest magnitude has these bits: the
// step 2^(b - 127) is the power of two with 64 <= top / step < 128, at least
// 2^-126, so that what codes stand for is no subnormal number; 255 where a value
// of the block is not finite.
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
  if (top >= kInfBits) return 255u;
  return (uint32_t)max((int)(top >> 23) - 6, 1);
}
// 2^(127 - b), what the block's values are multiplied by (0 for 255: codes 0)
__device__ __forceinline__ float block_inverse(uint32_t b) { return __uint_as_float(b == 255u ? 0u : (254u - b) << 23); }
// 2^(b - 127), or NaN for 255
__device__ __forceinline__ float block_step(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}


// Four codes of a block in a word: the nearest whole numbers, ties to even, of
// magnitude up to 127 (values past 127.5 steps are less than a step off).  Values
// are first held to 127 steps (0 in a block that is not finite, whose codes are 0);
// v / step + 1.5 * 2^23, rounded once, then has the code in its lowest byte.
struct BlockCode {
  float inverse, most;
  __device__ __forceinline__ explicit BlockCode(uint32_t b)
      : inverse(block_inverse(b)), most(b == 255u ? 0.0f : 127.0f * block_step(b)) {}
  __device__ __forceinline__ uint32_t one(float v) const {
    return __float_as_uint(fmaf(__builtin_amdgcn_fmed3f(v, -most, most), inverse, 12582912.0f));
  }
  __device__ __forceinline__ uint32_t operator()(float a, float b, float c, float d) const {
    const uint32_t ab = __builtin_amdgcn_perm(one(b), one(a), 0x0c0c0400u);
    const uint32_t cd = __builtin_amdgcn_perm(one(d), one(c), 0x0c0c0400u);
    return __builtin_amdgcn_perm(cd, ab, 0x05040100u);
  }
};

// The larger of a lane's value and that of the lane 32 (16) further on or back.
__device__ __forceinline__ uint32_t max_over_32(uint32_t v) {
  const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)s[0], (uint32_t)s[1]);
}
__device__ __forceinline__ uint32_t max_over_16(uint32_t v) {
  const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max((uint32_t)s[0], (uint32_t)s[1]);
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}

// A product's sum times its scales, in float32.  (The value is pinned before it
// is rounded to the output's type: a fused multiply and conversion in one kernel
// and not in another would give other bits.)
__device__ __forceinline__ float scale_sum(int sum, float sb, float sa) {
  float v = (float)sum * sb * sa;
  asm("" : "+v"(v));
  return v;
}

// Code j of a packed word, as a float.
__device__ __forceinline__ float unpack(uint32_t w, int j) { return (float)(int8_t)(w >> (8 * j)); }

// 8 values at p (any element alignment), the first `left` of them inside the row.
template <class T> __device__ __forceinline__ void load8(const T* p, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    if constexpr (sizeof(T) == 2) {
      typedef T T8 __attribute__((ext_vector_type(8)));
      typedef T8 T8u __attribute__((aligned(sizeof(T))));
      const T8 t = *reinterpret_cast<const T8u*>(p);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = to_f32(t[j]);
    } else {
      typedef float F4u __attribute__((ext_vector_type(4), aligned(4)));
      const F4u a = *reinterpret_cast<const F4u*>(p), b = *reinterpret_cast<const F4u*>(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? to_f32(p[j]) : 0.0f;
  }
}

__device__ __forceinline__ uint32_t top_of(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
  return m;
}

// What turns a row's values into codes, from the bits of its largest magnitude.
template <class T> struct RowCode {
  float lift, inverse;
  double inverse64;
  bool zero;
  __device__ __forceinline__ explicit RowCode(uint32_t top) {
    const float a = __uint_as_float(top);
    zero = top == 0u || top >= kInfBits;
    if constexpr (sizeof(T) == 2) {
      // (rows of tiny values are lifted by a power of two first)
      lift = a < 1e-30f ? 0x1p96f : 1.0f;
      inverse = zero ? 0.0f : 127.0f / (a * lift);
    } else {
      inverse64 = zero ? 0.0 : 127.0 / (double)a;
    }
  }
  __device__ __forceinline__ int operator()(float v) const {
    if (zero) return 0;
    if constexpr (sizeof(T) == 2) {
      const float t = v * lift * inverse;
      return (int)rintf(__uint_as_float((__float_as_uint(t) + 4u) & ~7u));
    } else {
      const double t = (double)v * inverse64;
      return (int)rint((t + 6144.0) - 6144.0);
    }
  }
};
__device__ __forceinline__ float row_scale(uint32_t top) {
  return top >= kInfBits ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
}

// i / per, by 32-bit division where that is enough
__device__ __forceinline__ int64_t row_of(int64_t i, int64_t per) {
  return ((uint64_t)(i | per) >> 32) == 0 ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
}

// Codes back to values of DT (16-bit types: rounded to nearest even; exact for
// blocks), 16 bytes of them a thread (float32 at 16384 x 4096: 32 bytes took 91 us,
// 3.7 TB/s), from thread `first` of `all`; columns d .. pad - 1 become zeros.
template <int DT, int Block>
__device__ __forceinline__ void dequantize_range(const Int8Rows& R, int64_t first, int64_t all) {
  typedef typename Elem<DT>::type E;
  constexpr int N = 16 / sizeof(E);
  typedef E EN __attribute__((ext_vector_type(N)));
  typedef EN ENu __attribute__((aligned(sizeof(E))));
  typedef uint32_t Words __attribute__((ext_vector_type(N / 4), aligned(1)));
  const int64_t groups = (R.d + 31) / 32, per = (R.pad + N - 1) / N, total = R.n * per;
  for (int64_t i = first; i < total; i += all) {
    const int64_t row = row_of(i, per), at = (i - row * per) * N;
    float step = 0.0f;
    if constexpr (Block == 0) step = static_cast<const float*>(R.scale)[row];
    else if (at < R.d) step = block_step(static_cast<const uint8_t*>(R.scale)[row * groups + at / 32]);
    const int8_t* c = R.codes + row * R.ldc + at;
    E* o = static_cast<E*>(const_cast<void*>(R.x)) + row * R.ldx + at;
    EN v;
    if (at + N <= R.d) {
      const Words w = *reinterpret_cast<const Words*>(c);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = from_f32<E>(unpack(w[j / 4], j & 3) * step);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = from_f32<E>(at + j < R.d ? (float)c[j] * step : 0.0f);
    }
    if (at + N <= R.pad) {
      *reinterpret_cast<ENu*>(o) = v;
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (at + j < R.pad) o[j] = v[j];
    }
  }
}

}  // namespace hess
