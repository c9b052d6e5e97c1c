// Element types of the feed-forward block and the distillation loss: storage
// in bf16, float32 or fp16, arithmetic in float32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hess_internal.hpp"

namespace hess {

template <int DT> struct Elem;
template <> struct Elem<kInBF16> {
  typedef __bf16 type;
  static constexpr int size = 2;
};
template <> struct Elem<kInF32> {
  typedef float type;
  static constexpr int size = 4;
};
template <> struct Elem<kInF16> {
  typedef _Float16 type;
  static constexpr int size = 2;
};

__device__ __forceinline__ float to_f32(__bf16 v) {
  return __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, v) << 16);
}
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }

// Round to nearest even; past the largest finite value to infinity.
template <class T> __device__ __forceinline__ T from_f32(float v) { return (T)v; }

}  // namespace hess
