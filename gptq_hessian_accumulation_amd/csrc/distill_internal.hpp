// Internal interface of the top-logit distillation loss.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hess_internal.hpp"

namespace hess {

struct DistillParams {
  const void* z;         // student logits, n x vocab, row stride ldz
  int64_t ldz, n, vocab;
  const void* ids;       // n x k, int32 or int64
  int ids64;
  int64_t ldi;
  const void* values;    // n x k teacher logits
  int values_dtype;
  int64_t ldv;
  int k;
  const float* weight;   // n, or null
  float temperature;
  const float* dloss;    // backward: n
  float* loss;           // forward: n
  float* stats;          // n x 2: maximum, sum of exponentials; forward: written (or null); backward: read
  void* dz;              // gradient, row stride lddz, or null
  int64_t lddz;
  void* work;
};

// Rows of one launch of `parts` workgroups of `threads` each a row: a grid
// takes fewer than 2^32 threads.
constexpr int64_t distill_rows_per_launch(int threads, int64_t parts) {
  return (((int64_t)1 << 32) - 1) / (threads * parts);
}

// Rows r .. r + most - 1 of a call, logits of esize bytes.
inline DistillParams distill_rows(DistillParams P, int esize, int64_t r, int64_t most) {
  auto skip = [](auto*& p, int64_t bytes) {
    if (p) p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(reinterpret_cast<uintptr_t>(p) + bytes);
  };
  skip(P.z, r * P.ldz * esize);
  skip(P.dz, r * P.lddz * esize);
  skip(P.ids, r * P.ldi * (P.ids64 ? 8 : 4));
  skip(P.values, r * P.ldv * (P.values_dtype == kInF32 ? 4 : 2));
  skip(P.weight, r * 4);
  skip(P.dloss, r * 4);
  skip(P.loss, r * 4);
  skip(P.stats, r * 8);
  P.n = P.n - r < most ? P.n - r : most;
  return P;
}

int64_t distill_workspace(int64_t n, int64_t vocab, int dtype);
hipError_t launch_distill(const DistillParams& P, int dtype, hipStream_t stream);
hipError_t launch_distill_backward(const DistillParams& P, int dtype, hipStream_t stream);

}  // namespace hess
