// Internal interface of the top-logit distillation loss.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

int64_t distill_workspace(int64_t n, int64_t vocab, int dtype);
hipError_t launch_distill(const DistillParams& P, int dtype, hipStream_t stream);
hipError_t launch_distill_backward(const DistillParams& P, int dtype, hipStream_t stream);

}  // namespace hess
