// Distillation from a teacher's top logits on gfx950.  For each row, with
// p = softmax(values / T) over the present entries and q = softmax(z / T):
//
//   loss = w sum_i p_i (log p_i - log q[id_i]),   q_j = exp(z_j / T - m) / s
//   dz_j = c w / T (q_j - sum over i with id_i = j of p_i)
//
// with m = max(z / T) and s = sum exp(z / T - m).
//
// One workgroup a row.  Exponentials are float32, joined across the workgroup
// in float64; the k teacher terms are float64, because the loss is a difference of logarithms that cancel where
// student and teacher agree.  1 / T is rounded once to float32 and used for
// both softmaxes, so that the rounding acts as a temperature off by 2^-25 and
// not as an offset between the two.

#include <cmath>

#include "distill_internal.hpp"
#include "elem.hpp"

namespace hess {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kTop = 1024;

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}
// Sum / maximum over the workgroup, the same value in every thread.
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = red[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) t += red[w];
  return t;
}
__device__ __forceinline__ double block_max(double v, double* red) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = red[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) t = fmax(t, red[w]);
  return t;
}

__device__ __forceinline__ int64_t load_id(const DistillParams& P, int64_t row, int i) {
  return P.ids64 ? static_cast<const int64_t*>(P.ids)[row * P.ldi + i]
                 : static_cast<const int32_t*>(P.ids)[row * P.ldi + i];
}
__device__ __forceinline__ float load_value(const DistillParams& P, int64_t row, int i) {
  const int64_t o = row * P.ldv + i;
  if (P.values_dtype == kInBF16) return to_f32(static_cast<const __bf16*>(P.values)[o]);
  if (P.values_dtype == kInF16) return to_f32(static_cast<const _Float16*>(P.values)[o]);
  return static_cast<const float*>(P.values)[o];
}

template <int DT, bool Backward> __global__ void __launch_bounds__(kThreads) distill_row(DistillParams P) {
  typedef typename Elem<DT>::type T;
  __shared__ double red[kWaves];
  __shared__ int s_id[kTop];
  __shared__ float s_p[kTop], s_z[kTop];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(P.z) + row * P.ldz;
  T* dz = static_cast<T*>(P.dz) + (P.dz ? row * P.lddz : 0);
  const float w = P.weight ? P.weight[row] : 1.0f;
  const float it = (float)(1.0 / (double)P.temperature);

  // the teacher's entries; id -1: absent, as is one of value -infinity (p = 0)
  double vmax = -INFINITY;
  int any = 0, bad = 0;
  for (int i = tid; i < P.k; i += kThreads) {
    const int64_t id = load_id(P, row, i);
    const float v = id >= 0 ? load_value(P, row, i) : -INFINITY;
    const bool present = v != -INFINITY;
    any |= present;
    bad |= id >= P.vocab;
    s_id[i] = (present && id < P.vocab) ? (int)id : -1;
    if (s_id[i] >= 0) {
      s_p[i] = v;
      s_z[i] = to_f32(z[id]);
      vmax = fmax(vmax, (double)v * it);
    }
  }
  any = __syncthreads_or(any);
  bad = __syncthreads_or(bad);
  if (w == 0.0f || !any) {
    if (!Backward && tid == 0) P.loss[row] = 0.0f;
    if (!Backward && P.stats && tid < 2) P.stats[2 * row + tid] = 0.0f;
    if (P.dz)
      for (int64_t j = tid; j < P.vocab; j += kThreads) dz[j] = from_f32<T>(0.0f);
    return;
  }
  vmax = block_max(vmax, red);
  double psum = 0.0;
  for (int i = tid; i < P.k; i += kThreads)
    if (s_id[i] >= 0) psum += exp((double)s_p[i] * it - vmax);
  psum = block_sum(psum, red);
  const double lsep = vmax + log(psum);

  float m, sum;
  if constexpr (Backward) {
    m = P.stats[2 * row];
    sum = P.stats[2 * row + 1];
  } else {
    m = -INFINITY;
    for (int64_t j = tid; j < P.vocab; j += kThreads) m = fmaxf(m, to_f32(z[j]) * it);
    m = (float)block_max((double)m, red);
    // nothing above -infinity: the differences below would be NaN for -infinity itself
    if (m == -INFINITY) m = 0.0f;
    sum = 0.0f;
    for (int64_t j = tid; j < P.vocab; j += kThreads) sum += expf(fmaf(to_f32(z[j]), it, -m));
    sum = (float)block_sum((double)sum, red);
  }
  const double logsum = log((double)sum);

  double term = 0.0;
  for (int i = tid; i < P.k; i += kThreads) {
    if (s_id[i] < 0) continue;
    const double lp = (double)s_p[i] * it - lsep;
    const double p = exp(lp);
    if (p != 0.0) term += p * (lp - ((double)s_z[i] * it - m - logsum));
    s_p[i] = (float)p;
  }
  if constexpr (!Backward) {
    term = block_sum(term, red);
    if (tid == 0) {
      P.loss[row] = bad ? NAN : (float)(term * w);
      if (P.stats) {
        P.stats[2 * row] = m;
        P.stats[2 * row + 1] = sum;
      }
    }
  }
  if (!P.dz) return;
  __syncthreads();
  const float c = bad ? NAN : (Backward ? P.dloss[row] : 1.0f) * w / P.temperature;
  const float inv = 1.0f / sum;
  for (int64_t j = tid; j < P.vocab; j += kThreads)
    dz[j] = from_f32<T>(c * (expf(fmaf(to_f32(z[j]), it, -m)) * inv));
  __syncthreads();
  for (int i = tid; i < P.k; i += kThreads) {
    const int id = s_id[i];
    if (id < 0) continue;
    float p = 0.0f;
    for (int j = 0; j < P.k; ++j) p += s_id[j] == id ? s_p[j] : 0.0f;
    dz[id] = from_f32<T>(c * (expf(fmaf(s_z[i], it, -m)) * inv - p));
  }
}

template <bool Backward> hipError_t launch(const DistillParams& P, int dtype, hipStream_t stream) {
  const unsigned grid = (unsigned)P.n;
  if (dtype == kInBF16) distill_row<kInBF16, Backward><<<grid, kThreads, 0, stream>>>(P);
  else if (dtype == kInF16) distill_row<kInF16, Backward><<<grid, kThreads, 0, stream>>>(P);
  else distill_row<kInF32, Backward><<<grid, kThreads, 0, stream>>>(P);
  return hipGetLastError();
}

}  // namespace

int64_t distill_workspace(int64_t n, int64_t vocab, int dtype) { return 0; }

hipError_t launch_distill(const DistillParams& P, int dtype, hipStream_t stream) {
  return launch<false>(P, dtype, stream);
}
hipError_t launch_distill_backward(const DistillParams& P, int dtype, hipStream_t stream) {
  return launch<true>(P, dtype, stream);
}

}  // namespace hess
