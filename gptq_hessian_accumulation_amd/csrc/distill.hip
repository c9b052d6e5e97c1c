// Distillation from a teacher's top logits on gfx950.  For each row, with
// p = softmax(values / T) over the present entries and q = softmax(z / T):
//
//   loss = w sum_i p_i (log p_i - log q[id_i]),   q_j = exp((z_j - m) / T) / s
//   dz_j = c w / T (q_j - sum over i with id_i = j of p_i)
//
// with m = max z and s = sum exp((z - m) / T).
//
// Three kernels, all bound by the bytes of z and dz:
//  * loss and gradient in one pass over rows that fit the register file: a
//    workgroup holds a whole row (up to 16 vectors of 16 bytes a thread) and
//    reads it once;
//  * the loss alone: one workgroup a row, a running maximum and sum;
//  * the gradient from the row's statistics: chunks of rows, one pass.
// Longer rows take the second and the third for loss and gradient.
//
// Measured (a large copy reaches 4.8 TB/s, a read 5.6): 8192 x 131072 bf16,
// loss and gradient, 0.87 ms, 4.9 TB/s; 1024 x 65537 float32, loss alone, 51
// us, 5.2 TB/s; 2047 x 50001 bf16 with a quarter of the rows masked, 93 us, 3.8
// TB/s.  Few rows and short rows are bound by one row's chain of loads, joins
// and float64 logarithms, about 8 us.  A second pass over the row instead of
// registers reads it again from the last-level cache: 512 x 262144, which does
// not fit, takes 170 us, 3.1 TB/s.
//
// Exponentials are 2^x of float32 arguments (z - m) log2(e) / T (the
// difference first, so that values near the type's largest stay finite);
// threads' sums are float32 and joined in float64; the k teacher terms are
// float64, because the loss is a difference of logarithms that cancel where
// student and teacher agree.  log2(e) / T is rounded once to float32 and used
// for both softmaxes, so that the rounding acts as a temperature off by 2^-24
// and not as an offset between the two.

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "distill_internal.hpp"
#include "elem.hpp"

namespace hess {

namespace {

constexpr int kTop = 1024;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));

// Sum and maximum over groups of Lanes lanes, in every lane.
template <int Lanes = 64, class T> __device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = Lanes / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <int Lanes = 64> __device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = Lanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// 16 bytes of a row of T: its values, and loads and stores at any alignment.
template <int DT> struct Vec {
  typedef typename Elem<DT>::type T;
  static constexpr int N = 16 / Elem<DT>::size;
  typedef T TN __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef typename std::conditional<sizeof(T) == 2, u32x4_at2, u32x4_at4>::type U;
  // elements j .. j + N - 1 of a row of n; past it -infinity
  static __device__ __forceinline__ u32x4 load(const T* row, int64_t j, int64_t n) {
    if (j + N <= n) return *reinterpret_cast<const U*>(row + j);
    TN t;
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = (T)(-INFINITY);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (j + e < n) t[e] = row[j + e];
    return __builtin_bit_cast(u32x4, t);
  }
  static __device__ __forceinline__ void store(T* row, int64_t j, int64_t n, const float (&v)[N]) {
    TN t;
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = from_f32<T>(v[e]);
    if (j + N <= n) {
      *reinterpret_cast<U*>(row + j) = __builtin_bit_cast(u32x4, t);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (j + e < n) row[j + e] = t[e];
    }
  }
  static __device__ __forceinline__ void store_whole(T* p, const float (&v)[N]) {
    TN t;
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = from_f32<T>(v[e]);
    *reinterpret_cast<U*>(p) = __builtin_bit_cast(u32x4, t);
  }
  static __device__ __forceinline__ void get(const u32x4& r, float (&v)[N]) {
    const TN t = __builtin_bit_cast(TN, r);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = to_f32(t[e]);
  }
};

// A thread's teacher entries i = tid + q Threads of one row.  id -1: absent,
// as is an entry of value -infinity (p = 0).  An id past the vocabulary (bad)
// takes no part either, but makes the row NaN whatever its value and whatever
// stands beside it: only a row with neither kind is one without entries.
template <int Threads> struct Entries {
  static constexpr int kPer = kTop / Threads;
  int id[kPer];
  float v[kPer], z[kPer];
  int bad;
  // entries fill the waves in order: whether this one has any
  static __device__ __forceinline__ bool mine(int k) { return (int)(threadIdx.x & ~63u) < k; }
  uint32_t raw_lo[kPer], raw_hi[kPer], raw_v[kPer];

  // Issues the loads (nothing waits for them here) ...
  __device__ __forceinline__ void load(const DistillParams& P, int64_t row) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = threadIdx.x + q * Threads;
      raw_lo[q] = raw_hi[q] = raw_v[q] = 0;
      if (q * Threads < P.k && i < P.k) {
        if (P.ids64) {
          const uint2 t = static_cast<const uint2*>(P.ids)[row * P.ldi + i];
          raw_lo[q] = t.x;
          raw_hi[q] = t.y;
        } else {
          raw_lo[q] = static_cast<const uint32_t*>(P.ids)[row * P.ldi + i];
        }
        if (P.values_dtype == kInF32) raw_v[q] = static_cast<const uint32_t*>(P.values)[row * P.ldv + i];
        else raw_v[q] = static_cast<const uint16_t*>(P.values)[row * P.ldv + i];
      }
    }
  }
  // ... and takes what they brought.
  __device__ __forceinline__ void decode(const DistillParams& P) {
    bad = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      id[q] = -1;
      v[q] = -INFINITY;
      if (q * Threads >= P.k) continue;
      const int64_t t = P.ids64 ? (int64_t)(((uint64_t)raw_hi[q] << 32) | raw_lo[q]) : (int64_t)(int32_t)raw_lo[q];
      const float x = P.values_dtype == kInF32    ? __uint_as_float(raw_v[q])
                      : P.values_dtype == kInBF16 ? __uint_as_float(raw_v[q] << 16)
                                                  : (float)__builtin_bit_cast(_Float16, (uint16_t)raw_v[q]);
      const bool here = (int)threadIdx.x + q * Threads < P.k;
      bad |= here && t >= P.vocab;
      const bool present = here && t >= 0 && t < P.vocab && x != -INFINITY;
      id[q] = present ? (int)t : -1;
      v[q] = present ? x : -INFINITY;
    }
  }
  // the student's logits of the entries in [lo, hi)
  template <class T> __device__ __forceinline__ void gather(const T* zr, int k, int lo, int hi) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      z[q] = 0.0f;
      if (q * Threads < k && id[q] >= lo && id[q] < hi) z[q] = to_f32(zr[id[q]]);
    }
  }
};

// What the waves of a workgroup exchange for one row.
template <int Waves> struct Joined {
  float m[Waves], s[Waves], vm[Waves];
  double ps[Waves], term[Waves];
  int flags[Waves], dup;
};

// The waves' shares joined, in every thread: vm, and log of the whole sum.  A
// share without a maximum is empty (sum 0) or holds nothing but NaN (sum NaN):
// either sum is taken as it is.
template <int Waves>
__device__ __forceinline__ void teacher_join(const Joined<Waves>& J, double it, float& vm, double& logps) {
  const int l = threadIdx.x & (Waves - 1);
  const float x = J.vm[l];
  vm = wave_max<Waves>(x);
  logps = log(wave_sum<Waves>(x == -INFINITY ? J.ps[l] : J.ps[l] * exp(((double)x - (double)vm) * it)));
}

// A wave's share of the teacher's softmax: its largest value, and the sum of
// exponentials above it.
template <int Threads>
__device__ __forceinline__ void teacher_share(const Entries<Threads>& E, int k, double it, float& vm, double& ps) {
  vm = -INFINITY;
  ps = 0.0;
  if (!E.mine(k)) return;
#pragma unroll
  for (int q = 0; q < E.kPer; ++q) vm = fmaxf(vm, E.v[q]);
  vm = wave_max(vm);
#pragma unroll
  for (int q = 0; q < E.kPer; ++q)
    if (q * Threads < k && E.id[q] >= 0) ps += exp(((double)E.v[q] - (double)vm) * it);
  ps = wave_sum(ps);
}

// Its terms of the loss; p, float32, to s_p where that is wanted.
template <int Threads, int Waves>
__device__ __forceinline__ double teacher_terms(const Entries<Threads>& E, int k, const Joined<Waves>& J, double it, float m,
                                                float sum, float* s_p) {
  float vm;
  double logps;
  teacher_join(J, it, vm, logps);
  const double logsum = log((double)sum);
  double term = 0.0;
#pragma unroll
  for (int q = 0; q < E.kPer; ++q) {
    if (q * Threads >= k || E.id[q] < 0) continue;
    const double lp = ((double)E.v[q] - (double)vm) * it - logps;
    const double p = exp(lp);
    if (p != 0.0) term += p * (lp - (((double)E.z[q] - (double)m) * it - logsum));
    if (s_p) s_p[threadIdx.x + q * Threads] = (float)p;
  }
  return wave_sum(term);
}

// Whether two entries of ids[0 .. k) name the same word: groups of threads
// compare each entry with a part of them (four at a time, the same ones in
// every lane of a group; ids is 16-byte aligned and padded to a multiple of 4
// with negative values).
template <int Threads> __device__ __forceinline__ bool any_twice(const int* ids, int k) {
  const int lg = k <= 64 ? 6 : 32 - __clz(k - 1);
  const int groups = max(1, Threads >> lg);
  const int g = __builtin_amdgcn_readfirstlane(threadIdx.x >> lg);
  const int quads = (k + 3) >> 2;
  bool twice = false;
  if (g < groups) {
    const int q0 = quads * g / groups, q1 = quads * (g + 1) / groups;
    for (int i = threadIdx.x & ((1 << lg) - 1); i < k; i += Threads) {
      const int id = ids[i];
      for (int q = q0; q < q1; ++q) {
        const int4 x = reinterpret_cast<const int4*>(ids)[q];
        const int at = i - 4 * q;
        twice |= id >= 0 && ((x.x == id && at != 0) || (x.y == id && at != 1) || (x.z == id && at != 2) ||
                             (x.w == id && at != 3));
      }
    }
  }
  return twice;
}

// The entries' own elements of the gradient: c (q - p), p summed over the
// entries of one word where any is named twice.
template <int DT, int Threads>
__device__ __forceinline__ void scatter(const DistillParams& P, const Entries<Threads>& E, const int* ids,
                                        const float* ps, bool twice, typename Elem<DT>::type* dz, float m, float cl,
                                        float inv, float c, int lo, int hi) {
  typedef typename Elem<DT>::type T;
#pragma unroll
  for (int q = 0; q < E.kPer; ++q) {
    const int id = E.id[q];
    if (q * Threads >= P.k || id < lo || id >= hi) continue;
    float p;
    if (twice) {
      p = 0.0f;
      for (int j = 0; j < P.k; j += 4) {
        const int4 x = *reinterpret_cast<const int4*>(ids + j);
        const float4 y = *reinterpret_cast<const float4*>(ps + j);
        p += x.x == id ? y.x : 0.0f;
        p += x.y == id ? y.y : 0.0f;
        p += x.z == id ? y.z : 0.0f;
        p += x.w == id ? y.w : 0.0f;
      }
    } else {
      p = ps[threadIdx.x + q * Threads];
    }
    dz[id] = from_f32<T>(c * (__builtin_amdgcn_exp2f((E.z[q] - m) * cl) * inv - p));
  }
}

// Adds N values to a running maximum and sum of exponentials (float32).
template <int N> __device__ __forceinline__ void online(const float (&v)[N], float cl, float& m, float& s) {
  float a = m;
#pragma unroll
  for (int e = 0; e < N; ++e) a = fmaxf(a, v[e]);
  float t = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) t += __builtin_amdgcn_exp2f((v[e] - a) * cl);
  s = s * __builtin_amdgcn_exp2f((m - a) * cl) + t;
  m = a;
}

// The waves' maxima and sums joined, in every thread.
template <int Waves> __device__ __forceinline__ void student_join(const Joined<Waves>& J, float cl, float& m, float& s) {
  const int l = threadIdx.x & (Waves - 1);
  const float x = J.m[l];
  m = wave_max<Waves>(x);
  s = (float)wave_sum<Waves>((double)(J.s[l] * __builtin_amdgcn_exp2f((x - m) * cl)));
}

struct Scales {
  float cl;   // log2(e) / T
  double it;  // the same scale to base e
};
__device__ __forceinline__ Scales scales(const DistillParams& P) {
  const float cl = (float)(1.4426950408889634 / (double)P.temperature);
  return {cl, (double)cl * 0.69314718055994531};
}

// Loss and gradient of a row of at most Threads * NV whole vectors; the fewer
// than one vector's elements after them go to the first threads, one each.
template <int DT, int Threads, int NV>
__global__ void __launch_bounds__(Threads, 4) distill_resident(DistillParams P) {
  typedef typename Elem<DT>::type T;
  typedef Vec<DT> V;
  constexpr int kWaves = Threads / 64;
  __shared__ Joined<kWaves> J;
  __shared__ __attribute__((aligned(16))) int s_id[kTop];
  __shared__ __attribute__((aligned(16))) float s_p[kTop];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int vocab = (int)P.vocab, nvec = vocab / V::N;
  const int last = nvec * V::N + tid;  // this thread's element past the vectors
  const auto [cl, it] = scales(P);
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(P.z) + row * P.ldz;
  T* dz = static_cast<T*>(P.dz) + row * P.lddz;
  const float w = P.weight ? P.weight[row] : 1.0f;

  // Vector i of this thread: waves past the row's end do nothing, lanes past
  // it take the last vector (and are left out of the sums and stores).  The
  // thread index is made opaque in each loop, so that offsets are computed
  // where they are used and not kept for all vectors at once.
  auto wave_in = [&](int i) { return i * Threads + wave * 64 < nvec; };
  auto opaque_tid = [&] {
    int t = tid;
    asm volatile("" : "+v"(t));
    return t;
  };

  u32x4 v[NV];
  float rest = -INFINITY, m = -FLT_MAX, sum = 0.0f, c = 0.0f;
  Entries<Threads> E;
  int all = 0;
  if (w != 0.0f) {
    E.load(P, row);
    int t = opaque_tid();
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (wave_in(i)) v[i] = *reinterpret_cast<const typename V::U*>(z + min(i * Threads + t, nvec - 1) * V::N);
    if (last < vocab) rest = to_f32(z[last]);
    E.decode(P);
    E.gather(z, P.k, 0, vocab);
    t = opaque_tid();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (wave_in(i)) {
        float x[V::N];
        V::get(v[i], x);
        float a = m, b = sum;
        online(x, cl, a, b);
        const bool in = i * Threads + t < nvec;
        m = in ? a : m;
        sum = in ? b : sum;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    const float one[1] = {rest};
    if (last < vocab) online(one, cl, m, sum);
    float vm;
    double ps;
    teacher_share(E, P.k, it, vm, ps);
    int present = 0;
#pragma unroll
    for (int q = 0; q < E.kPer; ++q) {
      present |= E.id[q] >= 0;
      if (q * Threads < P.k && tid + q * Threads < ((P.k + 3) & ~3)) s_id[tid + q * Threads] = E.id[q];
    }
    const float wm = wave_max(m);
    const float wsum = wave_sum(sum * __builtin_amdgcn_exp2f((m - wm) * cl));
    const int flags = (__any(present) ? 1 : 0) | (__any(E.bad) ? 2 : 0);
    if ((tid & 63) == 0) {
      J.m[wave] = wm;
      J.s[wave] = wsum;
      J.vm[wave] = vm;
      J.ps[wave] = ps;
      J.flags[wave] = flags;
      if (wave == 0) J.dup = 0;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kWaves; ++q) all |= J.flags[q];
    all = __builtin_amdgcn_readfirstlane(all);
  }
  if (all == 0) {
    const float g[V::N] = {};
#pragma unroll 1
    for (int j = tid; j < nvec; j += Threads) V::store_whole(dz + j * V::N, g);
    if (last < vocab) dz[last] = from_f32<T>(0.0f);
    if (tid == 0) P.loss[row] = 0.0f;
    if (P.stats && tid < 2) P.stats[2 * row + tid] = 0.0f;
    return;
  }
  student_join(J, cl, m, sum);
  if (E.mine(P.k)) {
    const double term = teacher_terms(E, P.k, J, it, m, sum, s_p);
    if ((tid & 63) == 0) J.term[wave] = term;
  }
  if (any_twice<Threads>(s_id, P.k)) J.dup = 1;
  c = (all & 2) ? NAN : w / P.temperature;
  const float inv = 1.0f / sum, f = c * inv;
  const int t = opaque_tid();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (wave_in(i)) {
      // opaque: the values unpacked above are not kept for here
      asm volatile("" : "+v"(v[i]));
      float g[V::N];
      V::get(v[i], g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) g[e] = __builtin_amdgcn_exp2f((g[e] - m) * cl) * f;
      if (i * Threads + t < nvec) V::store_whole(dz + (i * Threads + t) * V::N, g);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (last < vocab) dz[last] = from_f32<T>(__builtin_amdgcn_exp2f((rest - m) * cl) * f);
  __syncthreads();
  if (tid == 0) {
    double l = 0.0;
    for (int q = 0; q < kWaves && q * 64 < P.k; ++q) l += J.term[q];
    P.loss[row] = (all & 2) ? NAN : (float)(l * w);
    if (P.stats) {
      P.stats[2 * row] = m;
      P.stats[2 * row + 1] = sum;
    }
  }
  scatter<DT, Threads>(P, E, s_id, s_p, J.dup != 0, dz, m, cl, inv, c, 0, vocab);
}

// The loss, and the row's maximum and sum: one workgroup a row.
template <int DT, int Threads> __global__ void __launch_bounds__(Threads, 4) distill_loss(DistillParams P) {
  typedef typename Elem<DT>::type T;
  typedef Vec<DT> V;
  constexpr int kWaves = Threads / 64, kUnroll = 8;
  __shared__ Joined<kWaves> J;
  const int tid = threadIdx.x, wave = tid >> 6;
  const auto [cl, it] = scales(P);
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(P.z) + row * P.ldz;
  const float w = P.weight ? P.weight[row] : 1.0f;
  bool zero = w == 0.0f;
  float m = -FLT_MAX, sum = 0.0f, vm;
  double ps;
  Entries<Threads> E;
  int all = 0;
  if (!zero) {
    E.load(P, row);
    // blocks of kUnroll vectors a thread; in the last one, lanes past the row
    // take its last vector and leave it out.  The fewer than one vector's
    // elements after the vectors go to the first threads, one each.
    const int64_t nvec = P.vocab / V::N;
    for (int64_t b0 = 0; b0 < nvec; b0 += kUnroll * Threads) {
      const bool whole = b0 + kUnroll * Threads <= nvec;
      u32x4 v[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        v[i] = *reinterpret_cast<const typename V::U*>(z + min(b0 + i * Threads + tid, nvec - 1) * V::N);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        if (!whole && b0 + i * Threads + (tid & ~63) >= nvec) continue;
        float x[V::N], a = m, s = sum;
        V::get(v[i], x);
        online(x, cl, a, s);
        const bool in = b0 + i * Threads + tid < nvec;
        m = in ? a : m;
        sum = in ? s : sum;
      }
    }
    if (nvec * V::N + tid < P.vocab) {
      const float one[1] = {to_f32(z[nvec * V::N + tid])};
      online(one, cl, m, sum);
    }
    E.decode(P);
    E.gather(z, P.k, 0, (int)P.vocab);
    teacher_share(E, P.k, it, vm, ps);
    int present = 0;
#pragma unroll
    for (int q = 0; q < E.kPer; ++q) present |= E.id[q] >= 0;
    const float wm = wave_max(m);
    const float wsum = wave_sum(sum * __builtin_amdgcn_exp2f((m - wm) * cl));
    const int flags = (__any(present) ? 1 : 0) | (__any(E.bad) ? 2 : 0);
    if ((tid & 63) == 0) {
      J.m[wave] = wm;
      J.s[wave] = wsum;
      J.vm[wave] = vm;
      J.ps[wave] = ps;
      J.flags[wave] = flags;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kWaves; ++q) all |= J.flags[q];
    zero = all == 0;
  }
  if (zero) {
    if (tid == 0) P.loss[row] = 0.0f;
    if (P.stats && tid < 2) P.stats[2 * row + tid] = 0.0f;
    return;
  }
  student_join(J, cl, m, sum);
  if (E.mine(P.k)) {
    const double term = teacher_terms(E, P.k, J, it, m, sum, nullptr);
    if ((tid & 63) == 0) J.term[wave] = term;
  }
  __syncthreads();
  if (tid == 0) {
    double t = 0.0;
    for (int q = 0; q < kWaves && q * 64 < P.k; ++q) t += J.term[q];
    P.loss[row] = (all & 2) ? NAN : (float)(t * w);
    if (P.stats) {
      P.stats[2 * row] = m;
      P.stats[2 * row + 1] = sum;
    }
  }
}

// The gradient from the row's maximum and sum: workgroup (row, part) does a
// chunk of the row and the teacher's entries inside it.
template <int DT, int Threads> __global__ void __launch_bounds__(Threads, 4) distill_grad(DistillParams P, int parts) {
  typedef typename Elem<DT>::type T;
  typedef Vec<DT> V;
  constexpr int kWaves = Threads / 64, kUnroll = 8;
  __shared__ Joined<kWaves> J;
  __shared__ __attribute__((aligned(16))) int s_id[kTop];
  __shared__ __attribute__((aligned(16))) float s_p[kTop];
  const int tid = threadIdx.x, wave = tid >> 6;
  const auto [cl, it] = scales(P);
  const int64_t row = blockIdx.x / (unsigned)parts;
  const int part = blockIdx.x - (unsigned)row * (unsigned)parts;
  const int64_t per = ((P.vocab + (int64_t)parts * V::N - 1) / ((int64_t)parts * V::N)) * V::N;
  const int64_t lo = part * per, hi = min(P.vocab, lo + per);
  const T* z = static_cast<const T*>(P.z) + row * P.ldz;
  T* dz = static_cast<T*>(P.dz) + row * P.lddz;
  const float w = P.weight ? P.weight[row] : 1.0f;
  bool zero = w == 0.0f;
  float m = 0.0f, c = 0.0f, inv = 0.0f;
  Entries<Threads> E;
  if (!zero) {
    E.load(P, row);
    m = P.stats[2 * row];
    inv = 1.0f / P.stats[2 * row + 1];
    E.decode(P);
    E.gather(z, P.k, (int)lo, (int)hi);
    float vm;
    double ps;
    teacher_share(E, P.k, it, vm, ps);
    int present = 0;
#pragma unroll
    for (int q = 0; q < E.kPer; ++q) {
      present |= E.id[q] >= 0;
      if (q * Threads < P.k && tid + q * Threads < ((P.k + 3) & ~3)) s_id[tid + q * Threads] = E.id[q];
    }
    const int flags = (__any(present) ? 1 : 0) | (__any(E.bad) ? 2 : 0);
    if ((tid & 63) == 0) {
      J.vm[wave] = vm;
      J.ps[wave] = ps;
      J.flags[wave] = flags;
      if (wave == 0) J.dup = 0;
    }
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int q = 0; q < kWaves; ++q) all |= J.flags[q];
    zero = all == 0;
    c = (all & 2) ? NAN : (P.dloss ? P.dloss[row] : 1.0f) * w / P.temperature;
    if (!zero && E.mine(P.k)) {
      double logps;
      teacher_join(J, it, vm, logps);
#pragma unroll
      for (int q = 0; q < E.kPer; ++q)
        if (q * Threads < P.k && E.id[q] >= 0) s_p[tid + q * Threads] = (float)exp(((double)E.v[q] - (double)vm) * it - logps);
    }
    if (!zero && any_twice<Threads>(s_id, P.k)) J.dup = 1;
  }
  // blocks of kUnroll whole vectors a thread, then the rest vector by vector
  const float f = c * inv;
  int64_t j = lo + (int64_t)tid * V::N;
  const int64_t step = (int64_t)Threads * V::N, block = kUnroll * step;
  auto slope = [&](const u32x4& r, float (&g)[V::N]) {
    V::get(r, g);
#pragma unroll
    for (int e = 0; e < V::N; ++e) g[e] = __builtin_amdgcn_exp2f((g[e] - m) * cl) * f;
  };
  const float none[V::N] = {};
  for (int64_t b0 = lo; b0 + block <= hi; b0 += block, j += block) {
    if (zero) {
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) V::store_whole(dz + j + i * step, none);
    } else {
      u32x4 v[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) v[i] = *reinterpret_cast<const typename V::U*>(z + j + i * step);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        float g[V::N];
        slope(v[i], g);
        V::store_whole(dz + j + i * step, g);
      }
    }
  }
  // what is left: at most kUnroll vectors a thread, the last perhaps not whole
  const int64_t first = j - (int64_t)(tid & 63) * V::N;  // the wave's first element
  u32x4 v[kUnroll];
  if (!zero && hi - lo >= V::N) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (first + i * step < hi) v[i] = *reinterpret_cast<const typename V::U*>(z + min(j + i * step, hi - V::N));
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t at = j + i * step;
    if (at >= hi) break;
    float g[V::N];
    if (zero) {
#pragma unroll
      for (int e = 0; e < V::N; ++e) g[e] = 0.0f;
    } else {
      slope(at + V::N <= hi ? v[i] : V::load(z, at, hi), g);
    }
    V::store(dz, at, hi, g);
  }
  if (zero) return;
  __syncthreads();
  scatter<DT, Threads>(P, E, s_id, s_p, J.dup != 0, dz, m, cl, inv, c, (int)lo, (int)hi);
}

template <int DT> constexpr int64_t resident_limit() { return ((int64_t)1024 * 16 + 1) * Vec<DT>::N - 1; }

// Launches `go` on ranges of rows: `parts` workgroups of Threads each a row, and
// fewer than 2^32 threads a grid.
template <int DT, int Threads, class Go> void launch_rows(const DistillParams& P, int64_t parts, Go go) {
  const int64_t most = distill_rows_per_launch(Threads, parts);
  for (int64_t r = 0; r < P.n; r += most) {
    const DistillParams Q = distill_rows(P, Elem<DT>::size, r, most);
    go(Q, (unsigned)(Q.n * parts));
  }
}

template <int DT, int Threads, int NV> void launch_resident(const DistillParams& P, hipStream_t stream) {
  launch_rows<DT, Threads>(P, 1, [&](const DistillParams& Q, unsigned grid) {
    distill_resident<DT, Threads, NV><<<grid, Threads, 0, stream>>>(Q);
  });
}

template <int DT, int Threads> void launch_loss_of(const DistillParams& P, hipStream_t stream) {
  launch_rows<DT, Threads>(P, 1, [&](const DistillParams& Q, unsigned grid) {
    distill_loss<DT, Threads><<<grid, Threads, 0, stream>>>(Q);
  });
}
template <int DT> void launch_loss(const DistillParams& P, hipStream_t stream) {
  // few rows, or long ones: more threads a row
  if (P.n <= 512 && P.vocab > 16384) launch_loss_of<DT, 1024>(P, stream);
  else if (P.vocab > 8192) launch_loss_of<DT, 512>(P, stream);
  else if (P.vocab > 2048) launch_loss_of<DT, 256>(P, stream);
  else launch_loss_of<DT, 128>(P, stream);
}

template <int DT, int Threads> void launch_grad_of(const DistillParams& P, int64_t parts, hipStream_t stream) {
  launch_rows<DT, Threads>(P, parts, [&](const DistillParams& Q, unsigned grid) {
    distill_grad<DT, Threads><<<grid, Threads, 0, stream>>>(Q, (int)parts);
  });
}
template <int DT> void launch_grad(const DistillParams& P, hipStream_t stream) {
  // up to 16 vectors a thread; short rows take fewer threads (8192 rows of
  // 1000: 128 threads 29 us, 512 threads 56 us)
  const int64_t vecs = P.vocab / Vec<DT>::N;
  const int threads = vecs <= 1024 ? 128 : vecs <= 2048 ? 256 : 512;
  const int64_t parts = (vecs + 16 * threads) / (16 * threads);
  if (threads == 128) launch_grad_of<DT, 128>(P, parts, stream);
  else if (threads == 256) launch_grad_of<DT, 256>(P, parts, stream);
  else launch_grad_of<DT, 512>(P, parts, stream);
}

template <int DT> hipError_t launch(DistillParams P, hipStream_t stream) {
  if (!P.dz) {
    launch_loss<DT>(P, stream);
    return hipGetLastError();
  }
  const int64_t vecs = P.vocab / Vec<DT>::N;
  if (P.vocab > resident_limit<DT>()) {
    if (!P.stats) P.stats = static_cast<float*>(P.work);
    launch_loss<DT>(P, stream);
    launch_grad<DT>(P, stream);
  } else if (vecs <= 512) {
    launch_resident<DT, 128, 4>(P, stream);
  } else if (vecs <= 1024) {
    launch_resident<DT, 256, 4>(P, stream);
  } else if (P.n <= 256) {
    // a row for each CU: all its waves on it
    if (vecs <= 4096) launch_resident<DT, 1024, 4>(P, stream);
    else launch_resident<DT, 1024, 16>(P, stream);
  } else if (vecs <= 4096) {
    launch_resident<DT, 256, 16>(P, stream);
  } else if (vecs <= 8192) {
    launch_resident<DT, 512, 16>(P, stream);
  } else {
    launch_resident<DT, 1024, 16>(P, stream);
  }
  return hipGetLastError();
}

template <int DT> hipError_t backward(const DistillParams& P, hipStream_t stream) {
  launch_grad<DT>(P, stream);
  return hipGetLastError();
}

}  // namespace

// Rows too long for the registers keep their statistics between two launches.
int64_t distill_workspace(int64_t n, int64_t vocab, int dtype) {
  const int64_t limit = dtype == kInF32 ? resident_limit<kInF32>() : resident_limit<kInBF16>();
  return vocab > limit ? n * 8 : 0;
}

hipError_t launch_distill(const DistillParams& P, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) return launch<kInBF16>(P, stream);
  if (dtype == kInF16) return launch<kInF16>(P, stream);
  return launch<kInF32>(P, stream);
}
hipError_t launch_distill_backward(const DistillParams& P, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) return backward<kInBF16>(P, stream);
  if (dtype == kInF16) return backward<kInF16>(P, stream);
  return backward<kInF32>(P, stream);
}

}  // namespace hess
