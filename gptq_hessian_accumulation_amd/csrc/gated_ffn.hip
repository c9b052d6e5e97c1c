// The gated feed-forward block of a transformer layer on gfx950:
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) * u          x: n x d, Wg, Wu: f x d
//
// and its gradients, with dg = dh u act'(g) and du = dh act(g):
//
//   dx = dg Wg + du Wu,   dWg = dg^T x,   dWu = du^T x.
//
// All three are tiled matrix products with float32 accumulators.  A forward
// tile holds the same feature columns of both projections (each wave half
// gate, half up), so the activation and the product happen in registers and
// g and u never travel; they are written only when a backward pass will need
// them.  dx is one product over two segments of K (gate, then up), dWg and
// dWu one product with the gate and up rows stacked.

#include <algorithm>

#include "elem.hpp"
#include "ffn_internal.hpp"
#include "hess_device.hpp"
#include "../../include/hess.h"

namespace hess {

namespace {

// act(g) and act'(g) in float32.  The cumulative normal goes through erfc and
// tanh through the sigmoid (0.5 (1 + tanh s) = sigmoid(2 s)), so the left
// tails keep their relative accuracy.  Exact: float32 outputs, where the
// library exponential's last bits count; otherwise the hardware exponential.
template <bool Exact> __device__ __forceinline__ float sigmoidf(float v) {
  if constexpr (Exact) return 1.0f / (1.0f + expf(-v));
  else return __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

template <bool Exact> __device__ __forceinline__ float act_value(float g, int act) {
  if (act == HESS_SILU) return g * sigmoidf<Exact>(g);
  if (act == HESS_GELU) return g * (0.5f * erfcf(-0.70710678118654752f * g));
  return g * sigmoidf<Exact>(1.5957691216057308f * (g + 0.044715f * g * g * g));
}

template <bool Exact> __device__ __forceinline__ void act_both(float g, int act, float& a, float& da) {
  if (act == HESS_SILU) {
    const float s = sigmoidf<Exact>(g);
    a = g * s;
    da = s * (1.0f + g * (1.0f - s));
  } else if (act == HESS_GELU) {
    const float c = 0.5f * erfcf(-0.70710678118654752f * g);
    a = g * c;
    const float e = -0.5f * g * g;
    da = c + g * 0.39894228040143268f * (Exact ? expf(e) : __expf(e));
  } else {
    const float s = sigmoidf<Exact>(1.5957691216057308f * (g + 0.044715f * g * g * g));
    a = g * s;
    da = s + g * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * g * g);
  }
}

// Four consecutive outputs of one row; `left` of them lie inside the matrix.
template <class T> __device__ __forceinline__ void store4(T* p, const float (&v)[4], int left, bool vec) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  if (vec && left >= 4) {
    *reinterpret_cast<T4*>(p) = T4{from_f32<T>(v[0]), from_f32<T>(v[1]), from_f32<T>(v[2]), from_f32<T>(v[3])};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) p[j] = from_f32<T>(v[j]);
  }
}

// Outputs of row r, columns c .. c + 3 (dx, dw).
template <int DT, int Mode>
__device__ __forceinline__ void put4(const FfnGemm& P, int64_t r, int64_t c, const float (&v)[4]) {
  typedef typename Elem<DT>::type T;
  if (r >= P.M || c >= P.N) return;
  const int left = (int)min((int64_t)4, P.N - c);
  if constexpr (Mode == kFfnDx) {
    store4(static_cast<T*>(P.o0) + r * P.ldo0 + c, v, left, P.vec_out);
  } else {
    if (r < P.fp) {
      if (r < P.f) store4(static_cast<T*>(P.o0) + r * P.ldo0 + c, v, left, P.vec_out);
    } else if (r - P.fp < P.f) {
      store4(static_cast<T*>(P.o1) + (r - P.fp) * P.ldo1 + c, v, left, P.vec_out);
    }
  }
}

// Outputs of row r, features c .. c + 3 of the forward pass.
template <int DT>
__device__ __forceinline__ void put4_fwd(const FfnGemm& P, int64_t r, int64_t c, const float (&g)[4],
                                         const float (&u)[4]) {
  typedef typename Elem<DT>::type T;
  if (r >= P.M || c >= P.fp) return;
  float h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = act_value<DT == kInF32>(g[j], P.act) * u[j];
  if (c < P.N) store4(static_cast<T*>(P.o0) + r * P.ldo0 + c, h, (int)min((int64_t)4, P.N - c), P.vec_out);
  if (P.o1) {
    // columns f .. fp - 1 are the zeros their absent weight rows gave
    T* q = static_cast<T*>(P.o1) + r * 2 * P.fp + c;
    store4(q, g, 4, true);
    store4(q + P.fp, u, 4, true);
  }
}

// Tile t of the blocked order: groups of kGroupM tile rows, column by column
// inside a group, so that consecutive tiles (one XCD's, see item_of_block)
// share few operand panels.
constexpr int kGroupM = 8;
__device__ __forceinline__ void tile_coords(const FfnGemm& P, int t, int& I, int& J) {
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

// Column b of a forward tile's B panel: which projection, and which feature
// of the tile's edge / 2.  Each wave column (half the panel) holds its gate
// columns first, then the same features' up columns.
template <int Edge> __device__ __forceinline__ void fwd_column(int b, int& up, int& col) {
  const int w = b / (Edge / 2), in = b % (Edge / 2);
  up = in / (Edge / 4);
  col = w * (Edge / 4) + in % (Edge / 4);
}

// ---------------------------------------------------------------------------
// 128-tile kernel on the float32 matrix instruction.  4 waves, 64 x 64 each
// (2 x 2 blocks of v_mfma_f32_32x32x2_f32, B first, so that a lane holds four
// consecutive columns).  Operands are widened to float32 and staged k-major.
// ---------------------------------------------------------------------------

constexpr int kPad = 4;
constexpr int kLd = kFfnEdge + kPad;

template <int DT, int Mode> __global__ void __launch_bounds__(256) ffn_f32_tile(FfnGemm P) {
  typedef typename Elem<DT>::type T;
  __shared__ float sA[kFfnStep][kLd];
  __shared__ float sB[kFfnStep][kLd];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wr = wave >> 1, wc = wave & 1;
  const int nitems = gridDim.x;
  const int item = item_of_block(blockIdx.x, nitems);
  const int tail = P.ntiles - P.full;
  int t = item, part = 0;
  const bool whole = item < P.full;
  if (!whole) {
    part = (item - P.full) / tail;
    t = P.full + (item - P.full) % tail;
  }
  const int it0 = whole ? 0 : part * P.part_len;
  const int it1 = whole ? P.niter : min(P.niter, it0 + P.part_len);
  int I, J;
  tile_coords(P, t, I, J);
  const int64_t i0 = (int64_t)I * kFfnEdge;
  const int64_t j0 = (int64_t)J * (Mode == kFfnFwd ? kFfnEdge / 2 : kFfnEdge);
  const int per_seg = Mode == kFfnDx ? P.niter / 2 : P.niter;

  f32x16 acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[a][b] = f32x16{};

  // an operand whose K runs along a row: thread t takes row t / 2, 8 values
  // from k = 8 (t % 2); across rows: k = t / 16, 8 values from column 8 (t % 16)
  const int rk = tid >> 1, kk = (tid & 1) * 8;
  const int ck = tid >> 4, cc = (tid & 15) * 8;
  for (int it = it0; it < it1; ++it) {
    const int seg = Mode == kFfnDx && it >= per_seg;
    const int64_t k0 = (int64_t)(it - seg * per_seg) * kFfnStep;
    float va[8], vb[8];
    if constexpr (Mode == kFfnDw) {
      const T* p = static_cast<const T*>(P.a) + (k0 + ck) * P.lda + i0 + cc;
#pragma unroll
      for (int j = 0; j < 8; ++j) va[j] = (k0 + ck < P.K && i0 + cc + j < P.M) ? to_f32(p[j]) : 0.0f;
    } else {
      const T* p = static_cast<const T*>(P.a) + (i0 + rk) * P.lda + seg * P.fp + k0 + kk;
#pragma unroll
      for (int j = 0; j < 8; ++j) va[j] = (i0 + rk < P.M && k0 + kk + j < P.K) ? to_f32(p[j]) : 0.0f;
    }
    if constexpr (Mode == kFfnFwd) {
      int up, col;
      fwd_column<kFfnEdge>(rk, up, col);
      const int64_t row = j0 + col;
      const T* p = static_cast<const T*>(up ? P.b1 : P.b0) + row * (up ? P.ldb1 : P.ldb0) + k0 + kk;
#pragma unroll
      for (int j = 0; j < 8; ++j) vb[j] = (row < P.N && k0 + kk + j < P.K) ? to_f32(p[j]) : 0.0f;
    } else {
      const T* p = static_cast<const T*>(seg ? P.b1 : P.b0) + (k0 + ck) * (seg ? P.ldb1 : P.ldb0) + j0 + cc;
#pragma unroll
      for (int j = 0; j < 8; ++j) vb[j] = (k0 + ck < P.K && j0 + cc + j < P.N) ? to_f32(p[j]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (Mode == kFfnDw) sA[ck][cc + j] = va[j];
      else sA[kk + j][rk] = va[j];
      if constexpr (Mode == kFfnFwd) sB[kk + j][rk] = vb[j];
      else sB[ck][cc + j] = vb[j];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kFfnStep; k += 2) {
      float a[2], b[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        a[q] = sA[k + (lane >> 5)][64 * wr + 32 * q + (lane & 31)];
        b[q] = sB[k + (lane >> 5)][64 * wc + 32 * q + (lane & 31)];
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int s = 0; s < 2; ++s) acc[q][s] = mfma32x32x2_f32(b[s], a[q], acc[q][s]);
    }
  }

  const int r0 = 64 * wr + (lane & 31), c0 = 4 * (lane >> 5);
  if (!whole) {
    float* W = P.ws + ((int64_t)part * tail + (t - P.full)) * (kFfnEdge * kFfnEdge);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<float4*>(W + (r0 + 32 * q) * kFfnEdge + 64 * wc + 32 * s + 8 * b + c0) =
              float4{acc[q][s][4 * b], acc[q][s][4 * b + 1], acc[q][s][4 * b + 2], acc[q][s][4 * b + 3]};
    return;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float v[2][4];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[s][j] = acc[q][s][4 * b + j];
      if constexpr (Mode == kFfnFwd) {
        put4_fwd<DT>(P, i0 + r0 + 32 * q, j0 + 32 * wc + 8 * b + c0, v[0], v[1]);
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
          put4<DT, Mode>(P, i0 + r0 + 32 * q, j0 + 64 * wc + 32 * s + 8 * b + c0, v[s]);
      }
    }
}

// Split tiles: the parts' sums added in part order, then the epilogue.  Block
// (t, s) handles rows s * (1024 / Edge) .. of tile full + t; a thread takes
// four columns (forward: of both projections).
template <int DT, int Mode, int Edge> __global__ void __launch_bounds__(256) ffn_join(FfnGemm P) {
  const int tail = P.ntiles - P.full, t = blockIdx.x;
  int I, J;
  tile_coords(P, P.full + t, I, J);
  constexpr int kQuads = Mode == kFfnFwd ? Edge / 8 : Edge / 4;  // quads of columns per row
  const int id = blockIdx.y * 256 + threadIdx.x;
  const int row = id / kQuads, quad = id % kQuads;
  const float* W = P.ws + (int64_t)t * (Edge * Edge) + row * Edge;
  const int64_t stride = (int64_t)tail * (Edge * Edge);
  if constexpr (Mode == kFfnFwd) {
    constexpr int per = Edge / 16;  // quads per wave column and projection
    const int w = quad / per, q = quad % per;
    const int cg = w * (Edge / 2) + 4 * q;
    float g[4] = {}, u[4] = {};
    for (int p = 0; p < P.parts; ++p) {
      const float4 a = *reinterpret_cast<const float4*>(W + p * stride + cg);
      const float4 b = *reinterpret_cast<const float4*>(W + p * stride + cg + Edge / 4);
      g[0] += a.x, g[1] += a.y, g[2] += a.z, g[3] += a.w;
      u[0] += b.x, u[1] += b.y, u[2] += b.z, u[3] += b.w;
    }
    put4_fwd<DT>(P, (int64_t)I * Edge + row, (int64_t)J * (Edge / 2) + w * (Edge / 4) + 4 * q, g, u);
  } else {
    float v[4] = {};
    for (int p = 0; p < P.parts; ++p) {
      const float4 a = *reinterpret_cast<const float4*>(W + p * stride + 4 * quad);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    }
    put4<DT, Mode>(P, (int64_t)I * Edge + row, (int64_t)J * Edge + 4 * quad, v);
  }
}

// dg, du from dh and the saved pair, 8 columns a thread.
template <int DT, bool Vec>
__global__ void __launch_bounds__(256) ffn_dgu(const typename Elem<DT>::type* dh, int64_t lddh,
                                               const typename Elem<DT>::type* pre, typename Elem<DT>::type* out,
                                               int64_t f, int64_t fp, int act) {
  typedef typename Elem<DT>::type T;
  typedef T T8 __attribute__((ext_vector_type(8)));
  const int64_t row = blockIdx.y;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= fp) return;
  const T* q = pre + row * 2 * fp + c;
  const T8 g8 = *reinterpret_cast<const T8*>(q), u8 = *reinterpret_cast<const T8*>(q + fp);
  T8 h8;
  const T* hp = dh + row * lddh + c;
  if (Vec && c + 8 <= f) {
    h8 = *reinterpret_cast<const T8*>(hp);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) h8[j] = c + j < f ? hp[j] : (T)0.0f;
  }
  T8 dg, du;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float a, da;
    act_both<DT == kInF32>(to_f32(g8[j]), act, a, da);
    const float h = to_f32(h8[j]);
    dg[j] = c + j < f ? from_f32<T>(h * to_f32(u8[j]) * da) : (T)0.0f;
    du[j] = c + j < f ? from_f32<T>(h * a) : (T)0.0f;
  }
  T* o = out + row * 2 * fp + c;
  *reinterpret_cast<T8*>(o) = dg;
  *reinterpret_cast<T8*>(o + fp) = du;
}

template <class T> __global__ void __launch_bounds__(256) zero_rows(T* p, int64_t ld, int64_t cols, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256)
    p[i / cols * ld + i % cols] = T(0);
}

template <int DT, int Mode> hipError_t launch_mode(const FfnGemm& g, hipStream_t stream) {
  const int tail = g.ntiles - g.full;
  ffn_f32_tile<DT, Mode><<<g.full + tail * g.parts, 256, 0, stream>>>(g);
  if (tail > 0) {
    constexpr int quads = Mode == kFfnFwd ? kFfnEdge / 8 : kFfnEdge / 4;
    ffn_join<DT, Mode, kFfnEdge><<<dim3(tail, kFfnEdge * quads / 256), 256, 0, stream>>>(g);
  }
  return hipGetLastError();
}

template <int DT> hipError_t launch_dtype(const FfnGemm& g, int mode, hipStream_t stream) {
  if (mode == kFfnFwd) return launch_mode<DT, kFfnFwd>(g, stream);
  if (mode == kFfnDx) return launch_mode<DT, kFfnDx>(g, stream);
  return launch_mode<DT, kFfnDw>(g, stream);
}

template <int DT>
hipError_t dgu_dtype(const void* dh, int64_t lddh, const void* preact, void* dgu, int64_t n, int64_t f, int64_t fp,
                     int act, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const bool vec = ((reinterpret_cast<uintptr_t>(dh) | (uint64_t)(lddh * sizeof(T))) & 15u) == 0;
  const unsigned gx = (unsigned)((fp / 8 + 255) / 256);
  // a grid has at most 65,535 rows
  for (int64_t r0 = 0; r0 < n; r0 += 65535) {
    const unsigned rows = (unsigned)std::min<int64_t>(65535, n - r0);
    const T* d = static_cast<const T*>(dh) + r0 * lddh;
    const T* p = static_cast<const T*>(preact) + r0 * 2 * fp;
    T* o = static_cast<T*>(dgu) + r0 * 2 * fp;
    if (vec) ffn_dgu<DT, true><<<dim3(gx, rows), 256, 0, stream>>>(d, lddh, p, o, f, fp, act);
    else ffn_dgu<DT, false><<<dim3(gx, rows), 256, 0, stream>>>(d, lddh, p, o, f, fp, act);
  }
  return hipGetLastError();
}

}  // namespace

void ffn_schedule(FfnGemm& g, int mode, int edge, int step, int max_slots) {
  constexpr int kCUs = 256;
  const int cols = mode == kFfnFwd ? edge / 2 : edge;
  g.tm = (int)((g.M + edge - 1) / edge);
  g.tn = (int)((g.N + cols - 1) / cols);
  g.ntiles = g.tm * g.tn;
  const int per_seg = (int)((g.K + step - 1) / step);
  g.niter = mode == kFfnDx ? 2 * per_seg : per_seg;
  // whole tiles fill complete rounds of one workgroup per CU; the tiles of a
  // last, partly empty round are cut along K, as long as a part keeps at
  // least 256 values of K
  g.full = g.ntiles;
  g.parts = 1;
  g.part_len = g.niter;
  const int tail = g.ntiles % kCUs;
  if (tail > 0) {
    int parts = std::min(kCUs / tail, max_slots / tail);
    parts = std::min(parts, g.niter / std::max(1, 256 / step));
    if (parts >= 2) {
      g.part_len = (g.niter + parts - 1) / parts;
      g.parts = (g.niter + g.part_len - 1) / g.part_len;
      g.full = g.ntiles - tail;
    }
  }
}

hipError_t launch_ffn_gemm(const FfnGemm& g, int mode, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) return launch_dtype<kInBF16>(g, mode, stream);
  if (dtype == kInF16) return launch_dtype<kInF16>(g, mode, stream);
  return launch_dtype<kInF32>(g, mode, stream);
}

hipError_t launch_ffn_dgu(const void* dh, int64_t lddh, const void* preact, void* dgu, int64_t n, int64_t f,
                          int64_t fp, int act, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) return dgu_dtype<kInBF16>(dh, lddh, preact, dgu, n, f, fp, act, stream);
  if (dtype == kInF16) return dgu_dtype<kInF16>(dh, lddh, preact, dgu, n, f, fp, act, stream);
  return dgu_dtype<kInF32>(dh, lddh, preact, dgu, n, f, fp, act, stream);
}

hipError_t launch_zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int esize, hipStream_t stream) {
  const int64_t total = rows * cols;
  if (total == 0) return hipSuccess;
  const int grid = (int)std::min<int64_t>((total + 255) / 256, 4096);
  if (esize == 2) zero_rows<uint16_t><<<grid, 256, 0, stream>>>(static_cast<uint16_t*>(p), ld, cols, total);
  else zero_rows<uint32_t><<<grid, 256, 0, stream>>>(static_cast<uint32_t*>(p), ld, cols, total);
  return hipGetLastError();
}

}  // namespace hess
