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

#include "ffn_device.hpp"
#include "hess_device.hpp"

namespace hess {

namespace {

// ---------------------------------------------------------------------------
// 128-tile kernel on the float32 matrix instruction.  4 waves, 64 x 64 each
// (2 x 2 blocks of v_mfma_f32_32x32x2_f32, B first, so that a lane holds four
// consecutive columns).  Operands are widened to float32 and staged k-major.
// ---------------------------------------------------------------------------

constexpr int kPad = 4;
constexpr int kLd = kFfnEdge32 + kPad;

template <int Mode> __global__ void __launch_bounds__(256) ffn_f32_tile(FfnGemm P) {
  constexpr int DT = kInF32;
  typedef float T;
  __shared__ float sA[kFfnStep32][kLd];
  __shared__ float sB[kFfnStep32][kLd];
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
  const int64_t i0 = (int64_t)I * kFfnEdge32;
  const int64_t j0 = (int64_t)J * (Mode == kFfnFwd ? kFfnEdge32 / 2 : kFfnEdge32);
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
    const int64_t k0 = (int64_t)(it - seg * per_seg) * kFfnStep32;
    float va[8], vb[8];
    if constexpr (Mode == kFfnDw) {
      const T* p = static_cast<const T*>(P.a) + (k0 + ck) * P.lda + i0 + cc;
#pragma unroll
      for (int j = 0; j < 8; ++j) va[j] = (k0 + ck < P.K && i0 + cc + j < P.M) ? p[j] : 0.0f;
    } else {
      const T* p = static_cast<const T*>(P.a) + (i0 + rk) * P.lda + seg * P.fp + k0 + kk;
#pragma unroll
      for (int j = 0; j < 8; ++j) va[j] = (i0 + rk < P.M && k0 + kk + j < P.K) ? p[j] : 0.0f;
    }
    if constexpr (Mode == kFfnFwd) {
      int up, col;
      fwd_column(rk, up, col);
      const int64_t row = j0 + col;
      const T* p = static_cast<const T*>(up ? P.b1 : P.b0) + row * (up ? P.ldb1 : P.ldb0) + k0 + kk;
#pragma unroll
      for (int j = 0; j < 8; ++j) vb[j] = (row < P.N && k0 + kk + j < P.K) ? p[j] : 0.0f;
    } else {
      const T* p = static_cast<const T*>(seg ? P.b1 : P.b0) + (k0 + ck) * (seg ? P.ldb1 : P.ldb0) + j0 + cc;
#pragma unroll
      for (int j = 0; j < 8; ++j) vb[j] = (k0 + ck < P.K && j0 + cc + j < P.N) ? p[j] : 0.0f;
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
    for (int k = 0; k < kFfnStep32; k += 2) {
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
    float* W = P.ws + ((int64_t)part * tail + (t - P.full)) * (kFfnEdge32 * kFfnEdge32);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<float4*>(W + (r0 + 32 * q) * kFfnEdge32 + 64 * wc + 32 * s + 8 * b + c0) =
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
        put_fwd<DT>(P, i0 + r0 + 32 * q, j0 + 32 * wc + 8 * b + c0, v[0], v[1]);
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
          put<DT, Mode>(P, i0 + r0 + 32 * q, j0 + 64 * wc + 32 * s + 8 * b + c0, v[s]);
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
    const int w = quad >> 3, q = quad & 7;  // wave column, quad of its features
    const int cg = w * 64 + 4 * q;
    float g[4] = {}, u[4] = {};
    for (int p = 0; p < P.parts; ++p) {
      const float4 a = *reinterpret_cast<const float4*>(W + p * stride + cg);
      const float4 b = *reinterpret_cast<const float4*>(W + p * stride + cg + 32);
      g[0] += a.x, g[1] += a.y, g[2] += a.z, g[3] += a.w;
      u[0] += b.x, u[1] += b.y, u[2] += b.z, u[3] += b.w;
    }
    put_fwd<DT>(P, (int64_t)I * Edge + row, (int64_t)J * (Edge / 2) + w * 32 + 4 * q, g, u);
  } else {
    float v[4] = {};
    for (int p = 0; p < P.parts; ++p) {
      const float4 a = *reinterpret_cast<const float4*>(W + p * stride + 4 * quad);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    }
    put<DT, Mode>(P, (int64_t)I * Edge + row, (int64_t)J * Edge + 4 * quad, v);
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

template <int DT, int Mode, int Edge> void launch_join(const FfnGemm& g, hipStream_t stream) {
  constexpr int quads = Mode == kFfnFwd ? Edge / 8 : Edge / 4;
  ffn_join<DT, Mode, Edge><<<dim3(g.ntiles - g.full, Edge * quads / 256), 256, 0, stream>>>(g);
}

template <int DT, int Mode> void launch_joins(const FfnGemm& g, int edge, hipStream_t stream) {
  if (g.full == g.ntiles) return;
  if constexpr (DT != kInF32) {
    if (edge == 256) return launch_join<DT, Mode, 256>(g, stream);
  }
  launch_join<DT, Mode, 128>(g, stream);
}

template <int DT> hipError_t launch_type(const FfnGemm& g, int mode, int edge, hipStream_t stream) {
  if constexpr (DT == kInF32) {
    const int grid = g.full + (g.ntiles - g.full) * g.parts;
    if (mode == kFfnFwd) ffn_f32_tile<kFfnFwd><<<grid, 256, 0, stream>>>(g);
    else if (mode == kFfnDx) ffn_f32_tile<kFfnDx><<<grid, 256, 0, stream>>>(g);
    else ffn_f32_tile<kFfnDw><<<grid, 256, 0, stream>>>(g);
  } else {
    const hipError_t e = launch_ffn_tile16(g, mode, edge, DT, stream);
    if (e != hipSuccess) return e;
  }
  if (mode == kFfnFwd) launch_joins<DT, kFfnFwd>(g, edge, stream);
  else if (mode == kFfnDx) launch_joins<DT, kFfnDx>(g, edge, stream);
  else launch_joins<DT, kFfnDw>(g, edge, stream);
  return hipGetLastError();
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

namespace {

void schedule_for(FfnGemm& g, int mode, int edge, int step, int slots) {
  const int cols = mode == kFfnFwd ? edge / 2 : edge;
  g.tm = (int)((g.M + edge - 1) / edge);
  g.tn = (int)((g.N + cols - 1) / cols);
  g.ntiles = g.tm * g.tn;
  const int per_seg = (int)((g.K + step - 1) / step);
  g.niter = mode == kFfnDx ? 2 * per_seg : per_seg;
  // whole tiles fill complete rounds of the card's slots; the tiles of a
  // last, partly empty round are cut along K, as long as a part keeps at
  // least 256 values of K
  g.full = g.ntiles;
  g.parts = 1;
  g.part_len = g.niter;
  const int tail = g.ntiles % slots;
  if (tail > 0) {
    const int parts = std::min(slots / tail, g.niter / (256 / step));
    if (parts >= 2) {
      g.part_len = (g.niter + parts - 1) / parts;
      g.parts = (g.niter + g.part_len - 1) / g.part_len;
      g.full = g.ntiles - tail;
    }
  }
}

}  // namespace

int ffn_schedule(FfnGemm& g, int mode, int dtype) {
  constexpr int kCUs = 256;
  if (dtype == kInF32) {
    schedule_for(g, mode, kFfnEdge32, kFfnStep32, kCUs);
    return kFfnEdge32;
  }
  schedule_for(g, mode, 256, kFfnStep16, kCUs);
  if (g.ntiles >= kCUs / 2) return 256;
  schedule_for(g, mode, 128, kFfnStep16, 2 * kCUs);
  return 128;
}

hipError_t launch_ffn_gemm(const FfnGemm& g, int mode, int edge, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) return launch_type<kInBF16>(g, mode, edge, stream);
  if (dtype == kInF16) return launch_type<kInF16>(g, mode, edge, stream);
  return launch_type<kInF32>(g, mode, edge, stream);
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
