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

// dg, du from dh and the saved pair (of PT), 8 columns a thread; dh's rows may
// start anywhere.  Bound by its bytes (bf16, 8192 x 11264: 175 us with the pair
// in bf16, 5.3 TB/s, and 250 us with it in float32).
//
// Roundings: dg and du are rounded to the operands' type here, because the two
// products that follow take matrix instructions of that type; with the
// gradients' own last rounding that is an error of 1.4 times the last
// rounding alone (1.8 times where the pair was kept in a 16-bit type too).
// Without it the products would need a second 16-bit term of dg and du, twice
// the matrix work of the backward pass.
template <int DT, class PT>
__global__ void __launch_bounds__(256) ffn_dgu(const typename Elem<DT>::type* dh, int64_t lddh, const PT* pre,
                                               typename Elem<DT>::type* out, int64_t f, int64_t fp, int act) {
  typedef typename Elem<DT>::type T;
  typedef T T8 __attribute__((ext_vector_type(8)));
  typedef T8 T8u __attribute__((aligned(sizeof(T))));
  typedef PT P8 __attribute__((ext_vector_type(8)));
  const int64_t row = blockIdx.y;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= fp) return;
  const PT* q = pre + row * 2 * fp + c;
  const P8 g8 = *reinterpret_cast<const P8*>(q), u8 = *reinterpret_cast<const P8*>(q + fp);
  T8 h8;
  const T* hp = dh + row * lddh + c;
  if (c + 8 <= f) {
    h8 = *reinterpret_cast<const T8u*>(hp);
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

template <int DT, class PT>
hipError_t launch_dgu(const void* dh, int64_t lddh, const void* preact, void* dgu, int64_t n, int64_t f, int64_t fp,
                      int act, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const unsigned gx = (unsigned)((fp / 8 + 255) / 256);
  // a grid has at most 65,535 rows
  for (int64_t r0 = 0; r0 < n; r0 += 65535) {
    const unsigned rows = (unsigned)std::min<int64_t>(65535, n - r0);
    ffn_dgu<DT, PT><<<dim3(gx, rows), 256, 0, stream>>>(static_cast<const T*>(dh) + r0 * lddh, lddh,
                                                        static_cast<const PT*>(preact) + r0 * 2 * fp,
                                                        static_cast<T*>(dgu) + r0 * 2 * fp, f, fp, act);
  }
  return hipGetLastError();
}

}  // namespace

namespace {

// Places for workgroups on the card: a CU holds one of edge 256, two of edge
// 128, four of edge 64.
int slots_of(int edge) { return edge == 256 ? 256 : edge == 128 ? 512 : 1024; }

// What `groups` workgroups at once, at most one for each place, take per stage
// of K (us), from products timed at 64 .. 8192 tokens.  Float32 is bound by
// the matrix cores; 16-bit products of edge 256 are slowed by the card's power
// as it fills (0.50 us alone, 0.83 us on all CUs), and smaller edges reach
// 0.7 (128) and 0.4 (64) of its rate, but divide the work more evenly over the
// CUs: 300 tokens at 704 x 1000, bf16, take 7.7 us with edge 64, 11.5 with 128
// and 23 with 256; 1999 at 2560 x 9728 take 395, 232 and 187 (operands in the
// last-level cache; 209 with cold ones).
double stage_us(int edge, int groups, bool f32, int mode) {
  const int each = (groups + 255) / 256;  // on the busiest CU
  if (edge == 256) return f32 ? 3.7 : 0.50 + 0.33 * groups / 256;
  if (edge == 128) return f32 ? (each == 1 ? 1.03 : 0.97 * each) : (each > 1 ? 0.31 * each : mode == kFfnFwd ? 0.27 : 0.33);
  return f32 ? std::max(0.35, 0.27 * each) : std::max(0.20, 0.135 * each);
}

// The schedule for tiles of one edge, and its estimated time in us.
double schedule_for(FfnGemm& g, int mode, int edge, bool f32) {
  const int step = f32 ? 16 : 32, slots = slots_of(edge);
  const int cols = mode == kFfnFwd ? edge / 2 : edge;
  g.tm = (int)((g.M + edge - 1) / edge);
  g.tn = (int)((g.N + cols - 1) / cols);
  g.ntiles = g.tm * g.tn;
  const int per_seg = (int)((g.K + step - 1) / step);
  g.niter = mode == kFfnDx ? 2 * per_seg : per_seg;
  g.full = g.ntiles;
  g.parts = 1;
  g.part_len = g.niter;
  // whole tiles fill complete rounds of the card; the tiles of a last, partly
  // empty round may be cut along K into parts of at least 256 values, whose
  // sums go through the last-level cache (written and read at 12 TB/s) and a
  // second launch
  const double enter = edge == 256 ? 8.0 : 4.0, join = 3.0;
  const int tail = g.ntiles % slots;
  double us = (double)(g.ntiles / slots) * (g.niter * stage_us(edge, slots, f32, mode) + enter);
  if (tail == 0) return us;
  double best = 1e30;
  for (int parts = 1; parts <= std::max(1, std::min(2 * slots / tail, g.niter / (256 / step))); ++parts) {
    const int len = (g.niter + parts - 1) / parts, work = tail * parts;
    double t = work / slots * (len * stage_us(edge, slots, f32, mode) + enter);
    if (work % slots > 0) t += len * stage_us(edge, work % slots, f32, mode) + enter;
    if (parts > 1) t += join + (double)work * edge * edge * 8.0 / 12e6;
    if (t >= best) continue;
    best = t;
    if (parts > 1) {
      g.part_len = len;
      g.parts = (g.niter + len - 1) / len;
      g.full = g.ntiles - tail;
    }
  }
  return us + best;
}

}  // namespace

namespace {
FfnForced g_forced{0, 0, 1};
}
void ffn_force_schedule(FfnForced f) { g_forced = f; }

int ffn_schedule(FfnGemm& g, int mode, int dtype) {
  const FfnForced forced = g_forced;
  if (forced.edge != 0) {
    schedule_for(g, mode, forced.edge, dtype == kInF32);
    g.part_len = (g.niter + forced.parts - 1) / forced.parts;
    g.parts = (g.niter + g.part_len - 1) / g.part_len;
    // (the tiles cut along K are at most as many as the estimate would cut)
    g.full = g.parts == 1 ? g.ntiles : std::max(std::min(forced.whole, g.ntiles), g.ntiles - 1024);
    return forced.edge;
  }
  int edge = 0;
  double least = 1e30;
  FfnGemm chosen{};
  for (int e : {256, 128, 64}) {
    FfnGemm s = g;
    const double us = schedule_for(s, mode, e, dtype == kInF32);
    if (us >= least) continue;
    least = us;
    edge = e;
    chosen = s;
  }
  g = chosen;
  return edge;
}

hipError_t launch_ffn_dgu(const void* dh, int64_t lddh, const void* preact, bool pre32, void* dgu, int64_t n,
                          int64_t f, int64_t fp, int act, int dtype, hipStream_t stream) {
  if (dtype == kInF32) return launch_dgu<kInF32, float>(dh, lddh, preact, dgu, n, f, fp, act, stream);
  if (dtype == kInBF16)
    return pre32 ? launch_dgu<kInBF16, float>(dh, lddh, preact, dgu, n, f, fp, act, stream)
                 : launch_dgu<kInBF16, __bf16>(dh, lddh, preact, dgu, n, f, fp, act, stream);
  return pre32 ? launch_dgu<kInF16, float>(dh, lddh, preact, dgu, n, f, fp, act, stream)
               : launch_dgu<kInF16, _Float16>(dh, lddh, preact, dgu, n, f, fp, act, stream);
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
