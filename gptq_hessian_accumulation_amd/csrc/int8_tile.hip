// The product of int8 rows by tiles of edge 256, 128 or 64 with int32
// accumulators, on v_mfma_i32_16x16x64_i8.  A stage is 128 bytes of K, taken in
// two halves.
//
//  * 8 waves of 128 x 64 (edge 256) or 4 of 64 x 64 (edge 128) or 32 x 32 (edge
//    64); two waves share each SIMD (edge 128: two workgroups a CU; edge 64:
//    four).  The B operand goes first, so that a lane holds four consecutive
//    columns; two neighbouring blocks are exchanged between lane rows before
//    they are stored (eight columns, one 16-byte store).
//  * Both operands go from memory straight into LDS, whole 128-byte lines of a
//    row at a time (64 bytes ask L2 for twice the requests, 96 million instead
//    of 52 million at 16384 x 4096 x 11264).  A unit is one operand's share of a
//    stage; LDS holds five: those being multiplied, those of the next stage, and A
//    of the one after, so that a stage's loads are 1 to 1.75 stages ahead.  Where
//    LDS has room for it, nine units hold four stages.
//  * The waves meet once a stage.  Rows are kept 128 bytes each, their 16-byte
//    chunks XOR-swizzled by bits 1-3 of the row, and read with ds_read_b128 free of
//    bank conflicts.
//  * Rows past the matrix and chunks of K past it get an offset past every
//    descriptor's range and read as zeros.  Inside the last 16-byte chunk of K
//    the codes of A past K are zeros in memory, whatever those of B are.
//  * Sums are exact, so that a split along K and its order change nothing.
//
// Measured (bf16 outputs; the clock, and with it long products, varies by a tenth
// from card to card): 16384 x 4096 x 11264 590 to 640 us, 2.4 to 2.6 POPS (a
// library product of that size without scales 821 us, 1.84), 8192 x 8192 x 8192
// 404 us, 2.7 POPS (library 477).  Matrix cores busy in 65% of the cycles at a
// clock of 1.8 to 1.9 GHz, LDS in a quarter of them: the rest is the waves' meeting
// and the reads behind it.  With stages of 64 bytes, a meeting each, and loads three
// of them ahead: 643 us against 603 for the first in one trace, 55% busy; 1999 x
// 2560 x 9728 (edge 128), with the quantization of its rows, 68 us against 57 to 60
// (53 to 54 without).  Small products are bound by a launch's first loads and
// outputs: 300 x 704 x 1000 6 us.

#include <algorithm>
#include <type_traits>

#include "ffn_device.hpp"
#include "int8_device.hpp"
#include "int8_internal.hpp"

namespace hess {

namespace {

constexpr uint32_t kOOB = 0x80000000u;  // an offset past any descriptor's range
constexpr int64_t kAll = 0x7fffffff;

__device__ __forceinline__ i32x4 mma_i8(const u32x4& a, const u32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Tile t: groups of 8 tile rows, column by column inside a group.
__device__ __forceinline__ void coords(const Int8Gemm& P, int t, int& I, int& J) {
  const int per = 8 * P.tn, grp = t / per;
  const int rows = min(8, P.tm - grp * 8), in = t - grp * per;
  J = in / rows;
  I = grp * 8 + in - J * rows;
}

template <int DT, int Edge, int kUnits>
__global__ void __launch_bounds__(Edge == 256 ? 512 : 256, kUnits > 5 ? 1 : Edge == 64 ? 4 : 2) int8_tile(Int8Gemm P) {
  constexpr int kAhead = (kUnits - 1) / 2;          // stages that are loaded ahead
  constexpr int kColWaves = Edge == 256 ? 4 : 2;    // the tile's waves are 2 x kColWaves
  constexpr int kCols = Edge / kColWaves;           // columns of a wave
  constexpr int kBm = Edge / 32, kBn = kCols / 16;  // 16-wide blocks of a wave
  constexpr int kUnit = Edge * 128;
  constexpr int kLoads = kUnit / 1024 / (2 * kColWaves);  // 1-KB loads per wave and unit
  __shared__ __attribute__((aligned(1024))) char lds[kUnits * kUnit];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / kColWaves, wc = wave % kColWaves;
  const uint32_t lds0 = (uint32_t) reinterpret_cast<uintptr_t>((HESS_LDS char*)lds);

  // the whole tiles and the parts are dealt to the XCDs separately, so that
  // each has its share of either
  const int block = blockIdx.x;
  const int item = block < P.full ? item_of_block(block, P.full)
                                  : P.full + item_of_block(block - P.full, (int)gridDim.x - P.full);
  const int tail = P.ntiles - P.full;
  int t = item, part = 0;
  const bool whole = item < P.full;
  if (!whole) {
    part = (item - P.full) / tail;
    t = P.full + (item - P.full) % tail;
  }
  const int it0 = __builtin_amdgcn_readfirstlane(whole ? 0 : part * P.part_len);
  const int it1 = __builtin_amdgcn_readfirstlane(whole ? P.niter : min(P.niter, it0 + P.part_len));
  int I, J;
  coords(P, t, I, J);
  const int64_t i0 = (int64_t)I * Edge, j0 = (int64_t)J * Edge;

  // Offsets of this wave's loads: load i of a unit holds 8 rows, lane l row l / 8
  // of them and position l % 8, where chunk (l % 8) ^ (row / 2 % 8) lives.
  const int chunk = (lane & 7) ^ (lane >> 4);  // of even loads; of odd ones ^ 4
  uint32_t voffA[kLoads], voffB[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = 8 * (kLoads * wave + i) + (lane >> 3);
    const int c = chunk ^ (4 * (i & 1));  // (kLoads is even: so is kLoads * wave)
    voffA[i] = i0 + row < P.M ? (uint32_t)(row * P.lda + c * 16) : kOOB;
    voffB[i] = j0 + row < P.N ? (uint32_t)(row * P.ldb + c * 16) : kOOB;
  }
  const uint64_t baseA = reinterpret_cast<uint64_t>(P.a) + (uint64_t)(i0 * P.lda);
  const uint64_t baseB = reinterpret_cast<uint64_t>(P.b) + (uint64_t)(j0 * P.ldb);
  struct Next {
    u32x4 r;
    int lim;  // chunks of K left
  };
  auto describe = [&](uint64_t base, int j) {
    Next d;
    const int64_t k0 = (int64_t)j * 128;
    d.lim = (int)((P.K - k0 + 15) / 16);
    d.r = rsrc_words(base + (uint64_t)k0, j < it1 ? kAll : 0);
    return d;
  };
  // load i of the wave's kLoads of one unit
  auto load1 = [&](uint32_t unit, const Next& d, const uint32_t (&voff)[kLoads], int i) {
    const uint32_t off = (chunk ^ (4 * (i & 1))) < d.lim ? voff[i] : kOOB;
    lds_dma16(d.r, off, lds0 + unit + (uint32_t)((kLoads * wave + i) * 1024));
  };
  auto load_unit = [&](uint32_t unit, uint64_t base, const uint32_t (&voff)[kLoads], int j) {
    const Next d = describe(base, j);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load1(unit, d, voff, i);
  };

  // Operand block m of a wave's share: lane l holds row l % 16 of the block, chunk
  // l / 16 of the stage's half h (whose position differs in bit 2: 64 bytes).
  const int in_block = (lane & 15) * 128 + (((lane >> 4) ^ ((lane & 15) >> 1)) << 4);
  const int posA = wr * (Edge / 2) * 128 + in_block, posB = wc * kCols * 128 + in_block;
  auto read_a = [&](uint32_t unit, int h, int m) {
    return *reinterpret_cast<const u32x4*>(lds + unit + (posA ^ (64 * h)) + m * 2048);
  };
  auto read_b = [&](uint32_t unit, int h, int n) {
    return *reinterpret_cast<const u32x4*>(lds + unit + (posB ^ (64 * h)) + n * 2048);
  };

  i32x4 acc[kBm][kBn];
#pragma unroll
  for (int m = 0; m < kBm; ++m)
#pragma unroll
    for (int n = 0; n < kBn; ++n) acc[m][n] = i32x4{};

  // Stage j, half h, group by group: the matrix instructions of one A block, the
  // read of the A block kRot groups later (of the other half, or of the next stage,
  // at the end), reads of the following half's B (into c), and one load.  In half 0
  // the loads are of A of stage j + kAhead.  In half 1, once its last block of the
  // stage is read, the wave waits for its own loads of the next stage and meets the
  // others: the next stage is then complete and nobody reads this one, whose first
  // unit takes B of stage j + kAhead.
  constexpr int kRot = kBm < 4 ? kBm : 4;
  constexpr int kMeet = kBm - kRot;
  static_assert(kLoads <= kRot && kBn == kRot, "one load and one read of B in each of kRot groups");
  u32x4 a[kRot], b[kBn], c[kBn];
  uint32_t s0 = 0;  // the unit of A of this stage; those of B and of the next stages follow
  auto unit_at = [&](int k) {
    const uint32_t u = s0 + k * kUnit;
    return u >= kUnits * kUnit ? u - kUnits * kUnit : u;
  };

  // the scales of the lane's outputs, on their way before the first codes (rows and
  // columns past the matrix take its last one's)
  float sa[kBm], sb[kBn / 2][8];
#pragma unroll
  for (int m = 0; m < kBm; ++m) sa[m] = P.sa[min(i0 + wr * (Edge / 2) + (lane & 15) + 16 * m, P.M - 1)];
#pragma unroll
  for (int n = 0; n < kBn / 2; ++n)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      sb[n][j] = P.sb[min(j0 + wc * kCols + 16 * ((lane >> 4) & 1) + 8 * (lane >> 5) + 32 * n + j, P.N - 1)];

#pragma unroll
  for (int q = 0; q < kAhead; ++q) {
    load_unit(2 * q * kUnit, baseA, voffA, it0 + q);
    load_unit((2 * q + 1) * kUnit, baseB, voffB, it0 + q);
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(2 * kLoads * (kAhead - 1)));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int q = 0; q < kRot; ++q) a[q] = read_a(0, 0, q);
#pragma unroll
  for (int q = 0; q < kBn; ++q) b[q] = read_b(kUnit, 0, q);
  for (int j = it0; j < it1; ++j) {
    const uint32_t uB = unit_at(1), nA = unit_at(2), nB = unit_at(3), far = unit_at(kUnits - 1);
    {
      const Next d = describe(baseA, j + kAhead);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < kBm; ++m) {
#pragma unroll
        for (int n = 0; n < kBn; ++n) acc[m][n] = mma_i8(b[n], a[m % kRot], acc[m][n]);
        a[m % kRot] = m + kRot < kBm ? read_a(s0, 0, m + kRot) : read_a(s0, 1, m + kRot - kBm);
        if (m >= kMeet) c[m - kMeet] = read_b(uB, 1, m - kMeet);
        if (m < kLoads) load1(far, d, voffA, m);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    {
      const Next d = describe(baseB, j + kAhead);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < kBm; ++m) {
        if (m == kMeet) {
          // all loads but those of later stages than the next, and the wave's own reads
          __builtin_amdgcn_s_waitcnt(vm_wait((2 * kAhead - 3) * kLoads) & ~0x0f00);
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int n = 0; n < kBn; ++n) acc[m][n] = mma_i8(c[n], a[m % kRot], acc[m][n]);
        a[m % kRot] = m + kRot < kBm ? read_a(s0, 1, m + kRot) : read_a(nA, 0, m + kRot - kBm);
        if (m >= kMeet) {
          b[m - kMeet] = read_b(nB, 0, m - kMeet);
          if (m - kMeet < kLoads) load1(s0, d, voffB, m - kMeet);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    s0 = nA;
  }
  // the trailing loads write LDS: they end before the workgroup does
  __builtin_amdgcn_s_waitcnt(0x0070);
  __builtin_amdgcn_sched_barrier(0);

  if (!whole) {
    int* W = P.ws + ((int64_t)part * tail + (t - P.full)) * (Edge * Edge) +
             (wr * (Edge / 2) + (lane & 15)) * Edge + wc * kCols + 4 * (lane >> 4);
#pragma unroll
    for (int m = 0; m < kBm; ++m)
#pragma unroll
      for (int n = 0; n < kBn; ++n) *reinterpret_cast<i32x4*>(W + 16 * m * Edge + 16 * n) = acc[m][n];
    return;
  }
  // A tile's outputs.  Blocks n, n + 1: after exchanging the odd 16-lane rows of
  // the first with the even ones of the second, lane row g holds columns
  // 8 (g / 2) .. + 7 of block n + g % 2.
  typedef typename Elem<DT>::type T;
  int lv = lane;
  asm volatile("" : "+v"(lv));  // the offsets are computed here, not kept through the loop
  const int64_t c0 = j0 + wc * kCols + 16 * ((lv >> 4) & 1) + 8 * (lv >> 5);
#pragma unroll
  for (int m = 0; m < kBm; ++m) {
    const int64_t r = i0 + wr * (Edge / 2) + (lv & 15) + 16 * m;
    T* row = static_cast<T*>(P.y) + r * P.ldy;
#pragma unroll
    for (int n = 0; n < kBn; n += 2) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto s = __builtin_amdgcn_permlane16_swap((uint32_t)acc[m][n][j], (uint32_t)acc[m][n + 1][j], false, false);
        v[j] = scale_sum((int)s[0], sb[n / 2][j], sa[m]);
        v[4 + j] = scale_sum((int)s[1], sb[n / 2][4 + j], sa[m]);
      }
      const int64_t col = c0 + 16 * n;
      if (r < P.M && col < P.N) store_n(row + col, v, (int)min((int64_t)8, P.N - col));
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Split tiles: the parts' sums added, then the scales.  Block (t, s) handles
// rows s * (1024 / Edge) .. of tile full + t; a thread takes four columns.
template <int DT, int Edge> __global__ void __launch_bounds__(256) int8_join(Int8Gemm P) {
  typedef typename Elem<DT>::type T;
  const int tail = P.ntiles - P.full, t = blockIdx.x;
  int I, J;
  coords(P, P.full + t, I, J);
  constexpr int kQuads = Edge / 4;
  const int id = blockIdx.y * 256 + threadIdx.x, row = id / kQuads, quad = id % kQuads;
  const int64_t r = (int64_t)I * Edge + row, c = (int64_t)J * Edge + 4 * quad;
  if (r >= P.M || c >= P.N) return;
  const int* W = P.ws + (int64_t)t * (Edge * Edge) + row * Edge + 4 * quad;
  i32x4 s{};
  for (int p = 0; p < P.parts; ++p) s += *reinterpret_cast<const i32x4*>(W + (int64_t)p * tail * (Edge * Edge));
  const float sa = P.sa[r];
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = c + j < P.N ? scale_sum(s[j], P.sb[c + j], sa) : 0.0f;
  store_n(static_cast<T*>(P.y) + r * P.ldy + c, v, (int)min((int64_t)4, P.N - c));
}

// Up to one workgroup (edge 64: two) a CU: they are bound by the loads' latency,
// and LDS has room for four stages ahead instead of two.
template <int DT, int Edge> void launch_edge(const Int8Gemm& g, hipStream_t stream) {
  const int tail = g.ntiles - g.full, groups = g.full + tail * g.parts;
  constexpr int kDeep = Edge == 256 ? 5 : 9;
  if (groups <= (Edge == 64 ? 512 : 256))
    int8_tile<DT, Edge, kDeep><<<groups, Edge == 256 ? 512 : 256, 0, stream>>>(g);
  else
    int8_tile<DT, Edge, 5><<<groups, Edge == 256 ? 512 : 256, 0, stream>>>(g);
  if (tail > 0) int8_join<DT, Edge><<<dim3(tail, Edge * (Edge / 4) / 256), 256, 0, stream>>>(g);
}

template <int DT> void launch_type(const Int8Gemm& g, int edge, hipStream_t stream) {
  if (edge == 256) launch_edge<DT, 256>(g, stream);
  else if (edge == 128) launch_edge<DT, 128>(g, stream);
  else launch_edge<DT, 64>(g, stream);
}

// Places for workgroups on the card, and what `groups` workgroups at once take
// per stage of K (us), from products timed at 65 .. 16384 rows: us at 256 x 4096 x
// 4096 with edges 64 / 128 / 256 13.4 / 20.3 / 46.2, at 1999 x 2560 x 9728 99.7 /
// 68.3 / 71.7, at 8192 x 4096 x 11264 720 / 467 / 343.
int slots_of(int edge) { return edge == 256 ? 256 : edge == 128 ? 512 : 1024; }
double stage_us(int edge, int groups) {
  const int each = (groups + 255) / 256;  // on the busiest CU
  if (edge == 256) return 0.95 + 0.50 * groups / 256;
  if (edge == 128) return each > 1 ? 0.45 * each : 0.48 + 0.16 * groups / 256;
  return std::max(0.32, 0.165 * each);
}

// The schedule for tiles of one edge, and its estimated time in us: whole tiles
// fill complete rounds of the card, the tiles of a last, partly empty round may
// be cut along K.
double schedule_for(Int8Gemm& g, int edge) {
  const int slots = slots_of(edge);
  g.tm = (int)((g.M + edge - 1) / edge);
  g.tn = (int)((g.N + edge - 1) / edge);
  g.ntiles = g.tm * g.tn;
  g.niter = (int)((g.K + 127) / 128);
  g.full = g.ntiles;
  g.parts = 1;
  g.part_len = g.niter;
  const double enter = edge == 256 ? 8.0 : 4.0, join = 6.0;
  const int tail = g.ntiles % slots;
  double us = (double)(g.ntiles / slots) * (g.niter * stage_us(edge, slots) + enter);
  if (tail == 0) return us;
  double best = 1e30;
  for (int parts = 1; parts <= std::max(1, std::min(2 * slots / tail, g.niter / 2)); ++parts) {
    const int len = (g.niter + parts - 1) / parts, work = tail * parts;
    double t = work / slots * (len * stage_us(edge, slots) + enter);
    if (work % slots > 0) t += len * stage_us(edge, work % slots) + enter;
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

int int8_schedule(Int8Gemm& g) {
  const FfnForced forced = ffn_forced();
  if (forced.edge != 0) {
    schedule_for(g, forced.edge);
    g.part_len = (g.niter + forced.parts - 1) / forced.parts;
    g.parts = (g.niter + g.part_len - 1) / g.part_len;
    // (the tiles cut along K are at most as many as the estimate would cut)
    g.full = g.parts == 1 ? g.ntiles : std::max(std::min(forced.whole, g.ntiles), g.ntiles - 1024);
    return forced.edge;
  }
  int edge = 0;
  double least = 1e30;
  Int8Gemm chosen{};
  for (int e : {256, 128, 64}) {
    Int8Gemm s = g;
    const double us = schedule_for(s, e);
    if (us >= least) continue;
    least = us;
    edge = e;
    chosen = s;
  }
  g = chosen;
  return edge;
}

hipError_t launch_int8_tile(const Int8Gemm& g, int edge, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) launch_type<kInBF16>(g, edge, stream);
  else if (dtype == kInF16) launch_type<kInF16>(g, edge, stream);
  else launch_type<kInF32>(g, edge, stream);
  return hipGetLastError();
}

}  // namespace hess
