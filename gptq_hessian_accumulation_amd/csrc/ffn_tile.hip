// The gated feed-forward block's products: tiles of edge 256, 128 or 64 with
// float32 accumulators, on v_mfma_f32_16x16x32 (bf16 or fp16) or, for float32
// operands, v_mfma_f32_16x16x4_f32.  A stage is 64 bytes of K: 32 values of a
// 16-bit type, 16 of float32.
//
//  * 8 waves of 128 x 64 (edge 256) or 4 of 64 x 64 (edge 128) or 32 x 32
//    (edge 64, for small products), one matrix instruction (float32: four)
//    per 16 x 16 accumulator and stage.  Two waves share each SIMD (edge 128:
//    two workgroups a CU; edge 64: four), so that one's waits are covered by
//    the other's matrix instructions.  The B
//    operand goes first, so that a lane holds four consecutive columns; two
//    neighbouring blocks are exchanged between lane rows before they are
//    stored, which makes eight (one 16-byte store).
//  * Operands go from memory straight into LDS, five stages deep: the loads
//    of four iterations are in flight while one is multiplied, with one
//    barrier an iteration and hand-placed loads and operand reads among the
//    matrix instructions (the pipeline of the 256-tile Gram kernel).
//  * An operand whose rows run along K (x and the weights forward, the
//    gradient pair for dx) is kept row by row, 64 bytes a row, its 16-byte
//    chunks XOR-swizzled by bits 1-2 of the row, and read with ds_read_b128.
//    One whose rows run across K (the weights for dx, both operands of dW)
//    is kept k by k and read transposed with ds_read_b64_tr_b16 (float32:
//    value by value).
//  * Loads need no masks: rows and columns past the matrix get an offset past
//    every descriptor's range, k past the matrix or past the part of K a
//    workgroup was given lies outside the descriptor (or its chunk's offset
//    does), and all of these read as zeros.
//
// Measured (bf16 unless said; the card's clock, and with it every long product,
// varies by a tenth from card to card and over the first passes): forward of
// 16384 tokens at 4096 x 11264 2.34 to 2.43 ms, 1.24 to 1.29 PFLOP/s, with the
// activation (a library product of the same size alone: 1.44); 8192 tokens, dx
// 1.17 to 1.26 ms and dW 1.12 to 1.21 ms (library products 1.27 and 1.54);
// float32, 2000 x 2560 x 4000, 136 TFLOP/s of the 137 a large library product
// reaches.  16-bit products are bound by the card's
// power and the meetings of the waves: the matrix cores are busy in 64% of the
// cycles, at a clock that falls to 1.6 GHz; LDS is free of bank conflicts and
// busy in a quarter of them.  Small products are bound by a launch's fixed 4 to
// 8 us (first loads, outputs).  Slower here: 4 waves of 128 x 128 (the outputs
// of one wave a SIMD take 15 us a tile instead of 8), two groups of waves
// taking turns at multiplying and reading (two barriers a stage), workgroups
// that stay and load the next tile's first stages early.

#include <type_traits>

#include "ffn_device.hpp"
#include "hess_device.hpp"

namespace hess {

namespace {

constexpr uint32_t kOOB = 0x80000000u;  // an offset past any descriptor's range
constexpr int64_t kAll = 0x7fffffff;
constexpr int kStages = 5, kAhead = 4;

template <int DT, int Mode, int Edge>
__global__ void __launch_bounds__(Edge == 256 ? 512 : 256, Edge == 64 ? 4 : 2) ffn_tile(FfnGemm P) {
  constexpr bool kRowsA = Mode != kFfnDw;  // A's rows run along K
  constexpr bool kRowsB = Mode == kFfnFwd;
  constexpr int kColWaves = Edge == 256 ? 4 : 2;  // the tile's waves are 2 x kColWaves
  constexpr int kCols = Edge / kColWaves;         // columns of a wave
  constexpr int kBm = Edge / 32, kBn = kCols / 16;  // 16-wide blocks of a wave
  constexpr int kSize = Elem<DT>::size;
  constexpr int kStep = 64 / kSize, kPiece = 16 / kSize;  // values of K in a stage and a 16-byte chunk
  constexpr int kPanel = Edge * 64;
  constexpr int kStage = 2 * kPanel;
  constexpr int kLoads = kPanel / 1024 / (2 * kColWaves);  // 1-KB loads per wave, panel and stage
  constexpr int kRow = Edge * kSize;           // bytes of one k of a panel kept k by k
  constexpr int kPerK = 1024 / kRow;       // k's in one load of such a panel
  __shared__ __attribute__((aligned(1024))) char lds[kStages * kStage];
  // place of a chunk of columns in row k of a panel kept k by k; float32: the
  // lane rows of a read (k = 4 g + j) land in four 64-byte parts of the banks
  // (a 16-bit row of edge 64 has 8 chunks, the others 16 or more)
  auto place = [](int k, int c) {
    return kSize == 4 ? c ^ (4 * ((k >> 2) & 3)) : Edge == 64 ? c ^ (2 * (k & 3)) : chunk_pos(k, c);
  };

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
  tile_coords<Mode>(P, t, I, J);
  const int64_t i0 = (int64_t)I * Edge;
  const int64_t j0 = (int64_t)J * (Mode == kFfnFwd ? Edge / 2 : Edge);
  const int per_seg = Mode == kFfnDx ? P.niter / 2 : P.niter;
  const int64_t rowA = P.lda * kSize, rowB = P.ldb0 * kSize;

  // Offsets of this wave's loads.  Along K: load i holds 16 rows, lane l row
  // l / 4 of them and position l % 4, where chunk (l % 4) ^ (row / 2 % 4)
  // lives.  Across K: load i holds kPerK values of k, the lane a chunk of
  // columns of one of them.
  const int chunk = (lane & 3) ^ ((lane >> 3) & 3);
  uint32_t voffA[kLoads], voffB[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = 16 * (kLoads * wave + i) + (lane >> 2);
    const int k = kPerK * (kLoads * wave + i) + lane / (64 / kPerK);
    const int col = kPiece * place(k, lane % (64 / kPerK));
    if constexpr (kRowsA) voffA[i] = i0 + row < P.M ? (uint32_t)(row * rowA + chunk * 16) : kOOB;
    else voffA[i] = i0 + col < P.M ? (uint32_t)(k * rowA + col * kSize) : kOOB;
    if constexpr (kRowsB) {
      // the wave's B rows are of one projection (see fwd_column)
      const int feat = (wave >> 1) * (kCols / 2) + 16 * i + (lane >> 2);
      voffB[i] = j0 + feat < P.N ? (uint32_t)(feat * (int64_t)((wave & 1) ? P.ldb1 : P.ldb0) * kSize + chunk * 16) : kOOB;
    } else {
      const int64_t ld = Mode == kFfnDx ? 0 : rowB;  // dx: the segment's stride, added per iteration
      voffB[i] = j0 + col < P.N ? (uint32_t)(k * ld + col * kSize) : kOOB;
    }
  }
  // dx reads two weights, whose strides may differ; the wave's k rows are
  // few, so the offset is rebuilt when the segment changes
  uint32_t voffB1[kLoads];
  if constexpr (Mode == kFfnDx) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int k = kPerK * (kLoads * wave + i) + lane / (64 / kPerK);
      voffB1[i] = voffB[i] == kOOB ? kOOB : voffB[i] + (uint32_t)(k * P.ldb1 * kSize);
      if (voffB[i] != kOOB) voffB[i] += (uint32_t)(k * P.ldb0 * kSize);
    }
  }

  struct Next {
    u32x4 ra, rb;
    int lim;  // chunks of K left for the operands whose rows run along K
    int seg;
  };
  auto describe = [&](int j) {
    Next d;
    d.seg = Mode == kFfnDx && j >= per_seg;
    const int64_t k0 = (int64_t)(j - d.seg * per_seg) * kStep;
    const int64_t kend = Mode == kFfnDx ? P.fp : P.K;
    const bool live = j < it1;
    d.lim = (int)((kend - k0 + kPiece - 1) / kPiece);
    const int64_t valid = live ? max((int64_t)0, min((int64_t)kStep, P.K - k0)) : 0;
    const uint64_t a = reinterpret_cast<uint64_t>(P.a);
    if constexpr (kRowsA)
      d.ra = rsrc_words(a + (uint64_t)(i0 * rowA + (d.seg * P.fp + k0) * kSize), live ? kAll : 0);
    else
      d.ra = rsrc_words(a + (uint64_t)(k0 * rowA + i0 * kSize), valid * rowA);
    if constexpr (kRowsB) {
      const uint64_t b = reinterpret_cast<uint64_t>((wave & 1) ? P.b1 : P.b0);
      const int64_t ld = (wave & 1) ? P.ldb1 : P.ldb0;
      d.rb = rsrc_words(b + (uint64_t)((j0 * ld + k0) * kSize), live ? kAll : 0);
    } else {
      const uint64_t b = reinterpret_cast<uint64_t>(d.seg ? P.b1 : P.b0);
      const int64_t ld = d.seg ? P.ldb1 : P.ldb0;
      d.rb = rsrc_words(b + (uint64_t)((k0 * ld + j0) * kSize), valid * ld * kSize);
    }
    return d;
  };
  // load i of the wave's 2 kLoads of one stage
  auto load1 = [&](uint32_t stage, const Next& d, int i) {
    const bool isA = i < kLoads;
    const int q = isA ? i : i - kLoads;
    uint32_t off = isA ? voffA[q] : voffB[q];
    if (Mode == kFfnDx && !isA) off = d.seg ? voffB1[q] : off;
    if (isA ? kRowsA : kRowsB) off = chunk < d.lim ? off : kOOB;
    lds_dma16(isA ? d.ra : d.rb, off, stage + (isA ? 0 : kPanel) + (uint32_t)((kLoads * wave + q) * 1024));
  };
  auto load_stage = [&](uint32_t stage, int j) {
    const Next d = describe(j);
#pragma unroll
    for (int i = 0; i < 2 * kLoads; ++i) load1(stage, d, i);
  };

  // Operand block m of a wave's share: lane l holds row (or column) l % 16 of
  // the block, the l / 16-th chunk of K.  The block enters as 1024 m (rows)
  // or, by the XOR of the chunks, as a flip of address bits (16 m columns are
  // 2 m or 4 m chunks).
  const int tl = kPiece * (lane >> 4) + (kSize == 2 ? (lane & 15) >> 2 : 0);
  auto lane_pos = [&](bool rows, int col0) {
    if (rows) return col0 * 64 + (lane & 15) * 64 + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4);
    const int col = col0 + (kSize == 2 ? 4 * (lane & 3) : lane & 15);
    return tl * kRow + (place(tl, col / kPiece) << 4) + (col % kPiece) * kSize;
  };
  const int posA = lane_pos(kRowsA, wr * (Edge / 2)), posB = lane_pos(kRowsB, wc * kCols);
  auto read1 = [&](const char* stage, int pos, int m, bool rows) {
    if (rows) return *reinterpret_cast<const u32x4*>(stage + pos + m * 1024);
    const char* p = stage + (pos ^ (m << (kSize == 2 ? 5 : 6)));
    if constexpr (kSize == 2) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((HESS_LDS s16x4*)(p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((HESS_LDS s16x4*)(p + 4 * kRow));
      const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
      return u32x4{a.x, a.y, b.x, b.y};
    } else {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = *reinterpret_cast<const uint32_t*>(p + j * kRow);
      return o;
    }
  };
  auto read_a = [&](uint32_t stage, int m) { return read1(lds + stage, posA, m, kRowsA); };
  auto read_b = [&](uint32_t stage, int n) { return read1(lds + stage + kPanel, posB, n, kRowsB); };

  f32x4 acc[kBm][kBn];
#pragma unroll
  for (int m = 0; m < kBm; ++m)
#pragma unroll
    for (int n = 0; n < kBn; ++n) acc[m][n] = f32x4{};

  // Iteration j on the stage at cur (its first four A blocks are in a, its B
  // blocks in b), group by group: the matrix instructions of one A block, the
  // read of the A block four groups later (of the next stage at the end), a
  // read of the next stage's B (into c) and a load of iteration j + 4.  Before
  // the first read of the next stage the wave waits for its own loads of it
  // and meets the others (the next stage is then complete, and nobody reads
  // the one before cur); up to there it works on operands already read, so
  // that the matrix instructions run on from one iteration to the next.
  constexpr int kRot = kBm < 4 ? kBm : 4;  // A blocks in registers
  constexpr int kMeet = kBm - 6 > 0 ? kBm - 6 : 0;
  u32x4 a[kRot];
  auto step = [&](uint32_t cur, uint32_t nxt, uint32_t target, int j, const u32x4 (&b)[kBn], u32x4 (&c)[kBn]) {
    const Next d = describe(j + kAhead);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < kBm; ++m) {
      if (m == kMeet) {
        __builtin_amdgcn_s_waitcnt(vm_wait(2 * kLoads * (kAhead - 2)));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = 0; n < kBn; ++n) acc[m][n] = mma16<DT>(b[n], a[m % kRot], acc[m][n]);
      a[m % kRot] = m + kRot < kBm ? read_a(cur, m + kRot) : read_a(nxt, m + kRot - kBm);
      if (m >= kMeet && m < kMeet + kRot) {
        c[m - kMeet] = read_b(nxt, m - kMeet);
        load1(lds0 + target, d, m - kMeet);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(2 * kLoads == kRot && kBn == kRot, "one load and one read of B in each of kRot groups");

#pragma unroll
  for (int q = 0; q < kAhead; ++q) load_stage(lds0 + q * kStage, it0 + q);
  __builtin_amdgcn_s_waitcnt(vm_wait(2 * kLoads * (kAhead - 1)));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  u32x4 b[kBn], c[kBn];
#pragma unroll
  for (int q = 0; q < kRot; ++q) a[q] = read_a(0, q);
#pragma unroll
  for (int q = 0; q < kBn; ++q) b[q] = read_b(0, q);
  // two iterations a trip (two sets of B registers); an extra iteration
  // multiplies zeros.  The stages go round in scalar registers.
  uint32_t cur = 0, nxt = kStage, ld = kAhead * kStage;
  auto rotate = [&] {
    cur = nxt;
    nxt = nxt + kStage == kStages * kStage ? 0u : nxt + kStage;
    ld = ld + kStage == kStages * kStage ? 0u : ld + kStage;
  };
  for (int j = it0; j < it1; j += 2) {
    step(cur, nxt, ld, j, b, c);
    rotate();
    step(cur, nxt, ld, j + 1, c, b);
    rotate();
  }
  // the trailing loads write LDS: they end before the workgroup does
  __builtin_amdgcn_s_waitcnt(0x0070);
  __builtin_amdgcn_sched_barrier(0);

  if (!whole) {
    float* W = P.ws + ((int64_t)part * tail + (t - P.full)) * (Edge * Edge) +
               (wr * (Edge / 2) + (lane & 15)) * Edge + wc * kCols + 4 * (lane >> 4);
#pragma unroll
    for (int m = 0; m < kBm; ++m)
#pragma unroll
      for (int n = 0; n < kBn; ++n) {
        const f32x4 x = acc[m][n];
        *reinterpret_cast<float4*>(W + 16 * m * Edge + 16 * n) = float4{x[0], x[1], x[2], x[3]};
      }
    return;
  }
  // A tile's outputs.  Blocks n, n + 1: after exchanging the odd 16-lane rows
  // of the first with the even ones of the second, lane row g holds columns
  // 8 (g / 2) .. + 7 of block n + g % 2.  In: the tile lies inside the matrix.
  auto put_tile = [&](auto in) __attribute__((always_inline)) {
    constexpr bool In = decltype(in)::value;
    typedef typename Elem<DT>::type T;
    int lv = lane;
    asm volatile("" : "+v"(lv));  // the offsets are computed here, not kept through the loop
    const int cc = 16 * ((lv >> 4) & 1) + 8 * (lv >> 5);
    auto eight = [&](const f32x4& p, const f32x4& q, float (&o)[8]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(p[j]), __float_as_uint(q[j]), false, false);
        o[j] = __uint_as_float(s[0]);
        o[4 + j] = __uint_as_float(s[1]);
      }
    };
    // features of one row, forward
    auto put_features = [&](int64_t r, int64_t col, const float (&g)[8], const float (&u)[8]) {
      if constexpr (In) {
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = act_value<DT == kInF32>(g[e], P.act) * u[e];
        store_n(static_cast<T*>(P.o0) + r * P.ldo0 + col, h, 8);
        if (P.o1) put_preact<T>(P, r, col, g, u);
      } else {
        put_fwd<DT>(P, r, col, g, u);
      }
    };
    if constexpr (Mode == kFfnFwd && kBn == 2) {
      // one block of either projection: two rows of blocks are exchanged
      // instead, and lane row g holds row block g % 2
      float g[8], u[8];
      eight(acc[0][0], acc[1][0], g);
      eight(acc[0][1], acc[1][1], u);
      put_features(i0 + wr * (Edge / 2) + (lv & 15) + 16 * ((lv >> 4) & 1), j0 + wc * (kCols / 2) + 8 * (lv >> 5), g, u);
      return;
    }
#pragma unroll
    for (int m = 0; m < kBm; ++m) {
      const int64_t r = i0 + wr * (Edge / 2) + (lv & 15) + 16 * m;
      if constexpr (Mode == kFfnFwd) {
        float g[8], u[8];
        eight(acc[m][0], acc[m][1], g);
        eight(acc[m][kBn / 2], acc[m][kBn / 2 + 1], u);
        put_features(r, j0 + wc * (kCols / 2) + cc, g, u);
      } else {
#pragma unroll
        for (int n = 0; n < kBn; n += 2) {
          const int64_t col = j0 + wc * kCols + 16 * n + cc;
          float v[8];
          eight(acc[m][n], acc[m][n + 1], v);
          if constexpr (In) {
            T* o = static_cast<T*>(P.o0) + r * P.ldo0;
            if constexpr (Mode == kFfnDw)
              if (r >= P.fp) o = static_cast<T*>(P.o1) + (r - P.fp) * P.ldo1;
            store_n(o + col, v, 8);
          } else {
            put<DT, Mode>(P, r, col, v);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  const bool inside = i0 + Edge <= P.M && j0 + (Mode == kFfnFwd ? Edge / 2 : Edge) <= P.N &&
                      (Mode != kFfnDw || P.f == P.fp);
  if (inside) put_tile(std::true_type());
  else put_tile(std::false_type());
}

// Split tiles: the parts' sums added in part order, then the epilogue.  Block
// (t, s) handles rows s * (1024 / Edge) .. of tile full + t; a thread takes
// four columns (forward: of both projections).
template <int DT, int Mode, int Edge> __global__ void __launch_bounds__(256) ffn_join(FfnGemm P) {
  const int tail = P.ntiles - P.full, t = blockIdx.x;
  int I, J;
  tile_coords<Mode>(P, P.full + t, I, J);
  constexpr int kQuads = Mode == kFfnFwd ? Edge / 8 : Edge / 4;  // quads of columns per row
  const int id = blockIdx.y * 256 + threadIdx.x;
  const int row = id / kQuads, quad = id % kQuads;
  const float* W = P.ws + (int64_t)t * (Edge * Edge) + row * Edge;
  const int64_t stride = (int64_t)tail * (Edge * Edge);
  if constexpr (Mode == kFfnFwd) {
    constexpr int cols = Edge == 64 ? 32 : 64;  // of a wave: half gate, half up
    const int w = quad / (cols / 8), q = quad % (cols / 8);
    const int cg = w * cols + 4 * q;
    float g[4] = {}, u[4] = {};
    for (int p = 0; p < P.parts; ++p) {
      const float4 a = *reinterpret_cast<const float4*>(W + p * stride + cg);
      const float4 b = *reinterpret_cast<const float4*>(W + p * stride + cg + cols / 2);
      g[0] += a.x, g[1] += a.y, g[2] += a.z, g[3] += a.w;
      u[0] += b.x, u[1] += b.y, u[2] += b.z, u[3] += b.w;
    }
    put_fwd<DT>(P, (int64_t)I * Edge + row, (int64_t)J * (Edge / 2) + w * (cols / 2) + 4 * q, g, u);
  } else {
    float v[4] = {};
    for (int p = 0; p < P.parts; ++p) {
      const float4 a = *reinterpret_cast<const float4*>(W + p * stride + 4 * quad);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    }
    put<DT, Mode>(P, (int64_t)I * Edge + row, (int64_t)J * Edge + 4 * quad, v);
  }
}

template <int DT, int Mode, int Edge> void launch_edge(const FfnGemm& g, hipStream_t stream) {
  const int tail = g.ntiles - g.full;
  ffn_tile<DT, Mode, Edge><<<g.full + tail * g.parts, Edge == 256 ? 512 : 256, 0, stream>>>(g);
  if (tail == 0) return;
  constexpr int quads = Mode == kFfnFwd ? Edge / 8 : Edge / 4;
  ffn_join<DT, Mode, Edge><<<dim3(tail, Edge * quads / 256), 256, 0, stream>>>(g);
}

template <int DT, int Mode> hipError_t launch_mode(const FfnGemm& g, int edge, hipStream_t stream) {
  if (edge == 256) launch_edge<DT, Mode, 256>(g, stream);
  else if (edge == 128) launch_edge<DT, Mode, 128>(g, stream);
  else launch_edge<DT, Mode, 64>(g, stream);
  return hipGetLastError();
}

template <int DT> hipError_t launch_type(const FfnGemm& g, int mode, int edge, hipStream_t stream) {
  if (mode == kFfnFwd) return launch_mode<DT, kFfnFwd>(g, edge, stream);
  if (mode == kFfnDx) return launch_mode<DT, kFfnDx>(g, edge, stream);
  return launch_mode<DT, kFfnDw>(g, edge, stream);
}

// Matrix blockIdx.y: rows of `cols` 16-bit values to rows of `pad` (a multiple
// of 8), the rest zeros; 8 values a thread.
__global__ void __launch_bounds__(256) pack_rows16(PackRows P) {
  typedef uint16_t V __attribute__((ext_vector_type(8)));
  typedef V VU __attribute__((aligned(2)));
  const int m = blockIdx.y, cols = P.cols, per = P.pad / 8;
  const uint16_t* src = static_cast<const uint16_t*>(P.src[m]);
  uint16_t* dst = static_cast<uint16_t*>(P.dst[m]);
  const int64_t total = P.rows[m] * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 8;
    const uint16_t* p = src + r * P.ld[m] + c;
    V v;
    if (c + 8 <= cols) {
      v = *reinterpret_cast<const VU*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? p[j] : (uint16_t)0;
    }
    *reinterpret_cast<V*>(dst + r * P.pad + c) = v;
  }
}

}  // namespace

hipError_t launch_ffn_gemm(const FfnGemm& g, int mode, int edge, int dtype, hipStream_t stream) {
  if (dtype == kInBF16) return launch_type<kInBF16>(g, mode, edge, stream);
  if (dtype == kInF16) return launch_type<kInF16>(g, mode, edge, stream);
  return launch_type<kInF32>(g, mode, edge, stream);
}

hipError_t launch_pack_rows16(const PackRows& p, hipStream_t stream) {
  int64_t most = 0;
  for (int m = 0; m < p.count; ++m) most = p.rows[m] > most ? p.rows[m] : most;
  const int64_t total = most * (p.pad / 8);
  if (total == 0) return hipSuccess;
  const int grid = (int)(total < 256 * 2048 ? (total + 255) / 256 : 2048);
  pack_rows16<<<dim3(grid, p.count), 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace hess
