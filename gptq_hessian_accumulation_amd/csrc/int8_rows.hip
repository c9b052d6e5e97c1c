// Rows of activations or weights as int8 codes, and back, on gfx950.
//
// A scale a row (the operands of the 8-bit product): with a = max |x| of the
// row, code = rint(127 x / a), ties to even, scale = a / 127 in float32.  The
// code is the one exact arithmetic gives: for 16-bit types 127 x / a is formed
// in float32 (off by less than 3 units of its last place) and rounded to 2^-21
// relative first, which makes every tie exact, and other quotients of 11-bit
// numbers are at least 2^-19 from one; for float32 it is formed in float64 and
// rounded to 2^-40 (others are at least 2^-33 away).
// Blocks of 32 columns (checkpoints): steps are powers of two, so that codes
// take one exact multiplication and what they stand for is exact in bf16 and
// fp16.
// A row or block with an infinity or NaN has a NaN scale and codes 0.
//
// All bound by their bytes (a large copy reaches 4.9 TB/s on the same card).  16384 x
// 4096, calls one after another on changing inputs: bf16 to codes 40 us, 5.0 TB/s, a
// scale a row (46 to 47 us between long products, which leave the caches full and
// the clock low), 36 us in blocks, back 34 and 39 us; float32 61 and 63 us, back 62
// to 70 and 87 to 93 us.  A row is read once, into registers: rows past 16,384
// columns of a workgroup are read twice (512 x 65536 bf16 27 us, 3.7 TB/s).  Calls of
// a few hundred rows take 3.5 to 4.5 us, most of it the launch.

#include <algorithm>

#include "int8_device.hpp"
#include "int8_internal.hpp"

namespace hess {

namespace {

// 8 codes to p (any alignment), the first `left` of them inside what is written.
__device__ __forceinline__ void store8(int8_t* p, int64_t left, const uint2& q) {
  if (left >= 8) {
    *reinterpret_cast<uint2_at1*>(p) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = (int8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
  }
}

// Matrix m of a set of copies: 16 codes a thread, from thread `first` of `all`.
__device__ __forceinline__ void pack_range(const PackCodes& P, int m, int64_t first, int64_t all) {
  const int64_t per = P.pad / 16, total = P.rows[m] * per;
  for (int64_t i = first; i < total; i += all) {
    const int64_t r = row_of(i, per), c = (i - r * per) * 16;
    const int8_t* p = P.src[m] + r * P.ld[m] + c;
    u32x4 v{};
    if (c + 16 <= P.cols) {
      v = *reinterpret_cast<const u32x4_at1*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < P.cols) v[j / 4] |= (uint32_t)(uint8_t)p[j] << (8 * (j % 4));
    }
    *reinterpret_cast<u32x4*>(P.dst[m] + r * P.pad + c) = v;
  }
}
__global__ void __launch_bounds__(256) pack_codes(PackCodes P) {
  pack_range(P, blockIdx.y, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// A row a workgroup of T threads, P pieces of 8 values a thread in registers
// (rows longer than that are read twice).
template <int DT, int T, int P> __global__ void __launch_bounds__(T) quantize_rows(Int8Rows R, PackCodes C) {
  typedef typename Elem<DT>::type E;
  __shared__ uint32_t part[T / 64];
  const int64_t row = blockIdx.x;
  if (row >= R.n) {  // the workgroups behind the rows copy codes
    pack_range(C, 0, (row - R.n) * T + threadIdx.x, (int64_t)(gridDim.x - R.n) * T);
    return;
  }
  const E* x = static_cast<const E*>(R.x) + row * R.ldx;
  int8_t* c = R.codes + row * R.ldc;
  float v[P][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int64_t at = (int64_t)(i * T + threadIdx.x) * 8;
    if (at < R.d) load8(x + at, R.d - at, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    top = max(top, top_of(v[i]));
  }
  for (int64_t at = (int64_t)(P * T + threadIdx.x) * 8; at < R.d; at += T * 8) {
    float w[8];
    load8(x + at, R.d - at, w);
    top = max(top, top_of(w));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 64; ++w) top = max(top, part[w]);
  }
  const RowCode<E> code(top);
  if (threadIdx.x == 0) static_cast<float*>(R.scale)[row] = row_scale(top);
  auto put = [&](int64_t at, const float (&w)[8]) {
    int q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = code(w[j]);
    store8(c + at, R.pad - at, uint2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])});
  };
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int64_t at = (int64_t)(i * T + threadIdx.x) * 8;
    if (at < R.pad) put(at, v[i]);
  }
  for (int64_t at = (int64_t)(P * T + threadIdx.x) * 8; at < R.pad; at += T * 8) {
    float w[8] = {};
    if (at < R.d) load8(x + at, R.d - at, w);
    put(at, w);
  }
}

// Blocks of 32 columns: 8 values a thread, four neighbouring lanes a block, `wide`
// blocks a row: its `groups` of values, and those of zeros up to column pad.
template <int DT>
__global__ void __launch_bounds__(256) quantize_blocks(Int8Rows R, int64_t groups, int64_t wide, int64_t total) {
  typedef typename Elem<DT>::type E;
  // (whole waves run: total is a whole number of groups of four lanes)
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = row_of(i, wide * 4);
    const int64_t at = (i - row * wide * 4) * 8;
    float v[8] = {};
    if (at < R.d) load8(static_cast<const E*>(R.x) + row * R.ldx + at, R.d - at, v);
    uint32_t top = top_of(v);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t b = block_exponent(top);
    const BlockCode code(b);
    const uint2 q{code(v[0], v[1], v[2], v[3]), code(v[4], v[5], v[6], v[7])};
    if (at < R.pad) store8(R.codes + row * R.ldc + at, R.pad - at, q);
    if ((i & 3) == 0 && at < R.d) static_cast<uint8_t*>(R.scale)[row * groups + at / 32] = (uint8_t)b;
  }
}

template <int DT, int Block> __global__ void __launch_bounds__(256) dequantize(Int8Rows R) {
  dequantize_range<DT, Block>(R, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// The operands of a linear layer's gradients: blockIdx.y 0 and 1 the sets of rows,
// 2 the copy of dy.  xq and wq are rounded to dtype, since the matrix instructions
// take operands of one 16-bit type: gradients are then 0.0023 (bf16) or 0.00029
// (fp16) from the 64-bit values, where the last rounding alone leaves 0.0017 or
// 0.00021.  Their remainders as operands of their own would double the products,
// which are all but 37 of 1,290 us of an 8,192-token backward pass at 4096 x 11264;
// float32 has no such rounding.
template <int DT> __global__ void __launch_bounds__(256) grad_operands(GradOperands G) {
  typedef typename Elem<DT>::type E;
  typedef E E8 __attribute__((ext_vector_type(8)));
  typedef E8 E8u __attribute__((aligned(sizeof(E))));
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
  if (blockIdx.y < 2) {
    if (G.rows[blockIdx.y].x) dequantize_range<DT, 0>(G.rows[blockIdx.y], first, all);
    return;
  }
  const int64_t per = (G.pad + 7) / 8, total = G.n * per;
  for (int64_t i = first; i < total; i += all) {
    const int64_t row = row_of(i, per), at = (i - row * per) * 8;
    const E* p = static_cast<const E*>(G.src) + row * G.ld + at;
    E* o = static_cast<E*>(G.dst) + row * G.pad + at;
    if (at + 8 <= G.cols) {
      *reinterpret_cast<E8u*>(o) = *reinterpret_cast<const E8u*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < G.pad) o[j] = at + j < G.cols ? p[j] : (E)0.0f;
    }
  }
}

int grid_of(int64_t threads) { return (int)std::min<int64_t>((threads + 255) / 256, 8192); }

template <int DT, int T, int P> void launch_rows(const Int8Rows& r, const PackCodes& c, hipStream_t stream) {
  const int64_t most = (int64_t)1 << 20;  // workgroups of a launch (fewer than 2^32 threads)
  for (int64_t r0 = 0; r0 < r.n; r0 += most) {
    Int8Rows p = r;
    p.n = std::min(most, r.n - r0);
    p.x = static_cast<const char*>(r.x) + r0 * r.ldx * Elem<DT>::size;
    p.codes = r.codes + r0 * r.ldc;
    p.scale = static_cast<float*>(r.scale) + r0;
    const int extra = c.count > 0 && r0 == 0 ? (int)std::min<int64_t>((c.rows[0] * (c.pad / 16) + T - 1) / T, (1 << 18) / T) : 0;
    quantize_rows<DT, T, P><<<(unsigned)(p.n + extra), T, 0, stream>>>(p, c);
  }
}

// As few threads as hold a row in 2 or 4 pieces each: a wave up to 2,048 columns.
template <int DT> hipError_t quantize_type(const Int8Rows& r, int block, const PackCodes& c, hipStream_t stream) {
  if (block == 0) {
    if (r.d <= 1024) launch_rows<DT, 64, 2>(r, c, stream);
    else if (r.d <= 2048) launch_rows<DT, 64, 4>(r, c, stream);
    else if (r.d <= 4096) launch_rows<DT, 256, 2>(r, c, stream);
    else if (r.d <= 8192) launch_rows<DT, 256, 4>(r, c, stream);
    else launch_rows<DT, 1024, 2>(r, c, stream);
  } else {
    const int64_t groups = (r.d + 31) / 32, wide = std::max(groups, (r.pad + 31) / 32), total = r.n * wide * 4;
    quantize_blocks<DT><<<grid_of(total), 256, 0, stream>>>(r, groups, wide, total);
  }
  return hipGetLastError();
}

template <int DT> hipError_t dequantize_type(const Int8Rows& r, int block, hipStream_t stream) {
  const int64_t piece = 16 / Elem<DT>::size;
  const int grid = grid_of(r.n * ((r.pad + piece - 1) / piece));
  if (block == 0) dequantize<DT, 0><<<grid, 256, 0, stream>>>(r);
  else dequantize<DT, 32><<<grid, 256, 0, stream>>>(r);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize_and_pack(const Int8Rows& r, int dtype, const PackCodes& p, hipStream_t stream) {
  if (dtype == kInBF16) return quantize_type<kInBF16>(r, 0, p, stream);
  if (dtype == kInF16) return quantize_type<kInF16>(r, 0, p, stream);
  return quantize_type<kInF32>(r, 0, p, stream);
}

hipError_t launch_int8_quantize(const Int8Rows& r, int block, int dtype, hipStream_t stream) {
  if (r.n == 0) return hipSuccess;
  const PackCodes none{};
  if (dtype == kInBF16) return quantize_type<kInBF16>(r, block, none, stream);
  if (dtype == kInF16) return quantize_type<kInF16>(r, block, none, stream);
  return quantize_type<kInF32>(r, block, none, stream);
}

hipError_t launch_int8_grad_operands(const GradOperands& g, int dtype, hipStream_t stream) {
  int64_t most = g.src ? g.n * ((g.pad + 7) / 8) : 0;
  for (const Int8Rows& r : g.rows)
    if (r.x) most = std::max(most, r.n * ((r.pad + 7) / 8));
  const dim3 grid(grid_of(most), g.src ? 3 : 2);
  if (dtype == kInBF16) grad_operands<kInBF16><<<grid, 256, 0, stream>>>(g);
  else if (dtype == kInF16) grad_operands<kInF16><<<grid, 256, 0, stream>>>(g);
  else grad_operands<kInF32><<<grid, 256, 0, stream>>>(g);
  return hipGetLastError();
}

hipError_t launch_pack_codes(const PackCodes& p, hipStream_t stream) {
  int64_t most = 0;
  for (int m = 0; m < p.count; ++m) most = std::max(most, p.rows[m]);
  const int64_t total = most * (p.pad / 16);
  if (total == 0) return hipSuccess;
  pack_codes<<<dim3((unsigned)std::min<int64_t>((total + 255) / 256, 2048), p.count), 256, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_int8_dequantize(const Int8Rows& r, int block, int dtype, hipStream_t stream) {
  if (r.n == 0) return hipSuccess;
  if (dtype == kInBF16) return dequantize_type<kInBF16>(r, block, stream);
  if (dtype == kInF16) return dequantize_type<kInF16>(r, block, stream);
  return dequantize_type<kInF32>(r, block, stream);
}

}  // namespace hess
