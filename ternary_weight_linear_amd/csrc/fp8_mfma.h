// Block-scaled product of e4m3 codes on the matrix cores, shared by the linear layer and the
// experts' products:
//
//   y[m, n] = sum_b (sx[b, m] * sw[n / 128, b]) * sum_{k in b} q[m, k] w[n, k].
//
// A block's sum of 128 products comes from the matrix cores, the sum over blocks is one fp32
// FMA per block and output.
#pragma once

#include "fp8_internal.h"

namespace bl {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));

// The 32 codes that one lane holds of a 16-row x 128-input operand: lane 16 g + u has row u,
// inputs 16 g .. 16 g + 15 and 64 + 16 g .. 64 + 16 g + 15. (Any order of the inputs serves as
// long as both operands share it.)
struct Frag {
  u32x4 lo, hi;
};

// Row `row` (a pointer to its first code), block starting at input k0. Inputs from K on are
// zero; K % 16 == 0, so a 16-byte piece is whole or empty.
__device__ __forceinline__ Frag load_frag(const uint8_t* row, int64_t k0, int64_t K, int g) {
  Frag f;
  const int64_t a = k0 + 16 * g, b = a + 64;
  const u32x4 zero = {0, 0, 0, 0};
  f.lo = a < K ? *reinterpret_cast<const u32x4*>(row + a) : zero;
  f.hi = b < K ? *reinterpret_cast<const u32x4*>(row + b) : zero;
  return f;
}

// Eight e4m3 codes as fp16 (exact: every e4m3 value is an fp16 value).
__device__ __forceinline__ half8v to_half8(uint32_t a, uint32_t b) {
  const half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return half8v{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

struct FragH {
  half8v h[4];
};
__device__ __forceinline__ FragH to_half(const Frag& f) {
  FragH r;
  r.h[0] = to_half8(f.lo.x, f.lo.y);
  r.h[1] = to_half8(f.lo.z, f.lo.w);
  r.h[2] = to_half8(f.hi.x, f.hi.y);
  r.h[3] = to_half8(f.hi.z, f.hi.w);
  return r;
}

__device__ __forceinline__ uint32_t pack4(const f32x4& v, float r) {
  int c = 0;
  c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * r, v[1] * r, c, false);
  c = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * r, v[3] * r, c, true);
  return static_cast<uint32_t>(c);
}

// Sum over a block: D[row of a][row of b]; lane 16 g + u holds rows 4 g + i of a, row u of b.
// The codes go to the fp16 matrix cores, whose sums keep fp32's precision; the e4m3 form of
// the instruction keeps about 16 bits below the largest product (measured: relative error
// 1.4e-5 of a 128-term sum, against 9e-9 in fp16).
__device__ __forceinline__ f32x4 block_dot(const FragH& a, const FragH& b) {
  f32x4 c = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h[s], b.h[s], c, 0, 0, 0);
  return c;
}

// Where the rows of a product come from and go to.
struct RowMap {
  const int32_t* tiles;   // null: tile t is rows 16 MT t ..; else [tiles, 4] expert, first, rows
  const int32_t* n_tiles; // device count of tiles
  const int32_t* pair;    // sorted row -> slot m * k + j
  int gather_div;         // > 0: operand row of sorted row r is pair[r] / gather_div, else r
  int scatter;            // output row of sorted row r is pair[r], else r
};

struct ProductArgs {
  Fp8LinearArgs a;
  RowMap map;
  int64_t w_stride, sw_stride;   // elements between experts
  // gated products: codes [h_rows, N] and scales [ceil(N / 128), h_rows] of silu(gate) * up
  uint8_t* hq;
  float* hs;
  int64_t h_rows;
};

// One workgroup of eight waves: 16 rows of w by 16 MT rows of q; wave v takes blocks v, v + 8,
// ..., and the eight sums meet in LDS in the order of the waves.
template <int MT>
__global__ __launch_bounds__(512) void fp8_stream_kernel(ProductArgs p) {
  __shared__ f32x4 red[7][MT][64];
  const Fp8LinearArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, u = lane & 15;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  int64_t first = static_cast<int64_t>(blockIdx.y) * (16 * MT);
  int rows = 0, expert = 0;
  if (p.map.tiles) {
    if (static_cast<int>(blockIdx.y) >= *p.map.n_tiles) return;
    expert = p.map.tiles[4 * blockIdx.y];
    first = p.map.tiles[4 * blockIdx.y + 1];
    rows = p.map.tiles[4 * blockIdx.y + 2];
  } else {
    rows = static_cast<int>(a.M - first < 16 * MT ? a.M - first : 16 * MT);
  }
  const int64_t KB = (a.K + kFp8Block - 1) / kFp8Block;
  const int64_t n = n0 + u < a.N ? n0 + u : a.N - 1;
  const uint8_t* wrow = a.w + expert * p.w_stride + n * a.K;
  const float* sw = a.sw + expert * p.sw_stride + (n0 / kFp8Block) * KB;
  const uint8_t* qrow[MT];
  int64_t srow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int r = 16 * t + u < rows ? 16 * t + u : rows - 1;
    int64_t at = first + r;
    if (p.map.gather_div > 0) at = p.map.pair[at] / p.map.gather_div;
    srow[t] = at;
    qrow[t] = a.q + at * a.K;
  }
  f32x4 acc[MT] = {};
  for (int64_t kb = wave; kb < KB; kb += 8) {
    const FragH w = to_half(load_frag(wrow, kb * kFp8Block, a.K, g));
    const float s = sw[kb];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const FragH q = to_half(load_frag(qrow[t], kb * kFp8Block, a.K, g));
      const float f = a.sx[kb * a.M + srow[t]] * s;
      acc[t] += block_dot(w, q) * f;
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int t = 0; t < MT; ++t) red[wave - 1][t][lane] = acc[t];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    for (int v = 0; v < 7; ++v) acc[t] += red[v][t][lane];
    if (16 * t + u >= rows) continue;
    int64_t at = first + 16 * t + u;
    if (p.map.scatter) at = p.map.pair[at];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + 4 * g + i < a.N) store_as(a.y, a.ydtype, at * a.ldy + n0 + 4 * g + i, acc[t][i]);
  }
}

}  // namespace
}  // namespace bl
