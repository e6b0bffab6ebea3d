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
//
// EXACT: the codes go to the fp16 matrix instruction, whose sums keep fp32's precision. The
// e4m3 instruction takes the codes as they are at twice the rate, but cuts each eight products
// that follow each other at 2^-13 of the power of two of the largest before it adds them: a sum
// errs by up to 7 2^-13 (8.5e-4) of its magnitudes. Measured: 2e-5 of them on normal values, 3e-4
// with one loud channel (the fp16 instruction 9e-9). That is below bf16's rounding, 2^-9 of the
// result, but not fp16's 2^-12, nor may it move codes of a quantised result: the e4m3
// instruction serves bf16 results only.
typedef int i32x8 __attribute__((ext_vector_type(8)));

template <bool EXACT>
struct OperandT { using type = i32x8; };
template <>
struct OperandT<true> { using type = FragH; };
template <bool EXACT>
using Operand = typename OperandT<EXACT>::type;

template <bool EXACT>
__device__ __forceinline__ Operand<EXACT> operand(const Frag& f) {
  if constexpr (EXACT) return to_half(f);
  else return i32x8{(int)f.lo.x, (int)f.lo.y, (int)f.lo.z, (int)f.lo.w, (int)f.hi.x, (int)f.hi.y, (int)f.hi.z, (int)f.hi.w};
}

__device__ __forceinline__ f32x4 block_dot(const FragH& a, const FragH& b) {
  f32x4 c = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h[s], b.h[s], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4 block_dot(const i32x8& a, const i32x8& b) {
  const f32x4 c = {0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);   // no scales
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
  // tiled linear product: tiles from `whole` on have K in `parts` (2 or more; else none has), and
  // leave fp32 sums [parts, tiles, BM, BN] in part
  int whole, parts;
  float* part;
};

// Vectors at any multiple of their element's size: global memory takes unaligned accesses.
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

__device__ __forceinline__ uint32_t pack16(int dtype, float lo, float hi) {
  return dtype == BL_BF16 ? bf16_bits(lo) | static_cast<uint32_t>(bf16_bits(hi)) << 16
                          : half_bits(lo) | static_cast<uint32_t>(half_bits(hi)) << 16;
}

// Four consecutive outputs of a row, in one store where the row has them all.
__device__ __forceinline__ void store4(const Fp8LinearArgs& a, int64_t row, int64_t n, const f32x4& v) {
  const int64_t at = row * a.ldy + n;
  if (n + 3 < a.N) {
    if (a.ydtype == BL_F32) *reinterpret_cast<f32x4_at4*>(static_cast<float*>(a.y) + at) = v;
    else
      *reinterpret_cast<u32x2_at2*>(static_cast<uint16_t*>(a.y) + at) =
          u32x2{pack16(a.ydtype, v[0], v[1]), pack16(a.ydtype, v[2], v[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) store_as(a.y, a.ydtype, at + e, v[e]);
  }
}

// Source of a streaming product's activations: e4m3 codes with their scales in memory, or
// values of a bl_dtype that each workgroup quantises into LDS first.
constexpr int kSrcCodes = -1;
// What the streaming kernel computes.
constexpr int kStreamLinear = 0;   // rows of q times w
constexpr int kStreamGated = 1;    // NT / 2 gate and NT / 2 up fragments: silu(gate) * up
constexpr int kStreamSlots = 2;    // one token's weighted sum over its slots (x is [M k, K])

struct StreamArgs {
  ProductArgs p;
  const void* x;           // SRC >= 0: values, rows ldx apart
  int64_t ldx;
  const int32_t* index;    // direct tiles: tile t is slot t, its expert index[t]; null: as p.map says
  const float* weight;     // kStreamSlots
  int E, k;
};

constexpr int kStreamWaves = 8;
constexpr int kStreamThreads = 64 * kStreamWaves;

// LDS bytes of `rows` quantised rows: codes (rows 64 bytes past a multiple of 128, so that
// they start in different banks), then scales.
__host__ __device__ inline int staged_row(int KB) { return KB * kFp8Block + 64; }
__host__ __device__ inline int staged_bytes(int rows, int KB) { return rows * (staged_row(KB) + 4 * KB); }

// Eight consecutive values of a bl_dtype at p (16-byte aligned).
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::type* p, float (&v)[8]) {
  if constexpr (DT == BL_F32) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = to_float<DT>(static_cast<uint16_t>(a[j] & 0xFFFFu));
      v[2 * j + 1] = to_float<DT>(static_cast<uint16_t>(a[j] >> 16));
    }
  }
}

// The maximum of |v| over the 16 lanes of a block, as bits, at least the floor.
__device__ __forceinline__ uint32_t block_top(const float (&v)[8]) {
  uint32_t a = kFp8FloorBits;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(v[i]));
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), off)));
  return a;
}

__device__ __forceinline__ u32x2 pack8(const float (&v)[8], float r) {
  return u32x2{pack4(f32x4{v[0], v[1], v[2], v[3]}, r), pack4(f32x4{v[4], v[5], v[6], v[7]}, r)};
}

struct QuantArgs {
  const void* x;              // rows of K values (GATED: 2 K), ldx apart
  int64_t M, K, KB, ldx;
  const int32_t* rows_used;   // device count of rows, or null: M
  uint8_t* q;                 // [M, K]
  float* scale;               // [KB, M]
};

// Quantises 16 blocks of 128 values from block `first` on (inputs run first), one per 16 lanes:
// a 16-byte load per lane (two of fp32), a maximum over the lanes, an 8-byte store.
template <int DT, bool GATED>
__device__ __forceinline__ void quant_blocks(const QuantArgs& a, int64_t first) {
  using T = typename Elem<DT>::type;
  const int64_t blk = first + (threadIdx.x >> 4);
  const int64_t m = blk / a.KB, kb = blk - m * a.KB;
  const int64_t k = kb * kFp8Block + (threadIdx.x & 15) * 8;
  if (m >= (a.rows_used ? *a.rows_used : a.M)) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (k < a.K) {
    const T* x = static_cast<const T*>(a.x) + m * a.ldx + k;
    load8<DT>(x, v);
    if constexpr (GATED) {
      float u[8];
      load8<DT>(x + a.K, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = silu_mul(v[i], u[i]);
    }
  }
  const float am = __uint_as_float(block_top(v));
  if (k < a.K) *reinterpret_cast<u32x2*>(a.q + m * a.K + k) = pack8(v, code_factor(am));
  if ((threadIdx.x & 15) == 0) a.scale[kb * a.M + m] = am / kFp8Max;
}

// Streaming product for few rows: the weights are read once, straight into registers, and
// decide the time. A workgroup of eight waves is S ranges of K by 8 / S groups of 16 NT weight
// rows; range r takes blocks r, r + S, ..., so the workgroup reads the next 128 S codes of each
// row together, and the ranges meet in LDS in order. The loads of several waves per SIMD hide
// each other's latency: keeping a second block's loads in flight per wave measured slower in
// every shape (more registers, a block too many read at the end). Workgroups start at different
// blocks (rot): weight rows are usually a power of two apart, and all workgroups at the same
// input would meet in a few of the memory's channels. The fp16 instruction costs nothing here:
// with the e4m3 one the times are the same.
// Kernel trace, weights that no cache holds, us (weight bytes / time): 1 x 8192 x 8192 17.1 (3.9
// TB/s; 14.4 where 200 MB of weights take turns), 16 x 8192 x 8192 18.3, 16 x 28672 x 8192 43.7 (5.4
// TB/s), 1 x 28672 x 8192 40.4 (5.8 TB/s). Reading that much and nothing else in one launch: 67 MB
// 12.1, 235 MB 36.7.
template <int MT, int NT, int S, int SRC, int MODE>
__global__ __launch_bounds__(kStreamThreads) void fp8_stream_kernel(StreamArgs s) {
  constexpr bool GATED = MODE == kStreamGated;
  constexpr int G = kStreamWaves / S;               // groups of weight rows
  constexpr int NC = GATED ? NT / 2 : NT;           // fragments of output columns of a group
  __shared__ f32x4 red[S][G * NT * MT][64];
  extern __shared__ __attribute__((aligned(16))) uint8_t staged[];
  const ProductArgs& p = s.p;
  const Fp8LinearArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, u = lane & 15;
  const int range = wave % S, group = wave / S;
  const int by = blockIdx.y, bx = blockIdx.x;       // tile of rows; workgroups along the columns run first
  const int64_t n0 = (static_cast<int64_t>(bx) * G + group) * (16 * NC);
  int64_t first = static_cast<int64_t>(by) * (16 * MT);
  int rows = 0, expert = 0;
  if constexpr (MODE == kStreamSlots) {
    first = static_cast<int64_t>(by) * s.k;
    rows = 1;
  } else if (s.index) {
    first = by;
    rows = 1;
    expert = s.index[first];
    if (expert < 0 || expert >= s.E) return;
  } else if (p.map.tiles) {
    if (by >= *p.map.n_tiles) return;
    expert = p.map.tiles[4 * by];
    first = p.map.tiles[4 * by + 1];
    rows = p.map.tiles[4 * by + 2];
  } else {
    rows = static_cast<int>(a.M - first < 16 * MT ? a.M - first : 16 * MT);
  }
  const int KB = static_cast<int>((a.K + kFp8Block - 1) / kFp8Block);
  const int64_t scale_rows = (a.N + kFp8Block - 1) / kFp8Block * KB;
  const uint8_t* wrow[NT];
  const float* sw[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t c = n0 + 16 * (i % NC);
    const int64_t n = (c + u < a.N ? c + u : a.N - 1) + (i >= NC ? a.N : 0);
    wrow[i] = a.w + expert * p.w_stride + n * a.K;
    sw[i] = a.sw + expert * p.sw_stride + (i >= NC ? scale_rows : 0) +
            (c < a.N ? c : a.N - 1) / kFp8Block * KB;
  }
  const uint8_t* qrow[MT];
  const float* srow[MT];
  if constexpr (SRC == kSrcCodes) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      int64_t at = first + (16 * t + u < rows ? 16 * t + u : rows - 1);
      if (p.map.gather_div > 0) at = p.map.pair[at] / p.map.gather_div;
      qrow[t] = a.q + at * a.K;
      srow[t] = a.sx + at;
    }
  }

  struct Stage {
    Frag w[NT], q[MT];
    float sw[NT], sx[MT];
    int kb, row;           // staged rows: which block of which
    bool some;
  };
  // kStreamSlots: item it is block it % KB of slot it / KB; a slot that names no expert is read
  // at expert 0 (in bounds) and left out of the sum
  const int items = MODE == kStreamSlots ? s.k * KB : KB;
  const int rot = MODE == kStreamSlots ? 0 : bx % KB;
  auto load = [&](Stage& st, int it) __attribute__((always_inline)) {
    int kb = it + rot < KB || MODE == kStreamSlots ? it + rot : it + rot - KB;
    int64_t wo = 0, so = 0;
    float weigh = 1.0f;
    st.row = 0;
    if constexpr (MODE == kStreamSlots) {
      st.row = it / KB;
      kb = it - st.row * KB;
      // uniform loads through the scalar cache: a vector load here would put its latency before
      // that of the weights it leads to
      using ConstInt = const __attribute__((address_space(4))) int32_t;
      using ConstFloat = const __attribute__((address_space(4))) float;
      int e = ((ConstInt*)s.index)[first + st.row];
      st.some = e >= 0 && e < s.E;
      weigh = ((ConstFloat*)s.weight)[first + st.row];
      e = st.some ? e : 0;
      wo = e * p.w_stride;
      so = e * p.sw_stride;
    }
    st.kb = kb;
    const int64_t k0 = static_cast<int64_t>(kb) * kFp8Block;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      st.w[i] = load_frag(wrow[i] + wo, k0, a.K, g);
      st.sw[i] = sw[i][so + kb] * weigh;
    }
    if constexpr (SRC == kSrcCodes) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        st.q[t] = load_frag(qrow[t], k0, a.K, g);
        st.sx[t] = srow[t][kb * a.M];
      }
    }
  };
  f32x4 acc[NT][MT] = {};
  const int staged_rows = MODE == kStreamSlots ? s.k : rows;
  const auto* staged_scale = reinterpret_cast<const float*>(staged + staged_rows * staged_row(KB));
  auto multiply = [&](const Stage& st) __attribute__((always_inline)) {
    if constexpr (MODE == kStreamSlots) {
      if (!st.some) return;
    }
    FragH q[MT];
    float sx[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if constexpr (SRC == kSrcCodes) {
        q[t] = to_half(st.q[t]);
        sx[t] = st.sx[t];
      } else {
        const int r = MODE == kStreamSlots ? st.row : min(u, rows - 1);
        const uint8_t* at = staged + r * staged_row(KB) + st.kb * kFp8Block + 16 * g;
        q[t] = to_half(Frag{*reinterpret_cast<const u32x4*>(at), *reinterpret_cast<const u32x4*>(at + 64)});
        sx[t] = staged_scale[r * KB + st.kb];
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const FragH w = to_half(st.w[i]);
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[i][t] += block_dot(w, q[t]) * (sx[t] * st.sw[i]);
    }
  };

  // kStreamSlots runs one workgroup per CU: four blocks per wave are read at a time
  constexpr int D = MODE == kStreamSlots ? 4 : 1;
  Stage st[D];
  auto load_all = [&](int it) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < D; ++d) load(st[d], min(it + d * S, items - 1));
  };
  if constexpr (SRC != kSrcCodes) {
    // 16 lanes per block of 128 values, as in fp8_quant_act_kernel; the first pass's loads go
    // out before the first weights', so that waiting for them does not wait for those
    const int blocks = staged_rows * KB;
    using T = typename Elem<SRC == kSrcCodes ? 0 : SRC>::type;
    constexpr int step = kStreamThreads / 16, P = 2;   // blocks per pass, passes loaded ahead
    float v[P][8];
    auto fetch = [&](int b, float (&x)[8]) __attribute__((always_inline)) {
      const int r = b / KB, k = (b - r * KB) * kFp8Block + (threadIdx.x & 15) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
      int64_t at = first + r;
      if (MODE != kStreamSlots && p.map.gather_div > 0) at /= p.map.gather_div;
      if (b < blocks && k < a.K) load8<SRC == kSrcCodes ? 0 : SRC>(static_cast<const T*>(s.x) + at * s.ldx + k, x);
    };
    auto put = [&](int b, const float (&x)[8]) __attribute__((always_inline)) {
      const float am = __uint_as_float(block_top(x));
      if (b >= blocks) return;
      const int r = b / KB, kb = b - r * KB;
      *reinterpret_cast<u32x2*>(staged + r * staged_row(KB) + kb * kFp8Block + (threadIdx.x & 15) * 8) =
          pack8(x, code_factor(am));
      if ((threadIdx.x & 15) == 0) const_cast<float*>(staged_scale)[b] = am / kFp8Max;
    };
    const int b0 = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < P; ++i) fetch(b0 + i * step, v[i]);
    load_all(range);
#pragma unroll
    for (int i = 0; i < P; ++i) put(b0 + i * step, v[i]);
    for (int b = b0 + P * step; b - b0 < blocks; b += step) {
      fetch(b, v[0]);
      put(b, v[0]);
    }
    __syncthreads();
  } else {
    load_all(range);
  }
  for (int it = range; it < items; it += D * S) {
    if (it > range) load_all(it);
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (it + d * S < items) multiply(st[d]);
  }

  auto finish = [&](int64_t n, int t, f32x4 r, const f32x4& up) __attribute__((always_inline)) {
    if constexpr (GATED) {
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = silu_mul(r[e], up[e]);
    }
    if (16 * t + u >= rows) return;
    int64_t at = first + 16 * t + u;
    if constexpr (MODE == kStreamSlots) at = by;
    else if (p.map.scatter) at = p.map.pair[at];
    store4(a, at, n + 4 * g, r);
  };
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) red[range][(group * NT + i) * MT + t][lane] = acc[i][t];
  __syncthreads();
  // wave v finishes the workgroup's output fragments v, v + 8, ...
  for (int f = wave; f < G * NC * MT; f += kStreamWaves) {
    const int t = f % MT, i = f / MT % NC, gr = f / (MT * NC);
    auto total = [&](int n) __attribute__((always_inline)) {
      f32x4 sum = red[0][(gr * NT + n) * MT + t][lane];
#pragma unroll
      for (int v = 1; v < S; ++v) sum += red[v][(gr * NT + n) * MT + t][lane];
      return sum;
    };
    const f32x4 r = total(i);
    finish((static_cast<int64_t>(bx) * G + gr) * (16 * NC) + 16 * i, t, r, GATED ? total(i + NC) : r);
  }
}

// Starts the kernel over the columns of w and `tiles` tiles of rows; staged: rows to quantise.
template <int MT, int NT, int S, int SRC, int MODE>
hipError_t start_stream(const StreamArgs& st, int64_t tiles, int staged, hipStream_t s) {
  constexpr int cols = 16 * NT * (kStreamWaves / S) / (MODE == kStreamGated ? 2 : 1);
  const int lds = SRC == kSrcCodes ? 0 : staged_bytes(staged, static_cast<int>(fp8_blocks(st.p.a.K)));
  const int64_t along = (st.p.a.N + cols - 1) / cols;
  if (tiles > 65535 || !grid_fits(along, kStreamThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<uint32_t>(along), static_cast<uint32_t>(tiles));
  fp8_stream_kernel<MT, NT, S, SRC, MODE><<<grid, kStreamThreads, lds, s>>>(st);
  return hipGetLastError();
}
template <int NT, int S, int MODE>
hipError_t start_stream_x(const StreamArgs& st, int xdtype, int64_t tiles, int staged, hipStream_t s) {
  return xdtype == BL_F16    ? start_stream<1, NT, S, BL_F16, MODE>(st, tiles, staged, s)
         : xdtype == BL_BF16 ? start_stream<1, NT, S, BL_BF16, MODE>(st, tiles, staged, s)
                             : start_stream<1, NT, S, BL_F32, MODE>(st, tiles, staged, s);
}

}  // namespace
}  // namespace bl
