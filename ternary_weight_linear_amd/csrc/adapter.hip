// Low-rank adapters of many requests beside a shared projection, and their gradients. The contract
// is bl_adapter_forward and bl_adapter_backward in include/libbitlinear.h. Row m has adapter
// e = index[m], whose matrices are a[e] [R, K] and b[e] [R, N], both with rows along the long axis:
//
//   forward    h = a x,            y  = base + s b^T h
//   backward   dh = s b dy,        dx = base + a^T dh,     da = sum_m dh x^T,   db = sum_m s h dy^T
//
// so three products serve both directions: a product over the long axis (shrink), one along it
// (expand) and a sum over rows (outer). Rows are sorted by adapter, in tiles of 32 rows of one
// adapter each.
#include <algorithm>

#include "adapter_internal.h"

namespace bl {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));

constexpr int kTile = 32;                           // sorted rows of one adapter

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int rank_pad(int64_t R) { return static_cast<int>(div_up(R, 16) * 16); }
inline int64_t max_tiles(int64_t M, int64_t L) { return M / kTile + std::min(M, L + 1); }

// ------------------------------------------------------------------------------------------
// eight consecutive values of a row
// ------------------------------------------------------------------------------------------
template <int DT>
struct Eight {
  u32x4 w;
};
template <>
struct Eight<BL_F32> {
  f32x4 w[2];
};

// Values at .. at + 7 of a row of n; those from n on are 0. VEC: whole pieces, 16-byte aligned.
template <int DT, bool VEC>
__device__ __forceinline__ Eight<DT> load8(const typename Elem<DT>::type* row, int64_t at, int64_t n) {
  Eight<DT> v{};
  if constexpr (VEC) {
    if (at < n) v = *reinterpret_cast<const Eight<DT>*>(row + at);
  } else if constexpr (DT == BL_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j < n) v.w[j / 4][j % 4] = row[at + j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j < n) v.w[j / 2] |= static_cast<uint32_t>(row[at + j]) << (16 * (j & 1));
  }
  return v;
}

template <int DT>
__device__ __forceinline__ float value(const Eight<DT>& v, int j) {
  if constexpr (DT == BL_F32) return v.w[j / 4][j % 4];
  else return to_float<DT>(static_cast<uint16_t>(v.w[j / 2] >> (16 * (j & 1))));
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(typename Elem<DT>::type* row, int64_t at, int64_t n, const float (&v)[8]) {
  if constexpr (DT == BL_F32) {
    if constexpr (VEC) {
      if (at >= n) return;
      *reinterpret_cast<f32x4*>(row + at) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(row + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < n) row[at + j] = v[j];
    }
  } else {
    uint16_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = DT == BL_BF16 ? bf16_bits(v[j]) : half_bits(v[j]);
    if constexpr (VEC) {
      if (at >= n) return;
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = b[2 * j] | static_cast<uint32_t>(b[2 * j + 1]) << 16;
      *reinterpret_cast<u32x4*>(row + at) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < n) row[at + j] = b[j];
    }
  }
}

// ------------------------------------------------------------------------------------------
// rows sorted by adapter
// ------------------------------------------------------------------------------------------
// The sort is stable, so that sums over an adapter's rows have one order. A chunk of 8192 rows per
// workgroup, 512 per wave; more than one chunk: a first launch counts, the second places. Bucket L
// holds the rows without an adapter. Each bucket starts a tile of its own.
constexpr int kSortWaves = 16, kSortSteps = 8;
constexpr int kSortChunk = kSortWaves * 64 * kSortSteps;

struct SortArgs {
  const int32_t* index;
  int64_t M;
  int L, chunks;
  int32_t* order;
  int32_t* tile;
  int32_t* start;
  int32_t* counts;      // [chunks, L + 1]
};

inline size_t sort_lds(int64_t L) { return static_cast<size_t>(L + 1) * (kSortWaves * 2 + 8); }

// MODE 0: the only chunk. 1: this chunk's counts. 2: its places, from all chunks' counts.
template <int MODE>
__global__ __launch_bounds__(64 * kSortWaves) void adapter_sort_kernel(SortArgs a) {
  extern __shared__ int lds[];
  __shared__ int sums[kSortWaves];
  const int B = a.L + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* total = lds;                                 // [B] rows of each bucket
  int* place = lds + B;                             // [B] first place of this chunk's rows
  uint16_t* cnt = reinterpret_cast<uint16_t*>(lds + 2 * B);   // [waves, B]
  for (int i = threadIdx.x; i < B * kSortWaves; i += blockDim.x) cnt[i] = 0;
  __syncthreads();

  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kSortChunk + wave * 64 * kSortSteps + lane;
  int e[kSortSteps], rank[kSortSteps];
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i) {
    const int64_t m = m0 + 64 * i;
    e[i] = -1;
    if (m < a.M) {
      const int v = a.index[m];
      e[i] = v >= 0 && v < a.L ? v : a.L;
    }
  }
  // rank of each row among those of its bucket in its wave; one round per bucket of 64 rows
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i) {
    rank[i] = 0;
    uint64_t left = __ballot(e[i] >= 0);
    while (left) {
      const int b = __builtin_amdgcn_readlane(e[i], __builtin_ctzll(left));
      const uint64_t same = __ballot(e[i] == b);
      const int before = cnt[wave * B + b];
      if (e[i] == b) rank[i] = before + __popcll(same & ((1ull << lane) - 1));
      __builtin_amdgcn_wave_barrier();
      if (lane == 0) cnt[wave * B + b] = static_cast<uint16_t>(before + __popcll(same));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      left &= ~same;
    }
  }
  __syncthreads();
  // counts per wave become the rows of earlier waves
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = cnt[w * B + b];
      cnt[w * B + b] = static_cast<uint16_t>(sum);
      sum += n;
    }
    if constexpr (MODE == 1) a.counts[static_cast<int64_t>(blockIdx.x) * B + b] = sum;
    total[b] = sum;
    place[b] = 0;
  }
  if constexpr (MODE == 1) return;
  if constexpr (MODE == 2) {
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
      int all = 0, before = 0;
      for (int c = 0; c < a.chunks; ++c) {
        const int n = a.counts[static_cast<int64_t>(c) * B + b];
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
        all += n;
      }
      total[b] = all;
      place[b] = before;
    }
  }
  __syncthreads();
  // first tile of each bucket: each thread has a run of buckets
  const int per = (B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
  const int b0 = min(static_cast<int>(threadIdx.x) * per, B), b1 = min(b0 + per, B);
  int tiles = 0;
  for (int b = b0; b < b1; ++b) tiles += (total[b] + kTile - 1) / kTile;
  int at = tiles;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int t = __shfl_up(at, off);
    if (lane >= off) at += t;
  }
  if (lane == 63) sums[wave] = at;
  __syncthreads();
  for (int w = 0; w < wave; ++w) at += sums[w];
  at -= tiles;
  const bool first = blockIdx.x == 0;
  for (int b = b0; b < b1; ++b) {
    const int n = (total[b] + kTile - 1) / kTile;
    place[b] += at * kTile;
    if (first) {
      a.start[b] = at;
      if (b == a.L) a.start[B] = at + n;
      for (int t = 0; t < n; ++t) a.tile[at + t] = b;
      for (int i = total[b]; i < n * kTile; ++i) a.order[static_cast<int64_t>(at) * kTile + i] = -1;
    }
    at += n;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i)
    if (e[i] >= 0) a.order[place[e[i]] + cnt[wave * B + e[i]] + rank[i]] = static_cast<int32_t>(m0 + 64 * i);
}

// ------------------------------------------------------------------------------------------
// shrink: part[split, row, r] = sum over the split's k of S[row, k] w[e, r, k]
// ------------------------------------------------------------------------------------------
struct Sorted {
  const int32_t* order;
  const int32_t* tile;
  const int32_t* start;
  int L;
  int64_t rows;           // places: 32 max_tiles
};

struct ShrinkArgs {
  Sorted o;
  const void* s;
  int64_t D, ld;
  const void* w;          // [L, R, D]
  int R, RP, splits;
  float* part;
};

template <int DT>
__device__ __forceinline__ f32x4 dot32(const Eight<DT>& s, const Eight<DT>& w, f32x4 acc) {
  if constexpr (DT == BL_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, s.w), __builtin_bit_cast(half8v, w.w), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, s.w), __builtin_bit_cast(bf8v, w.w), acc, 0, 0, 0);
}

template <int SD, int WD, int NR, bool VEC>
__global__ __launch_bounds__(256) void adapter_shrink_kernel(ShrinkArgs a) {
  __shared__ float red[4][kTile][16 * NR];
  const int t = blockIdx.x;
  if (t >= a.o.start[a.o.L]) return;
  const int e = a.o.tile[t];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.z * 16 * NR;
  using S = typename Elem<SD>::type;
  using W = typename Elem<WD>::type;
  const S* row[2];
  int64_t n[2];                                     // no row: nothing is read
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = a.o.order[static_cast<int64_t>(t) * kTile + 16 * i + c];
    row[i] = static_cast<const S*>(a.s) + static_cast<int64_t>(m < 0 ? 0 : m) * a.ld;
    n[i] = m < 0 ? 0 : a.D;
  }
  const W* w[NR];
  int64_t nw[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + 16 * i + c;
    w[i] = static_cast<const W*>(a.w) + (static_cast<int64_t>(e) * a.R + min(r, a.R - 1)) * a.D;
    nw[i] = r < a.R ? a.D : 0;
  }
  f32x4 acc[2][NR] = {};
  const int64_t units = (a.D + 63) / 64;
  const int64_t u0 = units * blockIdx.y / a.splits, u1 = units * (blockIdx.y + 1) / a.splits;
#pragma unroll 2
  for (int64_t u = u0 + wave; u < u1; u += 4) {
    Eight<SD> sv[2][2];
    Eight<WD> wv[2][NR];
    const int64_t k = u * 64 + g * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) sv[j][i] = load8<SD, VEC>(row[i], k + 8 * j, n[i]);
#pragma unroll
      for (int i = 0; i < NR; ++i) wv[j][i] = load8<WD, VEC>(w[i], k + 8 * j, nw[i]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          if constexpr (SD == WD && SD != BL_F32) {
            acc[i][q] = dot32<SD>(sv[j][i], wv[j][q], acc[i][q]);
          } else {
#pragma unroll
            for (int l = 0; l < 8; ++l)
              acc[i][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(value<SD>(sv[j][i], l), value<WD>(wv[j][q], l), acc[i][q], 0, 0, 0);
          }
        }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < NR; ++q)
#pragma unroll
      for (int l = 0; l < 4; ++l) red[wave][16 * i + 4 * g + l][16 * q + c] = acc[i][q][l];
  __syncthreads();
  float* out = a.part + (blockIdx.y * a.o.rows + static_cast<int64_t>(t) * kTile) * a.RP + r0;
  for (int i = threadIdx.x; i < kTile * 16 * NR; i += 256) {
    const int m = i / (16 * NR), r = i % (16 * NR);
    if (r0 + r < a.RP) out[m * a.RP + r] = red[0][m][r] + red[1][m][r] + red[2][m][r] + red[3][m][r];
  }
}

// ------------------------------------------------------------------------------------------
// expand: y[row, n] = base[row, n] + sum_r c[row, r] w[e, r, n]
// ------------------------------------------------------------------------------------------
struct ExpandArgs {
  Sorted o;
  const float* c;         // [splits, rows, RP], summed here
  int splits;
  int R, RP;
  const float* scale;     // [L] or null
  float* h;               // [M, R] or null: the sums without the scale
  const void* w;          // [L, R, N]
  int64_t N;
  const void* base;
  int64_t ldbase;
  void* y;
  int64_t ldy;
};

template <int WD, int YD, bool VEC>
__global__ __launch_bounds__(256) void adapter_expand_kernel(ExpandArgs a) {
  extern __shared__ float cl[];                     // [32][RP + 4]
  __shared__ int rows[kTile];
  const int t = blockIdx.x;
  if (t >= a.o.start[a.o.L + 1]) return;
  const int e = a.o.tile[t], lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int pitch = a.RP + 4;
  const bool none = e >= a.o.L;
  if (none && a.base == a.y && (!a.h || blockIdx.y)) return;
  if (threadIdx.x < kTile) rows[threadIdx.x] = a.o.order[static_cast<int64_t>(t) * kTile + threadIdx.x];
  const float f = a.scale && !none ? a.scale[e] : 1.0f;
  for (int i = threadIdx.x; i < kTile * a.RP; i += 256) {
    const int m = i / a.RP, r = i % a.RP;
    float v = 0.0f;
    if (!none)
      for (int s = 0; s < a.splits; ++s) v += a.c[(s * a.o.rows + static_cast<int64_t>(t) * kTile + m) * a.RP + r];
    if (a.h && blockIdx.y == 0 && r < a.R) {
      const int row = a.o.order[static_cast<int64_t>(t) * kTile + m];
      if (row >= 0) a.h[static_cast<int64_t>(row) * a.R + r] = v;
    }
    cl[m * pitch + r] = v * f;
  }
  __syncthreads();
  const int64_t n0 = (static_cast<int64_t>(blockIdx.y) * 4 + wave) * 128, n = n0 + 8 * c;
  if (n0 >= a.N) return;
  using W = typename Elem<WD>::type;
  using Y = typename Elem<YD>::type;
  f32x4 acc[2][8] = {};
  if (!none) {
    const W* w = static_cast<const W*>(a.w) + static_cast<int64_t>(e) * a.R * a.N;
    for (int r0 = 0; r0 < a.RP; r0 += 16) {
      Eight<WD> wv[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int r = r0 + 4 * s + g;
        wv[s] = load8<WD, VEC>(w + static_cast<int64_t>(min(r, a.R - 1)) * a.N, n, r < a.R ? a.N : 0);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float c0 = cl[c * pitch + r0 + 4 * s + g], c1 = cl[(16 + c) * pitch + r0 + 4 * s + g];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = value<WD>(wv[s], j);
          acc[0][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(c0, v, acc[0][j], 0, 0, 0);
          acc[1][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(c1, v, acc[1][j], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const int row = rows[16 * i + 4 * g + l];
      if (row < 0) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[i][j][l];
      if (a.base) {
        const Eight<YD> b = load8<YD, VEC>(static_cast<const Y*>(a.base) + row * a.ldbase, n, a.N);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = none ? value<YD>(b, j) : value<YD>(b, j) + v[j];
      }
      store8<YD, VEC>(static_cast<Y*>(a.y) + row * a.ldy, n, a.N, v);
    }
}

// ------------------------------------------------------------------------------------------
// dh and the scaled h, sorted; places without a row are 0
// ------------------------------------------------------------------------------------------
struct FinishArgs {
  Sorted o;
  const float* part;      // [splits, rows, RP]
  int splits, R, RP;
  const float* scale;
  const float* h;         // [M, R]
  float* dh;              // [rows, RP]
  float* hs;              // [rows, RP]
};

__global__ __launch_bounds__(256) void adapter_finish_kernel(FinishArgs a) {
  const int t = blockIdx.x;
  if (t >= a.o.start[a.o.L]) return;
  const int e = a.o.tile[t];
  const float f = a.scale ? a.scale[e] : 1.0f;
  const int64_t at = static_cast<int64_t>(t) * kTile;
  for (int i = threadIdx.x; i < kTile * a.RP; i += 256) {
    const int m = i / a.RP, r = i % a.RP;
    const int row = a.o.order[at + m];
    float v = 0.0f, h = 0.0f;
    if (row >= 0 && r < a.R) {
      for (int s = 0; s < a.splits; ++s) v += a.part[(s * a.o.rows + at + m) * a.RP + r];
      h = a.h[static_cast<int64_t>(row) * a.R + r];
    }
    a.dh[at * a.RP + i] = v * f;
    a.hs[at * a.RP + i] = h * f;
  }
}

// ------------------------------------------------------------------------------------------
// outer: grad[e, r, d] = sum over the adapter's rows of c[row, r] S[row, d]
// ------------------------------------------------------------------------------------------
// Tiles are split evenly over workgroups. An adapter that lies within one split is written at
// once; the pieces of the others go to sum[2 split], where the adapter began in an earlier split,
// or sum[2 split + 1], and meet in adapter_gather_kernel in their order.
struct OuterArgs {
  Sorted o;
  const float* c;         // [rows, RP]
  const void* s;
  int64_t D, ld;
  int R, RP, splits;
  float* sum;             // [2 splits, R, D]
  float* grad;            // [L, R, D]
  int add;
};

template <int SD, int NR, bool VEC>
__global__ __launch_bounds__(256) void adapter_outer_kernel(OuterArgs a) {
  __shared__ float red[16 * NR][128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int64_t d0 = static_cast<int64_t>(blockIdx.x) * 128;
  const int r0 = blockIdx.z * 16 * NR;
  const int64_t tiles = a.o.start[a.o.L];
  const int t1 = static_cast<int>(tiles * (blockIdx.y + 1) / a.splits);
  using S = typename Elem<SD>::type;
  for (int t = static_cast<int>(tiles * blockIdx.y / a.splits); t < t1;) {
    const int e = a.o.tile[t], first = a.o.start[e], last = a.o.start[e + 1];
    const int end = min(last, t1);
    f32x4 acc[NR][8] = {};
    for (int i = t + wave; i < end; i += 4) {
      const int64_t at = static_cast<int64_t>(i) * kTile;
      Eight<SD> sv[8];
      float cv[8][NR];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int row = a.o.order[at + 4 * s + g];
        sv[s] = load8<SD, VEC>(static_cast<const S*>(a.s) + static_cast<int64_t>(row < 0 ? 0 : row) * a.ld, d0 + 8 * c, row < 0 ? 0 : a.D);
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          const int r = r0 + 16 * q + c;
          cv[s][q] = r < a.RP ? a.c[(at + 4 * s + g) * a.RP + r] : 0.0f;
        }
      }
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = value<SD>(sv[s], j);
#pragma unroll
          for (int q = 0; q < NR; ++q) acc[q][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(cv[s][q], v, acc[q][j], 0, 0, 0);
        }
    }
    // the waves' sums, one after another
    for (int w = 0; w < 4; ++w) {
      if (wave == w) {
#pragma unroll
        for (int q = 0; q < NR; ++q)
#pragma unroll
          for (int l = 0; l < 4; ++l)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float& p = red[16 * q + 4 * g + l][8 * c + j];
              p = w ? p + acc[q][j][l] : acc[q][j][l];
            }
      }
      __syncthreads();
    }
    const bool whole = first >= t && last <= end;
    float* out = whole ? a.grad + static_cast<int64_t>(e) * a.R * a.D
                       : a.sum + (2 * static_cast<int64_t>(blockIdx.y) + (first >= t ? 1 : 0)) * a.R * a.D;
    for (int i = threadIdx.x; i < 16 * NR * 128; i += 256) {
      const int r = r0 + i / 128;
      const int64_t d = d0 + i % 128;
      if (r < a.R && d < a.D) {
        float* p = out + r * a.D + d;
        *p = whole && a.add ? *p + red[i / 128][i % 128] : red[i / 128][i % 128];
      }
    }
    __syncthreads();
    t = end;
  }
}

__global__ __launch_bounds__(256) void adapter_gather_kernel(OuterArgs a) {
  const int64_t n = static_cast<int64_t>(a.R) * a.D;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 1024 + threadIdx.x;
  const int64_t tiles = a.o.start[a.o.L];
  for (int e = blockIdx.y; e < a.o.L; e += gridDim.y) {
    const int64_t first = a.o.start[e], last = a.o.start[e + 1];
    float* grad = a.grad + e * n;
    if (first == last) {
      if (!a.add)
        for (int i = 0; i < 4; ++i)
          if (at + 256 * i < n) grad[at + 256 * i] = 0.0f;
      continue;
    }
    // the split of tile t is the largest s whose first tile, floor(s tiles / splits), is not past t
    const int64_t s0 = ((first + 1) * a.splits - 1) / tiles, s1 = (last * a.splits - 1) / tiles;
    if (s0 == s1) continue;
    for (int i = 0; i < 4; ++i) {
      const int64_t d = at + 256 * i;
      if (d >= n) break;
      float v = a.sum[(2 * s0 + 1) * n + d];
      for (int64_t s = s0 + 1; s <= s1; ++s) v += a.sum[2 * s * n + d];
      grad[d] = a.add ? grad[d] + v : v;
    }
  }
}

// ------------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------------
int shrink_splits(int64_t M, int64_t L, int64_t R, int64_t D) {
  const int64_t groups = max_tiles(M, L) * div_up(rank_pad(R), 64);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({1024 / groups, div_up(D, 64) / 8, 16})));
}
int outer_splits(int64_t M, int64_t R, int64_t D) {
  const int64_t groups = div_up(D, 128) * div_up(rank_pad(R), 64);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({1024 / groups, div_up(M, 4 * kTile), 32})));
}

struct Scratch {
  Sorted o;
  int32_t* order;
  int32_t* tile;
  int32_t* start;
  int32_t* counts;
  float *part, *c, *sum;
};
Scratch scratch(const AdapterWs& L, char* ws, const AdapterRows& r) {
  Scratch s{};
  s.order = reinterpret_cast<int32_t*>(ws + L.order_off);
  s.tile = reinterpret_cast<int32_t*>(ws + L.tile_off);
  s.start = reinterpret_cast<int32_t*>(ws + L.start_off);
  s.counts = reinterpret_cast<int32_t*>(ws + L.count_off);
  s.part = reinterpret_cast<float*>(ws + L.part_off);
  s.c = reinterpret_cast<float*>(ws + L.c_off);
  s.sum = reinterpret_cast<float*>(ws + L.sum_off);
  s.o = Sorted{s.order, s.tile, s.start, static_cast<int>(r.L), max_tiles(r.M, r.L) * kTile};
  return s;
}

hipError_t sort_rows(const AdapterRows& r, const Scratch& w, hipStream_t s) {
  SortArgs a{r.index, r.M, static_cast<int>(r.L), static_cast<int>(div_up(r.M, kSortChunk)), w.order, w.tile, w.start, w.counts};
  const size_t lds = sort_lds(r.L);
  if (a.chunks == 1) {
    adapter_sort_kernel<0><<<1, 64 * kSortWaves, lds, s>>>(a);
    return hipGetLastError();
  }
  adapter_sort_kernel<1><<<a.chunks, 64 * kSortWaves, lds, s>>>(a);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  adapter_sort_kernel<2><<<a.chunks, 64 * kSortWaves, lds, s>>>(a);
  return hipGetLastError();
}

// Whether rows of n values of either type are whole, aligned pieces of eight.
bool vec_rows(const void* p, int64_t n, int64_t ld) {
  return !p || (n % 8 == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0);
}

template <int SD, int WD, bool VEC>
hipError_t start_shrink_nr(const ShrinkArgs& a, int64_t tiles, hipStream_t s) {
  const int nr = std::min(a.RP / 16, 4);
  const dim3 grid(static_cast<uint32_t>(tiles), a.splits, static_cast<uint32_t>(div_up(a.RP, 64)));
  if (nr == 1) adapter_shrink_kernel<SD, WD, 1, VEC><<<grid, 256, 0, s>>>(a);
  else if (nr == 2) adapter_shrink_kernel<SD, WD, 2, VEC><<<grid, 256, 0, s>>>(a);
  else if (nr == 3) adapter_shrink_kernel<SD, WD, 3, VEC><<<grid, 256, 0, s>>>(a);
  else adapter_shrink_kernel<SD, WD, 4, VEC><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <int SD, int WD>
hipError_t start_shrink_vec(const ShrinkArgs& a, int64_t tiles, hipStream_t s) {
  return vec_rows(a.s, a.D, a.ld) && vec_rows(a.w, a.D, a.D) ? start_shrink_nr<SD, WD, true>(a, tiles, s)
                                                              : start_shrink_nr<SD, WD, false>(a, tiles, s);
}
// sd is wd, or fp32.
hipError_t start_shrink(const ShrinkArgs& a, int sd, int wd, int64_t tiles, hipStream_t s) {
  if (wd == BL_F16) return sd == BL_F16 ? start_shrink_vec<BL_F16, BL_F16>(a, tiles, s) : start_shrink_vec<BL_F32, BL_F16>(a, tiles, s);
  if (wd == BL_BF16) return sd == BL_BF16 ? start_shrink_vec<BL_BF16, BL_BF16>(a, tiles, s) : start_shrink_vec<BL_F32, BL_BF16>(a, tiles, s);
  return start_shrink_vec<BL_F32, BL_F32>(a, tiles, s);
}

template <int WD, int YD>
hipError_t start_expand_vec(const ExpandArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(tiles), static_cast<uint32_t>(div_up(a.N, 512)));
  const size_t lds = static_cast<size_t>(kTile) * (a.RP + 4) * 4;
  if (vec_rows(a.w, a.N, a.N) && vec_rows(a.base, a.N, a.ldbase) && vec_rows(a.y, a.N, a.ldy))
    adapter_expand_kernel<WD, YD, true><<<grid, 256, lds, s>>>(a);
  else
    adapter_expand_kernel<WD, YD, false><<<grid, 256, lds, s>>>(a);
  return hipGetLastError();
}
// yd is wd, or fp32.
hipError_t start_expand(const ExpandArgs& a, int wd, int yd, int64_t tiles, hipStream_t s) {
  if (wd == BL_F16) return yd == BL_F16 ? start_expand_vec<BL_F16, BL_F16>(a, tiles, s) : start_expand_vec<BL_F16, BL_F32>(a, tiles, s);
  if (wd == BL_BF16) return yd == BL_BF16 ? start_expand_vec<BL_BF16, BL_BF16>(a, tiles, s) : start_expand_vec<BL_BF16, BL_F32>(a, tiles, s);
  return start_expand_vec<BL_F32, BL_F32>(a, tiles, s);
}

template <int SD, bool VEC>
hipError_t start_outer_nr(const OuterArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(div_up(a.D, 128)), a.splits, static_cast<uint32_t>(div_up(a.RP, 64)));
  const int nr = std::min(a.RP / 16, 4);
  if (nr == 1) adapter_outer_kernel<SD, 1, VEC><<<grid, 256, 0, s>>>(a);
  else if (nr == 2) adapter_outer_kernel<SD, 2, VEC><<<grid, 256, 0, s>>>(a);
  else if (nr == 3) adapter_outer_kernel<SD, 3, VEC><<<grid, 256, 0, s>>>(a);
  else adapter_outer_kernel<SD, 4, VEC><<<grid, 256, 0, s>>>(a);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const dim3 each(static_cast<uint32_t>(div_up(static_cast<int64_t>(a.R) * a.D, 1024)), static_cast<uint32_t>(a.o.L));
  adapter_gather_kernel<<<each, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <int SD>
hipError_t start_outer_vec(const OuterArgs& a, hipStream_t s) {
  return vec_rows(a.s, a.D, a.ld) ? start_outer_nr<SD, true>(a, s) : start_outer_nr<SD, false>(a, s);
}
hipError_t start_outer(const OuterArgs& a, int sd, hipStream_t s) {
  return sd == BL_F16 ? start_outer_vec<BL_F16>(a, s) : sd == BL_BF16 ? start_outer_vec<BL_BF16>(a, s) : start_outer_vec<BL_F32>(a, s);
}

}  // namespace

AdapterWs adapter_ws(int64_t M, int64_t L, int64_t R, int64_t K, int64_t N, bool backward) {
  AdapterWs w{};
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += (static_cast<size_t>(bytes) + 255) & ~size_t(255);
    return at;
  };
  const int64_t tiles = max_tiles(M, L), rows = tiles * kTile, RP = rank_pad(R), D = backward ? N : K;
  w.order_off = take(rows * 4);
  w.tile_off = take(tiles * 4);
  w.start_off = take((L + 2) * 4);
  w.count_off = take(M > kSortChunk ? div_up(M, kSortChunk) * (L + 1) * 4 : 0);
  w.part_off = take(shrink_splits(M, L, R, D) * rows * RP * 4);
  w.c_off = take(backward ? 2 * rows * RP * 4 : 0);
  w.sum_off = take(backward ? 2 * std::max(outer_splits(M, R, K) * R * K, outer_splits(M, R, N) * R * N) * 4 : 0);
  w.total = off;
  return w;
}

hipError_t launch_adapter_forward(const AdapterForwardArgs& a, char* ws, hipStream_t s) {
  const AdapterRows& r = a.rows;
  const Scratch w = scratch(adapter_ws(r.M, r.L, r.R, a.K, a.N, false), ws, r);
  const int64_t tiles = max_tiles(r.M, r.L);
  const int R = static_cast<int>(r.R), RP = rank_pad(r.R), splits = shrink_splits(r.M, r.L, r.R, a.K);
  hipError_t e = sort_rows(r, w, s);
  if (e != hipSuccess) return e;
  e = start_shrink(ShrinkArgs{w.o, a.x, a.K, a.ldx, a.a, R, RP, splits, w.part}, a.dtype, a.dtype, tiles, s);
  if (e != hipSuccess) return e;
  return start_expand(ExpandArgs{w.o, w.part, splits, R, RP, a.scale, a.h, a.b, a.N, a.base, a.ldbase, a.y, a.ldy},
                      a.dtype, a.ydtype, tiles, s);
}

hipError_t launch_adapter_backward(const AdapterBackwardArgs& a, char* ws, hipStream_t s) {
  const AdapterRows& r = a.rows;
  const Scratch w = scratch(adapter_ws(r.M, r.L, r.R, a.K, a.N, true), ws, r);
  const int64_t tiles = max_tiles(r.M, r.L);
  const int R = static_cast<int>(r.R), RP = rank_pad(r.R), splits = shrink_splits(r.M, r.L, r.R, a.N);
  float *dh = w.c, *hs = w.c + w.o.rows * RP;
  hipError_t e = sort_rows(r, w, s);
  if (e != hipSuccess) return e;
  e = start_shrink(ShrinkArgs{w.o, a.dy, a.N, a.lddy, a.b, R, RP, splits, w.part}, a.dydtype, a.dtype, tiles, s);
  if (e != hipSuccess) return e;
  adapter_finish_kernel<<<static_cast<uint32_t>(tiles), 256, 0, s>>>(FinishArgs{w.o, w.part, splits, R, RP, a.scale, a.h, dh, hs});
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.dx) {
    e = start_expand(ExpandArgs{w.o, dh, 1, R, RP, nullptr, nullptr, a.a, a.K, a.base, a.ldbase, a.dx, a.lddx}, a.dtype, a.dxdtype, tiles, s);
    if (e != hipSuccess) return e;
  }
  e = start_outer(OuterArgs{w.o, dh, a.x, a.K, a.ldx, R, RP, outer_splits(r.M, r.R, a.K), w.sum, a.da, a.add}, a.dtype, s);
  if (e != hipSuccess) return e;
  return start_outer(OuterArgs{w.o, hs, a.dy, a.N, a.lddy, R, RP, outer_splits(r.M, r.R, a.N), w.sum, a.db, a.add}, a.dydtype, s);
}

}  // namespace bl
