// Low-rank adapters of many requests beside a shared projection, and their gradients. The contract
// is bl_adapter_forward and bl_adapter_backward in include/libbitlinear.h. Row m has adapter
// e = index[m], whose matrices are a[e] [R, K] and b[e] [R, N], both with rows along the long axis:
//
//   forward    h = a x,            y  = base + s b^T h
//   backward   dh = s b dy,        dx = base + a^T dh,     da = sum_m dh x^T,   db = sum_m s h dy^T
//
// so three products serve both directions: a product over the long axis (shrink), one along it
// (expand) and a sum over rows (outer). Rows are sorted by adapter, in tiles of 32 rows of one
// adapter each; few rows of a forward pass go each by itself. All of it moves far more bytes than it
// computes, so each kernel's loads decide: how many are in flight, and how many lines a load touches
// (a quarter wave is served one line a clock).
#include <algorithm>
#include <type_traits>

#include "adapter_internal.h"
#include "bl_internal.h"

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
// The hardware reads and writes 16 bytes at any address that its elements' alignment allows, so rows of
// any length and stride go eight values at a time; a row's last piece may be shorter.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <int DT>
struct Eight {
  u32x4 w;
};
template <>
struct Eight<BL_F32> {
  f32x4 w[2];
};

template <int DT>
__device__ __forceinline__ Eight<DT> load_whole(const typename Elem<DT>::type* p) {
  Eight<DT> v;
  if constexpr (DT == BL_F32) {
    v.w[0] = *reinterpret_cast<const f32x4_any*>(p);
    v.w[1] = *reinterpret_cast<const f32x4_any*>(p + 4);
  } else {
    v.w = *reinterpret_cast<const u32x4_any*>(p);
  }
  return v;
}
// Dwords v moved down by s (of N) dwords, zeros behind them.
template <int N>
__device__ __forceinline__ void move_down(uint32_t (&v)[N], int s) {
#pragma unroll
  for (int step = N / 2; step > 0; step >>= 1)
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = s & step ? (j + step < N ? v[j + step] : 0) : v[j];
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = s < N ? v[j] : 0;
}
// Values at .. at + N - 1 of a row of n as dwords; those from n on are 0. Where the row ends inside, its
// last N values are loaded and moved down, so that no load is under a condition.
template <int DT, int N>
__device__ __forceinline__ void load_end(const typename Elem<DT>::type* row, int64_t at, int64_t n,
                                         uint32_t (&v)[N * sizeof(typename Elem<DT>::type) / 4]) {
  constexpr int W = N * sizeof(*row) / 4;           // dwords
  if (n < N) {                                      // uniform: a row shorter than a piece
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (at + j < n) {
        if constexpr (DT == BL_F32) v[j] = __float_as_uint(row[at + j]);
        else v[j / 2] |= static_cast<uint32_t>(row[at + j]) << (16 * (j & 1));
      }
    return;
  }
  const int64_t from = min(at, n - N);
  const int s = static_cast<int>(min(at - from, static_cast<int64_t>(2 * N)));
#pragma unroll
  for (int j = 0; j < W; j += 4) {
    const u32x4 w = *reinterpret_cast<const u32x4_any*>(row + from + 4 * j / static_cast<int>(sizeof(*row)));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[j + k] = w[k];
  }
  if constexpr (DT == BL_F32) {
    move_down<W>(v, s);
  } else {
    move_down<W>(v, s / 2);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t next = j + 1 < W ? v[j + 1] : 0;
      v[j] = s & 1 ? __builtin_amdgcn_alignbit(next, v[j], 16) : v[j];
    }
  }
}
// Values at .. at + 7 of a row of n; those from n on are 0. WHOLE: there are none.
template <int DT, bool WHOLE>
__device__ __forceinline__ Eight<DT> load8(const typename Elem<DT>::type* row, int64_t at, int64_t n) {
  if constexpr (WHOLE) return load_whole<DT>(row + at);
  uint32_t w[sizeof(Eight<DT>) / 4];
  load_end<DT, 8>(row, at, n, w);
  Eight<DT> v;
  if constexpr (DT == BL_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v.w[j / 4][j % 4] = __uint_as_float(w[j]);
  } else {
    v.w = u32x4{w[0], w[1], w[2], w[3]};
  }
  return v;
}
// A piece of 16 bytes of a row, its first value at `at`; values from n on are 0.
template <int DT, bool WHOLE>
__device__ __forceinline__ u32x4 load16(const typename Elem<DT>::type* row, int64_t at, int64_t n) {
  if constexpr (WHOLE) return *reinterpret_cast<const u32x4_any*>(row + at);
  uint32_t w[4];
  load_end<DT, 16 / sizeof(*row)>(row, at, n, w);
  return u32x4{w[0], w[1], w[2], w[3]};
}
template <int DT>
__device__ __forceinline__ Eight<DT> zero_unless(bool keep, Eight<DT> v) {
  return keep ? v : Eight<DT>{};
}

template <int DT>
__device__ __forceinline__ float value(const Eight<DT>& v, int j) {
  if constexpr (DT == BL_F32) return v.w[j / 4][j % 4];
  else return to_float<DT>(static_cast<uint16_t>(v.w[j / 2] >> (16 * (j & 1))));
}

template <int DT>
__device__ __forceinline__ uint16_t bits16(float v) {
  return DT == BL_BF16 ? bf16_bits(v) : half_bits(v);
}

// Places lo .. n - 1 of a row alone.
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type* row, int64_t at, int64_t lo, int64_t n, const float (&v)[8]) {
  if constexpr (DT == BL_F32) {
    if (at >= lo && at + 8 <= n) {
      *reinterpret_cast<f32x4_any*>(row + at) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_any*>(row + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
      return;
    }
  } else if (at >= lo && at + 8 <= n) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = bits16<DT>(v[2 * j]) | static_cast<uint32_t>(bits16<DT>(v[2 * j + 1])) << 16;
    *reinterpret_cast<u32x4_any*>(row + at) = w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (at + j >= lo && at + j < n) {
      if constexpr (DT == BL_F32) row[at + j] = v[j];
      else row[at + j] = bits16<DT>(v[j]);
    }
}

// Column j of eight rows of eight 16-bit values, as one matrix operand: one byte permutation for
// each pair of rows.
__device__ __forceinline__ u32x4 column(const u32x4 (&row)[8], int j) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __builtin_amdgcn_perm(row[2 * i + 1][j / 2], row[2 * i][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
  return v;
}

// 16 x 16 products over 32 values of 16 bits each.
template <int DT>
__device__ __forceinline__ f32x4 dot32(u32x4 a, u32x4 b, f32x4 acc) {
  if constexpr (DT == BL_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), acc, 0, 0, 0);
}

// ------------------------------------------------------------------------------------------
// fp32 coefficients as 16-bit parts
// ------------------------------------------------------------------------------------------
// h and dh are fp32, and what they are multiplied by has 16 bits. The 16-bit matrix instructions are 16
// times as fast as the fp32 one, so a coefficient is cut into three bf16 parts of 8 bits each, which
// hold all of its 24 bits that are not below 2^-133. fp16 values are cut into two bf16 parts, of 8 and
// 3 bits, so that their products are whole too: six instructions where fp16 parts would take two, but
// those have no range for rows or ranks far quieter than the loudest beside them. (4096 x 8192, fp16,
// six / two: rank 64 86 us / 82, gradients, rank 32, 105 / 107, where two need exponents.)
constexpr int kParts = 3;
template <int DT>
constexpr int kValueParts = DT == BL_F16 ? 2 : 1;

// Infinities and NaN are in the first part alone.
__device__ __forceinline__ void split(float v, uint16_t (&part)[kParts]) {
  const bool odd = abs_bits(v) >= 0x7F800000u;
  const uint32_t hi = odd ? static_cast<uint32_t>(bf16_bits(v)) << 16 : __float_as_uint(v) & 0xFFFF0000u;
  const float r = odd ? 0.0f : v - __uint_as_float(hi);
  const uint32_t mid = __float_as_uint(r) & 0xFFFF0000u;
  const float lo = r - __uint_as_float(mid);
  part[0] = static_cast<uint16_t>(hi >> 16);
  part[1] = static_cast<uint16_t>(mid >> 16);
  part[2] = static_cast<uint16_t>(__float_as_uint(lo) >> 16);
}
// Eight 16-bit values as bf16 parts. What is infinite or NaN is NaN in the second part.
template <int DT>
__device__ __forceinline__ void value_parts(u32x4 v, u32x4 (&part)[kValueParts<DT>]) {
  if constexpr (DT == BL_F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f[2] = {to_float<BL_F16>(static_cast<uint16_t>(v[i])), to_float<BL_F16>(static_cast<uint16_t>(v[i] >> 16))};
      uint32_t b[2], r[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        b[j] = __float_as_uint(f[j]);
        r[j] = __float_as_uint(f[j] - __uint_as_float(b[j] & 0xFFFF0000u));
      }
      part[0][i] = __builtin_amdgcn_perm(b[1], b[0], 0x07060302u);
      part[1][i] = __builtin_amdgcn_perm(r[1], r[0], 0x07060302u);
    }
  } else {
    part[0] = v;
  }
}
// acc += the product of coefficients and values, the least parts first.
template <int DT>
__device__ __forceinline__ f32x4 dot_parts(const u32x4 (&c)[kParts], const u32x4 (&v)[kValueParts<DT>], f32x4 acc) {
#pragma unroll
  for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
    for (int q = kValueParts<DT> - 1; q >= 0; --q) acc = dot32<BL_BF16>(c[p], v[q], acc);
  return acc;
}

// Coefficients of the sorted rows, in what the passes after it need of: fp32 [rows, RP]; parts as operands
// whose rows are rows, [rows / 16, RK / 32, 3, 64 lanes, 8] (RK: R up to 32); parts as operands whose rows
// are ranks, [tiles, RP / 16, 3, 64 lanes, 8]. So an operand is 1 KB in one piece. What a row or a rank
// has not is 0.
struct Coefs {
  float* f;
  uint16_t* by_row;
  uint16_t* by_rank;
};

// ------------------------------------------------------------------------------------------
// rows sorted by adapter
// ------------------------------------------------------------------------------------------
// A tile's word: its adapter (L: none), which of the adapter's tiles it is, modulo 16, and how many follow
// it, up to 15. So a kernel can take several tiles of an adapter at a time: the workgroups of the others
// end at once.
__host__ __device__ __forceinline__ int tile_word(int e, int pos, int left) { return e | (pos & 15) << 16 | (left < 15 ? left : 15) << 20; }
__device__ __forceinline__ int tile_adapter(int w) { return w & 0xFFFF; }
__device__ __forceinline__ int tile_pos(int w) { return w >> 16 & 15; }
__device__ __forceinline__ int tile_left(int w) { return w >> 20; }

// The sort is stable, so that sums over an adapter's rows have one order. A chunk of up to 8192 rows
// per workgroup; more than one chunk: a first launch counts, the second places. Bucket L holds the
// rows without an adapter. Each bucket starts a tile of its own. The counters of the call's later
// launches are cleared on the way. A chain of waits bounds it: 4.3 us in the trace up to 1024 rows, 7
// for 4096.
constexpr int kSortWaves = 16, kSortSteps = 8;
constexpr int kSortChunk = kSortWaves * 64 * kSortSteps;

struct SortArgs {
  const int32_t* index;
  int64_t M;
  int L, chunks, steps;   // 64 rows per step and wave
  int32_t* order;
  int32_t* tile;
  int32_t* start;
  int32_t* counts;        // [chunks, L + 1]
  uint32_t* arrived;      // [ncnt]
  int64_t ncnt;
};

inline size_t sort_lds(int64_t L) { return static_cast<size_t>(L + 1) * (kSortWaves * 2 + 12) + 4; }

// Lanes whose bucket is this lane's, from a ballot of each of its bits.
__device__ __forceinline__ uint64_t same_bucket(int e, int bits) {
  uint64_t same = __ballot(e >= 0);
  for (int i = 0; i < bits; ++i) {
    const uint64_t set = __ballot((e >> i) & 1);
    same &= (e >> i) & 1 ? set : ~set;
  }
  return same;
}

// MODE 0: the only chunk. 1: this chunk's counts. 2: its places, from all chunks' counts.
template <int MODE>
__global__ __launch_bounds__(64 * kSortWaves) void adapter_sort_kernel(SortArgs a) {
  extern __shared__ int sort_mem[];
  __shared__ int sums[kSortWaves];
  const int B = a.L + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* total = sort_mem;                                 // [B] rows of each bucket
  int* place = sort_mem + B;                             // [B] first place of this chunk's rows
  int* start = sort_mem + 2 * B;                         // [B + 1] first tile of each bucket, and the end
  uint16_t* cnt = reinterpret_cast<uint16_t*>(sort_mem + 3 * B + 1);   // [waves, B]
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kSortChunk + wave * 64 * a.steps + lane;
  int e[kSortSteps], rank[kSortSteps];
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i) {
    const int64_t m = m0 + 64 * i;
    e[i] = -1;
    if (i < a.steps && m < a.M) {
      const int v = a.index[m];
      e[i] = v >= 0 && v < a.L ? v : a.L;
    }
  }
  for (int i = threadIdx.x; i < B * kSortWaves; i += blockDim.x) cnt[i] = 0;
  if constexpr (MODE != 1)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.ncnt; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
      a.arrived[i] = 0;
  __syncthreads();
  // rank of each row among those of its bucket in its wave: the first lane of each bucket counts
  const int bits = 32 - __builtin_clz(a.L);
  uint16_t* mine = cnt + wave * B;
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i) {
    rank[i] = 0;
    if (i >= a.steps) continue;
    const uint64_t same = same_bucket(e[i], bits);
    const uint64_t below = same & ((1ull << lane) - 1);
    if (e[i] >= 0) {
      const int before = mine[e[i]];
      rank[i] = before + __popcll(below);
      __builtin_amdgcn_wave_barrier();
      if (below == 0) mine[e[i]] = static_cast<uint16_t>(before + __popcll(same));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // counts per wave become the rows of earlier waves
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    int n[kSortWaves], sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) n[w] = cnt[w * B + b];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      cnt[w * B + b] = static_cast<uint16_t>(sum);
      sum += n[w];
    }
    if constexpr (MODE == 1) a.counts[static_cast<int64_t>(blockIdx.x) * B + b] = sum;
    int before = 0;
    if constexpr (MODE == 2) {
      sum = 0;
#pragma unroll 8
      for (int c = 0; c < a.chunks; ++c) {
        const int v = a.counts[static_cast<int64_t>(c) * B + b];
        before += c < static_cast<int>(blockIdx.x) ? v : 0;
        sum += v;
      }
    }
    total[b] = sum;
    place[b] = before;
  }
  if constexpr (MODE == 1) return;
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
  for (int b = b0; b < b1; ++b) {
    start[b] = at;
    place[b] += at * kTile;
    at += (total[b] + kTile - 1) / kTile;
    if (b == a.L) start[B] = at;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i)
    if (e[i] >= 0) a.order[place[e[i]] + mine[e[i]] + rank[i]] = static_cast<int32_t>(m0 + 64 * i);
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= B; b += blockDim.x) a.start[b] = start[b];
    const int all = start[B];
    for (int t = threadIdx.x; t < all; t += blockDim.x) {
      int lo = 0, hi = B - 1;                       // the last bucket that starts at t or before; empty ones end where they start
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (start[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      a.tile[t] = tile_word(lo, t - start[lo], start[lo + 1] - 1 - t);
    }
    for (int i = threadIdx.x; i < B * kTile; i += blockDim.x) {
      const int b = i / kTile, p = total[b] + i % kTile;
      if (p < (start[b + 1] - start[b]) * kTile) a.order[static_cast<int64_t>(start[b]) * kTile + p] = -1;
    }
  }
}

// Values that are loaded together, before a branch on one of them: the loads of the others would wait
// for its answer otherwise.
__device__ __forceinline__ void loaded() {}
template <typename... T>
__device__ __forceinline__ void loaded(int& v, T&... more) {
  asm volatile("" : "+v"(v));
  loaded(more...);
}

struct Sorted {
  const int32_t* order;
  const int32_t* tile;
  const int32_t* start;
  int L;
  int64_t rows;           // places: 32 max_tiles
};

// ------------------------------------------------------------------------------------------
// shrink: sums[row, r] = sum over k of S[row, k] w[e, r, k], and the coefficients made of them
// ------------------------------------------------------------------------------------------
// A workgroup has a tile of 32 rows, up to 64 ranks and one of the splits of k; its waves take blocks
// of 128 bytes of a row in turn. An operand's lanes 0 .. 15 are 16 rows, and a load whose lanes touch
// so many lines gets 16 bytes a clock: so eight lanes load a row's 128 bytes, and the operand is picked
// up from LDS of the wave's own. Where there are several workgroups to a tile, the last one that ends
// adds their sums, in order, and makes the coefficients (memory-side stores, no cache write-back: about
// 1 us to arrive, 1 to gather, 1.5 to 4.5 for the coefficients). 4096 x 8192, bf16, rank 32: 24 us, of
// which 15 are the loop at 4.5 TB/s of rows; rank 64 31 us (operands straight from memory 39). 64 ranks
// to a workgroup, since each block of ranks reads the rows again (with 32, the whole call, bf16: 4096 x
// 8192, rank 64 80 -> 82 us, rank 128 131 -> 135, 2000 x 8640, rank 40 37 -> 41). Registers for two
// workgroups to a CU: for one 79 -> 83, for three, which spill, 140 (rank 64).
constexpr int kShrinkWaves = 4;
struct ShrinkArgs {
  Sorted o;
  const void* s;
  int64_t D, ld;
  const void* w;          // [L, R, D]
  int R, RP, splits, by_chip;
  float* part;            // [splits, rows, RP]
  uint32_t* arrived;      // [max_tiles]
  const float* scale;     // [L] or null
  float* h_out;           // [M, R] or null: the sums
  const float* h_in;      // [M, R] or null: coefficients of its own, times the scale too
  Coefs c, hc;            // of the sums times the scale, and of h_in
};

// Values of a tile in LDS, v [32][RP + 1], as the coefficients that the later passes take.
template <int DT>
__device__ __forceinline__ void write_coefs(const Coefs& c, int64_t t, int RP, const float* v) {
  const int pitch = RP + 1, tid = threadIdx.x;
  if (c.f)
    for (int i = tid; i < kTile * RP; i += 64 * kShrinkWaves) c.f[t * kTile * RP + i] = v[i / RP * pitch + i % RP];
  if constexpr (DT != BL_F32) {
    const auto parts_of = [&](auto at, u32x4 (&w)[kParts]) {   // of eight values
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint16_t part[kParts];
        split(at(j), part);
#pragma unroll
        for (int p = 0; p < kParts; ++p) w[p][j / 2] |= static_cast<uint32_t>(part[p]) << (16 * (j & 1));
      }
    };
    if (c.by_row) {
      const int RK = (RP + 31) / 32 * 32, m = tid / 8;
      for (int k = tid % 8; k < RK / 8; k += 8) {
        u32x4 w[kParts] = {};
        parts_of([&](int j) { return 8 * k + j < RP ? v[m * pitch + 8 * k + j] : 0.0f; }, w);
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          uint16_t* to = c.by_row + (((t * 2 + m / 16) * (RK / 32) + k / 4) * kParts + p) * 512;
          *reinterpret_cast<u32x4*>(to + (k % 4 * 16 + m % 16) * 8) = w[p];
        }
      }
    }
    if (c.by_rank) {
      const int q = tid % 4;
      for (int r = tid / 4; r < RP; r += 16 * kShrinkWaves) {
        u32x4 w[kParts] = {};
        parts_of([&](int j) { return v[(8 * q + j) * pitch + r]; }, w);
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          uint16_t* to = c.by_rank + ((t * (RP / 16) + r / 16) * kParts + p) * 512;
          *reinterpret_cast<u32x4*>(to + (q * 16 + r % 16) * 8) = w[p];
        }
      }
    }
  }
}

// CD: the type of what the coefficients will multiply, HD: of what h_in's will.
template <int SD, int WD, int NR, int CD, int HD>
__global__ __launch_bounds__(64 * kShrinkWaves, 2) void adapter_shrink_kernel(ShrinkArgs a) {
  extern __shared__ __align__(16) float lds[];      // the waves' rooms, [4][32][16 NR], then [32][RP + 1]
  __shared__ int last, place_row[kTile];
  constexpr int V = kShrinkWaves, kThreads = 64 * V;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.z * 16 * NR;
  using S = typename Elem<SD>::type;
  using W = typename Elem<WD>::type;
  int end = a.o.start[a.o.L], t = blockIdx.y, part = blockIdx.x;
  if (a.by_chip) {
    // workgroups go to the eight chips in turn: each gets a run of the tiles, and so few adapters
    const int all = end * a.splits, per = (all + 7) / 8, id = t * a.splits + part;
    const int mine = id % 8 * per + id / 8;
    if (id / 8 >= per || mine >= all) return;
    t = mine / a.splits;
    part = mine % a.splits;
  }
  const int32_t* order = a.o.order + static_cast<int64_t>(t) * kTile;
  int word = a.o.tile[t], some = order[0], m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = order[8 * i + lane / 8];
  loaded(end, word, some, m[0], m[1], m[2], m[3]);
  if (t >= end) return;
  const int e = tile_adapter(__builtin_amdgcn_readfirstlane(word));
  if (wave == 0 && lane % 8 == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) place_row[8 * i + lane / 8] = m[i];
  }
  // Places without a row and ranks past the last one repeat another: their sums are not used. Load i
  // of a block brings rows 8 i + lane / 8 (16-bit w beside fp32 rows: 16 i + lane / 4).
  constexpr int KU = SD == BL_F32 ? 32 : 64;        // values of a block
  constexpr int WL = SD == BL_F32 && WD != BL_F32 ? 4 : 8;   // lanes of a row of w
  constexpr int WN = 16 * NR * WL / 64;             // loads of a block of w
  constexpr int SV = 16 / sizeof(S), WV = 16 / sizeof(W);    // values of a lane's piece
  const S* row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = static_cast<const S*>(a.s) + static_cast<int64_t>(m[i] < 0 ? some : m[i]) * a.ld;
  const W* w[WN];
#pragma unroll
  for (int i = 0; i < WN; ++i)
    w[i] = static_cast<const W*>(a.w) + (static_cast<int64_t>(e) * a.R + min(r0 + 64 / WL * i + lane / WL, a.R - 1)) * a.D;
  f32x4 acc[2][NR] = {};
  struct Block {
    u32x4 s[4], w[WN];
  };
  const auto load = [&](Block& v, int64_t u, auto whole) {
    __builtin_amdgcn_sched_barrier(0);              // or the loads sink to where they are used
#pragma unroll
    for (int i = 0; i < 4; ++i) v.s[i] = load16<SD, decltype(whole)::value>(row[i], u * KU + lane % 8 * SV, a.D);
#pragma unroll
    for (int i = 0; i < WN; ++i) v.w[i] = load16<WD, decltype(whole)::value>(w[i], u * KU + lane % WL * WV, a.D);
    __builtin_amdgcn_sched_barrier(0);
  };
  // pieces of 16 bytes, [32][8] and [16 NR][WL], in an XOR order that spreads 16 rows over all banks
  u32x4* room = reinterpret_cast<u32x4*>(lds) + wave * (kTile * 8 + 16 * NR * WL);
  u32x4* wroom = room + kTile * 8;
  const auto place = [](int r, int p, int lanes) { return r * lanes + (p ^ (lanes == 8 ? r >> 1 & 7 : r >> 2 & 3)); };
  const auto spread = [&](const Block& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) room[place(8 * i + lane / 8, lane % 8, 8)] = v.s[i];
#pragma unroll
    for (int i = 0; i < WN; ++i) wroom[place(64 / WL * i + lane / WL, lane % WL, WL)] = v.w[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  const auto multiply = [&]() {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x4 sv[2], wv[NR];
#pragma unroll
      for (int i = 0; i < 2; ++i) sv[i] = room[place(16 * i + c, 4 * j + g, 8)];
#pragma unroll
      for (int q = 0; q < NR; ++q) wv[q] = wroom[WL == 8 ? place(16 * q + c, 4 * j + g, 8) : place(16 * q + c, 2 * j + (g >> 1), 4)];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          if constexpr (SD != BL_F32) {
            acc[i][q] = dot32<SD>(sv[i], wv[q], acc[i][q]);
          } else {
#pragma unroll
            for (int l = 0; l < 4; ++l) {
              float wl;
              if constexpr (WD == BL_F32) wl = __uint_as_float(wv[q][l]);
              else wl = to_float<WD>(static_cast<uint16_t>((g & 1 ? wv[q][2 + l / 2] : wv[q][l / 2]) >> (16 * (l & 1))));
              acc[i][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(sv[i][l]), wl, acc[i][q], 0, 0, 0);
            }
          }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  const int64_t units = (a.D + KU - 1) / KU, full = a.D / KU;
  const int64_t u0 = units * part / a.splits, u1 = units * (part + 1) / a.splits, uf = min(u1, full);
  int64_t u = u0 + wave;
  int64_t n = u < uf ? (uf - u + V - 1) / V : 0;    // whole blocks of this wave
  Block v0, v1;
  if (n) {
    // two blocks in flight; no load is under a condition of its own, so each wait is for the older ones
    // alone
    load(v0, u, std::true_type{});
    load(v1, n > 1 ? u + V : u, std::true_type{});
    for (; n > 2; n -= 2) {
      spread(v0);
      load(v0, u += 2 * V, std::true_type{});
      multiply();
      spread(v1);
      load(v1, n > 3 ? u + V : u, std::true_type{});
      multiply();
    }
    spread(v0);
    multiply();
    if (n == 2) {
      spread(v1);
      multiply();
    }
  }
  if (u1 > full && (full - u0) % V == wave) {       // the block that is not whole
    load(v0, full, std::false_type{});
    spread(v0);
    multiply();
  }
  __syncthreads();

  // the waves' sums
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < NR; ++q)
#pragma unroll
      for (int l = 0; l < 4; ++l) lds[(wave * kTile + 16 * i + 4 * g + l) * 16 * NR + 16 * q + c] = acc[i][q][l];
  __syncthreads();
  constexpr int kEach = kTile * 16 * NR / kThreads;
  float sum[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = tid + kThreads * i;
    sum[i] = lds[at] + lds[at + kTile * 16 * NR] + lds[at + 2 * kTile * 16 * NR] + lds[at + 3 * kTile * 16 * NR];
  }
  const int groups = a.splits * static_cast<int>(gridDim.z), pitch = a.RP + 1;
  const float f = a.scale ? a.scale[e] : 1.0f;
  if (groups > 1) {
    float* out = a.part + (part * a.o.rows + static_cast<int64_t>(t) * kTile) * a.RP;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = tid + kThreads * i, r = r0 + at % (16 * NR);
      if (r < a.RP) atomic_store_agent(out + at / (16 * NR) * a.RP + r, sum[i]);
    }
    wait_own_memory_ops();
    __syncthreads();
    if (tid == 0) last = arrive_agent(a.arrived + t) + 1 == static_cast<uint32_t>(groups);
    __syncthreads();
    if (!last) return;
    // about 32 loads in flight at a time: of PL places (all of a thread's, up to rank 64) those of NS
    // splits
    constexpr int PL = 2 * NR, NS = 32 / PL;
    const float* in = a.part + static_cast<int64_t>(t) * kTile * a.RP;
    const int64_t step = a.o.rows * a.RP;
    for (int i0 = tid; i0 < kTile * a.RP; i0 += PL * kThreads) {
      float v[PL] = {};
      for (int s0 = 0; s0 < a.splits; s0 += NS) {
        float p[NS][PL];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int i = 0; i < PL; ++i)
            p[s][i] = atomic_load_agent(in + min(s0 + s, a.splits - 1) * step + min(i0 + i * kThreads, kTile * a.RP - 1));
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int i = 0; i < PL; ++i) v[i] += s0 + s < a.splits ? p[s][i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int at = i0 + i * kThreads;
        if (at < kTile * a.RP) lds[at / a.RP * pitch + at % a.RP] = v[i];
      }
    }
  } else {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = tid + kThreads * i, r = at % (16 * NR);
      if (r < a.RP) lds[at / (16 * NR) * pitch + r] = sum[i];
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < kTile * a.RP; i += kThreads) {
    const int r = i % a.RP, at = place_row[i / a.RP];
    float& v = lds[i / a.RP * pitch + r];
    const bool there = at >= 0 && r < a.R;
    if (there && a.h_out) a.h_out[static_cast<int64_t>(at) * a.R + r] = v;
    v = there ? v * f : 0.0f;
  }
  // h_in: eight loads in flight, under way while the sums' coefficients are made
  float h[8];
  const auto load_h = [&](int i0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = min(i0 + i * kThreads, kTile * a.RP - 1), r = k % a.RP, at = place_row[k / a.RP];
      h[i] = a.h_in[static_cast<int64_t>(max(at, 0)) * a.R + min(r, a.R - 1)];
      h[i] = at >= 0 && r < a.R ? h[i] * f : 0.0f;
    }
  };
  if (a.h_in) load_h(tid);
  __syncthreads();
  write_coefs<CD>(a.c, t, a.RP, lds);
  if (a.h_in) {
    __syncthreads();
    for (int i0 = tid; i0 < kTile * a.RP; i0 += 8 * kThreads) {
      if (i0 != tid) load_h(i0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = i0 + i * kThreads;
        if (k < kTile * a.RP) lds[k / a.RP * pitch + k % a.RP] = h[i];
      }
    }
    __syncthreads();
    write_coefs<HD>(a.hc, t, a.RP, lds);
  }
}

// ------------------------------------------------------------------------------------------
// expand: y[row, n] = base[row, n] + sum_r c[row, r] w[e, r, n]
// ------------------------------------------------------------------------------------------
struct ExpandArgs {
  Sorted o;
  Coefs c;
  int R, RP;
  float* h;               // [M, R] or null: rows without an adapter get zeros
  const void* w;          // [L, R, N]
  int64_t N;
  const void* base;
  int64_t ldbase;
  void* y;
  int64_t ldy;
  int tiles;              // 1, 2 or 4
};

// A wave has 16 rows and 128 columns at a time: lane 16 g + c columns 8 c .. 8 c + 7 of them, so that
// w, base and y go 16 bytes at a time, and matrix instruction j makes columns 8 c + j.
template <int YD, bool WHOLE>
__device__ __forceinline__ void load_base(const ExpandArgs& a, const int (&row)[4], int64_t n, Eight<YD> (&base)[4]) {
  using Y = typename Elem<YD>::type;
  if (!a.base) return;
#pragma unroll
  for (int l = 0; l < 4; ++l)                       // a place without a row reads row 0
    base[l] = load8<YD, WHOLE>(static_cast<const Y*>(a.base) + max(row[l], 0) * a.ldbase, n, a.N);
}
template <int YD>
__device__ __forceinline__ void store_rows(const ExpandArgs& a, const int (&row)[4], int64_t n, int64_t lo, const Eight<YD> (&base)[4],
                                           const f32x4 (&acc)[8]) {
  using Y = typename Elem<YD>::type;
#pragma unroll
  for (int l = 0; l < 4; ++l) {
    if (row[l] < 0) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = acc[j][l];
      if (a.base) v[j] = value<YD>(base[l], j) + v[j];
    }
    store8<YD>(static_cast<Y*>(a.y) + row[l] * a.ldy, n, lo, a.N, v);
  }
}
// Rows without an adapter are base's.
template <int YD, bool WHOLE>
__device__ __forceinline__ void copy_rows(const ExpandArgs& a, const int (&row)[4], int64_t n, int64_t lo) {
  using Y = typename Elem<YD>::type;
  Eight<YD> base[4] = {};
  load_base<YD, WHOLE>(a, row, n, base);
#pragma unroll
  for (int l = 0; l < 4; ++l) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = value<YD>(base[l], j);
    if (row[l] >= 0) store8<YD>(static_cast<Y*>(a.y) + row[l] * a.ldy, n, lo, a.N, v);
  }
}

// The rows of up to `count` tiles. KB blocks of 32 ranks of w stay in registers over them; 0: any rank,
// w is loaded again for each tile (fp32: always so). Reading base and writing y bound it: 4096 x 8192,
// bf16, rank 32 31 us (134 MB, 4.3 TB/s), rank 64 38; with two halves' rows per wave and w loaded by
// each tile 57.
template <int WD, int YD, int KB, bool WHOLE>
__device__ __forceinline__ void expand_tiles(const ExpandArgs& a, int64_t at, int count, int e, int64_t n0, int64_t lo, int lane) {
  const int c = lane & 15, g = lane >> 4;
  const int64_t n = n0 + 8 * c;
  using W = typename Elem<WD>::type;
  constexpr int VP = kValueParts<WD>;
  const W* w = static_cast<const W*>(a.w) + static_cast<int64_t>(e) * a.R * a.N;
  const int RK = (a.RP + 31) / 32 * 32;
  int row[4];
  const auto rows = [&](int64_t p, int (&r)[4]) {
#pragma unroll
    for (int l = 0; l < 4; ++l) r[l] = a.o.order[p + 4 * g + l];
  };
  const auto load_w = [&](int r0, u32x4 (&v)[8]) {  // 32 ranks: rows 8 g .. 8 g + 7 of them
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int r = r0 + 8 * g + s;
      if constexpr (WD != BL_F32)
        v[s] = zero_unless(r < a.R, load8<WD, WHOLE>(w + static_cast<int64_t>(min(r, a.R - 1)) * a.N, n, a.N)).w;
    }
  };
  Eight<YD> base[4] = {};
  rows(at, row);
  load_base<YD, WHOLE>(a, row, n, base);
  // as operands: column j of block k. Two blocks of fp16 columns in parts would take 128 registers:
  // they are cut for each tile (4096 x 8192, rank 64: 86 us for the whole call where 93)
  constexpr bool kCut = WD != BL_F16 || KB == 1;
  u32x4 wv[KB ? KB : 1][8][kCut ? VP : 1];
  if constexpr (KB > 0) {
    u32x4 raw[KB][8];
#pragma unroll
    for (int k = 0; k < KB; ++k) load_w(32 * k, raw[k]);
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const u32x4 v = column(raw[k], j);
        if constexpr (kCut) value_parts<WD>(v, wv[k][j]);
        else wv[k][j][0] = v;
      }
  }
  for (int i = 0; i < count; ++i, at += kTile) {
    f32x4 acc[8] = {};
    int next[4];
    rows(i + 1 < count ? at + kTile : at, next);
    if constexpr (WD == BL_F32) {
      const float* co = a.c.f + at * a.RP;
      for (int r0 = 0; r0 < a.RP; r0 += 16) {
        Eight<WD> v[4];
        float cv[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int r = r0 + 4 * s + g;
          v[s] = zero_unless(r < a.R, load8<WD, WHOLE>(w + static_cast<int64_t>(min(r, a.R - 1)) * a.N, n, a.N));
          cv[s] = co[c * a.RP + r];
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(cv[s], value<WD>(v[s], j), acc[j], 0, 0, 0);
      }
    } else {
      const u32x4* co = reinterpret_cast<const u32x4*>(a.c.by_row) + at / 16 * (RK / 32) * kParts * 64 + lane;
      if constexpr (KB > 0) {
        u32x4 cv[KB][kParts];
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int p = 0; p < kParts; ++p) cv[k][p] = co[(k * kParts + p) * 64];
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if constexpr (kCut) {
              acc[j] = dot_parts<WD>(cv[k], wv[k][j], acc[j]);
            } else {
              u32x4 v[VP];
              value_parts<WD>(wv[k][j][0], v);
              acc[j] = dot_parts<WD>(cv[k], v, acc[j]);
            }
          }
      } else {
        for (int r0 = 0; r0 < RK; r0 += 32) {
          u32x4 raw[8], cv[kParts];
          load_w(r0, raw);
#pragma unroll
          for (int p = 0; p < kParts; ++p) cv[p] = co[(r0 / 32 * kParts + p) * 64];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            u32x4 v[VP];
            value_parts<WD>(column(raw, j), v);
            acc[j] = dot_parts<WD>(cv, v, acc[j]);
          }
        }
      }
    }
    Eight<YD> more[4] = {};
    load_base<YD, WHOLE>(a, next, n, more);
    store_rows<YD>(a, row, n, lo, base, acc);
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      row[l] = next[l];
      base[l] = more[l];
    }
  }
}

// A workgroup has up to `tiles` tiles and 256 columns, its waves the tiles' halves. Tiles come after
// the columns: rows are read and written whole by workgroups that run together. Registers for three
// workgroups to a CU (two of fp32 results, and of two blocks of fp16): for two the same within 1 us,
// for four, which spill, 4096 x 8192, rank 64 79 -> 140 us.
template <int WD, int YD, int KB>
__global__ __launch_bounds__(256, YD == BL_F32 || (WD == BL_F16 && KB == 2) ? 2 : 3) void adapter_expand_kernel(ExpandArgs a) {
  const int t = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t at = static_cast<int64_t>(t) * kTile + 16 * (wave & 1);
  int end = a.o.start[a.o.L + 1], word = a.o.tile[t], first = a.o.order[at], row[4];
#pragma unroll
  for (int l = 0; l < 4; ++l) row[l] = a.o.order[at + 4 * (lane >> 4) + l];
  loaded(end, word, first, row[0], row[1], row[2], row[3]);
  if (t >= end) return;
  word = __builtin_amdgcn_readfirstlane(word);
  const int e = tile_adapter(word);
  // the last columns are taken with those before them, to be 128, and stored alone
  const int64_t lo = (static_cast<int64_t>(blockIdx.x) * 2 + (wave >> 1)) * 128, n0 = max(min(lo, a.N - 128), int64_t(0));
  const int64_t n = n0 + 8 * (lane & 15);
  if (e >= a.o.L) {
    if (a.h && blockIdx.x == 0)
      for (int i = threadIdx.x; i < kTile * a.R; i += 256) {
        const int m = a.o.order[static_cast<int64_t>(t) * kTile + i / a.R];
        if (m >= 0) a.h[static_cast<int64_t>(m) * a.R + i % a.R] = 0.0f;
      }
    if (a.base == a.y || lo >= a.N) return;
    if (a.N >= 128) copy_rows<YD, true>(a, row, n, lo);
    else copy_rows<YD, false>(a, row, n, lo);
    return;
  }
  if (tile_pos(word) % a.tiles) return;
  const int count = min(a.tiles, tile_left(word) + 1);
  if (lo >= a.N || (count == 1 && first < 0)) return;   // a half without rows
  if (a.N >= 128) expand_tiles<WD, YD, KB, true>(a, at, count, e, n0, lo, lane);
  else expand_tiles<WD, YD, 0, false>(a, at, count, e, n0, lo, lane);
}

// ------------------------------------------------------------------------------------------
// outer: grad[e, r, d] = sum over the adapter's rows of c[row, r] S[row, d]
// ------------------------------------------------------------------------------------------
// A workgroup has 128 columns, up to 32 ranks and an even share of the tiles, which its waves take in
// turn. An adapter that lies within one share is written at once. The pieces of one that does not go to
// sum[2 share], where the adapter began in an earlier share, or sum[2 share + 1]; the workgroup that
// ends last adds them in their order. Each share has at most one adapter that goes on after it, so the
// share where an adapter begins names its counter. A wave has two tiles' loads in flight, which bounds
// it: 4096 rows of 8192 and 8192, bf16, rank 32 34 us for both sums (134 MB, 3.9 TB/s; with one tile at
// a time 100). fp32 rows have one in flight and the fp32 instruction: 1024 rows of 8640 in fp32 beside 3200
// in fp16, rank 8, 19 us (42 MB) where each sum by itself takes 19 and 15.
struct OuterArgs {
  Sorted o;
  Coefs c;
  const void* s;
  int64_t D, ld;
  int R, RP, splits;
  float* sum;             // [2 splits, R, D]
  uint32_t* arrived;      // [splits, blocks of ranks, blocks of columns]
  float* grad;            // [L, R, D]
  int add;
};
// One launch takes both sums: the first `columns` workgroups along x are p[0]'s.
struct OuterPair {
  OuterArgs p[2];
  uint32_t columns;
};

// What a wave takes of a tile: lane 16 g + c rows 8 g .. 8 g + 7 (fp32: 4 i + g), columns 8 c .. 8 c + 7.
template <int SD, int NR>
struct OuterTile {
  int row[8];
  Eight<SD> s[8];
  u32x4 c[NR][kParts];                              // 16-bit parts
  float f[SD == BL_F32 ? 8 : 1][NR];

  __device__ __forceinline__ void load_rows(const OuterArgs& a, int64_t t, int g) {
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = a.o.order[t * kTile + (SD == BL_F32 ? 4 * i + g : 8 * g + i)];
  }
  template <bool WHOLE>
  __device__ __forceinline__ void load(const OuterArgs& a, int64_t t, int64_t d, int r0, int c16, int g) {
    using S = typename Elem<SD>::type;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      s[i] = load8<SD, WHOLE>(static_cast<const S*>(a.s) + static_cast<int64_t>(max(row[i], 0)) * a.ld, d, a.D);
    if constexpr (SD == BL_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          const int r = r0 + 16 * q + c16;
          f[i][q] = r < a.RP ? a.c.f[(t * kTile + 4 * i + g) * a.RP + r] : 0.0f;
        }
    } else {
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int rb = min(r0 / 16 + q, a.RP / 16 - 1);   // past the last rank: not used
#pragma unroll
        for (int p = 0; p < kParts; ++p)
          c[q][p] = reinterpret_cast<const u32x4*>(a.c.by_rank)[((t * (a.RP / 16) + rb) * kParts + p) * 64 + 16 * g + c16];
      }
    }
  }
  // A place without a row holds row 0's values, which the sums must not see.
  __device__ __forceinline__ void multiply(const int (&rows)[8], f32x4 (&acc)[NR][8]) {
    if constexpr (SD == BL_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const Eight<SD> v = zero_unless(rows[i] >= 0, s[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int q = 0; q < NR; ++q)
            acc[q][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[i][q], value<SD>(v, j), acc[q][j], 0, 0, 0);
      }
    } else {
      u32x4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = zero_unless(rows[i] >= 0, s[i]).w;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u32x4 v[kValueParts<SD>];
        value_parts<SD>(column(w, j), v);
#pragma unroll
        for (int q = 0; q < NR; ++q) acc[q][j] = dot_parts<SD>(c[q], v, acc[q][j]);
      }
    }
  }
};

// Tiles t, t + STEP .. before end: each is loaded while the one before is multiplied, its rows' numbers one
// tile earlier still. Past the last tile the loads repeat it, so that none is under a condition.
template <int SD, int NR, bool TWO, bool WHOLE, int STEP>
__device__ __forceinline__ void outer_tiles(const OuterArgs& a, int t, int end, int64_t d, int r0, int c, int g, f32x4 (&acc)[NR][8]) {
  if (t >= end) return;
  const int last = t + (end - 1 - t) / STEP * STEP;
  if constexpr (!TWO || !WHOLE) {
    OuterTile<SD, NR> v;
    int rows[8];
    v.load_rows(a, t, g);
    for (; t <= last; t += STEP) {
      v.template load<WHOLE>(a, t, d, r0, c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) rows[k] = v.row[k];
      v.load_rows(a, min(t + STEP, last), g);
      v.multiply(rows, acc);
    }
    return;
  }
  if (t == last) {                                  // the only one
    OuterTile<SD, NR> v;
    v.load_rows(a, t, g);
    v.template load<WHOLE>(a, t, d, r0, c, g);
    v.multiply(v.row, acc);
    return;
  }
  OuterTile<SD, NR> v[2];
  v[0].load_rows(a, t, g);
  v[1].load_rows(a, min(t + STEP, last), g);
  v[0].template load<WHOLE>(a, t, d, r0, c, g);
  for (;;)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      OuterTile<SD, NR>&now = v[i], &next = v[1 - i];
      int rows[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) rows[k] = now.row[k];
      __builtin_amdgcn_sched_barrier(0);
      next.template load<WHOLE>(a, min(t + STEP, last), d, r0, c, g);
      now.load_rows(a, min(t + 2 * STEP, last), g);
      __builtin_amdgcn_sched_barrier(0);
      now.multiply(rows, acc);
      if ((t += STEP) > last) return;
    }
}

// red [4 waves][16 NR][32].
template <int SD, int NR, bool TWO>
__device__ __forceinline__ void outer(const OuterArgs& a, uint32_t column, f32x4 (*red)[32], int& last_one) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
  if (static_cast<int>(blockIdx.y) >= a.splits) return;
  // the last columns are taken with those before them, to be 128, and written alone
  const int64_t lo = static_cast<int64_t>(column) * 128, d0 = max(min(lo, a.D - 128), int64_t(0));
  const int r0 = blockIdx.z * 16 * NR;
  const int64_t tiles = a.o.start[a.o.L], n = static_cast<int64_t>(a.R) * a.D;
  const auto each = [&](auto f) {                   // of this workgroup's values: (row and column in red, place in [R, D])
    const int64_t d = d0 + tid % 128;
    if (d < lo || d >= a.D) return;
#pragma unroll
    for (int i = 0; i < 8 * NR; ++i) {
      const int r = r0 + 2 * i + tid / 128;
      if (r < a.R) f(tid + 256 * i, r * a.D + d);
    }
  };
  const float* flat = reinterpret_cast<const float*>(red);
  const auto sum = [&](int i) { return flat[i] + flat[i + 2048 * NR] + flat[i + 2 * 2048 * NR] + flat[i + 3 * 2048 * NR]; };
  // adapters without rows, shared out over the shares
  if (!a.add)
    for (int e0 = blockIdx.y; e0 < a.o.L; e0 += 64 * a.splits) {
      const int mine = min(e0 + lane * a.splits, a.o.L - 1);
      uint64_t empty = __ballot(e0 + lane * a.splits < a.o.L && a.o.start[mine] == a.o.start[mine + 1]);
      for (; empty; empty &= empty - 1) {
        const int64_t e = e0 + __builtin_ctzll(empty) * a.splits;
        each([&](int, int64_t at) { a.grad[e * n + at] = 0.0f; });
      }
    }

  // no share without a tile: the last to end is known by how many shares an adapter lies in
  const int64_t shares = min(static_cast<int64_t>(a.splits), tiles);
  if (blockIdx.y >= shares) return;
  const int t0 = static_cast<int>(tiles * blockIdx.y / shares), t1 = static_cast<int>(tiles * (blockIdx.y + 1) / shares);
  // (us of the gradients, bf16, for a quarter / third / half of the share: 4096 x 4096, rank 32, 16
  // adapters 92 / 84 / 83, 32 of rank 16 85 / 80 / 80; 12000 x 4096, rank 32, 8 adapters 163 / 163 /
  // 184, 16 188 / 165 / 165; none: 2048 x 2048, rank 8, 200 adapters 47 -> 68)
  const int few = max(4, (t1 - t0) / 3);
  int turn = 0;
  int words = 0, words_at = t0 - 64;                // of 64 tiles, one a lane
  for (int t = t0; t < t1;) {
    if (t - words_at >= 64) words = a.o.tile[min(static_cast<int64_t>((words_at = t) + lane), tiles - 1)];
    const int word = __builtin_amdgcn_readlane(words, t - words_at), e = tile_adapter(word);
    // its first tile and the one after its last: known but at the share's start, and of long ones
    const int first = t == t0 ? a.o.start[e] : t, last = tile_left(word) < 15 ? t + tile_left(word) + 1 : a.o.start[e + 1];
    const int end = min(last, t1);
    float* grad = a.grad + e * n;
    f32x4 acc[NR][8] = {};
    if (first >= t && last <= end && end - t <= few) {
      // an adapter of few of the share's tiles is one wave's, which writes it from its registers
      if (turn++ % 4 == wave) {
        if (a.D >= 128) outer_tiles<SD, NR, TWO, true, 1>(a, t, end, d0 + 8 * c, r0, c, g, acc);
        else outer_tiles<SD, NR, TWO, false, 1>(a, t, end, d0 + 8 * c, r0, c, g, acc);
#pragma unroll
        for (int q = 0; q < NR; ++q)
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            const int r = r0 + 16 * q + 4 * g + l;
            if (r >= a.R) continue;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = acc[q][j][l];
            if (a.add) {
              const Eight<BL_F32> old = load8<BL_F32, false>(grad + r * a.D, d0 + 8 * c, a.D);
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = value<BL_F32>(old, j) + v[j];
            }
            store8<BL_F32>(grad + r * a.D, d0 + 8 * c, lo, a.D, v);
          }
      }
      t = end;
      continue;
    }
    if (a.D >= 128) outer_tiles<SD, NR, TWO, true, 4>(a, t + wave, end, d0 + 8 * c, r0, c, g, acc);
    else outer_tiles<SD, NR, TWO, false, 4>(a, t + wave, end, d0 + 8 * c, r0, c, g, acc);
    // the waves' sums, added in their order as they are read
#pragma unroll
    for (int q = 0; q < NR; ++q)
#pragma unroll
      for (int l = 0; l < 4; ++l)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          red[wave * 16 * NR + 16 * q + 4 * g + l][2 * c + j] =
              f32x4{acc[q][4 * j][l], acc[q][4 * j + 1][l], acc[q][4 * j + 2][l], acc[q][4 * j + 3][l]};
    __syncthreads();
    if (first >= t && last <= end) {
      each([&](int i, int64_t at) { grad[at] = a.add ? grad[at] + sum(i) : sum(i); });
    } else {
      float* out = a.sum + (2 * static_cast<int64_t>(blockIdx.y) + (first >= t ? 1 : 0)) * n;
      each([&](int i, int64_t at) { atomic_store_agent(out + at, sum(i)); });
      wait_own_memory_ops();
      __syncthreads();
      // the share of tile t is the largest s whose first tile, floor(s tiles / shares), is not past t
      const int64_t s0 = ((first + 1) * shares - 1) / tiles, s1 = (last * shares - 1) / tiles;
      if (tid == 0)
        last_one = arrive_agent(a.arrived + (s0 * gridDim.z + blockIdx.z) * ((a.D + 127) / 128) + column) == static_cast<uint32_t>(s1 - s0);
      __syncthreads();
      if (last_one) {
        // eight places' values of four shares in flight at a time
        const int parts = static_cast<int>(s1 - s0) + 1;
        for (int i0 = tid; i0 < 16 * NR * 128; i0 += 8 * 256) {
          int64_t at[8];
          bool here[8];
          float v[8] = {};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = i0 + 256 * i, r = r0 + k / 128;
            const int64_t d = d0 + k % 128;
            here[i] = r < a.R && d >= lo && d < a.D;
            at[i] = here[i] ? r * a.D + d : static_cast<int64_t>(min(r0, a.R - 1)) * a.D;
          }
          for (int q = 0; q < parts; q += 4) {
            float p[4][8];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const int64_t share = s0 + min(q + s, parts - 1);
              const float* in = a.sum + (2 * share + (share == s0 ? 1 : 0)) * n;
#pragma unroll
              for (int i = 0; i < 8; ++i) p[s][i] = atomic_load_agent(in + at[i]);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] += q + s < parts ? p[s][i] : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (here[i]) grad[at[i]] = a.add ? grad[at[i]] + v[i] : v[i];
        }
      }
    }
    __syncthreads();
    t = end;
  }
}

// Types of the first and the second sum of a pair. Registers: two workgroups to a CU, or one with two
// tiles of 16-bit values in flight beyond rank 16; fp32 leaves none for a second tile. (us of the
// gradients of 4096 x 8192, rank 32, for one / two: bf16 100 / 127, fp32 223 / 207; 1024 x 4096, rank
// 8, bf16 44 / 41.) 32 ranks to a workgroup: with 16, whose rows are read twice as often, 4096 x 8192,
// rank 32 101 -> 115 us, 8 adapters of rank 64 142 -> 156.
template <int SD, int TD, int NR>
__global__ __launch_bounds__(256, SD == BL_F32 || NR == 1 ? 2 : 1) void adapter_outer_kernel(OuterPair pair) {
  __shared__ f32x4 red[4 * 16 * NR][32];
  __shared__ int last_one;
  constexpr bool kTwo = SD != BL_F32;
  const bool second = blockIdx.x >= pair.columns;
  const uint32_t column = second ? blockIdx.x - pair.columns : blockIdx.x;
  if constexpr (SD == TD) {
    const OuterArgs a = second ? pair.p[1] : pair.p[0];   // in registers: not loaded again at every use
    outer<SD, NR, kTwo>(a, column, red, last_one);
  } else if (second) {
    const OuterArgs a = pair.p[1];
    outer<TD, NR, NR == 1>(a, column, red, last_one);
  } else {
    const OuterArgs a = pair.p[0];
    outer<SD, NR, kTwo>(a, column, red, last_one);
  }
}

// ------------------------------------------------------------------------------------------
// few rows: each by itself, nothing sorted
// ------------------------------------------------------------------------------------------
struct RowsArgs {
  AdapterForwardArgs f;
  int R;
};

// h[m, r] for RW ranks of a row: every thread has pieces of eight values of the row and of each rank. One
// row of 8192, rank 16: 3.2 us in the trace, 48 rows 5, 320 rows of 4096, rank 32 10 (84 MB of matrices
// from the caches).
template <int DT, int RW>
__global__ __launch_bounds__(256) void adapter_rows_shrink_kernel(RowsArgs p) {
  __shared__ float red[4][RW];
  const AdapterForwardArgs& a = p.f;
  using T = typename Elem<DT>::type;
  const int tid = threadIdx.x, r0 = blockIdx.y * RW;
  const int64_t m = blockIdx.x;
  const int e = a.rows.index[m];
  float* h = a.h + m * p.R + r0;
  if (e < 0 || e >= a.rows.L) {
    if (tid < RW && r0 + tid < p.R) h[tid] = 0.0f;
    return;
  }
  const T* x = static_cast<const T*>(a.x) + m * a.ldx;
  const T* w[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) w[i] = static_cast<const T*>(a.a) + (static_cast<int64_t>(e) * p.R + min(r0 + i, p.R - 1)) * a.K;
  float sum[RW] = {};
  const auto add = [&](int64_t k, auto whole) {
    const Eight<DT> xv = load8<DT, decltype(whole)::value>(x, k, a.K);
    Eight<DT> wv[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) wv[i] = load8<DT, decltype(whole)::value>(w[i], k, a.K);
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[i] += value<DT>(xv, j) * value<DT>(wv[i], j);
  };
  const int64_t full = a.K / 2048 * 2048;
#pragma unroll 4
  for (int64_t k = 0; k < full; k += 2048) add(k + 8 * tid, std::true_type{});
  if (full + 8 * tid < a.K) add(full + 8 * tid, std::false_type{});
#pragma unroll
  for (int i = 0; i < RW; ++i) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum[i] += __shfl_xor(sum[i], off);
    if (tid % 64 == 0) red[tid / 64][i] = sum[i];
  }
  __syncthreads();
  if (tid < RW && r0 + tid < p.R) h[tid] = red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid];
}

// 512 columns of a row of y: each wave takes every fourth rank. One row of 8192, rank 16: 3.6 us in the
// trace, 48 rows of 28672 9.5 (50 MB, 5.2 TB/s).
template <int WD, int YD>
__global__ __launch_bounds__(256) void adapter_rows_expand_kernel(RowsArgs p) {
  __shared__ f32x4 red[4][64][2];
  const AdapterForwardArgs& a = p.f;
  using W = typename Elem<WD>::type;
  using Y = typename Elem<YD>::type;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t m = blockIdx.y, n0 = static_cast<int64_t>(blockIdx.x) * 512, n = n0 + 8 * lane, at = n0 + 2 * tid;
  const int e = a.rows.index[m];
  const bool none = e < 0 || e >= a.rows.L;
  if (none && a.base == a.y) return;
  const Y* base = static_cast<const Y*>(a.base) + m * a.ldbase;
  float b[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (a.base && at + i < a.N) b[i] = to_float<YD>(base[at + i]);
  float v[2] = {};
  if (!none) {
    const W* w = static_cast<const W*>(a.b) + static_cast<int64_t>(e) * p.R * a.N;
    const float* h = a.h + m * p.R;
    float sum[8] = {};
    const auto ranks = [&](auto whole) {
#pragma unroll 8
      for (int r = wave; r < p.R; r += 4) {
        const float c = h[r];
        const Eight<WD> wv = load8<WD, decltype(whole)::value>(w + r * a.N, n, a.N);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += c * value<WD>(wv, j);
      }
    };
    if (n0 + 512 <= a.N) ranks(std::true_type{});
    else ranks(std::false_type{});
    red[wave][lane][0] = f32x4{sum[0], sum[1], sum[2], sum[3]};
    red[wave][lane][1] = f32x4{sum[4], sum[5], sum[6], sum[7]};
    __syncthreads();
    const float f = a.scale ? a.scale[e] : 1.0f;
    const float* flat = reinterpret_cast<const float*>(red);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 2 * tid + i;
      v[i] = f * (flat[k] + flat[512 + k] + flat[1024 + k] + flat[1536 + k]);
      if (a.base) v[i] = b[i] + v[i];
    }
  } else {
    v[0] = b[0];
    v[1] = b[1];
  }
  Y* y = static_cast<Y*>(a.y) + m * a.ldy;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (at + i < a.N) {
      if constexpr (YD == BL_F32) y[at + i] = v[i];
      else y[at + i] = bits16<YD>(v[i]);
    }
}

// ------------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------------
// Rows each by itself, in two launches that wait for nothing and need no scratch, or sorted. Each by
// itself a row reads its own copy of its adapter, R (K + N) values; a workgroup of four ranks takes as
// long as 8192 values whatever it reads, and a row's other workgroups as long as 12288. Sorted, the
// waits of three launches are most of the time until the rows themselves are. Up to kRowsMost by this
// count each goes by itself. (us from a graph, by itself / sorted, bf16, eight adapters: 64 rows of
// 8192 x 8192, rank 16 9.9 / 17.6, rank 64 17.9 / 23.5; 256 rows of 4096 x 4096, rank 64 21.7 / 23.0;
// 256 of 8192 x 28672, rank 8 28.8 / 24.5; 1024 of 1024 x 1024, rank 16 16.8 / 17.8, rank 64 38 / 22;
// 1024 of 512 x 512, rank 8 9.5 / 14.7; 4096 of 128 x 128, rank 8 21.6 / 16.3, rank 64 104 / 19. fp32
// reads twice as much on both ways: 256 of 4096 x 4096, rank 64 33.5 / 34.2, 64 of 8192 x 8192, rank 64
// 27.2 / 33.7. Over 464 shapes 1.1 % from the better way, 42 % at most; by R (K + N) alone 28 %, and 13
// times its time at most.)
constexpr int64_t kRowsMost = int64_t(11) << 23;
bool by_rows(int64_t M, int64_t R, int64_t K, int64_t N) {
  return M <= 65535 && M * (div_up(R, 4) * std::max<int64_t>(4 * K, 8192) + R * N + 12288) <= kRowsMost;
}

template <int DT>
hipError_t start_rows_shrink(const RowsArgs& p, hipStream_t s) {
  const auto M = static_cast<uint32_t>(p.f.rows.M);
  // one rank to a workgroup while that makes few of them, else four, which share the row's reads (us,
  // one / four, bf16: 16 rows of 8192, rank 16 7.9 / 8.9, 64 rows 11.0 / 12.4, 128 rows 13.3 / 14.7, of
  // 4096 11.2 / 11.2; 256 rows of 4096, rank 16 14.5 / 13.3, 320, rank 32 22.1 / 17.8, 900 of 1024,
  // rank 8 13.3 / 11.1)
  if (p.f.rows.M * p.R <= 1024) adapter_rows_shrink_kernel<DT, 1><<<dim3(M, p.R), 256, 0, s>>>(p);
  else adapter_rows_shrink_kernel<DT, 4><<<dim3(M, static_cast<uint32_t>(div_up(p.R, 4))), 256, 0, s>>>(p);
  return hipGetLastError();
}
template <int WD, int YD>
hipError_t start_rows_expand(const RowsArgs& p, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(div_up(p.f.N, 512)), static_cast<uint32_t>(p.f.rows.M));
  adapter_rows_expand_kernel<WD, YD><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}
hipError_t forward_by_rows(const AdapterForwardArgs& a, hipStream_t s) {
  const RowsArgs p{a, static_cast<int>(a.rows.R)};
  const hipError_t e = a.dtype == BL_F16    ? start_rows_shrink<BL_F16>(p, s)
                       : a.dtype == BL_BF16 ? start_rows_shrink<BL_BF16>(p, s)
                                            : start_rows_shrink<BL_F32>(p, s);
  if (e != hipSuccess) return e;
  if (a.dtype == BL_F16) return a.ydtype == BL_F16 ? start_rows_expand<BL_F16, BL_F16>(p, s) : start_rows_expand<BL_F16, BL_F32>(p, s);
  if (a.dtype == BL_BF16) return a.ydtype == BL_BF16 ? start_rows_expand<BL_BF16, BL_BF16>(p, s) : start_rows_expand<BL_BF16, BL_F32>(p, s);
  return start_rows_expand<BL_F32, BL_F32>(p, s);
}

// Splits for about 300 workgroups, 448 beyond rank 32, where the matrices' reads take as long as the
// rows': less than the 512 that the chip holds at once, since one that starts after the others doubles
// the time. (us, 300 / 448, bf16: 777 x 8640, rank 12 11.9 / 13.6, 4096 x 8192, rank 32 27.9 / 30.4,
// rank 64 38.5 / 31.3.)
int shrink_splits(int64_t M, int64_t L, int64_t R, int64_t D) {
  const int64_t groups = max_tiles(M, L) * div_up(rank_pad(R), 64), most = R <= 32 ? 300 : 448;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({most / groups, div_up(D, 64) / (2 * kShrinkWaves), 16})));
}
// Tiles of a workgroup of the product along the long axis: as many as leave 1024 workgroups or so. (us
// for 1 / 2 / 4 / 8, bf16: 4096 x 8192, rank 64 42 / 38 / 38 / 42, rank 32 34 / 31 / 32 / 36; 777 x
// 3200, rank 12, fp32 results 7.4 / 9.2 for 1 / 2.)
int expand_tiles_of(int64_t M, int64_t N) { return M * N >= int64_t(1) << 25 ? 4 : M * N >= int64_t(1) << 24 ? 2 : 1; }
// A run of tiles to each of the eight chips, or neighbours to different ones (us, by chip / not, bf16,
// 4096 rows of 8192: 64 adapters of rank 64 103 / 108, 8 79.1 / 80.6, of rank 32 70.5 / 71.0; fewer
// rows gain or lose as often: 1024 of 8192, rank 32 28.9 / 30.8, 1024 of 3200, rank 8 26.0 / 25.3, 400
// of 8640, rank 64 27.7 / 27.1).
int by_chip(const AdapterRows& r) { return r.M >= 64 * kTile; }
// Two workgroups to a CU, or the one that two tiles' registers of 16-bit values leave beyond rank 16. (us,
// 4096 rows of 8192, bf16, rank 32: 22 for 256 workgroups, 32 for 384, 30 for 512, 44 for 1024.)
// `blocks`: of 128 columns, of all that one launch takes.
int outer_splits(int64_t M, int64_t L, int64_t R, int64_t blocks, int dt) {
  const int64_t most = dt != BL_F32 && R > 16 ? 256 : 512, groups = blocks * div_up(rank_pad(R), 32);
  // four tiles to a share at least, or four adapters, whose gradients are written even if they have no rows
  const int64_t enough = std::max(div_up(M / kTile + std::min(M, L), 4), div_up(L, 4));
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({most / groups, enough, 32})));
}
// The most shares that a call's sums have, and the counters of one of them.
int64_t outer_shares(int64_t M, int64_t L, int64_t R, int64_t K, int64_t N) { return outer_splits(M, L, R, div_up(K, 128) + div_up(N, 128), BL_F32); }
int64_t outer_counters(int64_t shares, int64_t R, int64_t D) { return shares * div_up(D, 128) * div_up(rank_pad(R), 32); }

// Bytes of each layout of the coefficients.
struct CoefBytes {
  size_t f, by_row, by_rank;
};
CoefBytes coef_bytes(int64_t M, int64_t L, int64_t R) {
  const int64_t rows = max_tiles(M, L) * kTile, RP = rank_pad(R), RK = div_up(R, 32) * 32;
  return {static_cast<size_t>(rows * RP * 4), static_cast<size_t>(kParts * rows * RK * 2), static_cast<size_t>(kParts * rows * RP * 2)};
}

struct Scratch {
  Sorted o;
  int32_t* order;
  int32_t* tile;
  int32_t* start;
  int32_t* counts;
  uint32_t* arrived;
  float *part, *sum[2];
  Coefs c, hc;
};
Scratch scratch(const AdapterWs& L, char* ws, const AdapterRows& r) {
  Scratch s{};
  s.order = reinterpret_cast<int32_t*>(ws + L.order_off);
  s.tile = reinterpret_cast<int32_t*>(ws + L.tile_off);
  s.start = reinterpret_cast<int32_t*>(ws + L.start_off);
  s.counts = reinterpret_cast<int32_t*>(ws + L.count_off);
  s.arrived = reinterpret_cast<uint32_t*>(ws + L.arrived_off);
  s.part = reinterpret_cast<float*>(ws + L.part_off);
  for (int i = 0; i < 2; ++i) s.sum[i] = reinterpret_cast<float*>(ws + L.sum_off[i]);
  s.o = Sorted{s.order, s.tile, s.start, static_cast<int>(r.L), max_tiles(r.M, r.L) * kTile};
  const auto coefs = [&](const size_t (&at)[3]) {
    return Coefs{reinterpret_cast<float*>(ws + at[0]), reinterpret_cast<uint16_t*>(ws + at[1]), reinterpret_cast<uint16_t*>(ws + at[2])};
  };
  s.c = coefs(L.c_off);
  s.hc = coefs(L.hc_off);
  return s;
}

hipError_t sort_rows(const AdapterRows& r, const Scratch& w, int64_t counters, hipStream_t s) {
  const int chunks = static_cast<int>(div_up(r.M, kSortChunk));
  const int steps = chunks > 1 ? kSortSteps : static_cast<int>(div_up(r.M, 64 * kSortWaves));
  const SortArgs a{r.index, r.M, static_cast<int>(r.L), chunks, steps, w.order, w.tile, w.start, w.counts, w.arrived, counters};
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

template <int SD, int WD, int NR, int CD, int HD>
hipError_t start_shrink_as(const ShrinkArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 grid(a.splits, static_cast<uint32_t>(tiles) + (a.by_chip ? 7 : 0), static_cast<uint32_t>(div_up(a.RP, 64)));
  const size_t lds = std::max<size_t>(kShrinkWaves * (kTile * 8 + 16 * NR * 8) * 16, kTile * static_cast<size_t>(a.RP + 1) * 4);
  adapter_shrink_kernel<SD, WD, NR, CD, HD><<<grid, 64 * kShrinkWaves, lds, s>>>(a);
  return hipGetLastError();
}
template <int SD, int WD, int CD, int HD>
hipError_t start_shrink_nr(const ShrinkArgs& a, int64_t tiles, hipStream_t s) {
  const int nr = std::min(a.RP / 16, 4);
  if (nr == 1) return start_shrink_as<SD, WD, 1, CD, HD>(a, tiles, s);
  if (nr == 2) return start_shrink_as<SD, WD, 2, CD, HD>(a, tiles, s);
  if (nr == 3) return start_shrink_as<SD, WD, 3, CD, HD>(a, tiles, s);
  return start_shrink_as<SD, WD, 4, CD, HD>(a, tiles, s);
}
// sd is wd, or fp32. The sums' coefficients multiply values of wd, h_in's values of sd.
hipError_t start_shrink(const ShrinkArgs& a, int sd, int wd, int64_t tiles, hipStream_t s) {
  if (wd == BL_F16)
    return sd == BL_F16 ? start_shrink_nr<BL_F16, BL_F16, BL_F16, BL_F16>(a, tiles, s)
                       : start_shrink_nr<BL_F32, BL_F16, BL_F16, BL_F32>(a, tiles, s);
  if (wd == BL_BF16)
    return sd == BL_BF16 ? start_shrink_nr<BL_BF16, BL_BF16, BL_BF16, BL_BF16>(a, tiles, s)
                        : start_shrink_nr<BL_F32, BL_BF16, BL_BF16, BL_F32>(a, tiles, s);
  return start_shrink_nr<BL_F32, BL_F32, BL_F32, BL_F32>(a, tiles, s);
}

template <int WD, int YD>
hipError_t start_expand_as(const ExpandArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(div_up(a.N, 256)), static_cast<uint32_t>(tiles));
  if (WD == BL_F32 || a.RP > 64) adapter_expand_kernel<WD, YD, 0><<<grid, 256, 0, s>>>(a);
  else if (a.RP > 32) adapter_expand_kernel<WD, YD, WD == BL_F32 ? 0 : 2><<<grid, 256, 0, s>>>(a);
  else adapter_expand_kernel<WD, YD, WD == BL_F32 ? 0 : 1><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
// yd is wd, or fp32.
hipError_t start_expand(const ExpandArgs& a, int wd, int yd, int64_t tiles, hipStream_t s) {
  if (wd == BL_F16) return yd == BL_F16 ? start_expand_as<BL_F16, BL_F16>(a, tiles, s) : start_expand_as<BL_F16, BL_F32>(a, tiles, s);
  if (wd == BL_BF16) return yd == BL_BF16 ? start_expand_as<BL_BF16, BL_BF16>(a, tiles, s) : start_expand_as<BL_BF16, BL_F32>(a, tiles, s);
  return start_expand_as<BL_F32, BL_F32>(a, tiles, s);
}

template <int SD, int TD>
hipError_t start_outer_as(const OuterPair& a, uint32_t columns, hipStream_t s) {
  const dim3 grid(columns, std::max(a.p[0].splits, a.p[1].splits), static_cast<uint32_t>(div_up(a.p[0].RP, 32)));
  if (a.p[0].RP == 16) adapter_outer_kernel<SD, TD, 1><<<grid, 256, 0, s>>>(a);
  else adapter_outer_kernel<SD, TD, 2><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
// Types of the sums: the same, or fp32 and another.
hipError_t start_outer(const OuterPair& a, uint32_t columns, int sd, int td, hipStream_t s) {
  if (sd == td)
    return sd == BL_F16    ? start_outer_as<BL_F16, BL_F16>(a, columns, s)
           : sd == BL_BF16 ? start_outer_as<BL_BF16, BL_BF16>(a, columns, s)
                           : start_outer_as<BL_F32, BL_F32>(a, columns, s);
  return td == BL_F16 ? start_outer_as<BL_F32, BL_F16>(a, columns, s) : start_outer_as<BL_F32, BL_BF16>(a, columns, s);
}

// The layouts that a value of type dt is multiplied by: fp32 for fp32, else parts.
Coefs only(const Coefs& c, int dt, bool rows, bool ranks) {
  Coefs o{};
  if (dt == BL_F32) o.f = c.f;
  else if (rows) o.by_row = c.by_row;
  if (dt != BL_F32 && ranks) o.by_rank = c.by_rank;
  return o;
}

}  // namespace

AdapterWs adapter_ws(int64_t M, int64_t L, int64_t R, int64_t K, int64_t N, bool backward) {
  AdapterWs w{};
  if (!backward && by_rows(M, R, K, N)) return w;
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += (static_cast<size_t>(bytes) + 255) & ~size_t(255);
    return at;
  };
  const int64_t tiles = max_tiles(M, L), rows = tiles * kTile, RP = rank_pad(R), D = backward ? N : K;
  const CoefBytes b = coef_bytes(M, L, R);
  w.order_off = take(rows * 4);
  w.tile_off = take(tiles * 4);
  w.start_off = take((L + 2) * 4);
  w.count_off = take(M > kSortChunk ? div_up(M, kSortChunk) * (L + 1) * 4 : 0);
  const int64_t shares = outer_shares(M, L, R, K, N), splits = shrink_splits(M, L, R, D);
  w.counters = tiles + (backward ? outer_counters(shares, R, K) + outer_counters(shares, R, N) : 0);
  w.arrived_off = take(w.counters * 4);
  w.part_off = take(splits * div_up(RP, 64) > 1 ? splits * rows * RP * 4 : 0);   // a workgroup that has a tile alone meets none
  const size_t each[3] = {b.f, b.by_row, backward ? b.by_rank : 0};
  for (int i = 0; i < 3; ++i) w.c_off[i] = take(each[i]);
  if (backward) {
    w.hc_off[0] = take(b.f);
    w.hc_off[2] = take(b.by_rank);
    w.sum_off[0] = take(shares > 1 ? 2 * shares * R * K * 4 : 0);   // every adapter lies within the one share
    w.sum_off[1] = take(shares > 1 ? 2 * shares * R * N * 4 : 0);
  }
  w.total = off;
  return w;
}

hipError_t launch_adapter_forward(const AdapterForwardArgs& a, char* ws, hipStream_t s) {
  const AdapterRows& r = a.rows;
  if (by_rows(r.M, r.R, a.K, a.N)) return forward_by_rows(a, s);
  const AdapterWs L = adapter_ws(r.M, r.L, r.R, a.K, a.N, false);
  const Scratch w = scratch(L, ws, r);
  const int64_t tiles = max_tiles(r.M, r.L);
  const int R = static_cast<int>(r.R), RP = rank_pad(r.R), splits = shrink_splits(r.M, r.L, r.R, a.K);
  hipError_t e = sort_rows(r, w, L.counters, s);
  if (e != hipSuccess) return e;
  ShrinkArgs p{w.o, a.x, a.K, a.ldx, a.a, R, RP, splits, by_chip(r), w.part, w.arrived, a.scale, a.h, nullptr, only(w.c, a.dtype, true, false), {}};
  e = start_shrink(p, a.dtype, a.dtype, tiles, s);
  if (e != hipSuccess) return e;
  return start_expand(ExpandArgs{w.o, w.c, R, RP, a.h, a.b, a.N, a.base, a.ldbase, a.y, a.ldy, expand_tiles_of(r.M, a.N)}, a.dtype,
                      a.ydtype, tiles, s);
}

hipError_t launch_adapter_backward(const AdapterBackwardArgs& a, char* ws, hipStream_t s) {
  const AdapterRows& r = a.rows;
  const AdapterWs L = adapter_ws(r.M, r.L, r.R, a.K, a.N, true);
  const Scratch w = scratch(L, ws, r);
  const int64_t tiles = max_tiles(r.M, r.L);
  const int R = static_cast<int>(r.R), RP = rank_pad(r.R), splits = shrink_splits(r.M, r.L, r.R, a.N);
  hipError_t e = sort_rows(r, w, L.counters, s);
  if (e != hipSuccess) return e;
  ShrinkArgs p{w.o, a.dy, a.N, a.lddy, a.b, R, RP, splits, by_chip(r), w.part, w.arrived, a.scale, nullptr, a.h,
               only(w.c, a.dtype, a.dx != nullptr, true), only(w.hc, a.dydtype, false, true)};
  e = start_shrink(p, a.dydtype, a.dtype, tiles, s);
  if (e != hipSuccess) return e;
  uint32_t* arrived = w.arrived + tiles;
  const int64_t kb = div_up(a.K, 128), nb = div_up(a.N, 128);
  const int shares = outer_splits(r.M, r.L, r.R, kb + nb, a.dydtype);
  const OuterArgs da{w.o, w.c, a.x, a.K, a.ldx, R, RP, shares, w.sum[0], arrived, a.da, a.add};
  const OuterArgs db{w.o, w.hc, a.dy, a.N, a.lddy, R, RP, shares, w.sum[1], arrived + outer_counters(shares, r.R, a.K), a.db, a.add};
  // before dx, whose traffic would turn dy out of the caches; fp32, which takes longer, first
  e = start_outer(OuterPair{{db, da}, static_cast<uint32_t>(nb)}, static_cast<uint32_t>(kb + nb), a.dydtype, a.dtype, s);
  if (e != hipSuccess || !a.dx) return e;
  return start_expand(ExpandArgs{w.o, w.c, R, RP, nullptr, a.a, a.K, a.base, a.ldbase, a.dx, a.lddx, expand_tiles_of(r.M, a.K)}, a.dtype,
                      a.dxdtype, tiles, s);
}

}  // namespace bl
