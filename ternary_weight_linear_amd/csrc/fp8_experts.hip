// The experts' gated products (bl_fp8_experts): sort the (token, slot) pairs by expert,
// quantise x, multiply by the gate and up matrices, quantise silu(gate) * up, multiply by the
// down matrix, and add each token's slots with their weights.
#include <algorithm>

#include "fp8_gemm.h"

namespace bl {
namespace {

constexpr int kSortThreads = 256;

// The sort of the slots by expert. A chunk of slots per workgroup: each counts its chunk's
// slots per expert, and where there is more than one chunk, a second launch (which needs all
// counts) places them. Slots whose index is outside [0, E) get no row. The order of the rows of
// one expert within a chunk may differ from run to run; no output depends on it, since each
// row is multiplied by itself.
struct SortArgs {
  const int32_t* index;
  int P, E, chunk, chunks, tile;
  int32_t* head;      // [2] rows used, tiles
  int32_t* pair;      // [P] slot of each sorted row
  int32_t* tiles;     // [tiles, 4] expert, first row, rows
  int32_t* counts;    // [chunks, E], more than one chunk
};
// Up to 2048 slots one workgroup, which needs no second launch; else chunks of 512 (two slots
// per thread: the passes over a chunk wait on memory), at most 64.
inline int sort_chunk(int64_t P) {
  return static_cast<int>(P <= 2048 ? 2048 : P <= 512 * 64 ? 512 : (P + 63) / 64);
}
inline int sort_lds(int64_t E) { return static_cast<int>(E) * 8; }

__device__ __forceinline__ void count_slots(const SortArgs& a, int chunk, int* cnt) {
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int end = min((chunk + 1) * a.chunk, a.P);
  for (int i = chunk * a.chunk + threadIdx.x; i < end; i += kSortThreads) {
    const int e = a.index[i];
    if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
}

// From all slots per expert (cnt) and those of earlier chunks (next): the rows of this chunk's
// slots, and from chunk 0 the tiles. Each thread has a run of experts; runs are summed by a
// scan over the workgroup.
__device__ __forceinline__ void place_slots(const SortArgs& a, int chunk, const int* cnt, int* next) {
  __shared__ int sums[2][kSortThreads / 64];
  const int per = (a.E + kSortThreads - 1) / kSortThreads;
  const int e0 = threadIdx.x * per, e1 = min(e0 + per, a.E);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int rows = 0, nt = 0;
  for (int e = e0; e < e1; ++e) {
    rows += cnt[e];
    nt += (cnt[e] + a.tile - 1) / a.tile;
  }
  int row = rows, at = nt;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int r = __shfl_up(row, off), t = __shfl_up(at, off);
    if (lane >= off) {
      row += r;
      at += t;
    }
  }
  if (lane == 63) {
    sums[0][wave] = row;
    sums[1][wave] = at;
  }
  __syncthreads();
  for (int v = 0; v < wave; ++v) {
    row += sums[0][v];
    at += sums[1][v];
  }
  if (chunk == 0 && threadIdx.x == kSortThreads - 1) {
    a.head[0] = row;
    a.head[1] = at;
  }
  row -= rows;
  at -= nt;
  for (int e = e0; e < e1; ++e) {
    next[e] += row;
    if (chunk == 0)
      for (int r = 0; r < cnt[e]; r += a.tile, ++at) {
        a.tiles[4 * at] = e;
        a.tiles[4 * at + 1] = row + r;
        a.tiles[4 * at + 2] = min(a.tile, cnt[e] - r);
      }
    row += cnt[e];
  }
  __syncthreads();
  const int end = min((chunk + 1) * a.chunk, a.P);
  for (int i = chunk * a.chunk + threadIdx.x; i < end; i += kSortThreads) {
    const int e = a.index[i];
    if (e >= 0 && e < a.E) a.pair[atomicAdd(&next[e], 1)] = i;
  }
}

// One launch for what needs only the inputs: the first workgroups sort (or count) the slots,
// the others quantise x. 48 tokens of 4096, top 8 of 64: 4.7 us; 4096 tokens: 13 (and 7.4 for
// the placing), most of it waits of the passes over a chunk's slots.
template <int DT>
__global__ __launch_bounds__(kSortThreads) void experts_prepare_kernel(SortArgs a, QuantArgs q) {
  extern __shared__ int lds[];                     // [2, E]
  const int chunk = blockIdx.x;
  if (chunk >= a.chunks) {
    quant_blocks<DT, false>(q, static_cast<int64_t>(chunk - a.chunks) * (kSortThreads / 16));
    return;
  }
  int *cnt = lds, *next = lds + a.E;
  count_slots(a, chunk, cnt);
  if (a.chunks == 1) {
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) next[e] = 0;
    __syncthreads();
    place_slots(a, 0, cnt, next);
  } else {
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.counts[chunk * a.E + e] = cnt[e];
  }
}

__global__ __launch_bounds__(kSortThreads) void experts_place_kernel(SortArgs a) {
  extern __shared__ int lds[];                     // [2, E]
  const int chunk = blockIdx.x;
  int *cnt = lds, *next = lds + a.E;
  for (int i = threadIdx.x; i < 2 * a.E; i += kSortThreads) lds[i] = 0;
  __syncthreads();
  // the table is read as it lies, several words of it in flight per thread
  const int before = chunk * a.E;
#pragma unroll 8
  for (int i = threadIdx.x; i < a.chunks * a.E; i += kSortThreads) {
    const int n = a.counts[i], e = i % a.E;
    atomicAdd(&cnt[e], n);
    if (i < before) atomicAdd(&next[e], n);
  }
  __syncthreads();
  place_slots(a, chunk, cnt, next);
}

// y[m, n] = sum_j weight[m, j] part[m k + j, n], slots in their order. A thread has four columns
// (16 bytes) and up to eight slots' loads in flight: reading the parts bounds it (32768 x
// 4096: 124 us, 4.6 TB/s).
__global__ __launch_bounds__(256) void experts_combine_kernel(Fp8ExpertsArgs a, const float* __restrict__ part) {
  const int64_t m = blockIdx.x;
  const int64_t n = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * 4;
  if (n >= a.H) return;                             // H % 16 == 0: all four or none
  f32x4 sum = {0, 0, 0, 0};
  for (int64_t j0 = 0; j0 < a.k; j0 += 8) {
    f32x4 v[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t slot = m * a.k + j0 + j;
      const int e = j0 + j < a.k ? a.index[slot] : -1;
      w[j] = 0.0f;
      v[j] = f32x4{0, 0, 0, 0};
      if (e >= 0 && e < a.E) {
        w[j] = a.weight[slot];
        v[j] = *reinterpret_cast<const f32x4*>(part + slot * a.H + n);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += w[j] * v[j][i];
  }
  Fp8LinearArgs o{};
  o.N = a.H;
  o.y = a.y;
  o.ldy = a.ldy;
  o.ydtype = a.ydtype;
  store4(o, m, n, sum);
}

// The gate and up products take fp16 operands whatever the types: a sum that errs by more than
// fp32 does moves codes of silu(gate) * up (with the e4m3 instruction 1 of 3000, which put 1.2e-3
// of the result beside the 1.7e-3 of its rounding to bf16). 4096 tokens, top 8 of 64 experts of 4096
// x 1024: 630 us, 0.87 PFLOP/s; converting the codes bounds it, and a ninth of the tiles' rows
// are empty.
hipError_t start_up(const ProductArgs& p, int tile, int64_t nt, hipStream_t s) {
  if (tile == 64) return start_gemm<GemmShape<256, 64, 4, 2, 3, true, true>>(p, nt, s);
  return start_gemm<GemmShape<256, 128, 2, 4, 2, true, true>>(p, nt, s);
}
// Stages: three where the matrix instructions are fast, two where converting the codes is what
// takes long.
template <bool EXACT>
hipError_t start_down(const ProductArgs& p, int tile, int64_t nt, hipStream_t s) {
  if (tile == 64) return start_gemm<GemmShape<256, 64, 4, 2, 3, EXACT>>(p, nt, s);
  return start_gemm<GemmShape<256, 128, 2, 4, EXACT ? 2 : 3, EXACT>>(p, nt, s);
}

int64_t max_tiles(int64_t P, int64_t E, int tile) { return P / tile + (P < E ? P : E); }

// The tiled kernel's offsets within a matrix are 32 bits.
bool matrices_fit(int64_t H, int64_t I) {
  return 2 * I * H < (int64_t(1) << 31) && 256 * I < (int64_t(1) << 31);
}

// Tokens of one pass: a call of more runs pass after pass. The tiled kernel gathers rows of x's
// codes by 32-bit offsets, and the grids of the products stay in their limits (the streamed tiles
// of 16 rows lie along a dimension of 65535).
int64_t pass_tokens(int64_t M, int64_t H, int64_t k, int64_t I) {
  int64_t most = ((int64_t(1) << 31) - 1) / H;
  const int64_t slots = (int64_t(1) << 35) / I;
  most = std::min(most, std::max<int64_t>((matrices_fit(H, I) ? slots : std::min<int64_t>(slots, 1 << 19)) / k, 1));
  const int64_t passes = (M + most - 1) / most;
  return (M + passes - 1) / passes;
}

}  // namespace

ExpertsWs experts_ws(int64_t M_all, int64_t H, int64_t k, int64_t E, int64_t I) {
  ExpertsWs w{};
  const int64_t M = pass_tokens(M_all, H, k, I);
  const int64_t P = M * k, HB = fp8_blocks(H), IB = fp8_blocks(I);
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += (static_cast<size_t>(bytes) + 255) & ~size_t(255);
    return at;
  };
  w.q_off = take(M * H);
  w.sx_off = take(M * HB * 4);
  w.head_off = take(16);
  w.pair_off = take(P * 4);
  w.tile_off = take(max_tiles(P, E, 16) * 16);
  w.count_off = take((P + sort_chunk(P) - 1) / sort_chunk(P) * E * 4);
  w.hq_off = take(P * I);
  w.hs_off = take(P * IB * 4);
  w.sum_off = take(P * std::max(H, I) * 4);
  w.total = off;
  return w;
}

namespace {

hipError_t start_pass(const Fp8ExpertsArgs& a, char* ws, hipStream_t s) {
  const ExpertsWs L = experts_ws(a.M, a.H, a.k, a.E, a.I);
  const int64_t P = a.M * a.k, HB = fp8_blocks(a.H), IB = fp8_blocks(a.I);
  auto* q = reinterpret_cast<uint8_t*>(ws + L.q_off);
  auto* sx = reinterpret_cast<float*>(ws + L.sx_off);
  auto* head = reinterpret_cast<int32_t*>(ws + L.head_off);
  auto* pair = reinterpret_cast<int32_t*>(ws + L.pair_off);
  auto* tiles = reinterpret_cast<int32_t*>(ws + L.tile_off);
  auto* h = reinterpret_cast<float*>(ws + L.sum_off);
  auto* hq = reinterpret_cast<uint8_t*>(ws + L.hq_off);
  auto* hs = reinterpret_cast<float*>(ws + L.hs_off);
  float* part = h;                                  // h is done with before the down product starts
  const bool exact_down = a.ydtype != BL_BF16;
  // Rows per tile, by the average rows of an expert. Measured, us for tiles of 16 / 64 / 128 rows, 64
  // experts of 4096 x 1024, top 8, bf16: 16 rows an expert 208 / 210 / 221, 32 319 / 262 / 242, 64
  // 548 / 271 / 311, 96 782 / 351 / 322, 128 1015 / 396 / 347, 512 3833 / 1292 / 1076; 16 experts of
  // 2048 x 1024, top 2: 32 57 / 44 / 45, 128 148 / 86 / 67. Too few workgroups of a tile call for the
  // next smaller one: 8 experts of 1024 x 256, top 2: 32 28 / 29 / 30, 128 42 / 33 / 42; 9 of 2784 x
  // 336, top 8: 32 33 / 50 / 49; 49 of 2384 x 128: 151 251 / 80 / 89.
  const bool tiled = P > 16 * a.E && matrices_fit(a.H, a.I);
  const auto groups = [&](int64_t rows) {
    const int64_t most = (P + a.E - 1) / a.E;         // of one expert, were all alike
    return a.E * ((most + rows - 1) / rows) * ((a.I + 127) / 128);
  };
  int tile = !tiled ? 16 : P <= 96 * a.E ? 64 : 128;
  if (tile == 128 && groups(128) < 128) tile = 64;
  if (tile == 64 && P <= 40 * a.E && groups(64) <= 64) tile = 16;
  const int64_t nt = max_tiles(P, a.E, tile);
  // Few slots, most of them of different experts: a tile each, nothing to sort, and the rows are
  // quantised where they are used: two launches for five. A matrix that several slots share is
  // read once for each, so this ends where slots meet (us, this way / sorted, matrices of
  // 4096 x 1024: 24 slots of 64 experts 54 / 63, 32 of 64 75 / 67, 16 of 16 55 / 39, 8 of 16
  // 28 / 31, 8 of 4 31 / 30).
  constexpr int kStagedMost = 48 * 1024;
  const bool direct = (8 * P <= 3 * a.E || P <= 8) && a.H <= kStagedMost && a.k * a.I <= kStagedMost &&
                      staged_bytes(1, static_cast<int>(HB)) <= kStagedMost &&
                      staged_bytes(static_cast<int>(a.k), static_cast<int>(IB)) <= kStagedMost;

  // gate and up: silu(gate) * up of every sorted row, in fp32 (streamed) or as codes (tiled)
  StreamArgs up{};
  up.p.a = Fp8LinearArgs{q, sx, a.wgu, a.sgu, a.M, a.I, a.H, h, a.I, BL_F32};
  up.p.map = RowMap{tiles, head + 1, direct ? nullptr : pair, static_cast<int>(a.k), 0};
  up.p.w_stride = 2 * a.I * a.H;
  up.p.sw_stride = 2 * IB * HB;
  up.p.hq = hq;
  up.p.hs = hs;
  up.p.h_rows = P;
  up.x = a.x;
  up.ldx = a.ldx;
  up.E = static_cast<int>(a.E);
  up.k = static_cast<int>(a.k);
  StreamArgs down{};
  down.p.a = Fp8LinearArgs{hq, hs, a.wd, a.sd, P, a.H, a.I, part, a.H, BL_F32};
  down.p.map = RowMap{tiles, head + 1, pair, 0, 1};
  down.p.w_stride = a.H * a.I;
  down.p.sw_stride = HB * IB;
  down.x = h;
  down.ldx = a.I;
  down.E = up.E;
  down.k = up.k;
  hipError_t e;

  if (direct) {
    up.index = down.index = a.index;
    down.weight = a.weight;
    down.p.a.y = a.y;
    down.p.a.ydtype = a.ydtype;
    down.p.a.ldy = a.ldy;
    e = start_stream_x<2, 8, kStreamGated>(up, a.xdtype, P, 1, s);
    if (e != hipSuccess) return e;
    return start_stream<1, 1, 8, BL_F32, kStreamSlots>(down, a.M, static_cast<int>(a.k), s);
  }

  SortArgs sort{a.index, static_cast<int>(P), static_cast<int>(a.E), sort_chunk(P), 0, tile, head, pair, tiles,
                reinterpret_cast<int32_t*>(ws + L.count_off)};
  sort.chunks = static_cast<int>((P + sort.chunk - 1) / sort.chunk);
  const QuantArgs quant{a.x, a.M, a.H, HB, a.ldx, nullptr, q, sx};
  const dim3 prepare(static_cast<uint32_t>(sort.chunks + (a.M * HB + 15) / 16));
  if (a.xdtype == BL_F16) experts_prepare_kernel<BL_F16><<<prepare, kSortThreads, sort_lds(a.E), s>>>(sort, quant);
  else if (a.xdtype == BL_BF16) experts_prepare_kernel<BL_BF16><<<prepare, kSortThreads, sort_lds(a.E), s>>>(sort, quant);
  else experts_prepare_kernel<BL_F32><<<prepare, kSortThreads, sort_lds(a.E), s>>>(sort, quant);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (sort.chunks > 1) {
    experts_place_kernel<<<sort.chunks, kSortThreads, sort_lds(a.E), s>>>(sort);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (tile == 16) {
    e = start_stream<1, 4, 8, kSrcCodes, kStreamGated>(up, nt, 0, s);
    if (e != hipSuccess) return e;
    e = launch_fp8_quant_act(h, BL_F32, P, a.I, a.I, 0, head, hq, hs, s);
    if (e != hipSuccess) return e;
    e = start_stream<1, 4, 8, kSrcCodes, kStreamLinear>(down, nt, 0, s);
  } else {
    e = start_up(up.p, tile, nt, s);
    if (e != hipSuccess) return e;
    e = exact_down ? start_down<true>(down.p, tile, nt, s) : start_down<false>(down.p, tile, nt, s);
  }
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<uint32_t>(a.M), static_cast<uint32_t>((a.H + 1023) / 1024));
  experts_combine_kernel<<<grid, 256, 0, s>>>(a, part);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_experts(const Fp8ExpertsArgs& a, char* ws, hipStream_t s) {
  const int64_t tokens = pass_tokens(a.M, a.H, a.k, a.I);
  for (int64_t m = 0; m < a.M; m += tokens) {
    Fp8ExpertsArgs p = a;
    p.M = std::min(tokens, a.M - m);
    p.x = static_cast<const char*>(a.x) + m * a.ldx * dtype_bytes(a.xdtype);
    p.y = static_cast<char*>(a.y) + m * a.ldy * dtype_bytes(a.ydtype);
    p.index = a.index + m * a.k;
    p.weight = a.weight + m * a.k;
    const hipError_t e = start_pass(p, ws, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bl
