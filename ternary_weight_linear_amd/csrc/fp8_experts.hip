// The experts' gated products (bl_fp8_experts): sort the (token, slot) pairs by expert,
// quantise x, multiply by the gate and up matrices, quantise silu(gate) * up, multiply by the
// down matrix, and add each token's slots with their weights.
#include "fp8_gemm.h"

namespace bl {
namespace {

constexpr int kSortThreads = 1024;

// One workgroup: counts per expert, their running sum, the sorted rows and the tiles of at
// most `tile` rows. Slots whose index is outside [0, E) get no row. The order of the rows
// within an expert may differ from run to run; no output depends on it, since each row is
// multiplied by itself.
__global__ __launch_bounds__(kSortThreads) void experts_sort_kernel(
    const int32_t* __restrict__ index, int P, int E, int tile, int32_t* __restrict__ head,
    int32_t* __restrict__ pair, int32_t* __restrict__ tiles) {
  extern __shared__ int cnt[];              // [E] counts, then [E] next positions
  __shared__ int scan[2][kSortThreads];
  int* next = cnt + E;
  for (int e = threadIdx.x; e < E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < P; i += kSortThreads) {
    const int e = index[i];
    if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  // each thread sums its run of experts, then a scan over the threads
  const int per = (E + kSortThreads - 1) / kSortThreads;
  const int e0 = threadIdx.x * per;
  int rows = 0, nt = 0;
  for (int e = e0; e < min(e0 + per, E); ++e) {
    rows += cnt[e];
    nt += (cnt[e] + tile - 1) / tile;
  }
  scan[0][threadIdx.x] = rows;
  scan[1][threadIdx.x] = nt;
  __syncthreads();
  for (int off = 1; off < kSortThreads; off <<= 1) {
    int r = 0, t = 0;
    if (static_cast<int>(threadIdx.x) >= off) {
      r = scan[0][threadIdx.x - off];
      t = scan[1][threadIdx.x - off];
    }
    __syncthreads();
    scan[0][threadIdx.x] += r;
    scan[1][threadIdx.x] += t;
    __syncthreads();
  }
  int row = scan[0][threadIdx.x] - rows, at = scan[1][threadIdx.x] - nt;
  for (int e = e0; e < min(e0 + per, E); ++e) {
    next[e] = row;
    for (int r = 0; r < cnt[e]; r += tile, ++at) {
      tiles[4 * at] = e;
      tiles[4 * at + 1] = row + r;
      tiles[4 * at + 2] = min(tile, cnt[e] - r);
    }
    row += cnt[e];
  }
  if (threadIdx.x == kSortThreads - 1) {
    head[0] = scan[0][threadIdx.x];
    head[1] = scan[1][threadIdx.x];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < P; i += kSortThreads) {
    const int e = index[i];
    if (e >= 0 && e < E) pair[atomicAdd(&next[e], 1)] = i;
  }
}

// y[m, n] = sum_j weight[m, j] part[m k + j, n], slots in their order.
__global__ __launch_bounds__(256) void experts_combine_kernel(Fp8ExpertsArgs a,
                                                              const float* __restrict__ part) {
  const int64_t m = blockIdx.x;
  for (int64_t n = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x; n < a.H; n += 256 * gridDim.y) {
    float sum = 0.0f;
    for (int64_t j = 0; j < a.k; ++j) {
      const int e = a.index[m * a.k + j];
      if (e >= 0 && e < a.E) sum += a.weight[m * a.k + j] * part[(m * a.k + j) * a.H + n];
    }
    store_as(a.y, a.ydtype, m * a.ldy + n, sum);
  }
}

}  // namespace

int64_t experts_max_tiles(int64_t P, int64_t E, int tile) { return P / tile + (P < E ? P : E); }

ExpertsWs experts_ws(int64_t M, int64_t H, int64_t k, int64_t E, int64_t I) {
  ExpertsWs w{};
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
  w.tile_off = take(experts_max_tiles(P, E, 16) * 16);
  w.h_off = take(P * I * 4);
  w.hq_off = take(P * I);
  w.hs_off = take(P * IB * 4);
  w.part_off = take(P * H * 4);
  w.total = off;
  return w;
}

hipError_t launch_fp8_experts(const Fp8ExpertsArgs& a, char* ws, hipStream_t s) {
  const ExpertsWs L = experts_ws(a.M, a.H, a.k, a.E, a.I);
  const int64_t P = a.M * a.k, HB = fp8_blocks(a.H), IB = fp8_blocks(a.I);
  auto* q = reinterpret_cast<uint8_t*>(ws + L.q_off);
  auto* sx = reinterpret_cast<float*>(ws + L.sx_off);
  auto* head = reinterpret_cast<int32_t*>(ws + L.head_off);
  auto* pair = reinterpret_cast<int32_t*>(ws + L.pair_off);
  auto* tiles = reinterpret_cast<int32_t*>(ws + L.tile_off);
  auto* h = reinterpret_cast<float*>(ws + L.h_off);
  auto* hq = reinterpret_cast<uint8_t*>(ws + L.hq_off);
  auto* hs = reinterpret_cast<float*>(ws + L.hs_off);
  auto* part = reinterpret_cast<float*>(ws + L.part_off);
  // fp16 operands where the hidden layer's or the result's type would show the e4m3
  // instruction's sums (its error, 1.4e-5 of a block's, moves a few hidden codes: 1/2 of
  // bf16's rounding of the result, 4 times fp16's)
  const bool exact = a.xdtype != BL_BF16, exact_down = a.ydtype == BL_F32;
  // rows per tile, by the average rows of an expert; the tiled kernel's offsets are 32 bits
  const bool tiled = P > 48 * a.E && a.M * a.H < (int64_t(1) << 31) && 2 * a.I * a.H < (int64_t(1) << 31) &&
                     256 * a.I < (int64_t(1) << 31);
  const int tile = !tiled ? (P <= 16 * a.E ? 16 : 64) : P <= 192 * a.E || exact || exact_down ? 128 : 256;
  const int64_t nt = experts_max_tiles(P, a.E, tile);
  // few slots: a tile each, nothing to sort, and the rows are quantised where they are used
  constexpr int kStagedMost = 48 * 1024;
  const bool direct = (4 * P <= a.E || P <= 16) && a.H <= kStagedMost && a.k * a.I <= kStagedMost &&
                      staged_bytes(1, static_cast<int>(HB)) <= kStagedMost &&
                      staged_bytes(static_cast<int>(a.k), static_cast<int>(IB)) <= kStagedMost;

  // gate and up: silu(gate) * up of every sorted row, in fp32 (streamed) or as codes (tiled)
  StreamArgs up{};
  up.p.a = Fp8LinearArgs{q, sx, a.wgu, a.sgu, a.M, a.I, a.H, h, a.I, BL_F32, 1};
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
  down.p.a = Fp8LinearArgs{hq, hs, a.wd, a.sd, P, a.H, a.I, part, a.H, BL_F32, 1};
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
    down.p.a.vec = vec_rows(a.y, a.ldy, a.ydtype);
    e = start_stream_x<2, 8, kStreamGated>(up, a.xdtype, P, 1, s);
    if (e != hipSuccess) return e;
    return start_stream<1, 1, 8, BL_F32, kStreamSlots>(down, a.M, static_cast<int>(a.k), s);
  }

  experts_sort_kernel<<<1, kSortThreads, static_cast<size_t>(a.E) * 8, s>>>(
      a.index, static_cast<int>(P), static_cast<int>(a.E), tile, head, pair, tiles);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  e = launch_fp8_quant_act(a.x, a.xdtype, a.M, a.H, a.ldx, 0, nullptr, q, sx, s);
  if (e != hipSuccess) return e;
  if (tile <= 64) {
    e = tile == 16 ? start_stream<1, 4, 8, kSrcCodes, kStreamGated>(up, nt, 0, s)
                   : start_stream<4, 2, 8, kSrcCodes, kStreamGated>(up, nt, 0, s);
    if (e != hipSuccess) return e;
    e = launch_fp8_quant_act(h, BL_F32, P, a.I, a.I, 0, head, hq, hs, s);
    if (e != hipSuccess) return e;
    e = tile == 16 ? start_stream<1, 4, 8, kSrcCodes, kStreamLinear>(down, nt, 0, s)
                   : start_stream<4, 2, 8, kSrcCodes, kStreamLinear>(down, nt, 0, s);
  } else {
    e = exact         ? start_gemm<GemmShape<256, 128, 2, 4, true, true>>(up.p, nt, s)
        : tile == 128 ? start_gemm<GemmShape<256, 128, 2, 4, false, true>>(up.p, nt, s)
                      : start_gemm<GemmShape<256, 256, 2, 4, false, true>>(up.p, nt, s);
    if (e != hipSuccess) return e;
    e = exact_down    ? start_gemm<GemmShape<256, 128, 2, 4, true>>(down.p, nt, s)
        : tile == 128 ? start_gemm<GemmShape<256, 128, 2, 4, false>>(down.p, nt, s)
                      : start_gemm<GemmShape<256, 256, 2, 4, false>>(down.p, nt, s);
  }
  if (e != hipSuccess) return e;
  const uint32_t cols = static_cast<uint32_t>((a.H + 255) / 256);
  experts_combine_kernel<<<dim3(static_cast<uint32_t>(a.M), cols < 16 ? cols : 16), 256, 0, s>>>(a, part);
  return hipGetLastError();
}

}  // namespace bl
