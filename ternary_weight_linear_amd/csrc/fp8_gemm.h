// Tiled block-scaled product for many rows: operands staged through LDS.
#pragma once

#include "fp8_mfma.h"

namespace bl {
namespace {

// Offsets from here on are outside every buffer below: a load there gives zeros.
constexpr uint32_t kOutside = 0x80000000u;

// A buffer of 2 GiB at `base` (wave-uniform): the accesses are kept inside the operand by the
// row clamps, the buffer's own bound only turns the offset kOutside into zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_buffer(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(kOutside), 0x00020000);
}

// 16 (4) bytes per lane from base + offset + k0 into LDS at `to` + 16 (4) lane.
__device__ __forceinline__ void copy16_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, uint32_t k0, void* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16,
                                           static_cast<int>(offset), static_cast<int>(k0), 0, 0);
}
__device__ __forceinline__ void copy4_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, void* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 4,
                                           static_cast<int>(offset), 0, 0, 0);
}
// Waits until at most N of this wave's loads and copies are in flight.
template <int N>
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// The workgroup's waves meet. Unlike __syncthreads this does not wait for the copies in flight:
// wait_copies does, for those that are needed, and what a wave has read from LDS it has used in
// a matrix instruction by now. The fences only keep the compiler from moving accesses across.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// XCD x (workgroups are dealt to the eight XCDs in turn) takes a contiguous run of n tiles.
__device__ __forceinline__ int in_xcd_order(int i, int n) {
  const int xcd = i & 7, per = n / 8, more = n % 8;
  return xcd * per + min(xcd, more) + (i >> 3);
}
// Tiles lie in bands of 8 tiles of q; within a band q runs first.
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int id, int tiles_n, int tiles_m) {
  const int band = id / (8 * tiles_n), in = id - band * 8 * tiles_n;
  const int bm = min(8, tiles_m - band * 8);
  return {band * 8 + in % bm, in / bm};
}

template <int BN_, int BM_, int GN_, int GM_, int NS_, bool EXACT_, bool GATED_ = false>
struct GemmShape {
  static constexpr int BN = BN_, BM = BM_;          // tile: rows of w, rows of q
  static constexpr int GN = GN_, GM = GM_;          // waves along each
  static constexpr int WAVES = GN * GM, THREADS = 64 * WAVES;
  static constexpr int TN = BN / GN / 16, TM = BM / GM / 16;
  static constexpr bool EXACT = EXACT_;             // fp16 operands
  // A tile of w is BN / 2 gate rows and the BN / 2 up rows of the same channels, and the tile's
  // result is quantised silu(gate) * up. Each wave holds both rows of its channels.
  static constexpr bool GATED = GATED_;
  // bf16 results go out as rows of a wave's 128 columns (store_wide)
  static constexpr bool WIDE = !EXACT && !GATED && BN == 256 && WAVES == 8 && TN == 8 && TM % 2 == 0;
  static constexpr int NF = GATED ? 2 : 1;          // blocks of 128 rows of w that a wave reads
  static_assert(!GATED || BN == 256, "a gated tile is one block of 128 channels");
  static constexpr int NS = NS_;                    // stages: NS - 1 blocks' copies in flight
  static constexpr int CA = BN / 8 / WAVES, CB = BM / 8 / WAVES;   // copies per wave and block
  static constexpr int COPIES = CA + CB + 1;        // and one of its rows' scales
  static_assert(NS >= 2 && NS <= 4 && COPIES * (NS - 2) < 64, "what s_waitcnt can count");
  static_assert(BM / GM <= 64, "one copy holds a wave's scales");
};

// The fragment of 16 rows whose first byte for this lane is at `at` of a staged tile; the
// second 16 codes are in the piece four further on, which the XOR order puts 64 bytes away.
template <bool EXACT>
__device__ __forceinline__ Operand<EXACT> read_operand(const uint8_t* tile, uint32_t lo, uint32_t hi) {
  Frag f;
  f.lo = *reinterpret_cast<const u32x4*>(tile + lo);
  f.hi = *reinterpret_cast<const u32x4*>(tile + hi);
  return operand<EXACT>(f);
}

// Stores a wave's bf16 results through LDS of its own, 32 rows at a time, so that each row's 128
// columns go out as 256 consecutive bytes (from registers a row gets 32 bytes per store: four
// lanes of four columns). 16-byte pieces are in XOR order as in the tiles.
template <class S>
__device__ __forceinline__ void store_wide(const Fp8LinearArgs& a, const f32x4 (&acc)[S::TN][S::TM], uint8_t* room, int64_t first,
                                           int rows, int wm, int64_t n, int lane) {
  constexpr int PIECES = 2 * S::TN, ROWS = 64 / PIECES;   // 16-byte pieces of a row, rows per store
  const int g = lane >> 4, u = lane & 15;
#pragma unroll
  for (int jj = 0; jj < S::TM; jj += 2) {
#pragma unroll
    for (int j = jj; j < jj + 2; ++j) {
      const int row = 16 * (j - jj) + u;
#pragma unroll
      for (int i = 0; i < S::TN; ++i) {
        const u32x2 b = {pack16(a.ydtype, acc[i][j][0], acc[i][j][1]), pack16(a.ydtype, acc[i][j][2], acc[i][j][3])};
        *reinterpret_cast<u32x2*>(room + row * 16 * PIECES + 16 * ((2 * i + (g >> 1)) ^ (u % PIECES)) + 8 * (g & 1)) = b;
      }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int t = 0; t < 32 / ROWS; ++t) {
      const int row = ROWS * t + lane / PIECES, c = lane % PIECES, r = wm + 16 * jj + row;
      const u32x4 b = *reinterpret_cast<const u32x4*>(room + row * 16 * PIECES + 16 * (c ^ (row % PIECES)));
      if (r >= rows || n + 8 * c >= a.N) continue;
      uint16_t* to = static_cast<uint16_t*>(a.y) + (first + r) * a.ldy + n + 8 * c;
      // non-temporal: all CUs store at once, and 128 KB each would turn over the L2 (8192 x 8192 x
      // 1024: 98 us with ordinary stores, 94)
      if (n + 8 * c + 7 < a.N) {
        __builtin_nontemporal_store(b, reinterpret_cast<u32x4_at2*>(to));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + 8 * c + e < a.N) to[e] = static_cast<uint16_t>(b[e / 2] >> (16 * (e & 1)));
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// y = sum over blocks of (sx sw) (q w^T over the block's 128 inputs): every block's products start
// from zero in the matrix cores and are added, scaled, to fp32 sums in registers. A workgroup has
// BN x BM outputs; a block of both operands is copied straight into LDS while the one before it is
// multiplied. What bounds it: large tiles the matrix cores and the card's power (256 x 256,
// 4096 x 28672 x 8192: 820 to 840 us, 2.3 PFLOP/s), small ones L2, fp16 operands the conversion of
// the codes (512 x 3200 x 8640, K in five parts: 34 us). Of a 256 x 256 tile about 10 us are its start and its
// stores; one workgroup per CU that takes tile after tile and copies the next one's first block
// while it stores measured 1 to 3 % slower at every shape.
template <class S>
__global__ __launch_bounds__(S::THREADS) void fp8_gemm_kernel(ProductArgs p, int tiles_n, int tiles_m_arg) {
  // one array per operand and stage: the compiler can then tell that the copies into one
  // stage do not touch what is being read
  constexpr int N3 = S::NS > 2 ? 1 : 0, N4 = S::NS > 3 ? 1 : 0;
  __shared__ uint8_t bufA0[S::BN * 128], bufA1[S::BN * 128], bufA2[N3 ? S::BN * 128 : 1], bufA3[N4 ? S::BN * 128 : 1];
  __shared__ uint8_t bufB0[S::BM * 128], bufB1[S::BM * 128], bufB2[N3 ? S::BM * 128 : 1], bufB3[N4 ? S::BM * 128 : 1];
  __shared__ float bufS0[S::WAVES][64], bufS1[S::WAVES][64], bufS2[N3 ? S::WAVES : 1][64], bufS3[N4 ? S::WAVES : 1][64];
  __shared__ int to_rows[S::WAVES][64];             // output rows, where they are scattered
  const Fp8LinearArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, u = lane & 15;
  const int wn = (wave % S::GN) * (S::BN / S::GN), wm = (wave / S::GN) * (S::BM / S::GM);

  const int tiles_m = p.map.tiles ? *p.map.n_tiles : tiles_m_arg;
  const int total = tiles_n * tiles_m, whole = p.parts > 1 ? p.whole : total;
  const bool split = static_cast<int>(blockIdx.x) >= whole;   // K in parts: this is part z of tile whole + i
  int id = blockIdx.x, z = 0, i_of_rest = 0;
  if (split) {
    const int j = id - whole, rest = total - whole;
    if (p.parts <= 1) return;                       // (the grid is made for the most tiles there may be)
    z = j / rest;
    i_of_rest = in_xcd_order(j - z * rest, rest);
    id = whole + i_of_rest;
  } else {
    id = in_xcd_order(id, whole);
  }
  const TileAt tile = tile_at(id, tiles_n, tiles_m);
  const int tm = tile.m, tn = tile.n;

  const int64_t n0 = static_cast<int64_t>(tn) * S::BN;
  int64_t first = static_cast<int64_t>(tm) * S::BM;
  int rows = 0, expert = 0;
  if (p.map.tiles) {
    expert = __builtin_amdgcn_readfirstlane(p.map.tiles[4 * tm]);
    first = __builtin_amdgcn_readfirstlane(p.map.tiles[4 * tm + 1]);
    rows = __builtin_amdgcn_readfirstlane(p.map.tiles[4 * tm + 2]);
  } else {
    rows = static_cast<int>(a.M - first < S::BM ? a.M - first : S::BM);
  }
  const int64_t K = a.K, KB = (K + kFp8Block - 1) / kFp8Block;

  // staging: copy i of this wave fills rows 8 (i WAVES + wave) + lane / 8 of a tile; position
  // lane % 8 of a row holds the 16 codes of piece (lane % 8) ^ (row % 8)
  const int piece = (lane & 7) ^ (lane >> 3);
  uint32_t oa[S::CA], ob[S::CB];
  const auto ba = make_buffer(a.w + expert * p.w_stride + (S::GATED ? 0 : n0 * K));
  const auto bb = make_buffer(p.map.gather_div > 0 ? a.q : a.q + first * K);
  const int c0 = tn * (S::BN / 2);                  // GATED: the tile's first channel
#pragma unroll
  for (int i = 0; i < S::CA; ++i) {
    int n = 8 * (i * S::WAVES + wave) + (lane >> 3);
    if constexpr (S::GATED) {
      // row n of the tile: wave column n / (BN / GN), gate rows first, then up rows
      constexpr int W = S::BN / S::GN, half = W / 2;
      const int c = min(c0 + n / W * half + n % half, static_cast<int>(a.N) - 1);
      n = n % W < half ? c : static_cast<int>(a.N) + c;
    } else {
      n = min(n, static_cast<int>(min<int64_t>(a.N - 1 - n0, S::BN)));
    }
    oa[i] = static_cast<uint32_t>(n) * static_cast<uint32_t>(K) + 16 * piece;
  }
#pragma unroll
  for (int i = 0; i < S::CB; ++i) {
    int r = min(8 * (i * S::WAVES + wave) + (lane >> 3), rows - 1);
    if (p.map.gather_div > 0) r = p.map.pair[first + r] / p.map.gather_div;
    ob[i] = static_cast<uint32_t>(r) * static_cast<uint32_t>(K) + 16 * piece;
  }
  // scales: one copy brings those of the wave's up to 64 rows
  uint32_t os;
  {
    int64_t at = first + min(wm + min(lane, S::BM / S::GM - 1), rows - 1);
    if (p.map.gather_div > 0) at = p.map.pair[at] / p.map.gather_div;
    os = 4 * static_cast<uint32_t>(at);
  }
  // the wave's weight rows (GATED: of either half) lie in one block of 128 (BN / GN divides 128)
  const float* sw = a.sw + expert * p.sw_stride;
  const int64_t up_scales = (a.N + kFp8Block - 1) / kFp8Block * KB;
  sw += (S::GATED ? static_cast<int64_t>(tn) : min<int64_t>((n0 + wn) / kFp8Block, (a.N - 1) / kFp8Block)) * KB;

  // blocks [kb, blocks): all of them, or the workgroup's range of a split K
  const int per = split ? (static_cast<int>(KB) + p.parts - 1) / p.parts : static_cast<int>(KB);
  int kb = z * per;
  const int blocks = min(kb + per, static_cast<int>(KB));
  const bool cut = (KB - 1) * kFp8Block + 16 * piece >= K;   // this lane's piece of the last block is past K
  struct Weigh {
    float w[S::NF];
  };
  // Copy n (of COPIES) of block kb into a stage; past the last block, zeros (no memory is read)
  auto copy = [&](int n, int kb, uint8_t* ta, uint8_t* tb, float (*ts)[64]) __attribute__((always_inline)) {
    const bool skip = kb >= blocks || (cut && kb == KB - 1);
    const uint32_t k0 = static_cast<uint32_t>(kb) * kFp8Block;
    if (n < S::CA) copy16_to_lds(ba, skip ? kOutside : oa[n], k0, ta + 1024 * (n * S::WAVES + wave));
    else if (n < S::CA + S::CB) copy16_to_lds(bb, skip ? kOutside : ob[n - S::CA], k0, tb + 1024 * ((n - S::CA) * S::WAVES + wave));
    else copy4_to_lds(make_buffer(a.sx + min(kb, blocks - 1) * a.M), os, ts[wave]);
  };
  auto weigh = [&](int kb, Weigh& sc) __attribute__((always_inline)) {
    kb = min(kb, blocks - 1);
    sc.w[0] = sw[kb];
    if constexpr (S::GATED) sc.w[1] = sw[up_scales + kb];
  };
  auto stage = [&](int kb, uint8_t* ta, uint8_t* tb, float (*ts)[64], Weigh& sc) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < S::COPIES; ++n) copy(n, kb, ta, tb, ts);
    weigh(kb, sc);
  };

  const uint32_t in_row = u * 128 + 16 * (g ^ (u & 7));
  const uint32_t wa = wn * 128 + in_row, wa2 = wn * 128 + (in_row ^ 64);
  const uint32_t qa = wm * 128 + in_row, qa2 = wm * 128 + (in_row ^ 64);
  f32x4 acc[S::TN][S::TM] = {};
  // One block of inputs. While the matrix cores multiply weight fragment i by the TM fragments
  // of q, the products of fragment i - 1 are scaled and added (VALU) and fragment i + 1 is read.
  // With two stages the next block's copies go out between the first half of the products, not
  // ahead of the reads of LDS (2048 x 8192 x 8192: 115 -> 112 us, fp16 operands 1550 -> 1519);
  // with more stages they go out first (spread over the products 128 x 8192 x 8192 took 37 us
  // instead of 26).
  auto compute = [&](const uint8_t* ta, const uint8_t* tb, const float (*ts)[64], const Weigh& sc, int next,
                     uint8_t* na, uint8_t* nb, float (*ns)[64]) __attribute__((always_inline)) {
    constexpr int PER = (S::COPIES + (S::TN + 1) / 2 - 1) / ((S::TN + 1) / 2);
    float f[S::NF][S::TM];
#pragma unroll
    for (int j = 0; j < S::TM; ++j) {
      const float x = ts[wave][16 * j + u];
#pragma unroll
      for (int h = 0; h < S::NF; ++h) f[h][j] = x * sc.w[h];
    }
    Operand<S::EXACT> b[S::TM], w[2];
    f32x4 part[2][S::TM];
    w[0] = read_operand<S::EXACT>(ta, wa, wa2);
#pragma unroll
    for (int j = 0; j < S::TM; ++j) b[j] = read_operand<S::EXACT>(tb + 2048 * j, qa, qa2);
#pragma unroll
    for (int i = 0; i <= S::TN; ++i) {
      if (i + 1 < S::TN) w[(i + 1) & 1] = read_operand<S::EXACT>(ta + 2048 * (i + 1), wa, wa2);
      if constexpr (S::NS == 2) {
#pragma unroll
        for (int n = i * PER; n < (i + 1) * PER && n < S::COPIES; ++n) copy(n, next, na, nb, ns);
      }
      if (i < S::TN) {
        if constexpr (S::EXACT) {
          // the four instructions of a sum depend on each other: those of the TM sums take turns
#pragma unroll
          for (int j = 0; j < S::TM; ++j) part[i & 1][j] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < S::TM; ++j)
              part[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[i & 1].h[k], b[j].h[k], part[i & 1][j], 0, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < S::TM; ++j) part[i & 1][j] = block_dot(w[i & 1], b[j]);
        }
      }
      if (i > 0) {
#pragma unroll
        for (int j = 0; j < S::TM; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i - 1][j][e] = fmaf(part[(i - 1) & 1][j][e], f[(i - 1) * S::NF / S::TN][j], acc[i - 1][j][e]);
          asm volatile("" : "+v"(acc[i - 1][j]));   // the sum is formed here, not sunk to its next use
        }
      }
      // both LDS reads first, then the matrix instructions with the FMAs of the fragment before
      // (and the conversions of the next) between them
      if (i + 1 < S::TN) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int j = 0; j < (S::EXACT ? 4 : 1) * S::TM; ++j) {
        if (i < S::TN) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, S::EXACT ? 1 + 4 / S::TM : 4, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const bool busy = wm < rows;                      // a wave past the tile's rows only helps to copy
  Weigh w0, w1, w2, w3;
  // (a load of them between the stores of the results would wait for the stores)
  if (p.map.scatter)
    copy4_to_lds(make_buffer(p.map.pair + first), 4 * static_cast<uint32_t>(min(wm + min(lane, S::BM / S::GM - 1), rows - 1)),
                 to_rows[wave]);
  stage(kb, bufA0, bufB0, bufS0, w0);
  if constexpr (S::NS > 2) stage(kb + 1, bufA1, bufB1, bufS1, w1);
  if constexpr (S::NS > 3) stage(kb + 2, bufA2, bufB2, bufS2, w2);
  // Step kb: its copies have landed (this wave's, then every wave's, who are also done with the
  // stage of block kb - 1), block kb + NS - 1 goes there, block kb is multiplied.
#define BL_STEP(KB_, A, B, SC, W, NA, NB, NSC, NW)           \
  {                                                          \
    wait_copies<S::COPIES * (S::NS - 2)>();                  \
    meet();                                                  \
    if (S::NS > 2 || !busy) stage((KB_) + S::NS - 1, NA, NB, NSC, NW); \
    else weigh((KB_) + S::NS - 1, NW);                       \
    if (busy) compute(A, B, SC, W, (KB_) + S::NS - 1, NA, NB, NSC); \
  }
  if constexpr (S::NS == 2) {
    for (; kb + 2 <= blocks; kb += 2) {
      BL_STEP(kb, bufA0, bufB0, bufS0, w0, bufA1, bufB1, bufS1, w1)
      BL_STEP(kb + 1, bufA1, bufB1, bufS1, w1, bufA0, bufB0, bufS0, w0)
    }
    if (kb < blocks) BL_STEP(kb, bufA0, bufB0, bufS0, w0, bufA1, bufB1, bufS1, w1)
  } else if constexpr (S::NS == 3) {
    for (; kb + 3 <= blocks; kb += 3) {
      BL_STEP(kb, bufA0, bufB0, bufS0, w0, bufA2, bufB2, bufS2, w2)
      BL_STEP(kb + 1, bufA1, bufB1, bufS1, w1, bufA0, bufB0, bufS0, w0)
      BL_STEP(kb + 2, bufA2, bufB2, bufS2, w2, bufA1, bufB1, bufS1, w1)
    }
    if (kb < blocks) BL_STEP(kb, bufA0, bufB0, bufS0, w0, bufA2, bufB2, bufS2, w2)
    if (kb + 1 < blocks) BL_STEP(kb + 1, bufA1, bufB1, bufS1, w1, bufA0, bufB0, bufS0, w0)
  } else {
    for (; kb + 4 <= blocks; kb += 4) {
      BL_STEP(kb, bufA0, bufB0, bufS0, w0, bufA3, bufB3, bufS3, w3)
      BL_STEP(kb + 1, bufA1, bufB1, bufS1, w1, bufA0, bufB0, bufS0, w0)
      BL_STEP(kb + 2, bufA2, bufB2, bufS2, w2, bufA1, bufB1, bufS1, w1)
      BL_STEP(kb + 3, bufA3, bufB3, bufS3, w3, bufA2, bufB2, bufS2, w2)
    }
    if (kb < blocks) BL_STEP(kb, bufA0, bufB0, bufS0, w0, bufA3, bufB3, bufS3, w3)
    if (kb + 1 < blocks) BL_STEP(kb + 1, bufA1, bufB1, bufS1, w1, bufA0, bufB0, bufS0, w0)
    if (kb + 2 < blocks) BL_STEP(kb + 2, bufA2, bufB2, bufS2, w2, bufA1, bufB1, bufS1, w1)
  }
#undef BL_STEP
  wait_copies<0>();                                 // no copy outlives the workgroup
  __syncthreads();                                  // and every wave is past the tiles

  if constexpr (S::GATED) {
    // h = silu(gate) * up stays in fp32 up to its quantisation: the maximum of a row over the
    // tile's 128 channels meets over the lanes that share the row, then over the waves in LDS
    auto* top = reinterpret_cast<uint32_t*>(bufA0);   // [GN][BM]
    uint32_t mine[S::TM];
#pragma unroll
    for (int j = 0; j < S::TM; ++j) {
      mine[j] = kFp8FloorBits;
#pragma unroll
      for (int i = 0; i < S::TN / 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = c0 + wn / 2 + 16 * i + 4 * g + e;
          const float h = silu_mul(acc[i][j][e], acc[i + S::TN / 2][j][e]);
          acc[i][j][e] = c < a.N ? h : 0.0f;
          mine[j] = max(mine[j], abs_bits(acc[i][j][e]));
        }
      mine[j] = max(mine[j], static_cast<uint32_t>(__shfl_xor(static_cast<int>(mine[j]), 16)));
      mine[j] = max(mine[j], static_cast<uint32_t>(__shfl_xor(static_cast<int>(mine[j]), 32)));
    }
#pragma unroll
    for (int j = 0; j < S::TM; ++j)
      if (g == 0) top[wave % S::GN * S::BM + wm + 16 * j + u] = mine[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < S::TM; ++j) {
      const int r = wm + 16 * j + u;
      uint32_t m = top[r];
#pragma unroll
      for (int v = 1; v < S::GN; ++v) m = max(m, top[v * S::BM + r]);
      const float am = __uint_as_float(m), rcp = code_factor(am);
      if (r >= rows) continue;
      if (wn == 0 && g == 0) p.hs[tn * p.h_rows + first + r] = am / kFp8Max;
#pragma unroll
      for (int i = 0; i < S::TN / 2; ++i) {
        const int c = c0 + wn / 2 + 16 * i + 4 * g;
        if (c < a.N)                                  // N % 16 == 0: all four or none
          *reinterpret_cast<uint32_t*>(p.hq + (first + r) * a.N + c) = pack4(acc[i][j], rcp);
      }
    }
    return;
  }
  if (!S::GATED && split) {
    float* to = p.part + (static_cast<int64_t>(z) * (total - whole) + i_of_rest) * (S::BM * S::BN);
#pragma unroll
    for (int j = 0; j < S::TM; ++j) {
      const int r = wm + 16 * j + u;
      if (r >= rows) continue;
#pragma unroll
      for (int i = 0; i < S::TN; ++i) *reinterpret_cast<f32x4*>(to + r * S::BN + wn + 16 * i + 4 * g) = acc[i][j];
    }
    return;
  }
  if constexpr (S::WIDE) {
    if (a.ydtype == BL_BF16) {
      store_wide<S>(a, acc, (wave < 4 ? bufA0 : bufA1) + (wave & 3) * (1024 * S::TN), first, rows, wm, n0 + wn, lane);
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < S::TM; ++j) {
    const int r = wm + 16 * j + u;
    if (r >= rows) continue;
    const int64_t at = p.map.scatter ? to_rows[wave][16 * j + u] : first + r;
#pragma unroll
    for (int i = 0; i < S::TN; ++i) store4(a, at, n0 + wn + 16 * i + 4 * g, acc[i][j]);
  }
}

// y = the sum of the `parts` partial sums of each tile from `whole` on, in their order, four
// columns per thread. Reading them bounds it (five of 512 x 3200, 33 MB: 7 us).
template <class S>
__global__ __launch_bounds__(256) void sum_parts_kernel(ProductArgs p, int tiles_n, int tiles_m) {
  constexpr int PER = S::BM * S::BN / 1024;         // workgroups per tile
  const int i = blockIdx.x / PER, at = (blockIdx.x % PER * 256 + threadIdx.x) * 4;
  const int rest = tiles_n * tiles_m - p.whole;
  const TileAt t = tile_at(p.whole + i, tiles_n, tiles_m);
  const int64_t m = static_cast<int64_t>(t.m) * S::BM + at / S::BN, n = static_cast<int64_t>(t.n) * S::BN + at % S::BN;
  if (m >= p.a.M || n >= p.a.N) return;
  f32x4 sum = {0, 0, 0, 0};
  for (int z = 0; z < p.parts; ++z)
    sum += *reinterpret_cast<const f32x4*>(p.part + (static_cast<int64_t>(z) * rest + i) * (S::BM * S::BN) + at);
  store4(p.a, m, n, sum);
}

template <class S>
hipError_t start_gemm(const ProductArgs& p, int64_t tiles_m, hipStream_t s) {
  constexpr int64_t cols = S::GATED ? S::BN / 2 : S::BN;
  const int64_t tiles_n = (p.a.N + cols - 1) / cols;
  if (!grid_fits(tiles_n * tiles_m, S::THREADS)) return hipErrorInvalidConfiguration;
  fp8_gemm_kernel<S><<<dim3(static_cast<uint32_t>(tiles_n * tiles_m)), S::THREADS, 0, s>>>(
      p, static_cast<int>(tiles_n), static_cast<int>(tiles_m));
  return hipGetLastError();
}

// The product with K split over p.parts workgroups for each tile from p.whole on.
template <class S>
hipError_t start_split_gemm(const ProductArgs& p, hipStream_t s) {
  const int64_t tiles_n = (p.a.N + S::BN - 1) / S::BN, tiles_m = (p.a.M + S::BM - 1) / S::BM;
  const int64_t rest = tiles_n * tiles_m - p.whole;
  if (!grid_fits(p.whole + rest * p.parts, S::THREADS)) return hipErrorInvalidConfiguration;
  fp8_gemm_kernel<S><<<dim3(static_cast<uint32_t>(p.whole + rest * p.parts)), S::THREADS, 0, s>>>(
      p, static_cast<int>(tiles_n), static_cast<int>(tiles_m));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sum_parts_kernel<S><<<dim3(static_cast<uint32_t>(rest * (S::BM * S::BN / 1024))), 256, 0, s>>>(
      p, static_cast<int>(tiles_n), static_cast<int>(tiles_m));
  return hipGetLastError();
}

}  // namespace
}  // namespace bl
