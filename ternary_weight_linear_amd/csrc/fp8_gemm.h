// Tiled block-scaled product for many rows: operands staged through LDS.
#pragma once

#include "fp8_mfma.h"

namespace bl {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Offsets from here on are outside every buffer below: a load there gives zeros.
constexpr uint32_t kOutside = 0x80000000u;

// A buffer of 2 GiB at `base` (wave-uniform): the accesses are kept inside the operand by the
// row clamps, the buffer's own bound only turns the offset kOutside into zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_buffer(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(kOutside), 0x00020000);
}

// 16 bytes per lane from base + offset + k0 into LDS at `to` + 16 lane.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, uint32_t k0, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16,
                                           static_cast<int>(offset), static_cast<int>(k0), 0, 0);
}

template <int BN_, int BM_, int GN_, int GM_, bool EXACT_, bool GATED_ = false>
struct GemmShape {
  static constexpr int BN = BN_, BM = BM_;          // tile: rows of w, rows of q
  static constexpr int GN = GN_, GM = GM_;          // waves along each
  static constexpr int WAVES = GN * GM, THREADS = 64 * WAVES;
  static constexpr int TN = BN / GN / 16, TM = BM / GM / 16;
  static constexpr bool EXACT = EXACT_;             // fp16 operands
  // A tile of w is BN / 2 gate rows and the BN / 2 up rows of the same channels, and the tile's
  // result is quantised silu(gate) * up. Each wave holds both rows of its channels.
  static constexpr bool GATED = GATED_;
  static constexpr bool WIDE = !GATED && WAVES == 8 && TN == 8 && TM % 2 == 0;   // store_wide
  static constexpr int NF = GATED ? 2 : 1;          // blocks of 128 rows of w that a wave reads
  static_assert(!GATED || BN == 256, "a gated tile is one block of 128 channels");
  static constexpr int CA = BN / 8 / WAVES, CB = BM / 8 / WAVES;   // copies per wave and block
};

template <bool EXACT>
struct OperandT { using type = i32x8; };
template <>
struct OperandT<true> { using type = FragH; };

// The fragment of 16 rows whose first byte for this lane is at `at` of a staged tile; the
// second 16 codes are in the piece four further on, which the XOR order puts 64 bytes away.
template <bool EXACT>
__device__ __forceinline__ typename OperandT<EXACT>::type read_operand(const uint8_t* tile, uint32_t lo, uint32_t hi) {
  Frag f;
  f.lo = *reinterpret_cast<const u32x4*>(tile + lo);
  f.hi = *reinterpret_cast<const u32x4*>(tile + hi);
  if constexpr (EXACT) return to_half(f);
  else return i32x8{(int)f.lo.x, (int)f.lo.y, (int)f.lo.z, (int)f.lo.w, (int)f.hi.x, (int)f.hi.y, (int)f.hi.z, (int)f.hi.w};
}

__device__ __forceinline__ f32x4 block_dot(const i32x8& a, const i32x8& b) {
  const f32x4 c = {0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Stores a wave's 16-bit results through 8 KB of LDS of its own, 32 rows of 128 columns at a
// time, so that each row goes out as 256 consecutive bytes (from registers a row gets 32 bytes
// per store: four lanes of four columns). 16-byte pieces are in XOR order as in the tiles.
// kPartType: fp16 of value / scale, scale a power of two per row and 128 columns that brings
// their largest magnitude to [2^14, 2^15); values that are not finite stay so.
template <class S>
__device__ __forceinline__ void store_wide(const ProductArgs& p, const f32x4 (&acc)[S::TN][S::TM], uint8_t* room,
                                           int64_t first, int rows, int wm, int64_t n, int lane) {
  const Fp8LinearArgs& a = p.a;
  const int g = lane >> 4, u = lane & 15;
  __syncthreads();                                  // the last tile has been read
#pragma unroll
  for (int jj = 0; jj < S::TM; jj += 2) {
#pragma unroll
    for (int j = jj; j < jj + 2; ++j) {
      float f = 1.0f;
      if (a.ydtype == kPartType) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < S::TN; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = n + 16 * i + 4 * g + e < a.N ? abs_bits(acc[i][j][e]) : 0;
            m = max(m, b < 0x7F800000u ? b : 0);
          }
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
        // exponent of the scale, kept where the scale and its reciprocal are normal numbers
        const int e = min(max(static_cast<int>(m >> 23) - 14, 1), 253);
        f = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        const int r = wm + 16 * j + u;
        if (g == 0 && r < rows && n < a.N)
          p.part_scale[(n / kFp8Block) * a.M + p.map.pair[first + r]] = __uint_as_float(static_cast<uint32_t>(e) << 23);
      }
      const int row = 16 * (j - jj) + u;
#pragma unroll
      for (int i = 0; i < S::TN; ++i) {
        u32x2 b;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float v0 = acc[i][j][2 * h] * f, v1 = acc[i][j][2 * h + 1] * f;
          const uint32_t lo = a.ydtype == BL_BF16 ? bf16_bits(v0) : half_bits(v0);
          const uint32_t hi = a.ydtype == BL_BF16 ? bf16_bits(v1) : half_bits(v1);
          b[h] = lo | hi << 16;
        }
        *reinterpret_cast<u32x2*>(room + row * 256 + 16 * ((2 * i + (g >> 1)) ^ u) + 8 * (g & 1)) = b;
      }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int row = 4 * t + g, r = wm + 16 * jj + row;
      const u32x4 b = *reinterpret_cast<const u32x4*>(room + row * 256 + 16 * (u ^ (row & 15)));
      if (r >= rows || n + 8 * u >= a.N) continue;   // N % 8 == 0: all eight or none
      int64_t at = first + r;
      if (p.map.scatter) at = p.map.pair[at];
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.y) + at * a.ldy + n + 8 * u) = b;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <class S>
__global__ __launch_bounds__(S::THREADS) void fp8_gemm_kernel(ProductArgs p, int tiles_n, int tiles_m_arg) {
  // one array per operand and stage: the compiler can then tell that the copies into one
  // stage do not touch what is being read
  __shared__ uint8_t bufA0[S::BN * 128], bufA1[S::BN * 128], bufB0[S::BM * 128], bufB1[S::BM * 128];
  const Fp8LinearArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, u = lane & 15;
  const int wn = (wave % S::GN) * (S::BN / S::GN), wm = (wave / S::GN) * (S::BM / S::GM);

  const int tiles_m = p.map.tiles ? *p.map.n_tiles : tiles_m_arg;
  int id = blockIdx.x;
  {
    // XCD x (workgroups are dealt to the eight XCDs in turn) takes a contiguous run of tiles
    const int total = tiles_n * tiles_m, per = total / 8, more = total % 8;
    const int xcd = id & 7, i = id >> 3;
    if (i >= per + (xcd < more)) return;
    id = xcd * per + min(xcd, more) + i;
  }
  // bands of 8 tiles of q, within a band q runs first
  const int band = id / (8 * tiles_n), in = id - band * 8 * tiles_n;
  const int bm = min(8, tiles_m - band * 8);
  const int tm = band * 8 + in % bm, tn = in / bm;

  const int64_t n0 = static_cast<int64_t>(tn) * S::BN;
  int64_t first = static_cast<int64_t>(tm) * S::BM;
  int rows = 0, expert = 0;
  if (p.map.tiles) {
    expert = p.map.tiles[4 * tm];
    first = p.map.tiles[4 * tm + 1];
    rows = p.map.tiles[4 * tm + 2];
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
  const int kb_cut = K % kFp8Block ? static_cast<int>(KB) - 1 : -1;   // the block that K ends in
  const bool out = (KB - 1) * kFp8Block + 16 * piece >= K;
  auto stage = [&](int kb, uint8_t* ta, uint8_t* tb) __attribute__((always_inline)) {
    const bool skip = out && kb == kb_cut;
    const uint32_t k0 = static_cast<uint32_t>(kb) * kFp8Block;
#pragma unroll
    for (int i = 0; i < S::CA; ++i)
      copy_to_lds(ba, skip ? kOutside : oa[i], k0, ta + 1024 * (i * S::WAVES + wave));
#pragma unroll
    for (int i = 0; i < S::CB; ++i)
      copy_to_lds(bb, skip ? kOutside : ob[i], k0, tb + 1024 * (i * S::WAVES + wave));
  };

  uint32_t ox[S::TM];
#pragma unroll
  for (int j = 0; j < S::TM; ++j) {
    int64_t at = first + min(wm + 16 * j + u, rows - 1);
    if (p.map.gather_div > 0) at = p.map.pair[at] / p.map.gather_div;
    ox[j] = 4 * static_cast<uint32_t>(at);
  }
  // the wave's weight rows (GATED: of either half) lie in one block of 128 (BN / GN divides 128)
  const float* sw = a.sw + expert * p.sw_stride;
  const int64_t up_scales = (a.N + kFp8Block - 1) / kFp8Block * KB;
  sw += (S::GATED ? static_cast<int64_t>(tn) : min<int64_t>((n0 + wn) / kFp8Block, (a.N - 1) / kFp8Block)) * KB;

  const uint32_t in_row = u * 128 + 16 * (g ^ (u & 7));
  const uint32_t wa = wn * 128 + in_row, wa2 = wn * 128 + (in_row ^ 64);
  const uint32_t qa = wm * 128 + in_row, qa2 = wm * 128 + (in_row ^ 64);
  struct Scales {
    float x[S::TM], w[S::NF];
  };
  f32x4 acc[S::TN][S::TM] = {};
  // One block of inputs. While the matrix cores multiply weight fragment i by the TM fragments
  // of q, the products of fragment i - 1 are scaled and added (VALU) and fragment i + 1 is read.
  auto compute = [&](const uint8_t* ta, const uint8_t* tb, const Scales& sc) __attribute__((always_inline)) {
    float f[S::NF][S::TM];
#pragma unroll
    for (int h = 0; h < S::NF; ++h)
#pragma unroll
      for (int j = 0; j < S::TM; ++j) f[h][j] = sc.x[j] * sc.w[h];
    typename OperandT<S::EXACT>::type b[S::TM], w[2];
    f32x4 part[2][S::TM];
    w[0] = read_operand<S::EXACT>(ta, wa, wa2);
#pragma unroll
    for (int j = 0; j < S::TM; ++j) b[j] = read_operand<S::EXACT>(tb + 2048 * j, qa, qa2);
#pragma unroll
    for (int i = 0; i <= S::TN; ++i) {
      if (i + 1 < S::TN) w[(i + 1) & 1] = read_operand<S::EXACT>(ta + 2048 * (i + 1), wa, wa2);
#pragma unroll
      for (int j = 0; j < S::TM; ++j) {
        if (i < S::TN) part[i & 1][j] = block_dot(w[i & 1], b[j]);
        if (i > 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i - 1][j][e] = fmaf(part[(i - 1) & 1][j][e], f[(i - 1) * S::NF / S::TN][j], acc[i - 1][j][e]);
          asm volatile("" : "+v"(acc[i - 1][j]));   // the sum is formed here, not sunk to its next use
        }
      }
      // both LDS reads first, then each matrix instruction beside four FMAs of the one before
      if (i + 1 < S::TN) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int j = 0; j < S::TM; ++j) {
        if (i < S::TN) __builtin_amdgcn_sched_group_barrier(0x008, S::EXACT ? 4 : 1, 0);
        if (i > 0) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto scales = [&](int kb, Scales& sc) __attribute__((always_inline)) {
    sc.w[0] = sw[kb];
    if constexpr (S::GATED) sc.w[1] = sw[up_scales + kb];
    const auto sx = make_buffer(a.sx + kb * a.M);
#pragma unroll
    for (int j = 0; j < S::TM; ++j)
      sc.x[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sx, static_cast<int>(ox[j]), 0, 0));
  };
  // every copy of this wave has landed, then every wave's
  auto arrive = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0F70);             // vmcnt(0)
    __syncthreads();
  };

  const int blocks = static_cast<int>(KB);
  const bool busy = wm < rows;                      // a wave past the tile's rows only helps to copy
  Scales f0, f1;
  stage(0, bufA0, bufB0);
  scales(0, f0);
  for (int kb = 0; kb + 1 < blocks; kb += 2) {
    arrive();
    stage(kb + 1, bufA1, bufB1);
    scales(kb + 1, f1);
    if (busy) compute(bufA0, bufB0, f0);
    arrive();
    const int next = min(kb + 2, blocks - 1);     // past the end the last block again, never read
    stage(next, bufA0, bufB0);
    scales(next, f0);
    if (busy) compute(bufA1, bufB1, f1);
  }
  arrive();                                       // no copy outlives the workgroup
  if (busy && (blocks & 1)) compute(bufA0, bufB0, f0);

  if constexpr (S::GATED) {
    // h = silu(gate) * up stays in fp32 up to its quantisation: the maximum of a row over the
    // tile's 128 channels meets over the lanes that share the row, then over the waves in LDS
    auto* top = reinterpret_cast<uint32_t*>(bufA0);   // [GN][BM], every wave is past the tiles
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
    __syncthreads();
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
  if constexpr (S::WIDE) {
    if (a.ydtype != BL_F32 && a.vec8) {
      store_wide<S>(p, acc, (wave < 4 ? bufA0 : bufA1) + (wave & 3) * 8192, first, rows, wm, n0 + wn, lane);
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < S::TM; ++j) {
    const int r = wm + 16 * j + u;
    if (r >= rows) continue;
    int64_t at = first + r;
    if (p.map.scatter) at = p.map.pair[at];
#pragma unroll
    for (int i = 0; i < S::TN; ++i) store4(a, at, n0 + wn + 16 * i + 4 * g, acc[i][j]);
  }
}

template <class S>
hipError_t start_gemm(const ProductArgs& p, int64_t tiles_m, hipStream_t s) {
  constexpr int64_t cols = S::GATED ? S::BN / 2 : S::BN;
  const int64_t tiles_n = (p.a.N + cols - 1) / cols;
  fp8_gemm_kernel<S><<<dim3(static_cast<uint32_t>(tiles_n * tiles_m)), S::THREADS, 0, s>>>(
      p, static_cast<int>(tiles_n), static_cast<int>(tiles_m));
  return hipGetLastError();
}

}  // namespace
}  // namespace bl
