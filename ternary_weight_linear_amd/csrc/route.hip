// Routing to experts: scores, choice by biased score within the best groups, the k best, and
// their weights. The contract is bl_route_experts in include/libbitlinear.h.
//
// Two kernels. route_row16_kernel gives a row 16 lanes (a DPP row) and keeps its experts in
// registers, a contiguous run per lane and no lane in two groups: what a row needs of all its
// experts is four DPP steps. It takes up to 32 experts per lane, k <= 16 and 16 groups;
// route_kernel, one wave per row with the choices in LDS, takes the rest.
#include "fp8_internal.h"

namespace bl {
namespace {

constexpr int kRouteWaves = 4;

// Unsigned order = float order; -0 and +0 are equal. NaN is not passed.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t choice_key(float v, int e) {
  return (static_cast<uint64_t>(ordered_bits(v)) << 32) | static_cast<uint32_t>(~e);
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor(static_cast<unsigned long long>(v), off);
    v = v > o ? v : o;
  }
  return v;
}

// v of the lane N places round the 16 lanes of this lane's row.
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x120 + N, 0xF, 0xF, false));
}
template <int N>
__device__ __forceinline__ float ror(float v) {
  return __uint_as_float(ror<N>(__float_as_uint(v)));
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, ror<8>(v));
  v = max(v, ror<4>(v));
  v = max(v, ror<2>(v));
  return max(v, ror<1>(v));
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  v = min(v, ror<8>(v));
  v = min(v, ror<4>(v));
  v = min(v, ror<2>(v));
  return min(v, ror<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += ror<8>(v);
  v += ror<4>(v);
  v += ror<2>(v);
  return v + ror<1>(v);
}
// The value of lane (this lane ^ X) of its row.
template <int X>
__device__ __forceinline__ uint32_t row_xor(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(v), (X << 10) | 0x1F));
}
// The best two of a set (b1 >= b2) and of another lane's.
template <int X>
__device__ __forceinline__ void merge_best(uint32_t& b1, uint32_t& b2) {
  const uint32_t c1 = row_xor<X>(b1), c2 = row_xor<X>(b2);
  b2 = max(min(b1, c1), max(b2, c2));
  b1 = max(b1, c1);
}
// How many groups, of W lanes each, are better than this lane's; ties to the lower group.
template <int W, int N = W>
__device__ __forceinline__ int better_groups(uint32_t rank, uint32_t lane) {
  if constexpr (N >= 16) return 0;
  else {
    const uint32_t r = ror<N>(rank), l = ror<N>(lane);   // by every lane, before any condition
    return better_groups<W, N + W>(rank, lane) + static_cast<int>((r > rank) | ((r == rank) & (l < lane)));
  }
}
__device__ __forceinline__ float from_ordered(uint32_t b) {
  return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

// A group has 2^shift lanes of C <= NE experts each (without groups all 16 lanes): lane j holds
// experts e0 = (j >> shift) size + (j % 2^shift) C .. of its group, as far as that goes. Choice
// values are kept as unsigned keys in their order, 0 for what cannot be chosen.
// VALU work bounds it: the scores (an exponential and a division each) and, per round, two
// passes over the lane's NE keys. 16384 rows of 256 experts, 8 groups, top 8: 13.5 us a call among
// others (kernel trace 14.9, at least 14.0); 4096 rows of 60, top 4: 4.1; one row 6.7, a chain of
// waits.
template <int DT, int NE>
__global__ __launch_bounds__(256) void route_row16_kernel(RouteArgs a, int C, int shift, int vec) {
  __shared__ float scores[16][16 * NE + 16];        // expert e0 + i of lane j at 16 i + j
  __shared__ uint32_t chosen[16][16];               // place in scores, expert
  const uint32_t lane = threadIdx.x & 15, in = threadIdx.x >> 4;
  const int64_t m = group_id() * 16 + in;
  const int64_t mc = m < a.M ? m : a.M - 1;         // rows past the end work on the last one
  const int E = static_cast<int>(a.E), size = E / a.groups;
  const int group = static_cast<int>(lane) >> shift, within = (static_cast<int>(lane) & ((1 << shift) - 1)) * C;
  const int e0 = group * size + within;
  const int mine_n = group < a.groups ? min(C, size - within) : 0;   // may be negative
  const float none = -INFINITY;
  using T = typename Elem<DT>::type;
  const T* row = static_cast<const T*>(a.logits) + mc * a.ld;
  float c[NE], bias[NE] = {};                       // no bias adds 0, which changes nothing
  if (vec) {                                        // every lane has NE, whole and aligned pieces
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < NE / V; ++i) {
      const uint4 b = reinterpret_cast<const uint4*>(row + e0)[i];
      const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (DT == BL_F32) c[i * V + j] = __uint_as_float(w[j]);
        else c[i * V + j] = to_float<DT>(static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1))));
      }
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NE; i += 4) {
        const float4 b = *reinterpret_cast<const float4*>(a.bias + e0 + i);
        bias[i] = b.x;
        bias[i + 1] = b.y;
        bias[i + 2] = b.z;
        bias[i + 3] = b.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) c[i] = to_float<DT>(row[min(e0 + i, E - 1)]);   // all in flight at once
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NE; ++i) bias[i] = a.bias[min(e0 + i, E - 1)];
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) c[i] = i < mine_n ? c[i] : none;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) c[i] = c[i] > none ? fminf(c[i], 3.402823466e38f) : none;   // NaN compares false

  uint32_t key[NE];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float p = 1.0f / (1.0f + expf(-c[i])), v = p + bias[i];
      scores[in][16 * i + lane] = p;
      key[i] = c[i] > none && v > none ? ordered_bits(v) : 0;
    }
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      key[i] = c[i] > none ? ordered_bits(c[i]) : 0;
      top = max(top, key[i]);
    }
    const float mx = from_ordered(row_max(top));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      c[i] = c[i] > none ? expf(c[i] - mx) : 0.0f;
      sum += c[i];
    }
    sum = row_sum(sum);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      c[i] /= sum;
      scores[in][16 * i + lane] = c[i];
    }
    // without a bias the keys stay those of the logits: a softmax keeps their order
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float v = c[i] + bias[i];
        key[i] = key[i] && v > none ? ordered_bits(v) : 0;
      }
    }
  }

  if (a.groups > 1) {
    uint32_t b1 = 0, b2 = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      b2 = max(b2, min(b1, key[i]));
      b1 = max(b1, key[i]);
    }
    if (shift > 0) merge_best<1>(b1, b2);
    if (shift > 1) merge_best<2>(b1, b2);
    if (shift > 2) merge_best<4>(b1, b2);
    // a rank of 0 (nothing to choose) is below every other
    uint32_t rank = b1;
    if (a.sigmoid && b2) rank = ordered_bits(from_ordered(b1) + from_ordered(b2));
    const int better = shift == 0   ? better_groups<1>(rank, lane)
                       : shift == 1 ? better_groups<2>(rank, lane)
                       : shift == 2 ? better_groups<4>(rank, lane)
                                    : better_groups<8>(rank, lane);
    if (better >= a.kept) {
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] = 0;
    }
  }

  int found = 0;                                    // uniform over the row
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) best = max(best, key[i]);
    best = row_max(best);
    if (__ballot(best != 0) == 0) break;            // nothing left in any row of the wave
    // the lane's first expert at the best value, then the row's
    int at = NE;
#pragma unroll
    for (int i = NE - 1; i >= 0; --i) at = key[i] == best ? i : at;
    const uint32_t mine = at < NE ? static_cast<uint32_t>(e0 + at) : ~0u;
    at = mine == row_min(mine) && best ? at : NE;   // only the winner keeps its place
    found += best != 0;
    if (at < NE) chosen[in][j] = static_cast<uint32_t>(16 * at) + lane + (mine << 16);
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = at == i ? 0 : key[i];
  }
  // the lanes of a row are in one wave: they read what the others wrote without a barrier
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const bool some = static_cast<int>(lane) < found;
  const uint32_t at = some ? chosen[in][lane] : 0;
  const int idx = some ? static_cast<int>(at >> 16) : -1;
  float w = some ? scores[in][at & 0xFFFF] : 0.0f;
  if (a.renorm) {
    const float sum = row_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  if (static_cast<int>(lane) < a.k && m < a.M) {
    a.weight[m * a.k + lane] = w * a.factor;
    a.index[m * a.k + lane] = idx;
  }
}

// What the kernel above does not take (over 512 experts, 16 choices or 16 groups): a row per wave,
// its scores and choice values in LDS, one pass over them per choice (16384 rows of 480, top 20:
// 115 us).
template <int DT>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = group_id() * kRouteWaves + wave;
  if (m >= a.M) return;                     // waves never meet: no barrier below
  const int E = static_cast<int>(a.E);
  float* score = lds + wave * 2 * E;
  float* choice = score + E;
  const auto* row = static_cast<const typename Elem<DT>::type*>(a.logits) + m * a.ld;
  const float none = -INFINITY;

  float mx = none;
  for (int e = lane; e < E; e += 64) {
    float l = to_float<DT>(row[e]);
    l = l > none ? fminf(l, 3.402823466e38f) : none;   // NaN compares false
    choice[e] = l;
    mx = fmaxf(mx, l);
  }
  float inv = 1.0f;
  if (!a.sigmoid) {
    mx = wave_max(mx);
    float sum = 0.0f;
    for (int e = lane; e < E; e += 64) {
      const float l = choice[e];
      const float p = l > none ? expf(l - mx) : 0.0f;
      score[e] = p;
      sum += p;
    }
    inv = wave_sum(sum);
  }
  for (int e = lane; e < E; e += 64) {
    const float l = choice[e];
    float p, c;
    if (a.sigmoid) {
      p = 1.0f / (1.0f + expf(-l));
      c = a.bias ? p + a.bias[e] : p;
    } else {
      p = score[e] / inv;
      c = a.bias ? p + a.bias[e] : l;       // a softmax keeps the logits' order
    }
    score[e] = p;
    choice[e] = (l > none && c > none) ? c : none;
  }
  // the lanes read each other's choices from here on
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();

  uint64_t kept = ~0ull;                    // one bit per group
  const int size = E / a.groups;
  if (a.groups > 1) {
    // lane g ranks group g: its best choice, plus its second best for sigmoid scores
    float b1 = none, b2 = none;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const float c = choice[lane * size + i];
        b2 = fmaxf(b2, fminf(b1, c));
        b1 = fmaxf(b1, c);
      }
    float rank = b1;
    if (a.sigmoid && b2 > none) rank = b1 + b2;
    uint64_t key = lane < a.groups ? choice_key(rank, lane) : 0;
    kept = 0;
    for (int i = 0; i < a.kept; ++i) {
      const uint64_t best = wave_max_u64(key);
      const int g = static_cast<int>(~static_cast<uint32_t>(best));
      kept |= 1ull << g;
      if (g == lane) key = 0;
    }
  }

  auto own_best = [&]() {
    uint64_t best = 0;
    for (int e = lane; e < E; e += 64) {
      const float c = choice[e];
      if (c > none && ((kept >> (a.groups > 1 ? e / size : 0)) & 1)) {
        const uint64_t key = choice_key(c, e);
        best = best > key ? best : key;
      }
    }
    return best;
  };
  uint64_t mine = own_best();
  float w = 0.0f;
  int idx = -1;
  for (int j = 0; j < a.k; ++j) {
    const uint64_t best = wave_max_u64(mine);
    if (best == 0) break;                   // nothing is left (uniform over the wave)
    const int e = static_cast<int>(~static_cast<uint32_t>(best));
    if (j == lane) {
      idx = e;
      w = score[e];
    }
    if ((e & 63) == lane) {
      choice[e] = none;
      mine = own_best();
    }
  }
  if (a.renorm) {
    const float sum = wave_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  if (lane < a.k) {
    a.weight[m * a.k + lane] = w * a.factor;
    a.index[m * a.k + lane] = idx;
  }
}

}  // namespace

namespace {

template <int DT, int NE>
hipError_t start_row16(const RouteArgs& a, int C, int shift, hipStream_t s) {
  const size_t size = dtype_bytes(DT);
  const int vec = C == NE && 16 * C == a.E && C * size % 16 == 0 && a.ld * size % 16 == 0 &&
                  reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                  reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  route_row16_kernel<DT, NE><<<grid_of((a.M + 15) / 16), 256, 0, s>>>(a, C, shift, vec);
  return hipGetLastError();
}

template <int DT>
hipError_t start_route(const RouteArgs& a, hipStream_t s) {
  int shift = 4;                                    // lanes per group: the most that 16 lanes have
  while (shift >= 0 && (a.groups << shift) > 16) --shift;
  if (shift >= 0 && a.k <= 16) {
    const int64_t size = a.E / a.groups;
    const int C = static_cast<int>((size + (1 << shift) - 1) >> shift);
    if (C <= 4) return start_row16<DT, 4>(a, C, shift, s);
    if (C <= 8) return start_row16<DT, 8>(a, C, shift, s);
    if (C <= 16) return start_row16<DT, 16>(a, C, shift, s);
    if (C <= 32) return start_row16<DT, 32>(a, C, shift, s);
  }
  const dim3 grid = grid_of((a.M + kRouteWaves - 1) / kRouteWaves);
  route_kernel<DT><<<grid, 64 * kRouteWaves, static_cast<size_t>(kRouteWaves) * 2 * a.E * 4, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  return a.dtype == BL_F16 ? start_route<BL_F16>(a, s) : a.dtype == BL_BF16 ? start_route<BL_BF16>(a, s) : start_route<BL_F32>(a, s);
}

}  // namespace bl
