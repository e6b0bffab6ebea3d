// Routing to experts: scores, choice by biased score within the best groups, the k best, and
// their weights. The contract is bl_route_experts in include/libbitlinear.h.
//
// One wave per row. The row's scores and choices live in LDS; lane l owns experts l, l + 64,
// ... and keeps the best choice among them as a 64-bit key (ordered bits of the choice above
// the complement of the index, so the largest key is the best choice and, among equals, the
// lowest index). Each of k rounds takes the largest key of the wave; only its owner looks
// through its experts again.
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

template <int DT>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave;
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

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>((a.M + kRouteWaves - 1) / kRouteWaves));
  const size_t lds = static_cast<size_t>(kRouteWaves) * 2 * a.E * 4;
  if (a.dtype == BL_F16) route_kernel<BL_F16><<<grid, 64 * kRouteWaves, lds, s>>>(a);
  else if (a.dtype == BL_BF16) route_kernel<BL_BF16><<<grid, 64 * kRouteWaves, lds, s>>>(a);
  else route_kernel<BL_F32><<<grid, 64 * kRouteWaves, lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace bl
