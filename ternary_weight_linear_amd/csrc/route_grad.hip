// What training the router takes: the experts' balance loss with its counts, and the gradient of
// the logits. The contract is bl_route_balance and bl_route_backward in include/libbitlinear.h.
//
// A row has a group of 16 lanes (64 beyond 512 experts) and its experts in registers, V
// consecutive ones at a time per lane: expert (i LANES + lane) V + j is element i V + j.
#include <algorithm>

#include "adapter_internal.h"

namespace bl {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kMost = 3.402823466e38f;

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
template <int LANES>
__device__ __forceinline__ bool group_any(bool v) {
  const uint64_t all = __ballot(v);
  if constexpr (LANES == 64) return all != 0;
  else return (all >> (threadIdx.x & 48) & 0xFFFF) != 0;
}

template <int LANES, int V>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return (i / V * LANES + lane) * V + i % V;
}

// A row's logits; what is left out (-inf, NaN, past the last expert) is -inf.
template <int DT, int LANES, int NE, int V>
__device__ __forceinline__ void load_logits(const typename Elem<DT>::type* row, int E, int lane, float (&l)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = expert_of<LANES, V>(lane, i);
    if constexpr (V == 4 && DT == BL_F32) {
      f32x4 v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (e < E) v = *reinterpret_cast<const f32x4*>(row + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) l[i + j] = v[j];
    } else if constexpr (V == 4) {
      u32x2 v = {0, 0};
      if (e < E) v = *reinterpret_cast<const u32x2*>(row + e);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        l[i + j] = e < E ? to_float<DT>(static_cast<uint16_t>(v[j / 2] >> (16 * (j & 1)))) : -INFINITY;
    } else {
      l[i] = e < E ? to_float<DT>(row[e]) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) l[i] = l[i] > -INFINITY ? fminf(l[i], kMost) : -INFINITY;   // NaN compares false
}

// 1 / v by the hardware's instruction, which errs by one unit.
__device__ __forceinline__ float fast_inv(float v) { return __builtin_amdgcn_rcpf(v); }
// The gradient's scores are the routing's, by its expf. The loss's go into sums, which need no score
// below 2^-126: the hardware's instruction gives 0 there, and errs by |v| 2^-24 more (65536 rows of
// 1024, sigmoid 192 us where expf takes 222).
template <bool OF_ROUTING>
__device__ __forceinline__ float exponential(float v) {
  return OF_ROUTING ? expf(v) : __builtin_amdgcn_exp2f(v * 1.44269504088896341f);
}

// l becomes the normalised scores t (0 for what is left out). Sigmoid scores also give p and
// 1 - p, each without a difference. A row whose sigmoids are all below a half is normalised as
// exp(l - max) / (1 + exp(l)), so that none of them has to be large enough for fp32.
template <int LANES, int NE, bool SIGMOID, bool SCORES>
__device__ __forceinline__ void normalise(float (&l)[NE], float (&p)[NE], float (&q)[NE]) {
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NE; ++i) mx = fmaxf(mx, l[i]);
  mx = group_max<LANES>(mx);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const float v = l[i];
    if constexpr (SIGMOID) {
      const float z = exponential<SCORES>(-fabsf(v)), inv = fast_inv(1.0f + z);  // z = 0 for -inf
      const float ps = v >= 0.0f ? inv : z * inv;
      if constexpr (SCORES) {
        p[i] = ps;
        q[i] = v >= 0.0f ? z * inv : inv;
      }
      l[i] = mx > 0.0f ? ps : v > -INFINITY ? exponential<SCORES>(v - mx) * inv : 0.0f;
    } else {
      l[i] = v > -INFINITY ? exponential<SCORES>(v - mx) : 0.0f;
    }
    sum += l[i];
  }
  sum = group_sum<LANES>(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) l[i] *= inv;
}

__device__ __forceinline__ int64_t bounded(const int32_t* offsets, int64_t i, int64_t M) {
  const int64_t o = offsets[i];
  return o < 0 ? 0 : o > M ? M : o;
}
// The first sequence that ends past row m; S if none does. Few sequences: the group's lanes count those
// that end before, all at once.
template <int LANES>
__device__ __forceinline__ int64_t sequence_of(const int32_t* offsets, int64_t S, int64_t m, int lane) {
  if (S <= 2 * LANES) {
    int before = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = lane + LANES * i;
      const uint64_t all = __ballot(s < S && offsets[s < S ? s + 1 : 0] <= m);
      before += __popcll(LANES == 64 ? all : all >> (threadIdx.x & 48) & 0xFFFF);
    }
    return before;
  }
  int64_t lo = 0, hi = S;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (offsets[mid + 1] > m) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ------------------------------------------------------------------------------------------
// balance loss
// ------------------------------------------------------------------------------------------
// A workgroup sums a chunk of rows, sequence by sequence (those of a chunk are shared out over up to
// 16). Going from chunk to chunk and sequence to sequence, either number grows at each step: chunk +
// sequence numbers the partial sums. 16384 x 256, sigmoid, 11 sequences: 11 us in the trace (17 MB;
// scores are an exponential and a quotient each), its finish 7; 4096 x 60: 4.7 and 6.4, two chains of
// waits.
struct BalanceParts {
  int64_t chunk, chunks;
  float* t;               // [chunks + S - 1, E]
  int32_t* count;         // [chunks + S - 1, E]
  int32_t* rows;          // [chunks + S - 1]
};

constexpr int balance_threads(int lanes) { return lanes == 16 ? 1024 : 256; }

template <int DT, int LANES, int NE, int V, bool SIGMOID>
__global__ __launch_bounds__(balance_threads(LANES)) void route_balance_kernel(RouteRows r, BalanceParts w) {
  constexpr int T = balance_threads(LANES), G = T / LANES, W = T / 64;
  __shared__ float sums[W][LANES * NE];
  __shared__ int count[LANES * NE];
  __shared__ int counted[W];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, wave = threadIdx.x / 64, E = static_cast<int>(r.E);
  const int64_t c0 = blockIdx.x * w.chunk, c1 = min(c0 + w.chunk, r.M);
  const int64_t s0 = r.offsets ? sequence_of<64>(r.offsets, r.S, c0, threadIdx.x & 63) : 0;
  for (int64_t s = s0 + blockIdx.y; s < r.S; s += gridDim.y) {
    const int64_t begin = r.offsets ? bounded(r.offsets, s, r.M) : 0, end = r.offsets ? bounded(r.offsets, s + 1, r.M) : r.M;
    if (begin >= c1) break;
    const int64_t m0 = max(begin, c0), m1 = min(end, c1);
    if (m0 >= m1) continue;
    for (int i = threadIdx.x; i < E; i += T) count[i] = 0;
    __syncthreads();
    float acc[NE] = {};
    int n = 0;
    for (int64_t m = m0 + group; m < m1; m += G) {
      float l[NE], none[NE];
      load_logits<DT, LANES, NE, V>(static_cast<const typename Elem<DT>::type*>(r.logits) + m * r.ld, E, lane, l);
      bool any = false;
      for (int j = lane; j < r.k; j += LANES) {
        const int e = r.index[m * r.k + j];
        if (e >= 0 && e < E) {
          any = true;
          atomicAdd(&count[e], 1);
        }
      }
      any = group_any<LANES>(any);
      normalise<LANES, NE, SIGMOID, false>(l, none, none);
      n += any && lane == 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] += any ? l[i] : 0.0f;
    }
    // the wave's groups, then the waves
#pragma unroll
    for (int off = LANES; off < 64; off <<= 1) {
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] += __shfl_xor(acc[i], off);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off);
    if (threadIdx.x % 64 < LANES) {
#pragma unroll
      for (int i = 0; i < NE; ++i) sums[wave][expert_of<LANES, V>(lane, i)] = acc[i];
    }
    if (threadIdx.x % 64 == 0) counted[wave] = n;
    __syncthreads();
    const int64_t slot = blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += T) {
      float v = 0.0f;
#pragma unroll
      for (int g = 0; g < W; ++g) v += sums[g][e];
      w.t[slot * E + e] = v;
      w.count[slot * E + e] = count[e];
    }
    if (threadIdx.x == 0) {
      int rows = 0;
#pragma unroll
      for (int g = 0; g < W; ++g) rows += counted[g];
      w.rows[slot] = rows;
    }
    __syncthreads();
  }
}

// Sum of a value over the 1024 threads, in every thread.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  T all = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) all += lds[i];
  __syncthreads();
  return all;
}

// One workgroup per sequence: `parts` threads share an expert's partial sums, eight loads of each in
// flight at a time.
__global__ __launch_bounds__(1024) void route_balance_finish_kernel(RouteRows r, BalanceParts w, float* loss, int32_t* count, float* coef) {
  __shared__ double sum[1024];
  __shared__ int cnt[1024];
  __shared__ int64_t whole[16];
  const int64_t s = blockIdx.x;
  const int E = static_cast<int>(r.E);
  const int64_t begin = r.offsets ? bounded(r.offsets, s, r.M) : 0, end = r.offsets ? bounded(r.offsets, s + 1, r.M) : r.M;
  const int64_t first = begin / w.chunk + s, last = begin < end ? (end - 1) / w.chunk + s + 1 : first;   // slots
  int64_t n = 0;
  for (int64_t i = first + threadIdx.x; i < last; i += 1024) n += w.rows[i];
  const int width = E < 1024 ? E : 1024, parts = 1024 / width;
  const int part = threadIdx.x / width, e0 = threadIdx.x % width;
  double mine[2] = {};                              // of expert e0 and e0 + 1024
  int slots[2] = {};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = e0 + 1024 * q;
    double v = 0.0;
    int c = 0;
    if (part < parts && e < E)
      for (int64_t i = first + part; i < last; i += 8 * parts) {
        float tv[8];
        int cv[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int64_t at = min(i + k * parts, last - 1) * E + e;
          tv[k] = w.t[at];
          cv[k] = w.count[at];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i + k * parts < last) {
            v += tv[k];
            c += cv[k];
          }
      }
    sum[threadIdx.x] = v;
    cnt[threadIdx.x] = c;
    __syncthreads();
    if (part == 0 && e < E)
      for (int i = 0; i < parts; ++i) {
        mine[q] += sum[i * width + e0];
        slots[q] += cnt[i * width + e0];
      }
    __syncthreads();
    if (E <= 1024) break;
  }
  const int64_t rows = block_sum(n, whole);
  const double all = static_cast<double>(block_sum(static_cast<int64_t>(slots[0]) + slots[1], whole)) * static_cast<double>(rows);
  double v = 0.0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = e0 + 1024 * q;
    if (part == 0 && e < E) {
      const double f = all > 0.0 ? static_cast<double>(E) * slots[q] / all : 0.0;
      count[s * E + e] = slots[q];
      coef[s * E + e] = static_cast<float>(f);
      v += f * mine[q];
    }
  }
  v = block_sum(v, sum);
  if (threadIdx.x == 0) loss[s] = static_cast<float>(v);
}

// ------------------------------------------------------------------------------------------
// gradient of the logits
// ------------------------------------------------------------------------------------------
// With u = p / sum p over the slots (renormalised) and g = factor dweight, slot j adds to its
// expert's gradient
//   softmax   u_j (g_j - sum u g)    sigmoid   u_j (1 - p_j) (g_j - sum u g)       renormalised
//   softmax   p_j g_j                sigmoid   p_j (1 - p_j) g_j                   else,
// a softmax that is not renormalised takes p_e sum_j p_j g_j from every expert, and the balance loss
// adds t_e (c_e - sum t c), times 1 - p_e for sigmoid scores, with c = dloss coef. A row is read and
// written once: 16384 x 256, sigmoid, 12.6 us (33.5 MB, 2.7 TB/s; the scores' VALU work and three
// passes through LDS beside it), 4096 x 60 4.
template <int DT, int LANES, int NE, int V, bool SIGMOID, int KS>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBackwardArgs a) {
  constexpr int G = 256 / LANES;
  __shared__ __align__(16) float lds[G][LANES * NE];
  const RouteRows& r = a.r;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, E = static_cast<int>(r.E);
  const int64_t m = group_id() * G + group;
  const int64_t mc = m < r.M ? m : r.M - 1;         // rows past the end work on the last one
  float* row = lds[group];
  float t[NE], p[NE], q[NE];
  load_logits<DT, LANES, NE, V>(static_cast<const typename Elem<DT>::type*>(r.logits) + mc * r.ld, E, lane, t);
  int at[KS];
  float g[KS];
  bool any = false;
#pragma unroll
  for (int j = 0; j < KS; ++j) {
    const int slot = lane + LANES * j;
    at[j] = -1;
    g[j] = 0.0f;
    if (slot < r.k) {
      const int e = r.index[mc * r.k + slot];
      at[j] = e >= 0 && e < E ? e : -1;
      if (a.dweight && at[j] >= 0) g[j] = a.factor * a.dweight[mc * r.k + slot];
    }
    any |= at[j] >= 0;
  }
  any = group_any<LANES>(any);
  normalise<LANES, NE, SIGMOID, true>(t, p, q);

  // each slot's addend
  float v[KS] = {};
  float common = 0.0f;
  if (a.dweight) {
#pragma unroll
    for (int i = 0; i < NE; ++i) row[expert_of<LANES, V>(lane, i)] = SIGMOID ? p[i] : t[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    float ps[KS], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      ps[j] = at[j] >= 0 ? row[at[j]] : 0.0f;
      sum += ps[j];
    }
    if (a.renorm) {
      // quotients, as the routing has them: 1 / sum is infinite where the slots have next to no score
      sum = group_sum<LANES>(sum);
      float mean = 0.0f;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        ps[j] = sum > 0.0f ? ps[j] / sum : 0.0f;
        mean += ps[j] * g[j];
      }
      mean = group_sum<LANES>(mean);
#pragma unroll
      for (int j = 0; j < KS; ++j) v[j] = ps[j] * (g[j] - mean);
    } else {
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        v[j] = ps[j] * g[j];
        common += v[j];
      }
      common = SIGMOID ? 0.0f : group_sum<LANES>(common);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  float d[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) d[i] = 0.0f;
  if (a.coef) {
    int64_t s = 0;
    bool inside = any;
    if (r.offsets) {
      s = sequence_of<LANES>(r.offsets, r.S, mc, lane);
      inside = any && s < r.S && r.offsets[s < r.S ? s : 0] <= mc;
    }
    if (inside) {
      const float dl = a.dloss[s];
      float mean = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; i += V) {
        const int e = expert_of<LANES, V>(lane, i);
        if constexpr (V == 4) {
          f32x4 c = {0, 0, 0, 0};
          if (e < E) c = *reinterpret_cast<const f32x4*>(a.coef + s * E + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[i + j] = c[j];
        } else {
          d[i] = e < E ? a.coef[s * E + e] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) mean += t[i] * d[i];
      mean = group_sum<LANES>(mean);
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] = dl * t[i] * (d[i] - mean) * (SIGMOID ? q[i] : 1.0f);
    }
  }
  if (a.dweight) {
    if (!SIGMOID && !a.renorm) {
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] -= t[i] * common;
    }
    // the addends meet in LDS, in the order of the slots where two are of one expert
    uint32_t* tag = reinterpret_cast<uint32_t*>(row);
    bool twice = false;
#pragma unroll
    for (int j = 0; j < KS; ++j)
      if (at[j] >= 0) tag[at[j]] = lane + LANES * j;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < KS; ++j) twice |= at[j] >= 0 && tag[at[j]] != static_cast<uint32_t>(lane + LANES * j);
    twice = group_any<64>(twice);                   // uniform over the wave
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < NE; ++i) row[expert_of<LANES, V>(lane, i)] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (!twice) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
        if (at[j] >= 0) row[at[j]] = v[j];
    } else {
#pragma unroll
      for (int j = 0; j < KS; ++j)
        for (int i = 0; i < LANES; ++i) {
          if (lane == i && at[j] >= 0) row[at[j]] += v[j];
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < NE; ++i) d[i] += row[expert_of<LANES, V>(lane, i)] * (SIGMOID ? q[i] : 1.0f);
  }
  if (m >= r.M) return;
  const int64_t out = m * a.ldd;
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = expert_of<LANES, V>(lane, i);
    if (e >= E) continue;
    if constexpr (V == 4) {
      if (a.ddtype == BL_F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.dlogits) + out + e) = f32x4{d[i], d[i + 1], d[i + 2], d[i + 3]};
      } else {
        uint16_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = a.ddtype == BL_BF16 ? bf16_bits(d[i + j]) : half_bits(d[i + j]);
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dlogits) + out + e) =
            u32x2{b[0] | static_cast<uint32_t>(b[1]) << 16, b[2] | static_cast<uint32_t>(b[3]) << 16};
      }
    } else {
      store_as(a.dlogits, a.ddtype, out + e, d[i]);
    }
  }
}

// ------------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------------
bool vec_experts(const void* p, int64_t E, int64_t ld, size_t size) {
  return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * size) == 0;
}

// An fp32 sum of one group of lanes has 128 rows at most (2048 beyond 512 experts).
constexpr int64_t kMostChunk = 8192;
// Rows of a chunk, a row for every group of lanes at least: about 128 workgroups, 256 of many rows, and
// beyond 512 experts 128, 256 or 512. More chunks shorten the sums and lengthen their finish, which is
// one workgroup for each sequence. (us from a graph, one sequence, sigmoid, for 128 / 256 / 512: 16384
// x 256 20.5 / 23.7 / 23.6, 32768 x 256 25.3 / 26.0 / 38.6, 65536 x 256 36.4 / 32.4 / 44.2; 2048 x 1024
// 40 / 52 / 86, 8192 x 1024 74 / 69 / 94, 16384 x 1024 127 / 96 / 108, 65536 x 1024 429 / 248 / 193.)
int64_t balance_chunk(int64_t M, int64_t E) {
  const int64_t groups = E <= 512 ? 64 : 4;
  const int64_t most = M >= 32768 ? (E > 512 ? 512 : 256) : E > 512 && M >= 4096 ? 256 : 128;
  return (std::clamp<int64_t>(M / most, 1, kMostChunk) + groups - 1) / groups * groups;
}
struct BalanceWs {
  int64_t chunk, chunks;
  size_t count_off, rows_off, total;
};
BalanceWs balance_ws(int64_t M, int64_t E, int64_t S) {
  BalanceWs w{};
  w.chunk = balance_chunk(M, E);
  w.chunks = (M + w.chunk - 1) / w.chunk;
  const size_t slots = static_cast<size_t>(w.chunks + S - 1);
  w.count_off = (slots * E * 4 + 255) & ~size_t(255);
  w.rows_off = 2 * w.count_off;
  w.total = w.rows_off + ((slots * 4 + 255) & ~size_t(255));
  return w;
}

template <int DT, int LANES, int NE, int V>
hipError_t start_balance(const RouteRows& r, const BalanceParts& w, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(w.chunks), static_cast<uint32_t>(std::min<int64_t>(r.S, 16)));
  constexpr int T = balance_threads(LANES);
  if (r.sigmoid) route_balance_kernel<DT, LANES, NE, V, true><<<grid, T, 0, s>>>(r, w);
  else route_balance_kernel<DT, LANES, NE, V, false><<<grid, T, 0, s>>>(r, w);
  return hipGetLastError();
}
template <int DT, int V>
hipError_t start_balance_by(const RouteRows& r, const BalanceParts& w, hipStream_t s) {
  if (r.E <= 64) return start_balance<DT, 16, 4, V>(r, w, s);
  if (r.E <= 128) return start_balance<DT, 16, 8, V>(r, w, s);
  if (r.E <= 256) return start_balance<DT, 16, 16, V>(r, w, s);
  if (r.E <= 512) return start_balance<DT, 16, 32, V>(r, w, s);
  return start_balance<DT, 64, 32, V>(r, w, s);
}
template <int DT>
hipError_t start_balance_vec(const RouteRows& r, const BalanceParts& w, hipStream_t s) {
  return vec_experts(r.logits, r.E, r.ld, dtype_bytes(DT)) ? start_balance_by<DT, 4>(r, w, s) : start_balance_by<DT, 1>(r, w, s);
}

template <int DT, int LANES, int NE, int V, bool SIGMOID>
hipError_t start_backward(const RouteBackwardArgs& a, hipStream_t s) {
  const dim3 grid = grid_of((a.r.M + 256 / LANES - 1) / (256 / LANES));
  if (a.r.k <= LANES) route_backward_kernel<DT, LANES, NE, V, SIGMOID, 1><<<grid, 256, 0, s>>>(a);
  else route_backward_kernel<DT, LANES, NE, V, SIGMOID, LANES == 16 ? 4 : 1><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <int DT, int V, bool SIGMOID>
hipError_t start_backward_by(const RouteBackwardArgs& a, hipStream_t s) {
  if (a.r.E <= 64) return start_backward<DT, 16, 4, V, SIGMOID>(a, s);
  if (a.r.E <= 128) return start_backward<DT, 16, 8, V, SIGMOID>(a, s);
  if (a.r.E <= 256) return start_backward<DT, 16, 16, V, SIGMOID>(a, s);
  if (a.r.E <= 512) return start_backward<DT, 16, 32, V, SIGMOID>(a, s);
  return start_backward<DT, 64, 32, V, SIGMOID>(a, s);
}
template <int DT>
hipError_t start_backward_vec(const RouteBackwardArgs& a, hipStream_t s) {
  const bool vec = vec_experts(a.r.logits, a.r.E, a.r.ld, dtype_bytes(DT)) && vec_experts(a.dlogits, a.r.E, a.ldd, dtype_bytes(a.ddtype)) &&
                   reinterpret_cast<uintptr_t>(a.coef) % 16 == 0;
  if (vec) return a.r.sigmoid ? start_backward_by<DT, 4, true>(a, s) : start_backward_by<DT, 4, false>(a, s);
  return a.r.sigmoid ? start_backward_by<DT, 1, true>(a, s) : start_backward_by<DT, 1, false>(a, s);
}

}  // namespace

size_t route_balance_ws_bytes(int64_t M, int64_t E, int64_t S) { return balance_ws(M, E, S).total; }

hipError_t launch_route_balance(const RouteBalanceArgs& a, char* ws, hipStream_t s) {
  const BalanceWs L = balance_ws(a.r.M, a.r.E, a.r.S);
  const BalanceParts w{L.chunk, L.chunks, reinterpret_cast<float*>(ws), reinterpret_cast<int32_t*>(ws + L.count_off),
                       reinterpret_cast<int32_t*>(ws + L.rows_off)};
  const hipError_t e = a.r.dtype == BL_F16    ? start_balance_vec<BL_F16>(a.r, w, s)
                       : a.r.dtype == BL_BF16 ? start_balance_vec<BL_BF16>(a.r, w, s)
                                              : start_balance_vec<BL_F32>(a.r, w, s);
  if (e != hipSuccess) return e;
  route_balance_finish_kernel<<<static_cast<uint32_t>(a.r.S), 1024, 0, s>>>(a.r, w, a.loss, a.count, a.coef);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s) {
  return a.r.dtype == BL_F16    ? start_backward_vec<BL_F16>(a, s)
         : a.r.dtype == BL_BF16 ? start_backward_vec<BL_BF16>(a, s)
                                : start_backward_vec<BL_F32>(a, s);
}

}  // namespace bl
