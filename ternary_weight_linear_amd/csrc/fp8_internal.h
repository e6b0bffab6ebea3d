// Declarations and device helpers shared by the 8-bit floating point operators (e4m3 codes
// with one fp32 scale per block of 128) and the expert router.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "libbitlinear.h"

namespace bl {

constexpr int kFp8Block = 128;                      // inputs (and weight rows) per scale
constexpr float kFp8Max = 448.0f;                   // largest e4m3 value
constexpr uint32_t kFp8FloorBits = 0x0D800000u;     // 2^-100, the least block maximum used

inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }
inline size_t dtype_bytes(int dtype) { return dtype == BL_F32 ? 4 : 2; }

// A launch whose work-items along one dimension pass 2^32 runs modulo that, without an error.
inline bool grid_fits(int64_t groups, int threads) { return groups * threads < (int64_t(1) << 32); }
// So workgroups that may be many go over two dimensions (the last few of them may be too many).
inline dim3 grid_of(int64_t groups) {
  const int64_t x = groups < (int64_t(1) << 20) ? groups : int64_t(1) << 20;
  return dim3(static_cast<uint32_t>(x), static_cast<uint32_t>((groups + x - 1) / x));
}

// y = linear(q, w) on rows that are all multiplied by one weight matrix.
struct Fp8LinearArgs {
  const uint8_t* q;      // e4m3 codes [M, K]
  const float* sx;       // [KB, M]
  const uint8_t* w;      // e4m3 codes [N, K]
  const float* sw;       // [NB, KB]
  int64_t M, N, K;
  void* y;               // [M, N], rows ldy elements apart
  int64_t ldy;
  int ydtype;
};

struct Fp8ExpertsArgs {
  const void* x;         // [M, H], rows ldx elements apart
  int xdtype;
  int64_t M, H, ldx;
  const int32_t* index;  // [M, k]
  const float* weight;   // [M, k]
  int64_t k;
  const uint8_t* wgu;    // [E, 2, I, H]
  const float* sgu;      // [E, 2, IB, HB]
  const uint8_t* wd;     // [E, H, I]
  const float* sd;       // [E, HB, IB]
  int64_t E, I;
  void* y;               // [M, H], rows ldy elements apart
  int ydtype;
  int64_t ldy;
};

struct RouteArgs {
  const void* logits;    // [M, E], rows ld elements apart
  int dtype;
  int64_t M, E, ld;
  const float* bias;     // [E] or null
  int sigmoid;           // else softmax
  int groups, kept, k;
  int renorm;
  float factor;
  float* weight;         // [M, k]
  int32_t* index;        // [M, k]
};

// Carve-up of the experts' workspace (256-byte aligned regions, no fill needed).
struct ExpertsWs {
  size_t q_off, sx_off;        // quantised x: codes [M, H], scales [HB, M]
  size_t head_off;             // int32 [4]: rows used, tiles
  size_t pair_off;             // int32 [P] slot m * k + j of each sorted row
  size_t tile_off;             // int32 [tiles, 4]: expert, first row, rows
  size_t count_off;            // int32 [chunks, E]: slots per expert of each chunk of the sort
  size_t hq_off, hs_off;       // quantised silu(gate) * up: codes [P, I], scales [IB, P]
  size_t sum_off;              // fp32 [P, I] silu(gate) * up, where it is not quantised at once, and
                               // after that [P, H]: outputs before the weighted sum
  size_t total;
};
ExpertsWs experts_ws(int64_t M, int64_t H, int64_t k, int64_t E, int64_t I);

hipError_t launch_fp8_quant_act(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx,
                                int gated, const int32_t* rows_used, uint8_t* q, float* scale,
                                hipStream_t s);
hipError_t launch_fp8_quant_weight(const float* W, int64_t N, int64_t K, uint8_t* codes,
                                   float* scale, hipStream_t s);
// a.q and a.sx are scratch when x is given: they are filled from it where the product takes codes.
// part: fp8_part_bytes(M, N, K) of scratch for partial sums.
hipError_t launch_fp8_linear(const Fp8LinearArgs& a, const void* x, int xdtype, int64_t ldx, float* part,
                             hipStream_t s);
int64_t fp8_part_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_fp8_experts(const Fp8ExpertsArgs& a, char* ws, hipStream_t s);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

// ---- device helpers ------------------------------------------------------------------------

// Which workgroup of grid_of's this is.
__device__ __forceinline__ int64_t group_id() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }

template <int DT>
struct Elem;  // storage type of a bl_dtype
template <>
struct Elem<BL_F16> { using type = uint16_t; };
template <>
struct Elem<BL_BF16> { using type = uint16_t; };
template <>
struct Elem<BL_F32> { using type = float; };

template <int DT>
__device__ __forceinline__ float to_float(typename Elem<DT>::type v) {
  if constexpr (DT == BL_F32) return v;
  else if constexpr (DT == BL_BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else return static_cast<float>(__builtin_bit_cast(_Float16, v));
}

// fp32 to bf16 bits, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

__device__ __forceinline__ uint16_t half_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

__device__ __forceinline__ void store_as(void* y, int dtype, int64_t at, float v) {
  if (dtype == BL_F32) static_cast<float*>(y)[at] = v;
  else if (dtype == BL_BF16) static_cast<uint16_t*>(y)[at] = bf16_bits(v);
  else static_cast<uint16_t*>(y)[at] = half_bits(v);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What a block's values are multiplied by before they are rounded to codes, from its maximum.
// IEEE steps: they decide codes.
__device__ __forceinline__ float code_factor(float a) { return kFp8Max * (1.0f / a); }

// silu(g) * u in fp32
__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

}  // namespace bl
