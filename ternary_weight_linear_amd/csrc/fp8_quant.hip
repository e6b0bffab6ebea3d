// Block quantisers to e4m3: activations (one scale per row and 128 inputs) and weights (one
// scale per 128 x 128 block).
//
//   a = max(max |v| over the block, 2^-100),  q = e4m3(fl32(v * r)),  r = fl32(448 fl32(1 / a)),
//   scale = fl32(a / 448).
//
// |v r| <= 448 (1 + 2^-20), which rounds to 448, so no code overflows (1 / a is subnormal for
// a > 2^126, and still right to 21 bits). The maximum is taken over the bit patterns of |v| as
// unsigned integers: there NaN > inf > every finite value, so a block that holds NaN gets scale
// NaN and NaN codes.
#include "fp8_mfma.h"

namespace bl {
namespace {

// Memory bounds it, and small calls their launch (kernel trace): bf16 32768 x 8192 145 us (5.6
// TB/s), gated 2048 x 8640 22.7 (20.7 a call among others, 4.3 TB/s), fp16 16 x 8192 2.8.
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void fp8_quant_act_kernel(QuantArgs q) {
  quant_blocks<DT, GATED>(q, group_id() * 16);
}

// One workgroup per 128 x 128 block: thread t holds rows t / 16 + 16 i, inputs 8 (t % 16) ...,
// read once and kept in registers for the codes. Memory bounds it: 28672 x 8192 204 us (5.8 TB/s).
__global__ __launch_bounds__(256) void fp8_quant_weight_kernel(const float* __restrict__ W,
                                                               int64_t N, int64_t K, int64_t KB,
                                                               uint8_t* __restrict__ codes,
                                                               float* __restrict__ scale) {
  __shared__ uint32_t red[4];
  const int64_t nb = group_id() / KB, kb = group_id() - nb * KB;
  if (nb * kFp8Block >= N) return;
  const int r = threadIdx.x >> 4;
  const int64_t k = kb * kFp8Block + (threadIdx.x & 15) * 8;
  float v[8][8];
  uint32_t a = kFp8FloorBits;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = nb * kFp8Block + r + 16 * i;
    if (n < N && k < K) load8<BL_F32>(W + n * K + k, v[i]);
    else
      for (int e = 0; e < 8; ++e) v[i][e] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = max(a, abs_bits(v[i][e]));
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), off)));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  const float am = __uint_as_float(max(max(red[0], red[1]), max(red[2], red[3])));
  const float rcp = code_factor(am);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = nb * kFp8Block + r + 16 * i;
    if (n < N && k < K) *reinterpret_cast<u32x2*>(codes + n * K + k) = pack8(v[i], rcp);
  }
  if (threadIdx.x == 0) scale[nb * KB + kb] = am / kFp8Max;
}

template <int DT>
void start_quant(const void* x, int64_t M, int64_t K, int64_t ldx, int gated,
                 const int32_t* rows_used, uint8_t* q, float* scale, hipStream_t s) {
  const QuantArgs a{x, M, K, fp8_blocks(K), ldx, rows_used, q, scale};
  const dim3 grid = grid_of((M * a.KB + 15) / 16);
  if (gated) fp8_quant_act_kernel<DT, true><<<grid, 256, 0, s>>>(a);
  else fp8_quant_act_kernel<DT, false><<<grid, 256, 0, s>>>(a);
}

}  // namespace

hipError_t launch_fp8_quant_act(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx,
                                int gated, const int32_t* rows_used, uint8_t* q, float* scale,
                                hipStream_t s) {
  if (dtype == BL_F16) start_quant<BL_F16>(x, M, K, ldx, gated, rows_used, q, scale, s);
  else if (dtype == BL_BF16) start_quant<BL_BF16>(x, M, K, ldx, gated, rows_used, q, scale, s);
  else start_quant<BL_F32>(x, M, K, ldx, gated, rows_used, q, scale, s);
  return hipGetLastError();
}

hipError_t launch_fp8_quant_weight(const float* W, int64_t N, int64_t K, uint8_t* codes,
                                   float* scale, hipStream_t s) {
  const int64_t NB = fp8_blocks(N), KB = fp8_blocks(K);
  fp8_quant_weight_kernel<<<grid_of(NB * KB), 256, 0, s>>>(W, N, K, KB, codes, scale);
  return hipGetLastError();
}

}  // namespace bl
