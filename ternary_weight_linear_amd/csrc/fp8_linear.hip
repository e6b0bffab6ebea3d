// The block-scaled linear layer (bl_fp8_linear, bl_fp8_forward).
#include "fp8_mfma.h"

namespace bl {

hipError_t launch_fp8_linear(const Fp8LinearArgs& a, hipStream_t s) {
  ProductArgs p{a, RowMap{}, 0, 0};
  const uint32_t nt = static_cast<uint32_t>((a.N + 15) / 16);
  if (a.M <= 16)
    fp8_stream_kernel<1><<<dim3(nt, 1), 512, 0, s>>>(p);
  else
    fp8_stream_kernel<4><<<dim3(nt, static_cast<uint32_t>((a.M + 63) / 64)), 512, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace bl
