// The block-scaled linear layer (bl_fp8_linear, bl_fp8_forward).
#include "fp8_gemm.h"

namespace bl {

hipError_t launch_fp8_linear(const Fp8LinearArgs& a, hipStream_t s) {
  ProductArgs p{a, RowMap{}, 0, 0};
  const uint32_t nt = static_cast<uint32_t>((a.N + 15) / 16);
  if (a.M <= 16) {
    fp8_stream_kernel<1><<<dim3(nt, 1), 512, 0, s>>>(p);
  } else if (a.M <= 64 || 256 * a.K >= (int64_t(1) << 31)) {   // the tiled kernel's offsets are 32 bits
    fp8_stream_kernel<4><<<dim3(nt, static_cast<uint32_t>((a.M + 63) / 64)), 512, 0, s>>>(p);
  } else if (a.ydtype == BL_F32) {
    const int64_t tiles = ((a.N + 127) / 128) * ((a.M + 127) / 128);
    if (tiles >= 256) return start_gemm<GemmShape<128, 128, 2, 2, true>>(p, (a.M + 127) / 128, s);
    return start_gemm<GemmShape<64, 64, 2, 2, true>>(p, (a.M + 63) / 64, s);
  } else {
    const int64_t tiles = ((a.N + 255) / 256) * ((a.M + 255) / 256);
    if (tiles >= 256) return start_gemm<GemmShape<256, 256, 2, 4, false>>(p, (a.M + 255) / 256, s);
    const int64_t tiles2 = ((a.N + 127) / 128) * ((a.M + 127) / 128);
    if (tiles2 >= 256) return start_gemm<GemmShape<128, 128, 2, 2, false>>(p, (a.M + 127) / 128, s);
    return start_gemm<GemmShape<64, 64, 2, 2, false>>(p, (a.M + 63) / 64, s);
  }
  return hipGetLastError();
}

}  // namespace bl
