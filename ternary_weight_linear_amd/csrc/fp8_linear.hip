// The block-scaled linear layer (bl_fp8_linear, bl_fp8_forward).
#include "fp8_gemm.h"

namespace bl {
namespace {

// Rows of w per workgroup of the streaming kernel: the most that still gives most CUs (256) a
// workgroup. More rows read the activations less often; more workgroups than CUs bring nothing.
// Measured in us at K = 8192, M = 16, for 16 / 32 / 64 / 128 rows: N = 1024 9.7 / 13.2 / 20.5 /
// 26; N = 8192 18.3 / 14.2 / 21.4 / 25; N = 28672 - / 55.7 / 47.9 / 43.8; N = 11008, K = 4096
// 13.5 / 14.1 / 12.2 / -.
int stream_rows(int64_t N, int64_t tiles) {
  for (int r = 128; r > 16; r /= 2)
    if ((N + r - 1) / r * tiles >= 160) return r;
  return 16;
}

template <int MT>
hipError_t start_codes(const StreamArgs& st, hipStream_t s) {
  const int64_t tiles = (st.p.a.M + 16 * MT - 1) / (16 * MT);
  const int rows = stream_rows(st.p.a.N, tiles);
  if constexpr (MT <= 2) {
    if (rows == 128) return start_stream<MT, 4, 4, kSrcCodes, kStreamLinear>(st, tiles, 0, s);
    if (rows == 64) return start_stream<MT, 4, 8, kSrcCodes, kStreamLinear>(st, tiles, 0, s);
  }
  if (rows >= 32) return start_stream<MT, 2, 8, kSrcCodes, kStreamLinear>(st, tiles, 0, s);
  return start_stream<MT, 1, 8, kSrcCodes, kStreamLinear>(st, tiles, 0, s);
}

// One to four rows: each workgroup quantises them into LDS itself.
hipError_t start_values(const StreamArgs& st, int xdtype, hipStream_t s) {
  const int rows = static_cast<int>(st.p.a.M);
  switch (stream_rows(st.p.a.N, 1)) {
    case 128: return start_stream_x<4, 4, kStreamLinear>(st, xdtype, 1, rows, s);
    case 64: return start_stream_x<4, 8, kStreamLinear>(st, xdtype, 1, rows, s);
    case 32: return start_stream_x<2, 8, kStreamLinear>(st, xdtype, 1, rows, s);
    default: return start_stream_x<1, 8, kStreamLinear>(st, xdtype, 1, rows, s);
  }
}

}  // namespace

hipError_t launch_fp8_linear(const Fp8LinearArgs& args, const void* x, int xdtype, int64_t ldx, hipStream_t s) {
  Fp8LinearArgs a = args;
  a.vec = vec_rows(a.y, a.ldy, a.ydtype);
  a.vec8 = vec8_rows(a.y, a.N, a.ldy);
  StreamArgs st{};
  st.p.a = a;
  st.x = x;
  st.ldx = ldx;
  // (their codes and the reduction's 32 KB stay within 64 KB of LDS)
  if (x && a.M <= 4 && a.M * a.K <= 28672) return start_values(st, xdtype, s);
  if (x) {
    const hipError_t e = launch_fp8_quant_act(x, xdtype, a.M, a.K, ldx, 0, nullptr, const_cast<uint8_t*>(a.q),
                                              const_cast<float*>(a.sx), s);
    if (e != hipSuccess) return e;
  }
  if (a.M <= 16) return start_codes<1>(st, s);
  if (a.M <= 32) return start_codes<2>(st, s);
  // Up to 64 rows the streaming kernel reads 8 KB of codes of q per block and workgroup; the
  // tiled one shares them in LDS and wins once its 64 x 64 tiles fill the CUs (M = 64, K = 8192:
  // N = 8192 26.7 us streamed, 39.4 tiled; N = 28672 95.9 and 59.9). Its offsets are 32 bits.
  if ((a.M <= 64 && a.N < 64 * 256) || 256 * a.K >= (int64_t(1) << 31)) return start_codes<4>(st, s);
  const ProductArgs& p = st.p;
  if (a.ydtype == BL_F32) {
    const int64_t tiles = ((a.N + 127) / 128) * ((a.M + 127) / 128);
    if (tiles >= 256) return start_gemm<GemmShape<128, 128, 2, 2, true>>(p, (a.M + 127) / 128, s);
    return start_gemm<GemmShape<64, 64, 2, 2, true>>(p, (a.M + 63) / 64, s);
  }
  const int64_t tiles = ((a.N + 255) / 256) * ((a.M + 255) / 256);
  if (tiles >= 256) return start_gemm<GemmShape<256, 256, 2, 4, false>>(p, (a.M + 255) / 256, s);
  const int64_t tiles2 = ((a.N + 127) / 128) * ((a.M + 127) / 128);
  if (tiles2 >= 256) return start_gemm<GemmShape<128, 128, 2, 2, false>>(p, (a.M + 127) / 128, s);
  return start_gemm<GemmShape<64, 64, 2, 2, false>>(p, (a.M + 63) / 64, s);
}

}  // namespace bl
