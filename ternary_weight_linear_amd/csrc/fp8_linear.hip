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

int64_t tiles(int64_t M, int64_t N, int bn, int bm) { return ((N + bn - 1) / bn) * ((M + bm - 1) / bm); }

template <class S>
hipError_t start_whole(const ProductArgs& p, hipStream_t s) {
  return start_gemm<S>(p, (p.a.M + S::BM - 1) / S::BM, s);
}

// Tile of the tiled kernel. Large tiles read less from L2 (64 x 64 tiles are bound by it, at
// 11 to 15 TB/s), small ones fill the 256 CUs. Measured on MI355X, us, e4m3 instruction
// (256 x 256 / 128 x 128, four waves / 128 x 128, eight waves, four stages / 128 x 64 / 64 x 64):
//   4096 x 28672 x 8192  785 / 926 / - / - / -      2048 x 8192 x 8192  117 / 143 / 168 / 191 / -
//   512 x 8640 x 3200    - / 26.3 / 36 / 27.4 / 30  512 x 8192 x 8192   - / 57 / 43.0 / 52.8 / -
//   1024 x 4096 x 4096   - / 28.1 / 23.9 / 24.4 / 30   512 x 3200 x 8640 - / 57 / 38 / 30.7 / 32.6
//   96 x 28672 x 8192    - / 58.9 / 57.2 / 68.5 / 73.5
// and with K in parts where 64 x 64 tiles alone leave CUs idle (1 / 2 / 4 parts):
//   512 x 1024 x 8192 20.9 / 15.8 / 16.3   64 x 8192 x 8192 23.4 / 18.7 / 20.4
//   200 x 1024 x 8192 20.1 / 15.2 / 12.7   24 x 4096 x 11008 24.3 / 16.8 / 14.1
// fp16 operands: 4096 x 28672 x 8192 1545 (128 x 128); 512 x 3200 x 8640 45.5 (64 x 64), as with
// every other tile: converting the codes (a quarter-rate instruction per two of them, for each
// fragment that a wave reads) bounds it; staging q as fp16 halved that and lost as much to L2.
template <bool EXACT>
hipError_t start_tiled(const ProductArgs& p, float* part, hipStream_t s) {
  const int64_t M = p.a.M, N = p.a.N, t128 = tiles(M, N, 128, 128);
  const int parts = fp8_split_parts(M, N, p.a.K);
  if (parts > 1) return start_split_gemm<GemmShape<64, 64, 2, 2, EXACT ? 3 : 4, EXACT>>(p, parts, part, s);
  if constexpr (EXACT) {
    if (t128 >= 256) return start_whole<GemmShape<128, 128, 2, 2, 2, true>>(p, s);
    return start_whole<GemmShape<64, 64, 2, 2, 3, true>>(p, s);
  } else {
    if (t128 > 256) {
      // rounds over the chip: 256 large tiles take 1, 512 small ones 0.6 of it
      const double large = static_cast<double>((tiles(M, N, 256, 256) + 255) / 256), small = 0.6 * ((t128 + 511) / 512);
      if (large <= small) return start_whole<GemmShape<256, 256, 2, 4, 2, false>>(p, s);
      return start_whole<GemmShape<128, 128, 2, 2, 2, false>>(p, s);
    }
    if (t128 >= 200) return start_whole<GemmShape<128, 128, 2, 4, 4, false>>(p, s);
    if (tiles(M, N, 128, 64) >= 200 && tiles(M, N, 128, 64) <= 256)
      return start_whole<GemmShape<128, 64, 2, 2, 4, false>>(p, s);
    return start_whole<GemmShape<64, 64, 2, 2, 4, false>>(p, s);
  }
}

}  // namespace

int fp8_split_parts(int64_t M, int64_t N, int64_t K) {
  const int64_t t = tiles(M, N, 64, 64), KB = fp8_blocks(K);
  if (t > 128) return 1;
  int64_t parts = 256 / t < 8 ? 256 / t : 8;
  if (parts > KB / 8) parts = KB / 8;               // at least eight blocks each
  if (parts <= 1) return 1;
  const int64_t per = (KB + parts - 1) / parts;
  return static_cast<int>((KB + per - 1) / per);    // none empty
}

hipError_t launch_fp8_linear(const Fp8LinearArgs& a, const void* x, int xdtype, int64_t ldx, float* part,
                             hipStream_t s) {
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
  // fp32 results stream up to 32 rows (32 x 8192 x 8192: 20.5 us, tiled 23)
  if ((a.M <= 32 && a.ydtype == BL_F32) || 256 * a.K >= (int64_t(1) << 31))   // tiled: 32-bit offsets
    return start_codes<2>(st, s);
  return a.ydtype == BL_F32 ? start_tiled<true>(st.p, part, s) : start_tiled<false>(st.p, part, s);
}

}  // namespace bl
