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
  if (rows == 128) return start_stream<MT, 4, 4, kSrcCodes, kStreamLinear>(st, tiles, 0, s);
  if (rows == 64) return start_stream<MT, 4, 8, kSrcCodes, kStreamLinear>(st, tiles, 0, s);
  if (rows == 32) return start_stream<MT, 2, 8, kSrcCodes, kStreamLinear>(st, tiles, 0, s);
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

// Parts of K for 64 x 64 tiles that do not fill the CUs by themselves: up to eight, of at least
// eight blocks, by the share of the CUs' rounds that their workgroups fill less 4 % per part more
// (partial sums are written and read again), if that is a fifth better than without.
// Measured, us by parts: 168 tiles, K = 16384 1 38.7, 2 35.3, 3 29.3, 4 35.1 (fp16 operands 63,
// 51, 40, 42); 81 tiles, K = 19664 1 49.6, 2 32.5, 3 26.3, 6 29.8; 252 tiles 1 16.7, 2 20.2.
int split_parts(int64_t M, int64_t N, int64_t K) {
  const int64_t t = tiles(M, N, 64, 64), KB = fp8_blocks(K);
  if (t > 200) return 1;
  const auto fill = [t](int64_t parts) {
    const int64_t n = t * parts;
    return static_cast<double>(n) / static_cast<double>((n + 255) / 256 * 256) * (1.04 - 0.04 * static_cast<double>(parts));
  };
  int64_t best = 1;
  for (int64_t parts = 2; parts <= 8 && parts * 8 <= KB; ++parts)
    if (fill(parts) > fill(best) && fill(parts) > 1.2 * fill(1)) best = parts;
  const int64_t per = (KB + best - 1) / best;
  return static_cast<int>((KB + per - 1) / per);    // none empty
}

// The same for 128 x 128 tiles: the parts that make one round of the CUs, if they fill three
// quarters of it and have 32 blocks each (a part's first loads and its sums take about ten).
int large_parts(int64_t M, int64_t N, int64_t K) {
  const int64_t t = tiles(M, N, 128, 128);
  const int64_t parts = 256 / t < 8 ? 256 / t : 8;
  return parts > 1 && t * parts >= 192 && fp8_blocks(K) / parts >= 32 ? static_cast<int>(parts) : 1;
}

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
// 128 x 128 tiles, eight waves, K in parts (whole 64 x 64 / in parts): 1692 x 927 x 22848 103 / 73,
// 600 x 2000 x 12288 41 / 31, 300 x 4000 x 16384 62 / 46, 1000 x 1500 x 16384 50 / 46.5, with 16
// blocks a part only 128 x 8192 x 8192 26 / 28.5. fp16 operands gain nothing from it.
template <bool EXACT>
hipError_t start_tiled(const ProductArgs& p, float* part, hipStream_t s) {
  const int64_t M = p.a.M, N = p.a.N, t128 = tiles(M, N, 128, 128);
  const int parts = split_parts(M, N, p.a.K);
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
    const int large = large_parts(M, N, p.a.K);
    if (large > 1) return start_split_gemm<GemmShape<128, 128, 2, 4, 4, false>>(p, large, part, s);
    // (more than 512 small tiles are a third workgroup on some CUs: 1500 x 1500 x 8192, 144 large
    // or 576 small tiles, 37 / 45)
    if (t128 >= 200 || tiles(M, N, 64, 64) > 512) return start_whole<GemmShape<128, 128, 2, 4, 4, false>>(p, s);
    if (tiles(M, N, 128, 64) >= 200 && tiles(M, N, 128, 64) <= 256)
      return start_whole<GemmShape<128, 64, 2, 2, 4, false>>(p, s);
    return start_whole<GemmShape<64, 64, 2, 2, 4, false>>(p, s);
  }
}

}  // namespace

int fp8_split_parts(int64_t M, int64_t N, int64_t K) {
  const int small = split_parts(M, N, K), large = large_parts(M, N, K);
  return small > large ? small : large;
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
  // Up to 32 rows of short K still stream; over a long K the tiled kernel in parts has more loads
  // in flight (us, streamed / tiled, 16-bit results: 25 x 1750 x 3232 5.6 / 10.2, 32 x 4096 x 4096
  // 9.4 / 10.4, 32 x 8192 x 8192 20.6 / 17.4, 24 x 4096 x 11008 19.6 / 14.0; fp32: 32 x 8192 x 8192
  // 20.5 / 22, 25 x 910 x 20864 32.7 / 18.9). The tiled kernel's offsets are 32 bits.
  const int64_t stream_k = a.ydtype == BL_F32 ? 8192 : 4096;
  if ((a.M <= 32 && a.K <= stream_k) || 256 * a.K >= (int64_t(1) << 31)) return start_codes<2>(st, s);
  return a.ydtype == BL_F32 ? start_tiled<true>(st.p, part, s) : start_tiled<false>(st.p, part, s);
}

}  // namespace bl
