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

// Each workgroup quantises the rows into LDS itself.
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

// The tiled kernel's tiles and, in us, what one takes: `alone` per block of K with one workgroup
// on every CU, `shared` with `per_cu` of them (their LDS), a part `idle` of it however few CUs are
// busy, and `ends` for the start and the stores. Large tiles read less from L2 (64 x 64 tiles are
// bound by it, at 11 to 15 TB/s), small ones fill the CUs. Fitted to 1900 products measured on
// MI355X (17 to 4096 rows, 64 to 28672 columns, K of 256 to 28672, in one to eight parts of K), to
// 17 %; the tile and parts of the least estimate are on average 2 % (fp16 operands 3 %) from the
// best that was measured, at most 21 %. Some of them (256 x 256 / 256 x 128 / 128 x 128, four
// waves / 128 x 128, eight waves / 128 x 64 / 64 x 64):
//   4096 x 28672 x 8192  785 / - / 926 / - / - / -     2048 x 8192 x 8192  117 / - / 143 / 168 / 191 / -
//   192 x 28672 x 8192   103 / 72 / 80 / 84 / 101 / 112   1500 x 1500 x 8192  - / - / - / 37 / - / 45
//   512 x 8640 x 3200    - / - / 26 / 36 / 27 / 30     512 x 3200 x 8640   - / - / 57 / 38 / 31 / 33
// in parts, best (unsplit): 512 x 8192 x 28672 128 x 128 155, 256 x 256 128 with 4 (334);
//   300 x 4000 x 16384 64 x 64 62 (62), 128 x 128 46 with 2; 877 x 761 x 16384 64 x 64 29 with 3 (39)
// fp16 operands, 128 x 128 / 64 x 64: 4096 x 28672 x 8192 1545 / -, 128 x 28672 x 8192 79 / 97,
//   512 x 3200 x 8640 57 (41 with 5 parts) / 46; 96 x 8192 x 28672 78 with 4 parts (242) / 87 with 2 (133). With them
// converting the codes bounds it (a quarter-rate instruction per two of them, for each fragment
// that a wave reads); staging q as fp16 halved that and lost as much to L2.
struct Tile {
  int bn, bm, per_cu;
  float alone, shared, idle, ends;
};
constexpr Tile kTiles[] = {
    {64, 64, 2, 0.34f, 0.57f, 0.6f, 5.7f},     {128, 64, 1, 0.46f, 0.46f, 0.8f, 5.3f},
    {128, 128, 1, 0.70f, 0.70f, 0.7f, 6.1f},   {128, 128, 2, 1.00f, 1.30f, 0.5f, 7.4f},
    {256, 128, 1, 1.20f, 1.20f, 0.6f, 7.6f},   {256, 256, 1, 1.86f, 1.86f, 0.7f, 11.2f},
};
constexpr Tile kExactTiles[] = {{64, 64, 3, 0.54f, 0.95f, 0.6f, 5.0f}, {128, 128, 2, 1.40f, 1.90f, 0.5f, 12.0f}};

// Tiles run in rounds of 256 per_cu. Those of the last round, from `whole` on, may have K in parts:
// up to eight of at least six blocks, if they are then still one round. Their sums cost a launch
// and the partial sums' way to memory and back. Without / with the last round in parts:
// 1477 x 11045 x 15264 (264 tiles of 256 x 256) 438 / 311, 768 x 28672 x 8192 225 / 194.
struct Plan {
  int tile, parts, whole;
  int64_t part_bytes;
};
template <size_t N_TILES>
Plan make_plan(const Tile (&list)[N_TILES], int64_t M, int64_t N, int64_t K) {
  const int KB = static_cast<int>(fp8_blocks(K));
  Plan best{0, 1, 0, 0};
  float least = 0;
  for (int i = 0; i < static_cast<int>(N_TILES); ++i) {
    const Tile& t = list[i];
    const int64_t n = tiles(M, N, t.bn, t.bm), round = 256 * t.per_cu, full = n / round, rest = n - full * round;
    const float used = static_cast<float>(M) / static_cast<float>((M + t.bm - 1) / t.bm * t.bm);   // of its rows
    for (int parts = 1; parts <= 8; ++parts) {
      if (parts > 1 && (rest == 0 || rest * parts > round || KB < 6 * parts)) break;
      const int steps = (KB + parts - 1) / parts;
      if ((KB + steps - 1) / steps != parts) continue;   // the last part would be empty
      const float load = static_cast<float>(rest * parts) / 256;   // of the last round, per CU
      const float step = load <= 1 ? t.alone * (t.idle + (1 - t.idle) * load)
                                   : t.alone + (t.shared - t.alone) * (load - 1) / static_cast<float>(t.per_cu - 1);
      const int64_t bytes = parts > 1 ? rest * parts * t.bn * t.bm * 4 : 0;
      float us = static_cast<float>(full) * (static_cast<float>(KB) * t.shared + t.ends);
      if (load > 0) us += static_cast<float>(steps) * step + t.ends;
      if (parts > 1) us += 3.7f + static_cast<float>(bytes) * used * 2e-7f;
      if ((i == 0 && parts == 1) || us < least) {
        least = us;
        best = Plan{i, parts, static_cast<int>(full * round), bytes};
      }
    }
  }
  return best;
}

template <class S>
hipError_t start_plan(const ProductArgs& p, const Plan& plan, float* part, hipStream_t s) {
  ProductArgs q = p;
  q.whole = plan.whole;
  q.parts = plan.parts;
  q.part = part;
  return plan.parts > 1 ? start_split_gemm<S>(q, s) : start_gemm<S>(q, (p.a.M + S::BM - 1) / S::BM, s);
}

template <bool EXACT>
hipError_t start_tiled(const ProductArgs& p, float* part, hipStream_t s) {
  if constexpr (EXACT) {
    const Plan q = make_plan(kExactTiles, p.a.M, p.a.N, p.a.K);
    if (q.tile == 1) return start_plan<GemmShape<128, 128, 2, 2, 2, true>>(p, q, part, s);
    return start_plan<GemmShape<64, 64, 2, 2, 3, true>>(p, q, part, s);
  } else {
    const Plan q = make_plan(kTiles, p.a.M, p.a.N, p.a.K);
    switch (q.tile) {
      case 0: return start_plan<GemmShape<64, 64, 2, 2, 4, false>>(p, q, part, s);
      case 1: return start_plan<GemmShape<128, 64, 2, 2, 4, false>>(p, q, part, s);
      case 2: return start_plan<GemmShape<128, 128, 2, 4, 4, false>>(p, q, part, s);
      case 3: return start_plan<GemmShape<128, 128, 2, 2, 2, false>>(p, q, part, s);
      case 4: return start_plan<GemmShape<256, 128, 2, 4, 3, false>>(p, q, part, s);
      default: return start_plan<GemmShape<256, 256, 2, 4, 2, false>>(p, q, part, s);
    }
  }
}

}  // namespace

int64_t fp8_part_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 16) return 0;                            // streamed
  const int64_t a = make_plan(kTiles, M, N, K).part_bytes, b = make_plan(kExactTiles, M, N, K).part_bytes;
  return a > b ? a : b;
}

hipError_t launch_fp8_linear(const Fp8LinearArgs& a, const void* x, int xdtype, int64_t ldx, float* part,
                             hipStream_t s) {
  StreamArgs st{};
  st.p.a = a;
  st.x = x;
  st.ldx = ldx;
  // Few short rows: every workgroup quantises them itself, in one launch for two (us, this way /
  // with the quantiser's launch: 16 x 8192 x 1792 11.5 / 14.1, 8 x 8192 x 3584 12.1 / 14.1), up to
  // where more than four rows hold up long streams (16 x 28672 x 1792 15.6 / 14.2, 8 x 28672 x 3584
  // 21.9 / 20.7). Their codes and the reduction's 32 KB stay within 64 KB of LDS.
  if (x && a.M <= 16 && (a.M <= 4 || a.N * a.K <= (int64_t(1) << 25)) &&
      a.K <= 32768 && staged_bytes(static_cast<int>(a.M), static_cast<int>(fp8_blocks(a.K))) <= 32768)
    return start_values(st, xdtype, s);
  if (x) {
    const hipError_t e = launch_fp8_quant_act(x, xdtype, a.M, a.K, ldx, 0, nullptr, const_cast<uint8_t*>(a.q),
                                              const_cast<float*>(a.sx), s);
    if (e != hipSuccess) return e;
  }
  if (a.M <= 16) return start_codes<1>(st, s);
  // Up to 32 rows of short K still stream; over a long K the tiled kernel in parts has more loads
  // in flight (us, streamed / tiled, bf16 results: 25 x 1750 x 3232 5.6 / 10.2, 32 x 4096 x 4096
  // 9.4 / 10.4, 32 x 8192 x 8192 20.6 / 17.4, 24 x 4096 x 11008 19.6 / 14.0; fp16 operands: 32 x 8192 x 8192
  // 20.5 / 22, 25 x 910 x 20864 32.7 / 18.9). The tiled kernel's offsets are 32 bits.
  const bool exact = a.ydtype != BL_BF16;
  const int64_t stream_k = exact ? 8192 : 4096;
  if ((a.M <= 32 && a.K <= stream_k) || 256 * a.K >= (int64_t(1) << 31)) return start_codes<2>(st, s);
  return exact ? start_tiled<true>(st.p, part, s) : start_tiled<false>(st.p, part, s);
}

}  // namespace bl
