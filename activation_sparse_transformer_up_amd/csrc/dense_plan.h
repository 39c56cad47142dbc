// How the dense layers' products are cut up: their kinds, the tiles of each, the tile and the split of k that a
// product of given sizes takes. Host code only, apart from the kernels, so that it can be asked without a GPU.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace tw {
namespace {

// Kinds of products, and the tiles of each. Large tiles have the least traffic per operation, one workgroup
// of 8 waves per CU; the others are for products that large tiles would leave CUs idle in. Few rows make a
// product a stream of its weights, which needs many loads in flight per CU more than anything: the narrow
// tiles' rings keep 28 KB of weights per workgroup in flight (two per CU along k), the deep ones' 80 KB.
enum { kAlong, kAcross, kBoth };            // both operands along k; A across; both across
enum { kSmall, kMid, kLarge, kNarrow, kDeep };

constexpr int kCUs = 256;
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t kPartBytes = (int64_t)256 << 20;        // partial sums of one product
struct Tile { int m, n, wn; };              // columns, rows, rows of a wave
Tile tile_of(bool wide, int kind, int c, bool dual) {      // wide: bf16 operands or planes
  if (!wide) return c == kNarrow ? Tile{128, 32, 32} : Tile{64, 64, 32};
  if (kind == kAlong)
    return c == kSmall ? Tile{64, 64, 32} : c == kMid ? Tile{128, 128, 64} : c == kLarge ? Tile{256, 256, 64}
                                                                                      : Tile{dual ? 64 : 32, 32, 16};
  return c == kLarge ? Tile{256, 256, 128} : c == kMid ? Tile{256, 128, 64} : c == kNarrow ? Tile{64, 64, 16} : Tile{256, 64, 64};
}

// Nanoseconds of `tiles` tiles over `stages` stages: rounds of resident workgroups, each with its stages (all
// workgroups of a CU together; `alone` where at most half the places are taken) and its start and epilogue. Measured
// with every tile and split forced (us, x w of T x K by N; along k small / mid / large, across it small / mid /
// large, one split): 1000 x 2048 by 8192: 54 / 34 / 42, 45 / 36 / 44; 4096 x 2048 by 8192: 202 / 128 / 109, 171 / 141 /
// 106; 2048 x 4096 by 4096 across: 87 / 65 / 79; 1000 x 8192 by 2048 in four splits: 60 / 43 / 55, 60 / 46 / 57. Few rows
// (small / narrow): 1 x 4096 by 14336 along k 26.2 / 23.3, 64 rows 28.4 / 40; across it, 64 x 14336 by 4096 in 256
// workgroups: small 38, narrow 37, deep 31; one row small 34, narrow 25, deep 26. fp32 as it is / in planes: 2048 x
// 2048 by 2048 146 / 116, 4096 x 2048 by 2048 276 / 193, 2255 x 1648 by 6120 388 / 275, 997 x 1000 by 5456 (dual) 122 / 142.
struct Cost {
  int per_cu, stage, alone, start;
  bool turns = false;                       // by cost_of
};
constexpr Cost kCostAlong[4] = {{2, 330, 210, 2000}, {2, 840, 460, 4000}, {1, 1400, 1080, 8000}, {2, 270, 160, 1500}};     // 64-k stages
constexpr Cost kCostAcross[3] = {{2, 600, 590, 4500}, {1, 460, 390, 5000}, {1, 740, 530, 8000}};                        // 32-k stages
constexpr Cost kCostBoth[3] = {{2, 680, 620, 3500}, {}, {1, 740, 540, 8000}};
constexpr Cost kCostF = {3, 540, 690, 2000, true};                                  // fp32 as it is: 32-k stages
// fp32, 128 x 32: two per CU. 32 x 13768 by 6720, 53 tiles in 4 / 6 / 8 / 12 / 24 splits: 88 / 113 / 94 / 102 / 94 us, the
// 64 x 64 tile 102 / 110 / 118 / 101 / 105; 32 x 14336 by 4096 in 1 / 4 / 8 / 16: 295 / 82 / 50 / 51, 64 x 64 298 / 83 / 50 / 61; one
// row, where both wait for w, 191 / 57 / 45 / 46 and 193 / 56 / 45 / 51.
constexpr Cost kCostFew = {2, 1600, 720, 2000};
constexpr int kJoin = 6000;                 // the launch that adds partial sums, the host's part among it
constexpr double kStream = 5500;            // bytes per nanosecond from HBM
int64_t cost_of(const Cost &c, int64_t tiles, int64_t stages) {
  // turns: fp32 as it is, three 64 x 64 tiles per CU: the matrix instructions of a CU's workgroups take turns, whatever their rounds
  // (1000 x 2728 by 1000, 256 tiles, in 1 / 2 / 3 splits: 65 / 60 / 58 us; 300 x 8192 by 1024, 80 tiles, in 1 / 3 / 6: 176 / 66 / 58)
  if (c.turns) return stages * (c.stage * ceil_div(tiles, kCUs) + c.alone - c.stage) + c.start;
  const int64_t slots = kCUs * c.per_cu, left = tiles % slots;
  double more = left * 2 > slots ? (double)(left * 2 - slots) / slots : 0.0;
  if (c.per_cu > 1 && more > 0.0) more = 0.75 + 0.25 * more;          // some CUs have two: the others wait for them
  return tiles / slots * (stages * c.stage + c.start) +
         (left ? (int64_t)(stages * (c.alone + (c.stage - c.alone) * more)) + c.start : 0);
}

struct Split {
  int cls, S, ks;
  bool planes;                              // fp32 operands split into bf16 planes
  size_t part, ws;                          // bytes of the partial sums, and with them of the planes
};
// The tile and the split of k (1 to 64 times) of a product with the least cost. M columns (of each
// matrix of a dual A), K over all segments.
Split split_of(bool bf16, int kind, bool dual, int M, int N, int64_t K, int batch) {
  const int du = dual ? 2 : 1;
  Split best = {};
  int64_t least = 0;
  const int64_t elements = ((int64_t)M * du + N) * K * batch;
  const int64_t stream = (int64_t)((double)elements * (bf16 ? 2 : 4) / kStream);
  // np: products of planes; more: the launches that make them
  auto consider = [&](int c, const Cost &cost, int np = 1, int64_t more = 0) {
    const bool wide = bf16 || np > 1;
    const Tile t = tile_of(wide, kind, c, dual);
    const int ks = kind == kAlong && wide ? 64 : 32;
    const int64_t tiles = ceil_div((int64_t)M * du, t.m) * ceil_div(N, t.n) * batch;
    for (int S0 = 1; S0 <= 64; S0 += S0 < 8 ? 1 : S0 / 8 * 2) {
      const int64_t size = ceil_div(ceil_div(K, S0), 64) * 64, S = ceil_div(K, size);
      const int64_t part = S > 1 ? S * batch * N * M * du * 4 : 0;
      if (S0 > 1 && (tiles * S > kCUs * cost.per_cu || part > kPartBytes)) break;
      if (S < S0) continue;
      int64_t n = cost_of(cost, tiles * S, ceil_div(size, ks) * np);
      n = (n > stream ? n : stream) + (S > 1 ? kJoin + part / 5000 : 0) + more;
      if (least && n * 100 >= least * 97) continue;       // near ties go to the earlier tile and fewer splits
      least = n;
      best = {c, (int)S, (int)size, np > 1, (size_t)ceil_div(part, 256) * 256, 0};
    }
  };
  if (!bf16) {
    consider(kSmall, kCostF);
    if (kind == kAlong && N <= 32) consider(kNarrow, kCostFew);
    // planes: six products of twice the bytes, 10 bytes moved per element before them
    if (N > 128) {
      const int64_t more = 16000 + elements * 10 / 5000;
      const Cost *const cost = kind == kAlong ? kCostAlong : kind == kAcross ? kCostAcross : kCostBoth;
      consider(kLarge, cost[kLarge], 6, more);
      if (kind != kBoth) consider(kMid, cost[kMid], 6, more);
    }
  } else if (kind == kAlong) {
    if (N <= 64) consider(kNarrow, kCostAlong[kNarrow]);
    consider(kLarge, kCostAlong[kLarge]);
    consider(kMid, kCostAlong[kMid]);
    consider(kSmall, kCostAlong[kSmall]);
  } else if (kind == kAcross && N <= 64) {
    const int rows = N;                     // the rows' share of a stage
    consider(kNarrow, {1, 165 + rows * 7 / 5, 165 + rows * 7 / 5, 1500});
    consider(kDeep, {1, 680 + rows * 9 / 4, 680 + rows * 9 / 4, 2500});
  } else if (kind == kAcross) {
    consider(kLarge, kCostAcross[kLarge]);
    consider(kMid, kCostAcross[kMid]);
    consider(kSmall, kCostAcross[kSmall]);
  } else {
    consider(kLarge, kCostBoth[kLarge]);
    consider(kSmall, kCostBoth[kSmall]);
  }
  best.ws = best.part + (best.planes ? (size_t)ceil_div(elements * 6, 256) * 256 + 2048 : 0);
  return best;
}

// Rows of a strip of k_dense_rows; join: over partial sums of k. For column sums few strips, whose sums a further
// launch adds; one strip, without that launch, up to 256 rows (128 of a join, whose rows cost as many reads as there
// are splits). One strip's workgroups take 64 columns, where those of 256 would not be one per CU. us on the GPU, one
// strip of 256 columns a workgroup / of 64 / strips of 8 rows: db of 128 x 1024, bf16 gelu 8.5 / 4.0 / 5.7, fp32 gelu 21 / 7.1 /
// 6.4, fp32 relu 6.7 / 3.6 / 5.6; 256 x 14336, bf16 gelu 15 / 6.1 / 11, fp32 40 / 13 / 14; 256 x 60000 20 / 18 / 24 and 47 / 33 /
// 36; 16 rows 4.7 / 4.7 / 5.5. Gated backward with biases, joins of splits: fp32 64 x 1024 x 4096 70 / 63 / 64, 128 x 1000 x 2728
// 104 / 83 / 80 (the host's part of a launch is 4), 200 x 4096 x 1024 173 / 142 / 135, 256 x 4096 x 2048 298 / 271 / 263.
int strip_of(int N, bool sums, bool join) {
  if (sums && N <= (join ? 128 : 256)) return (int)(ceil_div(N, 8) * 8);
  const int64_t r = ceil_div(N, sums ? 64 : 1024);
  return (int)(ceil_div(r, 8) * 8);
}
int row_strips(int N, bool sums, bool join) { return (int)ceil_div(N, strip_of(N, sums, join)); }
// Whether a single strip's workgroups take 64 columns of M.
bool narrow_strip(int N, int M, bool join) { return row_strips(N, true, join) == 1 && N > 16 && ceil_div(M, 256) < kCUs; }

// Blocks of column sums that a product's epilogue leaves.
int sum_blocks(bool bf16, int kind, const Split &p, int N) {
  if (p.S > 1) return 4 * row_strips(N, true, true);
  const Tile t = tile_of(bf16 || p.planes, kind, p.cls, false);
  return (int)(ceil_div(N, t.n) * (t.n / t.wn));
}

}  // namespace
}  // namespace tw
