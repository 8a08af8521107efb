// Tile shapes, splits and workspace layout of the feed-forward operators, shared
// by the size queries and the launches.
#pragma once
#include <algorithm>

#include "launch.hpp"

namespace coalesce {
namespace {

constexpr int DZ_COLS = 256, DZ_ROWS = 8;  // columns and row lanes of a workgroup of the dZ pass (8 columns per thread)

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// How a product runs: tile shape (1 = 256 x 256, 2 = 128 x 128, 3 = 64 x 64; of
// a gated product 128, 64 and 64 output columns) and in how many ranges its K
// steps are split.
struct TilePlan {
  int variant, splits;
  double ns;  // estimated time
};

// The plan with the smallest estimated time.  A launch is `units` workgroup
// tiles (tiles x splits); a compute unit runs up to 1, 2 or 4 (gated: 3) of
// them at once, and one K step of all of them then takes step[units per CU]
// (ns; measured over products of 512 to 16384 rows and columns, bf16).  A tile
// has a fixed cost beside its K steps (the first copies, the epilogue), a
// split product writes and reads its fp32 partial results once more (at about
// 6 TB/s, mostly caches) in a second launch; and reading the operands from memory takes its time
// too: 4.5 TB/s with three or more tiles on each compute unit, 4.0 and 3.0 with
// two and one, in proportion below.
TilePlan plan_tiles(int64_t m, int64_t n, bool gated, int batch, int64_t ksteps, int num_cus) {
  static const int slots[2][3] = {{1, 2, 4}, {1, 2, 3}};
  static const double step[2][3][4] = {{{1500}, {780, 1200}, {550, 570, 720, 850}},
                                       {{1450}, {740, 1050}, {650, 700, 950}}};
  static const double fixed[3] = {6000, 4000, 3000};
  static const int ranges[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
  const double operand_bytes = (double)ksteps * 128.0 * ((double)m + (double)n * (gated ? 2 : batch));
  TilePlan best{3, 1, 1e300};
  for (int v = 1; v <= 3; ++v) {
    const int bm = v == 1 ? 256 : v == 2 ? 128 : 64;
    const int bn = !gated ? bm : v == 1 ? 128 : 64;
    const int64_t tiles = ((m + bm - 1) / bm) * ((n + bn - 1) / bn) * batch;
    const int per_cu = slots[gated][v - 1];
    for (int splits : ranges) {
      if (splits > 1 && (v == 1 || ksteps / splits < 4)) break;
      const int64_t units = tiles * splits;
      const int64_t rounds = units / ((int64_t)num_cus * per_cu), rest = units - rounds * num_cus * per_cu;
      const int in_rest = (int)((rest + num_cus - 1) / num_cus);  // 0 .. per_cu
      double t = (double)rounds * step[gated][v - 1][per_cu - 1] + (in_rest ? step[gated][v - 1][in_rest - 1] : 0.0);
      const double load = (double)units / num_cus;
      const double gb = load >= 3 ? 4500 : load >= 2 ? 4000 : load >= 1 ? 3000 : 3000 * load;
      t = std::max(t * (double)((ksteps + splits - 1) / splits), operand_bytes / gb) +
          ((double)rounds + (in_rest > 0)) * fixed[v - 1];
      if (splits > 1) t += 4000 + (double)splits * (double)m * (double)n * (gated ? 2 : batch) * 8.0 / 6000.0;
      if (t < best.ns) best = {v, splits, t};
      if (units > 2 * (int64_t)num_cus * per_cu) break;
    }
  }
  return best;
}

// The forward's plan: the few-row kernel with strips of `strip` columns, or (0)
// a tile plan.  The few-row kernel is bound by the reading of the weights, at
// 4.8 TB/s of whole 128-byte lines (strips of 64 columns; narrower ones draw
// 1.5 and 2 times the bytes), or by what one compute unit requests: about 3.5,
// 3.0 and 2.6 ns per row of a strip, which is a line or part of one, and X's
// rows add to that.  Measured, one token: gated 4096 x 16384 58 us against 62 of
// split tiles, 2048 x 5464 16.4 (strips of 32) against 20.8, 1001 x 2736 6.7
// (16) against 11.6; but 4096 x 4096, whose 64 strips leave most compute units
// idle, 29 to 36 against 22.8.
struct ForwardPlan {
  int strip;
  TilePlan tiles;
};
ForwardPlan plan_forward(int64_t m, int64_t n, int64_t k, bool gated, int num_cus) {
  ForwardPlan f{0, plan_tiles(m, n, gated, 1, (k + 63) / 64, num_cus)};
  if (m > 64) return f;
  static const double row_ns[3] = {3.5, 3.0, 2.6}, waste[3] = {1.0, 1.5, 2.0};
  const double nb = gated ? 2.0 : 1.0;
  double best = f.tiles.ns;
  for (int i = 0; i < 3; ++i) {
    const int strip = 64 >> i;
    const int64_t strips = (n + strip - 1) / strip, rounds = (strips + num_cus - 1) / num_cus;
    const double t = 2700.0 + std::max((double)k * (double)n * 2.0 * nb * waste[i] / 4800.0,
                                       (double)rounds * (double)k * (nb + (double)m / 64.0) * row_ns[i]);
    if (t < best) {
      best = t;
      f.strip = strip;
    }
  }
  if (f.strip) f.tiles.splits = 1;
  return f;
}

// Partial results of a split product: fp32 matrices of pitch ldp, range after
// range, those of a second product (of a gated product or a batch) behind the
// first's.
int64_t partial_pitch(int64_t n) { return (n + 3) / 4 * 4; }
size_t partial_bytes(const TilePlan& t, int64_t m, int64_t n, int products) {
  if (t.splits <= 1) return 0;
  return align256((size_t)t.splits * (size_t)m * (size_t)partial_pitch(n) * 4) * (size_t)products;
}

// Row chunks of the dZ pass: about 2048 workgroups, at least 8 rows each, and
// few enough for the grid's y extent.
int dz_chunk_rows(int64_t M, int64_t N) {
  const int64_t cols = (N + DZ_COLS - 1) / DZ_COLS;
  const int64_t want = std::max<int64_t>(1, 2048 / std::max<int64_t>(1, cols));
  int64_t rows = (M + want - 1) / want;
  rows = (rows + DZ_ROWS - 1) / DZ_ROWS * DZ_ROWS;
  return (int)std::max<int64_t>(rows, DZ_ROWS);
}

struct BwdPlan {
  int64_t ldw;       // pitch of dZ in elements
  int chunk_rows, chunks;
  size_t dz_bytes;   // one dZ matrix
  size_t sums_at, partial_at, total;
  TilePlan dx, dw;   // of the two products
};
BwdPlan bwd_plan(int64_t M, int64_t N, int64_t K, bool gated, int num_cus) {
  BwdPlan b{};
  // Rows on 128-byte lines, an odd number of lines each: dZ W^T reads a 128-byte
  // piece of each of 256 rows per K step, and with a pitch of a large power of
  // two they fall on few cache channels (dZ of 8192 x 16384 in dZ W^T: 1188
  // TFLOP/s at a pitch of 32 KB, 1341 with one more line; 16 or 64 bytes more,
  // off the lines, 1148 and 1232).
  b.ldw = (N + 63) / 64 * 64;
  if (b.ldw / 64 % 2 == 0) b.ldw += 64;
  b.chunk_rows = dz_chunk_rows(M, N);
  b.chunks = (M + b.chunk_rows - 1) / b.chunk_rows;
  b.dz_bytes = align256((size_t)M * (size_t)b.ldw * 2);
  b.sums_at = b.dz_bytes * (gated ? 2 : 1);
  b.partial_at = b.sums_at + align256((size_t)b.chunks * 2 * (size_t)N * 4);
  const int products = gated ? 2 : 1;
  b.dx = plan_tiles(M, K, false, 1, products * ((N + 63) / 64), num_cus);
  b.dw = plan_tiles(K, N, false, products, (M + 63) / 64, num_cus);
  // the two products run one after the other and share the space
  b.total = b.partial_at + std::max(partial_bytes(b.dx, M, K, 1), partial_bytes(b.dw, K, N, products));
  return b;
}

}  // namespace
}  // namespace coalesce
