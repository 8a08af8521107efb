// Tile shapes, splits and workspace layout of the feed-forward operators, shared
// by the size queries and the launches.
#pragma once
#include <algorithm>

#include "launch.hpp"

namespace coalesce {
namespace {

constexpr int DZ_COLS = 256, DZ_ROWS = 8;  // columns and row lanes of a workgroup of the dZ pass (8 columns per thread)

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// How a product runs: tile shape and in how many ranges its K steps are split.
struct TilePlan {
  int variant, splits;
  double ns;  // estimated time
};

// The compiled tile shapes (gemm16_core.hpp): rows, columns (of each matrix of
// a gated product), how many a compute unit holds, the time of one K step with
// 1, 2, ... of them on every compute unit, and the time a launch and a round of
// tiles take beside their K steps.  Measured in ns over products of 256 to 8192
// rows, bf16.  A step is bound by the matrix cores at 256 rows and more and more
// by the caches below (a 160-row tile draws 0.77 of the bytes per step for 0.63
// of the products), so the lower ones pay only where they fit the rows or fill
// the compute units better: gated 777 x 5461 x 2048 57.8 us in 256 rows, 48.5 in
// 160; 3000 x 4096 x 4096 180 in 256, 163 in 192.  Those lower than 256 exist
// where the m side lies along the contraction; 160 rows and the shapes called deep
// have three stages, which pays where a compute unit holds few tiles (bf16 with a
// bf16 residual: 64 x 64, 512 x 4096 x 4096 37.2 us without them, 30.4 with; 128 x
// 128, 2048 x 2048 x 4096 55.5 and 48.2).  The gated product has no deep ones.
struct TileShape {
  int bm, bn, slots;
  double step[4], launch, round;
};
constexpr int kShapes = 8, kShape256 = 1, kShape128 = 2, kShape64 = 3, kShape224 = 4, kShape192 = 5, kShape160 = 6,
              kShape64Deep = 7, kShape128Deep = 8;
static const TileShape kPlain[kShapes] = {
    {256, 256, 1, {1450}, 4000, 5000},          {128, 128, 2, {780, 1200}, 3000, 2000},
    {64, 64, 4, {430, 520, 700, 850}, 3000, 1500}, {224, 256, 1, {1290}, 4000, 5000},
    {192, 256, 1, {1180}, 4000, 5000},          {160, 256, 1, {1010}, 4000, 5000},
    {64, 64, 3, {380, 440, 700}, 3000, 1500},
    {128, 128, 1, {600}, 4000, 5000}};
static const TileShape kGated[kShapes] = {
    {256, 128, 1, {1450}, 4000, 5000}, {128, 64, 2, {740, 1050}, 3000, 2000}, {64, 64, 3, {600, 680, 950}, 3000, 1500},
    {224, 128, 1, {1290}, 4000, 5000}, {192, 128, 1, {1180}, 4000, 5000},     {160, 128, 1, {1010}, 4000, 5000},
    {64, 64, 0, {0}, 0, 0},            {128, 64, 0, {0}, 0, 0}};

// The plan with the smallest estimated time.  A launch is `units` workgroup
// tiles (tiles x splits), run in rounds of what the compute units hold.  A split
// product (128 x 128 or 64 x 64 tiles) writes and reads its fp32 partial results
// once more, at about 6 TB/s, mostly caches, in a second launch; and reading the
// operands from memory takes its time too: 4.5 TB/s with three or more tiles on
// each compute unit, 4.0 and 3.0 with two and one, in proportion below.  `rows`:
// the m side lies along the contraction, every shape may be used.
TilePlan plan_tiles(int64_t m, int64_t n, bool gated, int batch, int64_t ksteps, bool rows, int num_cus) {
  static const int ranges[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
  const double operand_bytes = (double)ksteps * 128.0 * ((double)m + (double)n * (gated ? 2 : batch));
  TilePlan best{kShape64, 1, 1e300};
  for (int v = 1; v <= kShapes; ++v) {
    const TileShape& s = gated ? kGated[v - 1] : kPlain[v - 1];
    if (s.slots == 0 || (!rows && (v == kShape224 || v == kShape192 || v == kShape160))) continue;
    const int64_t tiles = ((m + s.bm - 1) / s.bm) * ((n + s.bn - 1) / s.bn) * batch;
    for (int splits : ranges) {
      if (splits > 1 && ((v != kShape128 && v != kShape64 && v != kShape128Deep) || ksteps / splits < 4)) break;
      const int64_t units = tiles * splits, full = (int64_t)num_cus * s.slots;
      const int64_t rounds = units / full, rest = units - rounds * full;
      // the last round's step: between the times of the tile counts around its
      // load (the compute units share the caches, so the ones with a tile more
      // are not the slower for it)
      const double x = (double)rest / num_cus;
      const int i = std::min(std::max((int)x, 1), s.slots);
      const double last = rest == 0 ? 0.0 : i < s.slots && x > i ? s.step[i - 1] + (x - i) * (s.step[i] - s.step[i - 1])
                                                                 : s.step[i - 1];
      double t = (double)rounds * s.step[s.slots - 1] + last;
      const double load = (double)units / num_cus;
      const double gb = load >= 3 ? 4500 : load >= 2 ? 4000 : load >= 1 ? 3000 : 3000 * load;
      t = std::max(t * (double)((ksteps + splits - 1) / splits), operand_bytes / gb) + s.launch +
          ((double)rounds + (rest > 0)) * s.round;
      if (splits > 1) t += 4500 + (double)splits * (double)m * (double)n * (gated ? 2 : batch) * 8.0 / 6000.0;
      if (t < best.ns) best = {v, splits, t};
      if (units > 2 * full) break;
    }
  }
  return best;
}

// The forward's plan: the few-row kernel with strips of `strip` columns, or (0)
// a tile plan.  The few-row kernel is bound by the reading of the weights, at
// 4.8 TB/s of whole 128-byte lines (strips of 64 columns; narrower ones draw
// 1.5 and 2 times the bytes), or by what one compute unit requests: about 3.5,
// 3.0 and 2.6 ns per row of a strip, which is a line or part of one, and X's
// rows add to that.  Measured, one token: gated 4096 x 16384 55 us against 60 of
// split tiles, 2048 x 5464 16.4 (strips of 32) against 20.8, 1001 x 2736 6.7
// (16) against 11.6; but 4096 x 4096, whose 64 strips leave most compute units
// idle, 29 to 36 against 22.8.
struct ForwardPlan {
  int strip;
  TilePlan tiles;
};
ForwardPlan plan_forward(int64_t m, int64_t n, int64_t k, bool gated, int num_cus) {
  ForwardPlan f{0, plan_tiles(m, n, gated, 1, (k + 63) / 64, true, num_cus)};
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
  b.dx = plan_tiles(M, K, false, 1, products * ((N + 63) / 64), true, num_cus);
  b.dw = plan_tiles(K, N, false, products, (M + 63) / 64, false, num_cus);
  // the two products run one after the other and share the space
  b.total = b.partial_at + std::max(partial_bytes(b.dx, M, K, 1), partial_bytes(b.dw, K, N, products));
  return b;
}

}  // namespace
}  // namespace coalesce
