// How a product grouped by expert is cut into workgroups: tile shape and parts of the reduction, from the sizes alone.
// Host code without HIP, so that a test can ask which kernel a call takes.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace moe {

// Output tile rows are rows of the groups (kForward, kRows) or of the weight matrices (kWeights).
enum : int { kForward = 0, kRows = 1, kWeights = 2 };

struct GroupSizes {
  int n_groups, rows;  // rows: most of all groups
  int64_t w_stride;    // elements per matrix
  int cols;            // output columns
  int red;             // reduction length (kForward, kRows)
  int out_rows;        // rows of an output matrix (kWeights)
};

inline GroupSizes group_sizes(int dir, int n_groups, int rows, int N, int K) {
  GroupSizes p{};
  p.n_groups = n_groups;
  p.rows = rows;
  p.w_stride = static_cast<int64_t>(N) * K;
  p.cols = dir == kForward ? N : K;
  p.red = dir == kForward ? K : N;
  p.out_rows = N;
  return p;
}

namespace groups {

// Tile shapes, and what a call of each is expected to take, in us, as measured over sizes from one tile to thousands:
// `call` once; per tile and CU `ends` (first loads, last products, stores) and, per 64 indexes of a bf16 reduction (32
// of an fp32 one), `alone` where a CU has one tile at a time and `full` where its other tiles fill the gaps, of kForward,
// kRows and kWeights, which read none, one and both of their operands across; and no less than the matrices at the
// TB/s that kForward and kRows stream them with.  Over 150 calls, from one row to 2^28 weights, the shape and parts
// chosen here take 4 % longer than the best of all, as a geometric mean.  Two calls as examples, 64 groups of 512 rows,
// 1024 x 4096: kForward kWide 342, kBig 316 us; kRows, whose many short tiles leave kBig's stores uncovered, 363, 390.
struct Shape {
  int bm, bn;
  double call, ends, alone[3], full[3], forward, rows;
};
enum : int { kSmall, kNarrow, kMiddle, kWide, kBig, kFew, kShapes };
constexpr Shape kBf16Shapes[kShapes] = {
    {64, 64, 4.0, 0.9, {0.26, 0.26, 0.34}, {0.21, 0.21, 0.21}, 5.5, 5.4},
    {64, 128, 4.5, 1.2, {0.38, 0.38, 0.49}, {0.34, 0.34, 0.30}, 5.2, 5.9},
    {128, 128, 5.0, 2.0, {0.53, 0.53, 0.65}, {0.55, 0.55, 0.42}, 4.4, 5.5},
    {128, 256, 5.0, 3.0, {0.66, 0.66, 1.00}, {1.05, 1.05, 0.80}, 4.2, 6.6},
    {256, 256, 6.0, 3.0, {1.40, 1.44, 1.47}, {1.40, 1.44, 1.47}, 4.1, 5.2},
    {32, 64, 4.0, 0.9, {0.21, 0.21, 0.21}, {0.19, 0.19, 0.19}, 6.3, 5.5}};
constexpr Shape kF32Shapes[2] = {{64, 64, 4.0, 1.0, {0.55, 0.55, 0.55}, {0.50, 0.50, 0.50}, 5.5, 5.4},
                                 {64, 128, 4.5, 1.5, {1.00, 1.00, 1.00}, {0.95, 0.95, 0.95}, 5.2, 5.9}};

struct Plan {
  int shape, parts, high;
  int64_t blocks;
};

constexpr double kCus = 256;
constexpr int kMaxTileRows = (1 << 25) - 1;  // of kForward and kRows: 64 lanes' counts add up in 32 bits
constexpr int64_t kPartialBytes = 64 << 20;  // most that the parts of a call take of a workspace

// Shape, parts of the reduction and most workgroups of a call: the least of what the shapes are expected to take,
// where groups share the rows evenly, whole or in parts that a second launch adds up.
inline Plan plan(int dir, const GroupSizes& p, bool f32, bool out_f32) {
  const int shapes = f32 ? 2 : dir == kWeights ? kFew : kShapes;
  const int step = f32 ? 32 : 64, order = dir == kForward ? 0 : dir == kRows ? 1 : 2;
  const double busy = std::max(1.0, std::min<double>(p.n_groups, p.rows)), avg = p.rows / busy;
  // groups are seldom of one size, and the largest one's sum is what a call waits for: 33 us of a call of 16 groups of
  // very unequal sizes, 4903 rows in all, into 40 x 648 in one part, 19 in eight
  const double red = dir == kWeights ? std::min<double>(p.rows, 2.0 * avg) : p.red;
  const double out_rows = dir == kWeights ? static_cast<double>(p.n_groups) * p.out_rows : p.rows;
  const double steps = std::max(1.0, std::ceil(red / step));
  const double matrices = busy * p.w_stride * (f32 ? 4 : 2);
  Plan best{};
  double least = 0;
  for (int i = 0; i < shapes; ++i) {
    const Shape& h = f32 ? kF32Shapes[i] : kBf16Shapes[i];
    if (dir != kWeights && p.rows / h.bm + p.n_groups > kMaxTileRows) continue;  // 2^30 rows in the shortest tiles
    const double nt = std::ceil(static_cast<double>(p.cols) / h.bn);
    // a group's rows end inside a tile
    const double mt = dir == kWeights ? p.n_groups * std::ceil(static_cast<double>(p.out_rows) / h.bm)
                      : busy == 1 || avg <= h.bm * 0.75 ? busy * std::ceil(avg / h.bm) : busy * (avg / h.bm + 0.5);
    // rows that are not there are neither read nor multiplied
    const double used = dir == kWeights ? 1.0 : 0.6 + 0.4 * std::min(1.0, avg / h.bm);
    for (int parts = 1; parts <= 16; parts *= 2) {
      const double partial = out_rows * p.cols * 4 * parts;
      if (parts > 1 && (steps / parts < 4 || partial > kPartialBytes)) break;
      const double tiles = mt * nt * parts / kCus;  // of a CU
      // the one tile of a CU stores its values, and reads some to add, with nothing beside it: 20 GB/s a CU
      const double stores = i == kBig && !f32 ? h.bm * h.bn * (out_f32 ? 4 : 2) * 1.5 / 20e3 : 0.0;
      const double one = std::ceil(steps / parts) * h.alone[order] * used + h.ends + stores;
      const double full = std::ceil(steps / parts) * h.full[order] * used + h.ends;
      double us = h.call + std::max(one, i == kBig && !f32 ? std::ceil(tiles) * one : tiles * full);
      if (dir != kWeights) us = std::max(us, matrices / (dir == kForward ? h.forward : h.rows) / 1e6);
      if (parts > 1) us += 2.0 + partial * 2 / 8e6;
      if (best.parts == 0 || us < least) {
        least = us;
        best.shape = i;
        best.parts = parts;
      }
    }
  }
  const Shape& h = f32 ? kF32Shapes[best.shape] : kBf16Shapes[best.shape];
  const int64_t nt = (p.cols + h.bn - 1) / h.bn;
  const int64_t mt = dir == kWeights
                         ? static_cast<int64_t>(p.n_groups) * ((p.out_rows + h.bm - 1) / h.bm)
                         : (static_cast<int64_t>(p.rows) + static_cast<int64_t>(p.n_groups) * (h.bm - 1)) / h.bm;
  best.high = h.bm;
  best.blocks = mt * nt * best.parts;
  return best;
}

}  // namespace groups

}  // namespace moe
