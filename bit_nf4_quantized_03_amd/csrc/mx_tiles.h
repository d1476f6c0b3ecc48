// The rule that chooses the tile of a large microscaled product. Host code
// without any of HIP's.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace qnf4 {

inline int64_t mx_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tiles, and what a step of 128 elements costs with them in us: `light` for
// a workgroup while few compute units work, `full` on every compute unit (there
// per workgroup). `shared`: a compute unit holds two workgroups or more. All
// measured at K = 4096, N = 4096 (first an 8-bit X, then 4 bits).
//
// Large tiles re-read their operands less, small ones leave fewer compute units
// without work, so the tile is chosen by the time that these figures give.
// Times behind the rule (us, 8-bit X, N = K = 4096; its choice first): 4096
// rows 256 x 256 54, 256 x 128 61, 128 x 128 66; 2048 rows 256 x 128 32, 128 x
// 128 35, 256 x 256 43; 1000 rows 128 x 128 19, 128 x 64 23, 256 x 128 24; 301
// rows 128 x 64 12.3, 128 x 128 15.7, 64 x 64 17.3; 128 rows 64 x 64 9.6, 128 x
// 64 11.8. The 64 x 64 tile has two groups of waves with half the steps each
// and four stages: one workgroup fills a compute unit, but it is chosen where
// there is no second (with three stages, two to a unit, 128 rows 10.3; one
// group 11.6; 128 x 64 in two groups 12.2).
constexpr int kMxTiles = 5;
constexpr struct {
  int bn, bm, threads;
  bool shared;
  struct {
    double light, full;
  } cost[2];
} kMxTile[kMxTiles] = {{256, 256, 512, false, {{1.03, 1.53}, {0.61, 1.05}}},
                       {256, 128, 512, false, {{0.54, 0.88}, {0.41, 0.64}}},
                       {128, 128, 256, true, {{0.33, 0.47}, {0.29, 0.36}}},
                       {128, 64, 256, true, {{0.205, 0.305}, {0.19, 0.25}}},
                       {64, 64, 512, false, {{0.14, 0.185}, {0.12, 0.165}}}};
constexpr double kMxCus = 256;

// Workgroups of a launch. By expert, where the counts are on the GPU, as many
// as the rows can ask for: an expert's end in at most one partial tile.
inline int64_t mx_tile_groups(int bm, int bn, int64_t M, int64_t N, int experts) {
  return (experts ? M / bm + experts : mx_ceil(M, bm)) * mx_ceil(N, bn);
}

// The tile with the least cost. Its launch stays below 2^32 threads for every
// size that the entry points take (M and N up to 2^24, M N to 2^37, W's rows to
// 2^28): not because every tile's would, the 64 x 64 one reaches 2^34, but
// because the smaller tiles are dearer wherever there is that much work.
inline int mx_choose_tile(int64_t M, int64_t N, int experts, bool fp4) {
  int best = 0;
  double least = 0;
  for (int i = 0; i < kMxTiles; ++i) {
    const double tiles_n = static_cast<double>(mx_ceil(N, kMxTile[i].bn));
    double tiles_m = static_cast<double>(mx_ceil(M, kMxTile[i].bm)), spare = 0;
    if (experts) {
      // an expert's rows end in a partial tile, on average half of one; the
      // counts are on the GPU, and `spare` allows for a few more
      tiles_m = std::max(static_cast<double>(M) / kMxTile[i].bm + 0.5 * experts,
                         static_cast<double>(std::min<int64_t>(M, experts)));
      spare = 0.1;
    }
    const double load = tiles_m * tiles_n / kMxCus + spare;   // workgroups per compute unit
    const double light = kMxTile[i].cost[fp4].light, full = kMxTile[i].cost[fp4].full;
    double t;
    if (load <= 1) t = light + (full - light) * load;
    else t = full * (kMxTile[i].shared ? (load + std::ceil(load)) / 2 : std::ceil(load));
    if (i == 0 || t < least) least = t, best = i;
  }
  return best;
}

}  // namespace qnf4
