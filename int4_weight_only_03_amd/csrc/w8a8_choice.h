// Tiles of the 8-bit products' tile kernel: which sizes there are and which of them a call
// takes.  Host code, without HIP.
#pragma once

#include <algorithm>
#include <cmath>

#include "launch_limits.h"

namespace w4a16 {
namespace {

// R rows of one expert, or R slots over E of them (grouped)
struct TileCall {
  long R, E, N, K;
  bool grouped;
};

// Tiles of `slots` x `rows`, and the time of a launch in which every compute unit has one
// (us, 56 blocks of K) or `per_cu` of them, by measurement.
struct Choice {
  int slots, rows, per_cu;
  double one, all;
  int waves;  // of a workgroup
};
constexpr Choice kChoices[] = {
    {16, 32, 1, 7.7, 7.7, 8},      // 4 groups of waves over K, 4 images
    {32, 32, 1, 9.2, 9.2, 16},     // the same
    {32, 64, 1, 12.3, 12.3, 8},    // 2 groups, 4 images
    {64, 64, 1, 16.8, 16.8, 8},    // the same
    {64, 64, 2, 19.6, 30.0, 4},    // 4 images
    {64, 128, 1, 25.0, 25.0, 4},   // 4 images
    {128, 128, 1, 39.2, 39.2, 4},  // 4 images
    {128, 128, 2, 49.0, 66.0, 4},  // 2 images
    {256, 256, 1, 100.0, 100.0, 8},
};
constexpr Choice kExactChoices[] = {  // fp32 outputs: no more registers for larger tiles
    {16, 32, 1, 9.5, 9.5, 8},    {32, 32, 1, 12.0, 12.0, 16}, {32, 64, 1, 18.0, 18.0, 8},
    {64, 64, 1, 23.5, 23.5, 8},  {64, 64, 2, 31.3, 40.0, 4},  {128, 128, 2, 66.0, 110.0, 4},
};

// Workgroups of a launch, and the most that its grid takes (2^32 threads; dealt to 8 XCDs).
inline long tiles_of(int slots, int rows, const TileCall &p, long R) {
  const long items = p.grouped ? max_items(R, p.E, slots) : (R + slots - 1) / slots;
  return items * ((p.N + rows - 1) / rows);
}
inline long most_tiles(int waves) { return kMaxBlocks * 4 / waves - 8; }

// Time of a choice: rounds of tiles over 256 compute units.  An expert's last tile is on the
// average half empty, and one of 128 slots or more that is takes less time (32 experts of 4096
// x 7168, bf16, us with 128 and 256 slots: mean 64 197, 206; 94 268, 217; 128 273, 239; 188
// 343, 340; 256 404, 351).
inline double time_of(const Choice &c, const TileCall &p, long R) {
  const double experts = p.grouped ? double(std::min(p.R, p.E)) : 1.0;
  const double items = p.grouped ? experts * std::max(1.0, R / experts / c.slots + 0.5)
                                 : double((R + c.slots - 1) / c.slots);
  const double tiles = items * double((p.N + c.rows - 1) / c.rows);
  const double rounds = std::floor(tiles / (256 * c.per_cu));
  const double rest = tiles - rounds * 256 * c.per_cu;
  // A round that leaves half of the card idle is up to a fifth faster (256 x 256: 64 tiles 80,
  // 128 82, 168 83, 256 103).
  const double part = rest <= 256.0 ? c.one * (0.8 + 0.2 * std::max(0.0, rest / 128 - 1.0)) : c.all;
  const double t = rounds * c.all + (rest > 0.0 ? part : 0.0);
  return p.grouped && c.slots >= 128 ? t * (0.5 + 0.5 * std::min(1.0, R / experts / c.slots)) : t;
}

// The choice of the least time among those whose launch a grid takes; -1: none
struct Best {
  int choice;
  double time;
};
template <int kCount>
Best least(const Choice (&list)[kCount], const TileCall &p, long R) {
  Best best = {-1, INFINITY};
  for (int i = 0; i < kCount; ++i) {
    const double t = time_of(list[i], p, R);
    if (t < best.time && tiles_of(list[i].slots, list[i].rows, p, R) <= most_tiles(list[i].waves))
      best = {i, t};
  }
  return best;
}

// Rows of X that one launch takes, whole rounds of its tiles, before another takes the rest
// (all of them: one launch is the best).  Only where a round is worth it beside a launch (2
// us) and the host's own time.  us with one launch and with two, bf16: 1030 x 4096 x 7168 56,
// 43; 4100 165, 106; fp32 101, 80.
template <int kCount>
long rows_before_rest(const Choice (&list)[kCount], const TileCall &p) {
  const double blocks = double((p.K + 127) / 128) / 56.0;
  double least_time = least(list, p, p.R).time;
  long rows = p.R;
  if (p.grouped || least_time * blocks < 25.0) return rows;
  for (const Choice &c : list) {
    const long tiles_n = (p.N + c.rows - 1) / c.rows, round = 256L * c.per_cu;
    const long tiles = (p.R + c.slots - 1) / c.slots * tiles_n;
    const long first = tiles / round * round / tiles_n * c.slots;
    if (first <= 0 || first >= p.R) continue;
    const double t = least(list, p, first).time + least(list, p, p.R - first).time + 2.0 / blocks;
    if (t < least_time) {
      least_time = t;
      rows = first;
    }
  }
  return rows;
}

}  // namespace
}  // namespace w4a16
