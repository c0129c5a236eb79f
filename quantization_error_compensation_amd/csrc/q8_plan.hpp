// Which kernel a product of the 8-bit path takes, and the workspace it needs
// (host code).
//
// Up to 16 tokens, and up to 32 or 64 where that still pays, the weights are
// streamed by workgroups that hold 16 to 64 of their rows over the whole of K
// (k_q8_stream.hip); past that a workgroup multiplies a tile of tokens with a
// tile of rows (k_q8_gemm.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "q8.hpp"

namespace spear {

constexpr int kQ8Units = 256;            // compute units of gfx950
constexpr int kQ8CounterBytes = 65536;   // arrival counters at the head of the workspace
constexpr int kQ8MaxSplitTiles = 512;    // each tile with up to 8 waves of 4 parts
constexpr int64_t kQ8MaxPartials = (int64_t)64 << 20;
constexpr int kQ8MaxSplits = 8;

// ------------------------------------------------------------- few tokens
// x: loads of 8 tokens a block of K (1, 2, 4, 6, 8); tiles: 16-row tiles of the
// weights (of each projection) a workgroup; waves.
struct Q8Stream {
  int x, tiles, waves;  // x 0: the tile kernel
};

// The rows that the fullest compute unit streams, and the tokens' codes that
// come along with them, decide: a unit reads tiles * 2 KB of weights and x KB
// of tokens a block and workgroup.  More rows a workgroup read the tokens less
// often, fewer fill the units more evenly.  us for 1 / 2 / 4 tiles:
//   16 tokens  4096x4096 4.7 / 4.9 / 6.0   4096->6144 6.1 / 5.8 / 6.2
//              28672->8192 45.5 / 40.4 / 53.4   8192->10240 18.9 / 20.8 / 17.8
//   32 tokens  28672->8192 57.6 / 45.8 / 60.9   8192->10240 23.7 / 25.3 / 19.9
// Up to 8 tokens there is next to nothing to share: one tile (28672->8192 40.2,
// two 40.4).  One tile with at most 256 workgroups and K >= 8192: 8 waves
// instead of 4 (8192->1024, one token, 4.2 against 5.2; 11008->4096 10.1 against
// 11.1; but 4096x4096 4.7 against 4.5).
inline Q8Stream plan_q8_stream(const Q8Shape& s) {
  const int n = s.N / 16, parts = s.gated ? 2 : 1;
  // Past 32 tokens only layers that the tile kernel would have to split over K
  // to fill the units, whose join costs more than the tokens' repeated reads: 64
  // tokens, 4096x4096 6.3 against 9.0 us, 4096->6144 7.7 against 9.6, 8192->1024
  // 8.4 against 9.6; 11008->4096 17.4 against 14.9, 8192x8192 19.8 against 17.7.
  if (s.T > 64 || (s.T > 32 && (n > 384 || s.K > 8192))) return Q8Stream{0, 0, 0};
  Q8Stream best{s.T <= 8 ? 1 : s.T <= 16 ? 2 : s.T <= 32 ? 4 : s.T <= 48 ? 6 : 8, 1, 4};
  if (best.x > 1) {
    int64_t least = INT64_MAX;
    for (int tiles = 1; tiles <= (best.x <= 4 ? 4 : 2); tiles *= 2) {
      const int groups = (n + tiles - 1) / tiles;
      const int64_t cost = (int64_t)((groups + kQ8Units - 1) / kQ8Units) * (2 * tiles * parts + best.x);
      if (cost < least) {
        least = cost;
        best.tiles = tiles;
      }
    }
  }
  if (best.x <= 2 && best.tiles == 1 && n <= kQ8Units && s.K >= 8192) best.waves = 8;
  return best;
}

// ------------------------------------------------------------ many tokens
// The tile kernel's shapes: tokens x weight rows; held: workgroups that a
// compute unit holds; block: us that a unit needs for 128 codes of K of a tile;
// once: us that a tile's start and end add.
struct Q8Tile {
  int bm, bn, held;
  bool gated;  // a wave holds both projections of its columns
  double block, once;
};
constexpr Q8Tile kQ8Tiles[] = {
    {256, 256, 1, true, 1.33, 2.2},  {192, 256, 1, true, 1.20, 2.0},   {256, 128, 1, true, 0.73, 2.1},
    {128, 256, 1, true, 0.765, 2.2}, {128, 128, 1, false, 0.46, 2.4},  {64, 128, 2, true, 0.30, 3.3},
    {64, 64, 2, false, 0.19, 3.1},   {32, 128, 2, false, 0.235, 2.9}};
constexpr int kQ8TileCount = sizeof(kQ8Tiles) / sizeof(kQ8Tiles[0]);

struct Q8TilePlan {
  int tile, splits;
  int64_t tiles;
};

inline int64_t q8_tiles(const Q8Shape& s, const Q8Tile& t) {
  const int cols = s.gated ? t.bn / 2 : t.bn;
  return (int64_t)((s.T + t.bm - 1) / t.bm) * ((s.N + cols - 1) / cols);
}

// The shape and the number of splits of K with the least estimated time: the
// fullest unit's tiles, the memory traffic that does not hide behind them (as
// if at 10.6 TB/s), and with splits the partial sums' way through memory.  The
// constants are fitted to 3600 timings of 12 layers at 40 to 4096 tokens; the
// choice is 0.9% slower than the best of them on average, 15% at worst.  On 7106
// layers and token counts drawn at random (256 to 28672 wide) it is 1.8% slower on
// average and by more than 20% at 1.4% of them: 553 tokens gated 13888->1664 61.8
// us for 42.9 (44%, the worst), 136 tokens 9856->6528 35.7 for 25.4, 227 tokens
// gated 2304->4608 18.9 for 13.6, 307 tokens 13776->3248 48.3 for 35.1, and others
// of 80 to 620 tokens on layers of 1700 to 11000 rows; a fit to the drawn ones gains
// nothing on average.  Where K is no multiple of 128, rows do not begin on cache
// lines and every load takes two: 15 to 40% longer, for all shapes much alike, so
// that the choice is the same.  What it weighs, in us: large tiles fetch fewer bytes
// a product (3999 tokens gated 8192->28672: 1470 with 256 x 256, 1640 with 128 x
// 256, 2060 with 64 x 128); small ones fill the units (512 tokens 4096x4096: 14.6
// with 64 x 128, 26 with 256 x 128), and so do splits (512 tokens 28672->8192: 118
// with 256 x 128 in 2, 144 with 128 x 128 in 1; 256 tokens 8192x8192: 29 with 128 x
// 128 in 2, 34 with 64 x 128 in 1).
inline Q8TilePlan plan_q8_tiles(const Q8Shape& s) {
  Q8TilePlan best{0, 1, q8_tiles(s, kQ8Tiles[0])};
  double least = 1e300;
  const int blocks = (s.K + 127) / 128;
  const double rows = s.gated ? 2.0 * s.N : s.N;
  const double memory = (rows * s.K + (double)s.T * s.K + 2.0 * s.T * s.N) / 10.6e6;
  for (int i = 0; i < kQ8TileCount; ++i) {
    const Q8Tile& t = kQ8Tiles[i];
    if (s.gated && !t.gated) continue;
    const int64_t tiles = q8_tiles(s, t);
    if (i > 0 && tiles > 1 << 22) continue;  // a launch holds fewer than 2^32 threads
    for (int splits = 1; splits <= kQ8MaxSplits && splits <= blocks; ++splits) {
      if (splits > 1 && (tiles > kQ8MaxSplitTiles || tiles * splits * t.bm * t.bn * 4 > kQ8MaxPartials ||
                         (t.bm * t.bn > 256 * 128 && splits > 4)))
        break;
      const int64_t each = (tiles * splits + kQ8Units - 1) / kQ8Units;
      double us = (double)each * ((blocks + splits - 1) / splits) * t.block + memory +
                  (double)((each + t.held - 1) / t.held) * t.once;
      if (splits > 1) {
        const double area = t.bm * t.bn;
        us += 0.35 + 0.57 * splits + 0.09 * (splits - 1) * (double)each * area / 16384 +
              0.19 * (double)(tiles * splits) * area * 4e-6;
      }
      if (us < least) {
        least = us;
        best = Q8TilePlan{i, splits, tiles};
      }
    }
  }
  return best;
}

// Bytes of workspace for calls of up to s.T tokens: the counters and room for
// the partial sums of any of them (tiles round tokens and rows up to at most
// 255 more).
inline size_t q8_workspace_for(const Q8Shape& s) {
  if (s.T <= 32) return kQ8CounterBytes;
  const int64_t all = (int64_t)kQ8MaxSplits * (s.T + 256) * (s.rows() + 256) * 4;
  return (size_t)(kQ8CounterBytes + (all < kQ8MaxPartials ? all : kQ8MaxPartials));
}

}  // namespace spear
