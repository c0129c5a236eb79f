// The plan of the 8-bit products (csrc/q8_plan.hpp), built for the host: over
// many shapes the streaming variant exists and fits, the partial sums of every
// tile plan fit the workspace of any larger call, arrivals fit the counters and
// launches stay below 2^32 threads.  Called from tests/test_q8_plan.py.
#include <stdint.h>
#include <stdio.h>

#include "q8_plan.hpp"

using namespace spear;

extern "C" int q8_plan_faults(int K, int N, int gated, int T, int largest) {
  const Q8Shape s{K, N, T, gated != 0, false, false};
  const Q8Shape top{K, N, largest, gated != 0, false, false};
  const size_t room = q8_workspace_for(top);
  if (room < q8_workspace_for(s)) return 1;
  const Q8Stream f = plan_q8_stream(s);
  if (f.x) {
    const int variants[] = {114, 118, 214, 218, 224, 244, 414, 424, 444, 614, 624, 814, 824};
    bool known = false;
    for (int v : variants) known = known || v == f.x * 100 + f.tiles * 10 + f.waves;
    return !known || T > 8 * f.x ? 2 : 0;
  }
  const Q8TilePlan p = plan_q8_tiles(s);
  const Q8Tile& t = kQ8Tiles[p.tile];
  if (p.tile < 0 || p.tile >= kQ8TileCount || (s.gated && !t.gated)) return 3;
  if (p.tiles != q8_tiles(s, t) || p.splits < 1 || p.splits > kQ8MaxSplits || p.splits > (K + 127) / 128) return 4;
  if (p.splits > 1) {
    if (p.tiles > kQ8MaxSplitTiles) return 5;
    if (kQ8CounterBytes + p.tiles * p.splits * t.bm * t.bn * 4 > (int64_t)room) return 6;
  }
  if (p.tiles * p.splits * 512 >= (int64_t)1 << 32) return 7;
  return 0;
}

// Which kernel a product takes: a stream's loads of tokens * 100 + tiles * 10 +
// waves, or 10000 + 100 * (the tile's index, its form with loading waves being
// one of its own) + splits of K.
extern "C" int q8_plan_kernel(int K, int N, int gated, int T) {
  const Q8Shape s{K, N, T, gated != 0, false, false};
  const Q8Stream f = plan_q8_stream(s);
  if (f.x) return f.x * 100 + f.tiles * 10 + f.waves;
  const Q8TilePlan p = plan_q8_tiles(s);
  const bool loading_waves = kQ8Tiles[p.tile].bm == 256 && kQ8Tiles[p.tile].bn == 128 && T > 256;
  return 10000 + 100 * (loading_waves ? kQ8TileCount : p.tile) + p.splits;
}
