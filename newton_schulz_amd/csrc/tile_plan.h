// How the tiles of a product are handed to workgroups (host, and the device's
// side of it).
//
// A persistent grid of G workgroups walks the tiles; what is left after the
// whole rounds would keep few of them busy, so each of those tiles is cut along
// the contraction into `splits` parts, whose sums go to the workspace and are
// joined, in order, by a launch more.  8192 x 2560 out of 9728 (gradient of the
// inputs, 320 tiles of 256 x 256 on 256 CUs): 645 us in two rounds, 430 with
// the last 64 tiles in four parts each.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct TilePlan {
  int large;        // 256 x 256 products a workgroup (or 128 x 128)
  int tm, tn;       // tiles along the output's rows and columns
  int stages;       // of the contraction
  int splits;       // parts of a tile that is cut
  int part;         // stages of a part
  int whole;        // tiles that are not cut
  int units;        // tiles and parts of tiles
  int grid;
};

// What the kernel sees.
struct TileWork {
  int tm, tn, stages, splits, part, whole, units;
  char* parts;      // [cut tiles][splits] sums of a whole tile, rows contiguous
};

#ifdef __HIPCC__
struct TileUnit {
  int ti, tj;       // tile row and column
  int first, past;  // stages
  int slot;         // of the partial sums, or -1
};
__device__ __forceinline__ TileUnit tile_unit(const TileWork& w, int l) {
  TileUnit u;
  u.first = 0;
  u.past = w.stages;
  u.slot = -1;
  uint32_t t = static_cast<uint32_t>(l);
  if (l >= w.whole) {
    // neighbours work on the same stretch of the contraction
    const uint32_t cut = static_cast<uint32_t>(w.tm * w.tn - w.whole), i = t - static_cast<uint32_t>(w.whole), p = i / cut;
    t = static_cast<uint32_t>(w.whole) + i % cut;
    u.first = static_cast<int>(p) * w.part;
    u.past = min(u.first + w.part, w.stages);
    u.slot = static_cast<int>(i % cut) * w.splits + static_cast<int>(p);
  }
  // bands of four tile columns, row by row inside a band: the tiles that an XCD
  // works on at once share their operands in its L2
  constexpr uint32_t GN = 4;
  const uint32_t of_band = static_cast<uint32_t>(w.tm) * GN, band = t / of_band, r = t % of_band;
  const uint32_t wide = min(GN, static_cast<uint32_t>(w.tn) - band * GN);
  u.ti = static_cast<int>(wide == GN ? r / GN : r / wide);
  u.tj = static_cast<int>(band * GN + (wide == GN ? r % GN : r % wide));
  return u;
}
#endif

// What the pieces of a product take, in microseconds on an MI355X: a stage of a
// workgroup, its start and end, the join.
struct TileCost {
  double stage, ends;
};
// 256 x 256 products, one workgroup of eight waves a CU (2048 x 4096 x 2560: a
// stage in 1.9 us, the setup, the first loads and the stores 9); and 128 x 128,
// two of four waves (two stages at once in 1.5 us, 0.9 if alone; 5).
constexpr TileCost kLarge = {1.9, 9.0}, kSmallTwo = {1.5, 5.0}, kSmallOne = {0.9, 5.0};
constexpr double kJoin = 3.0, kJoinBytes = 5.3e6;  // bytes a microsecond

// Tiles of tile_m x tile_n, `slots` workgroups at a time, at most `room` bytes of
// partial sums.
inline TilePlan plan_tiles(int64_t m, int64_t n, int tile_m, int tile_n, int stages, int slots, size_t room, TileCost full,
                           TileCost few, double* cost) {
  TilePlan p = {};
  p.tm = static_cast<int>((m + tile_m - 1) / tile_m);
  p.tn = static_cast<int>((n + tile_n - 1) / tile_n);
  p.stages = stages;
  const int tiles = p.tm * p.tn, rounds = tiles / slots, rest = tiles % slots;
  const size_t bytes = static_cast<size_t>(tile_m) * tile_n * 4;
  auto time = [&](int units, int per) {
    const TileCost& c = 2 * units <= slots ? few : full;
    return ((units + slots - 1) / slots) * (per * c.stage + c.ends);
  };
  double best = rest ? time(rest, stages) : 0.0;
  p.splits = 1;
  p.part = stages;
  for (int s = 2; rest && s <= 32 && s <= stages; ++s) {
    const int part = (stages + s - 1) / s, parts = (stages + part - 1) / part;
    if (parts < s) continue;
    if (static_cast<size_t>(rest) * s * bytes > room) break;
    const double t = time(rest * s, part) + kJoin + static_cast<double>(static_cast<size_t>(rest) * s * bytes) / kJoinBytes;
    if (t < best) {
      best = t;
      p.splits = s;
      p.part = part;
    }
  }
  p.whole = p.splits > 1 ? tiles - rest : tiles;
  p.units = p.whole + (tiles - p.whole) * p.splits;
  p.grid = p.units < slots ? p.units : slots;
  *cost = rounds * (stages * full.stage + full.ends) + best;
  return p;
}
inline TileWork tile_work(const TilePlan& p, char* parts) { return {p.tm, p.tn, p.stages, p.splits, p.part, p.whole, p.units, parts}; }

// The plan of a product in tiles of 256 x 256 or 128 x 128; with an operand in
// three parts of half as many columns, whose stages take one and a half times as long.
inline TilePlan plan_product(int64_t m, int64_t n, int parts, int stages, int cus, size_t room) {
  const int of = parts > 1 ? 2 : 1;
  const double longer = parts > 1 ? 0.5 * parts : 1.0;
  auto times = [&](TileCost c) { return TileCost{c.stage * longer, c.ends}; };
  double large, small;
  TilePlan l = plan_tiles(m, n, 256, 256 / of, stages, cus, room, times(kLarge), times(kLarge), &large);
  const TilePlan s = plan_tiles(m, n, 128, 128 / of, stages, 2 * cus, room, times(kSmallTwo), times(kSmallOne), &small);
  l.large = 1;
  return large <= small ? l : s;
}
