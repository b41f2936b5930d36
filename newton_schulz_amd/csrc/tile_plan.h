// How the tiles of a product are handed to workgroups (host, and the device's
// side of it).
//
// A persistent grid of G workgroups walks the tiles; what is left after the
// whole rounds would keep few of them busy, so each of those tiles is cut along
// the contraction into `splits` parts, whose sums go to the workspace and are
// joined, in order, by a launch more.  8192 x 2560 out of 9728 (gradient of the
// inputs, 320 tiles of 256 x 256 on 256 CUs): 645 us in two rounds, see
// grad8.hip for what the split makes of it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct TilePlan {
  int large;        // 256 x 256 products a workgroup (or 128 x 128)
  int tm, tn;       // tiles along the output's rows and columns
  int stages;       // of the contraction
  int splits;       // parts of a tile that is cut
  int part;         // stages of a part
  int64_t whole;    // tiles that are not cut
  int64_t units;    // tiles and parts of tiles
  int grid;
};

// What the kernel sees.
struct TileWork {
  int tm, tn, stages, splits, part;
  int64_t whole, units;
  char* parts;      // [cut tiles][splits] sums of a whole tile, rows contiguous
};

#ifdef __HIPCC__
struct TileUnit {
  int64_t ti, tj;   // tile row and column
  int first, past;  // stages
  int64_t slot;     // of the partial sums, or -1
};
__device__ __forceinline__ TileUnit tile_unit(const TileWork& w, int64_t l) {
  TileUnit u;
  u.first = 0;
  u.past = w.stages;
  u.slot = -1;
  int64_t t = l;
  if (l >= w.whole) {
    // neighbours work on the same stretch of the contraction
    const int64_t cut = static_cast<int64_t>(w.tm) * w.tn - w.whole, p = (l - w.whole) / cut;
    t = w.whole + (l - w.whole) % cut;
    u.first = static_cast<int>(p) * w.part;
    u.past = min(u.first + w.part, w.stages);
    u.slot = (t - w.whole) * w.splits + p;
  }
  // bands of four tile columns, row by row inside a band: the tiles that an XCD
  // works on at once share their operands in its L2
  constexpr int GN = 4;
  const int64_t band = t / (static_cast<int64_t>(w.tm) * GN);
  const int64_t wide = min(static_cast<int64_t>(GN), w.tn - band * GN);
  const int64_t r = t - band * w.tm * GN;
  u.ti = r / wide;
  u.tj = band * GN + r % wide;
  return u;
}
#endif

// Tiles of tile_m x tile_n, `slots` workgroups at a time, at most `room` bytes of partial
// sums.  The costs are in stages of a workgroup: measured for 256-tiles, a tile's
// start and end take three stages' time, the second launch and its partial sums two
// and a sixteenth a part.
inline TilePlan plan_tiles(int64_t m, int64_t n, int tile_m, int tile_n, int stages, int slots, size_t room, double* cost) {
  constexpr double kEnds = 3.0, kJoin = 2.0, kJoinPart = 1.0 / 16;
  TilePlan p = {};
  p.tm = static_cast<int>((m + tile_m - 1) / tile_m);
  p.tn = static_cast<int>((n + tile_n - 1) / tile_n);
  p.stages = stages;
  const int64_t tiles = static_cast<int64_t>(p.tm) * p.tn, rounds = tiles / slots, rest = tiles % slots;
  const size_t bytes = static_cast<size_t>(tile_m) * tile_n * 4;
  double best = rest ? stages + kEnds : 0.0;
  p.splits = 1;
  p.part = stages;
  for (int s = 2; rest && s <= 32 && s <= stages; ++s) {
    const int part = (stages + s - 1) / s, parts = (stages + part - 1) / part;
    if (parts < s) continue;
    if (static_cast<size_t>(rest) * s * bytes > room) break;
    const double t = static_cast<double>((rest * s + slots - 1) / slots) * (part + kEnds) + kJoin + kJoinPart * static_cast<double>(rest) * s / 64;
    if (t < best) {
      best = t;
      p.splits = s;
      p.part = part;
    }
  }
  p.whole = p.splits > 1 ? tiles - rest : tiles;
  p.units = p.whole + (tiles - p.whole) * p.splits;
  p.grid = static_cast<int>(p.units < slots ? p.units : slots);
  *cost = static_cast<double>(rounds) * (stages + kEnds) + best;
  return p;
}
inline TileWork tile_work(const TilePlan& p, char* parts) { return {p.tm, p.tn, p.stages, p.splits, p.part, p.whole, p.units, parts}; }
