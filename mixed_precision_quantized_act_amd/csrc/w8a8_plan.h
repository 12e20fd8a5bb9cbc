// Which kernel and tiles take a qlinear_w8a8 call (host code, shared by the launch
// and a host-side test): the least of the times that a few measured constants
// give for each way.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qact {

// Few rows, or few outputs (w8a8_split.hip): tiles of 16 MT rows and 16 NT columns,
// W waves with rings of S lines of 128 elements per row.  Each is the fastest of all ways at
// some of 138 drawn sizes (rows x columns x K, us; the best of the others): 16 x 16 at 42 (2610 x
// 5 x 13392 1.45 times ahead), 32 x 32 at 12 (7176 x 24 x 8992 1.24), 64 x 16 at 17
// (9113 x 1 x 2032 5.4 and 6.5; 61 x 2943 x 288 4.1 and 4.5), 64 x 32 at 12 (64 x 7680
// x 1920 6.8 and 8.4), 64 x 64 at 11 (14022 x 47 x 12288 29 and 49; the rating takes 64 x 32
// there, 52).
#define QACT_W8_SPLITS(X) X(1, 1, 4, 4) X(2, 2, 4, 4) X(4, 1, 4, 3) X(4, 2, 4, 3) X(4, 4, 4, 2)
struct SplitShape {
  int mt, nt, waves, slots;
};
constexpr SplitShape kSplitShapes[] = {
#define QACT_W8_SHAPE(MT, NT, W, S) {MT, NT, W, S},
    QACT_W8_SPLITS(QACT_W8_SHAPE)
#undef QACT_W8_SHAPE
};
constexpr int kSplitK = 128;
constexpr int split_smem(const SplitShape& s) {
  const int ring = s.waves * s.slots * 16 * (s.mt + s.nt) * kSplitK, sums = s.waves * s.mt * s.nt * 1024;
  return ring > sums ? ring : sums;
}

// Many rows (qgemm_w8a8.hip): tiles of 128 x 128 (two fit a compute unit), 256 x
// 128, 192 x 256 and 256 x 256.  us: a tile's start and end and a unit of 64 of K, of
// a tile alone and with all compute units busy.  (256 x 128 one by one: 10374 x 590 x
// 3584 32.6, the best of the others 35.6; 12698 x 549 x 2320 32.1 and 33.6.)
//
// Over the same sizes what is chosen takes 1.02 times the best on the geometric mean.  The rating
// knows neither the outputs' type nor GELU (8192 x 8192 x 4096 to float32: 337, by 192 x 256 309).
enum W8Tile { kTile128, kTile256x128, kTile192x256, kTile256, kTiles };
constexpr int kTileRows[kTiles] = {128, 256, 192, 256}, kTileCols[kTiles] = {128, 128, 256, 256};
constexpr int kTileFit[kTiles] = {2, 1, 1, 1};
constexpr double kStartAlone[kTiles] = {2.5, 4.5, 5.5, 6.5}, kStartBusy[kTiles] = {3.2, 5.8, 6.2, 6.5};
constexpr double kUnitAlone[kTiles] = {0.21, 0.36, 0.42, 0.50}, kUnitBusy[kTiles] = {0.28, 0.48, 0.65, 0.80};
// 256 x 256 in a stream of whole rounds: start and end of the stream, end of a tile.  A unit
// costs a fiftieth more than one by one, so long K goes one by one, whose ends are
// exposed (8192 x 8192, 4 rounds, one by one and in a stream: K 16384 869 and 885, 8192
// 450 and 456, 4096 246 and 245, 2048 140 and 138; one round, 4096 x 4096 x 8192: 116 and
// 118).  All at the power limit, where rated times are up to a tenth too short.
constexpr double kStreamStart = 4.0, kStreamEnd = 3.0, kStreamUnit = 0.82;
constexpr int kStreamLeast = 6;                  // units

constexpr int64_t kW8Places = 256;               // compute units
constexpr int64_t kW8Most = (int64_t)1 << 30;    // workgroups of a launch
constexpr double kLaunch = 2.5;                  // us
// a workgroup's start and end, the rate at which a compute unit moves lines into its
// shared memory (bytes/us), the memory's (bytes/us), what joining cuts of K takes
constexpr double kSplitStart = 2.0, kLineRate = 75e3, kMemory = 4.9e6, kJoin = 3.0, kJoinRate = 4e6;

struct W8Plan {
  bool split;
  int shape;                       // of kSplitShapes, or a W8Tile (behind the stream's)
  int cuts;                        // of K (split)
  int64_t streamed;                // tiles of 256 x 256 taken in a stream
  double us;
};

inline int64_t w8_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t w8_part_bytes(int64_t M, int64_t N, int cuts) {
  return cuts > 1 ? (size_t)cuts * (size_t)(M * w8_up(N, 4)) * 16 : 0;
}

// The plan whose partial sums fit ws_bytes.
inline W8Plan w8_plan(int64_t M, int64_t N, int64_t K, size_t ws_bytes) {
  W8Plan best = {false, kTile128, 1, 0, 1e30};
  const auto rate = [&](const W8Plan& p) {
    if (p.us < best.us) best = p;
  };
  const double loaded = (double)(M + N) * (double)K / kMemory;
  for (int i = 0; i < (int)(sizeof(kSplitShapes) / sizeof(kSplitShapes[0])); ++i) {
    const SplitShape& s = kSplitShapes[i];
    const int64_t tiles = w8_up(M, 16 * s.mt) * w8_up(N, 16 * s.nt), lines = w8_up(K, kSplitK);
    if (tiles > kW8Most) continue;
    const int64_t fit = 160 * 1024 / split_smem(s), fits = fit < 8 ? fit : 8;
    for (int cuts = 1; cuts <= 16; ++cuts) {
      // a cut keeps every wave busy, and there is no point in more than a round of them
      if (cuts > 1 && (lines < (int64_t)cuts * s.waves || tiles * cuts > kW8Places * fits ||
                       w8_part_bytes(M, N, cuts) > ws_bytes))
        break;
      const int64_t groups = tiles * cuts, rounds = w8_up(groups, kW8Places * fits);
      const int64_t beside = groups < kW8Places ? 1 : groups < kW8Places * fits ? w8_up(groups, kW8Places) : fits;
      const double each = (double)(16 * (s.mt + s.nt)) * (double)(w8_up(lines, cuts) * kSplitK) / kLineRate;
      double us = kLaunch + (double)rounds * (kSplitStart + (double)beside * each);
      if (us < kLaunch + kSplitStart + loaded) us = kLaunch + kSplitStart + loaded;
      if (cuts > 1) us += kJoin + 2.0 * (double)w8_part_bytes(M, N, cuts) / kJoinRate;
      rate({true, i, cuts, 0, us});
    }
  }
  const double units = (double)w8_up(K, 64);
  const int64_t large = w8_up(M, 256) * w8_up(N, 256);
  for (int t = 0; t < kTiles; ++t) {
    const auto time = [&](int64_t n, int fit) {    // of n tiles one by one
      const int64_t places = kW8Places * fit, here = n < places ? n : places;
      const double busy = here < kW8Places ? (double)here / kW8Places : 1.0;
      const double beside = here < kW8Places ? 1.0 : (double)here / kW8Places;
      return (double)w8_up(n, places) * (kStartAlone[t] + busy * (kStartBusy[t] - kStartAlone[t]) +
                                         units * beside * (kUnitAlone[t] + busy * (kUnitBusy[t] - kUnitAlone[t])));
    };
    const int64_t tiles = w8_up(M, kTileRows[t]) * w8_up(N, kTileCols[t]);
    if (tiles <= kW8Most) rate({false, t, 1, 0, kLaunch + time(tiles, kTileFit[t])});
    // behind whole rounds of the stream
    if (t == kTile192x256 || large < kW8Places || units < kStreamLeast) continue;
    const int64_t rounds = t == kTile256 ? w8_up(large, kW8Places) : large / kW8Places;
    const int64_t streamed = t == kTile256 ? large : rounds * kW8Places;
    const int64_t rest = (large - streamed) * (256 / kTileRows[t]) * (256 / kTileCols[t]);
    rate({false, t, 1, streamed,
          kLaunch + kStreamStart + (double)rounds * (units * kStreamUnit + kStreamEnd) + time(rest, 1)});
  }
  return best;
}

}  // namespace qact
