// How the tile kernel's keys are cut into pieces (host code, shared by the
// kernel's launch and a host-side test that enumerates every workgroup).
#pragma once

#include <stdint.h>

namespace qact {

// How a row tile's keys are cut: n pieces, each `size` parts of `whole` and
// the last one what is left.
constexpr int kCuts = 64;
struct Pieces {
  int n, size, whole;
};

// First of piece p's tiles of keys (of `tiles`), and where it ends: piece n - 1 at
// the last.
constexpr int piece_begin(const Pieces& c, int tiles, int p) {
  return (int)((int64_t)tiles * (p * c.size) / c.whole);
}
constexpr int piece_end(const Pieces& c, int tiles, int p) {
  return p == c.n - 1 ? tiles : piece_begin(c, tiles, p + 1);
}

// One workgroup fits a compute unit: this many run at once.
constexpr int64_t kCutPlaces = 256;
// us: a workgroup's start and end; a tile of keys; what the partial sums cost,
// written and read again at 4 TB/s, and the launch that joins them.
constexpr double kTileStart = 8.0;
constexpr double tile_time(int D) { return D == 64 ? 0.97 : 1.7; }
constexpr double join_time(int64_t n, int64_t rows, int D) {
  return n > 1 ? 4.0 + (double)n * (double)rows * D * 4 * 1.5 / 4e6 : 0.0;
}

// The time in us of u row tiles whose `tiles` tiles of keys are cut so: that of
// the slowest place, and the join.  Equal pieces: all workgroups in rounds.
// Otherwise the large pieces run all at once and the last ones in rounds on the
// places beside them.  Of the cut as it is launched, in whole tiles of keys.
inline double cut_time(const Pieces& c, int64_t u, int64_t rows, int D, int64_t tiles) {
  const double each = tile_time(D), joined = join_time(c.n, rows, D);
  const double large = (double)((tiles * c.size + c.whole - 1) / c.whole) * each + kTileStart;
  if (c.size * c.n == c.whole) return (double)((u * c.n + kCutPlaces - 1) / kCutPlaces) * large + joined;
  const int64_t left = kCutPlaces - u * (c.n - 1);
  const double last = (double)((u + left - 1) / left) *
                      ((double)(tiles - piece_begin(c, (int)tiles, c.n - 1)) * each + kTileStart);
  return (large > last ? large : last) + joined;
}

// Row tiles that do not fill the compute units (or fill them badly) have their
// keys cut into pieces: at most 16 equal ones, or n - 1 large ones that all run
// at once and a small one for the places that are left.  At most `fit` pieces, the
// partial sums that the workspace holds.  (1350 rows, 30 heads of 64, 12376 keys:
// 180 row tiles, so one piece leaves 76 places idle.  Two pieces, the large one
// 0.70, 0.75, 0.80 and 0.85 of the keys: 218, 187, 181 and 190 us; 3, 4 and 7 equal
// ones: 237, 190 and 203.)
inline Pieces pieces_of(int64_t u, int64_t rows, int D, int64_t tiles, int64_t fit) {
  Pieces best = {1, 1, 1};
  double least = cut_time(best, u, rows, D, tiles);
  const auto rate = [&](const Pieces& c) {
    const double t = cut_time(c, u, rows, D, tiles);
    if (t < least) {
      least = t;
      best = c;
    }
  };
  for (int n = 2; n <= 16 && n <= fit && n <= tiles; ++n) {
    rate({n, 1, n});
    const int64_t left = kCutPlaces - u * (n - 1);             // places beside the large pieces
    if (left <= 0) continue;
    const double k = (double)((u + left - 1) / left);
    // the large part for which both kinds of places take the same time
    const double f = (k + (k - 1.0) * kTileStart / ((double)tiles * tile_time(D))) / (1.0 + k * (n - 1));
    const int size = (int)(f * kCuts + 0.5);
    if (size * (n - 1) < kCuts && size * n != kCuts) rate({n, size, kCuts});
  }
  return best;
}

}  // namespace qact
