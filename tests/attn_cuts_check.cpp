// The cut of the keys (csrc/attn_cuts.h) over many sizes: its pieces follow
// each other and end at the last key, fit the workspace, and take no longer
// than the plan says when their workgroups are dealt out in launch order; no
// equal cut is rated faster.  With arguments (u rows D tiles fit) it prints one plan.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <functional>
#include <queue>
#include <random>
#include <vector>

#include "attn_cuts.h"

using namespace qact;

// Workgroups (piece by piece) on the first place that is free.
static double dealt(const Pieces& c, int64_t u, int64_t rows, int D, int64_t tiles) {
  std::priority_queue<double, std::vector<double>, std::greater<double>> free;
  for (int64_t i = 0; i < kCutPlaces; ++i) free.push(0.0);
  double end = 0.0;
  for (int p = 0; p < c.n; ++p) {
    const double t = (double)(piece_end(c, (int)tiles, p) - piece_begin(c, (int)tiles, p)) * tile_time(D) + kTileStart;
    for (int64_t i = 0; i < u; ++i) {
      const double at = free.top() + t;
      free.pop();
      free.push(at);
      end = std::max(end, at);
    }
  }
  return end + join_time(c.n, rows, D);
}

int main(int argc, char** argv) {
  if (argc == 6) {
    const Pieces c = pieces_of(atoll(argv[1]), atoll(argv[2]), atoi(argv[3]), atoll(argv[4]), atoll(argv[5]));
    printf("%d %d %d\n", c.n, c.size, c.whole);
    return 0;
  }
  std::mt19937 g(7);
  const auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(g() % (uint64_t)(hi - lo + 1)); };
  int failures = 0, uneven = 0, cases = 0;
  for (; cases < 20000; ++cases) {
    const int D = g() % 2 ? 64 : 128;
    const int64_t u = g() % 4 ? pick(1, 300) : pick(1, 2000), rows = u * pick(64, 256);
    const int64_t tiles = g() % 3 ? pick(0, 64) : pick(0, 1000), fit = g() % 2 ? 1000 : pick(0, 20);
    const Pieces c = pieces_of(u, rows, D, tiles, fit);
    uneven += c.size * c.n != c.whole;
    bool ok = c.n == 1 || (c.n <= fit && c.n <= 16);
    const int all = (int)tiles;
    for (int t : {all, all / 2, all / 7, 1, 0, 1 << 24}) {      // of the plan's keys and of other streams'
      int at = 0;
      for (int p = 0; p < c.n; ++p) {
        ok = ok && piece_begin(c, t, p) == at && at <= piece_end(c, t, p) && (t != all || t == 0 || at < piece_end(c, t, p));
        at = piece_end(c, t, p);
      }
      ok = ok && at == t;
    }
    const double said = cut_time(c, u, rows, D, tiles), is = dealt(c, u, rows, D, tiles);
    ok = ok && is <= said * (1 + 1e-12);
    for (int n = 1; n <= 16 && (n == 1 || (n <= fit && n <= tiles)); ++n)
      ok = ok && is <= cut_time({n, 1, n}, u, rows, D, tiles) * (1 + 1e-12);
    if (!ok && ++failures <= 20)
      printf("u %ld rows %ld D %d tiles %ld fit %ld: %d %d %d, said %.1f is %.1f\n", (long)u, (long)rows, D, (long)tiles,
             (long)fit, c.n, c.size, c.whole, said, is);
  }
  printf("%d cases, %d of them uneven, %d failures\n", cases, uneven, failures);
  return failures != 0 || uneven == 0;
}
