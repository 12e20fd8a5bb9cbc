// Host-side check of csrc/attn_few_plan.h over many sizes: the tiles cover the rows, no
// split is without a step, a launch fits its grid.  Prints "ok <sizes>"; with arguments tree
// B Lq Hq Hkv D L: sixteens a wave, tiles, splits.
#include <cstdio>
#include <cstdlib>

#include "attn_few_plan.h"

using namespace qact;

int main(int argc, char** argv) {
  if (argc == 8) {
    long long x[7];
    for (int i = 0; i < 7; ++i) x[i] = std::atoll(argv[i + 1]);
    const FewPlan p = few_plan(x[0] != 0, false, x[1], x[2], (int)x[3], (int)x[4], (int)x[5], x[6]);
    std::printf("%d %lld %lld\n", p.sets, (long long)p.tiles, (long long)p.splits);
    return 0;
  }
  long n = 0;
  const int64_t streams[] = {1, 2, 3, 5, 16, 33, 64, 100, 500, 4096}, rows[] = {1, 2, 7, 13, 16, 17, 31, 32, 33, 48, 64, 100, 1024};
  const int heads[][2] = {{1, 1}, {8, 8}, {32, 8}, {30, 30}, {24, 8}, {128, 128}, {128, 1}};
  const int64_t lengths[] = {0, 1, 63, 64, 256, 257, 1000, 4099, 8191, 16000, 32768, 131072, 1 << 20, (int64_t)1 << 30};
  for (int kind = 0; kind < 3; ++kind)                         // a cache's, a tree's, bf16 of 128
    for (int64_t B : streams)
      for (int64_t Lq : rows)
        for (const auto& h : heads)
          for (int D = 64; D <= 128; D += 64)
            for (int64_t L : lengths) {
              if (B * Lq * h[0] >= 1 << 24) continue;
              const FewPlan p = few_plan(kind == 1, kind == 2, B, Lq, h[0], h[1], D, L);
              const int64_t r = Lq * (h[0] / h[1]), u = B * h[1] * p.tiles, w = (L + kFewKeys * kFewWaves - 1) / (kFewKeys * kFewWaves);
              bool ok = (p.sets == 1 || (p.sets == 2 && kind == 1 && r > kFewRows)) && p.splits >= 1;
              ok = ok && p.tiles * kFewRows * p.sets >= r && (p.tiles - 1) * kFewRows * p.sets < r;
              ok = ok && (p.splits == 1 || (p.splits <= w && p.splits * p.splits <= 8 * w));
              // (within a round or two, or what one more tile than there are places makes of it)
              ok = ok && (p.splits == 1 || u * p.splits < (p.sets == 2 ? 2 * kFewPlaces + 1 : kFewBlocks + u));
              ok = ok && u * p.splits < (int64_t)1 << 25;
              ok = ok && few_sums_bytes(p.splits, B * Lq * h[0], D) % (4 * (D + 2)) == 0;
              if (!ok) {
                std::printf("kind %d B %lld Lq %lld heads %d %d D %d L %lld: %d %lld %lld\n", kind, (long long)B, (long long)Lq,
                            h[0], h[1], D, (long long)L, p.sets, (long long)p.tiles, (long long)p.splits);
                return 1;
              }
              ++n;
            }
  std::printf("ok %ld\n", n);
  return 0;
}
