// Host-side check of csrc/w8a8_plan.h over many sizes: what is launched exists, fits
// and covers the outputs.  Prints "ok <sizes>"; with arguments M N K ws the plan:
// split, shape, cuts, streamed tiles.
#include <cstdio>
#include <cstdlib>

#include "w8a8_plan.h"

using namespace qact;

static void fail(const char* what, int64_t M, int64_t N, int64_t K, size_t ws) {
  std::printf("%s: M %lld N %lld K %lld ws %zu\n", what, (long long)M, (long long)N, (long long)K, ws);
  std::exit(1);
}

int main(int argc, char** argv) {
  if (argc == 5) {
    const W8Plan p = w8_plan(std::atoll(argv[1]), std::atoll(argv[2]), std::atoll(argv[3]), (size_t)std::atoll(argv[4]));
    std::printf("%d %d %d %lld\n", (int)p.split, p.shape, p.cuts, (long long)p.streamed);
    return 0;
  }
  const int shapes = (int)(sizeof(kSplitShapes) / sizeof(kSplitShapes[0]));
  for (const SplitShape& s : kSplitShapes)
    if (split_smem(s) > 160 * 1024) fail("shared memory", s.mt, s.nt, s.waves, s.slots);
  const int64_t sizes[] = {1, 2, 15, 16, 17, 63, 64, 65, 127, 200, 256, 257, 1000, 1350, 4096, 17776, 70001, 1 << 20,
                           (1 << 26) - 1};
  const int64_t depths[] = {16, 64, 112, 128, 320, 384, 1920, 2000, 8192, 7680, 65536, (1 << 17) - 16};
  const size_t spaces[] = {0, 4096, (size_t)1 << 20, (size_t)64 << 20, ~(size_t)0};
  long n = 0;
  for (int64_t M : sizes)
    for (int64_t N : sizes)
      for (int64_t K : depths) {
        if (((M + 255) / 256) * ((N + 127) / 128) > (1 << 24)) continue;         // (refused before)
        for (size_t ws : spaces) {
          const W8Plan p = w8_plan(M, N, K, ws);
          ++n;
          if (w8_part_bytes(M, N, p.cuts) > ws) fail("workspace", M, N, K, ws);
          if (ws == 0 && p.cuts != 1) fail("cuts without a workspace", M, N, K, ws);
          if (p.split) {
            if (p.shape < 0 || p.shape >= shapes || p.streamed) fail("shape", M, N, K, ws);
            const SplitShape& s = kSplitShapes[p.shape];
            const int64_t tiles = w8_up(M, 16 * s.mt) * w8_up(N, 16 * s.nt);
            if (tiles * p.cuts > kW8Most || tiles * 16 * s.mt * 16 * s.nt < M * N) fail("tiles", M, N, K, ws);
            // every cut has a line, the join's threads fit 32 bits
            const int64_t lines = w8_up(K, kSplitK), each = w8_up(lines, p.cuts);
            if (p.cuts > 1 && (w8_up(lines, each) > p.cuts || M * w8_up(N, 4) >= (int64_t)1 << 31)) fail("cuts", M, N, K, ws);
          } else {
            if (p.cuts != 1 || p.shape < 0 || p.shape >= kTiles) fail("tile", M, N, K, ws);
            const int64_t large = w8_up(M, 256) * w8_up(N, 256);
            if (p.streamed) {
              // whole rounds, or (the largest tile) all; the smaller tiles divide it
              if (K <= 64 * (kStreamLeast - 1) || p.streamed > large || large >= (int64_t)1 << 30) fail("stream", M, N, K, ws);
              if (p.shape != kTile256 && (p.streamed % kW8Places || 256 % kTileRows[p.shape] || 256 % kTileCols[p.shape]))
                fail("rounds", M, N, K, ws);
              if (p.shape == kTile256 && p.streamed != large) fail("left over", M, N, K, ws);
            } else if (w8_up(M, kTileRows[p.shape]) * w8_up(N, kTileCols[p.shape]) > kW8Most) {
              fail("launch", M, N, K, ws);
            }
          }
        }
      }
  std::printf("ok %ld\n", n);
  return 0;
}
