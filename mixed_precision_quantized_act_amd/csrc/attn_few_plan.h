// How attention of few query rows is laid out (host code, shared by the launch, by what a
// caller is told of the workspace and by a host-side test).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qact {

constexpr int kFewKeys = 64;     // keys of a wave's step
constexpr int kFewRows = 16;     // rows of a tile
constexpr int kFewWaves = 4;

// Workgroups to aim for: a few for each of the 256 compute units, so that
// streams of different lengths even out (16 streams of up to 32768 tokens, 8
// heads of 128: 256 143 us, 512 109, 1024 105, 2048 110).  Of bf16 heads of 128
// one workgroup runs at a time on a unit, and each round waits for its first
// keys: one round (16 tokens to 4000 states, 8 heads: 1024 69 us, 512 60, 256 56, 262
// MB at 4.7 TB/s).  Waves of two sixteens of rows run 512 workgroups at a time, and what is
// left of a round costs as much as one: 4 cuts or more of every tile fill one
// round, fewer two, and of 512 tiles none is cut (8 key heads of 128, 32768 keys, 32 rows: 4
// streams 512 workgroups 41 us, 768 53, 1024 50; 16 streams 133, 143 and 133;
// 64 rows, 16 streams: 512 241, 768 250, 1024 233; 40 streams of 24 rows, 8192 keys: 320
// 101, 960 91; 64 streams of 32 rows, 4096 keys: 512 69, 1024 81).
constexpr int64_t kFewBlocks = 1024, kFewBlocksWide = 256, kFewPlaces = 512;

inline int64_t few_tiles(int64_t Lq, int Hq, int Hkv, int sets) {
  return (Lq * (Hq / Hkv) + sets * kFewRows - 1) / (sets * kFewRows);
}

// Splits of keys up to L where s are wanted.  A step of a workgroup's waves takes about
// 1.8 us of a nearly empty chip and the join 0.22 us a split, so of w steps
// more than sqrt(8 w) splits cost more than they give (one stream of 32768: 32
// splits 21 us, 64 25, 128 37).
inline int64_t few_splits(int64_t s, int64_t L) {
  const int64_t w = (L + kFewKeys * kFewWaves - 1) / (kFewKeys * kFewWaves);
  s = s < w ? s : w;
  while (s > 1 && s * s > 8 * w) --s;
  if (s <= 1) return 1;
  const int64_t steps = (w + s - 1) / s;
  return (w + steps - 1) / steps;
}

struct FewPlan {
  int sets;                      // sixteens of rows that a wave takes
  int64_t tiles, splits;         // of a key head's rows, of the keys
};

// Keys that are the same for all rows but a tree's own, and bf16 heads of 128 (wide).
//
// Two sixteens spare every second key's decoding, but take twice the registers and
// make the steps longer: only of a tree, where a SIMD has 20 steps of 64 keys of 128
// elements, 40 of 64 (32 rows of a key head, 128 key heads of 128, 16000 keys: 109 -> 87
// us; 32 of them 39.1 and 39.7; 8 and 4000 keys 13.0 and 16.3.  Heads of 64: 62 -> 57,
// 25.1 and 28.8, 11.6 and 13.2.  Four at a time, 64 rows: 269 us where two take 212.)
inline FewPlan few_plan(bool tree, bool wide, int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  const int64_t steps = B * Hkv * few_tiles(Lq, Hq, Hkv, 1) * ((L + kFewKeys - 1) / kFewKeys);
  const bool two = tree && Lq * (Hq / Hkv) > kFewRows && steps * D >= (int64_t)1024 * 20 * 128;
  FewPlan p = {two ? 2 : 1, few_tiles(Lq, Hq, Hkv, two ? 2 : 1), 1};
  const int64_t u = B * Hkv * p.tiles, blocks = wide ? kFewBlocksWide : kFewBlocks;
  p.splits = few_splits(!two ? (blocks + u - 1) / u : 4 * u <= kFewPlaces ? kFewPlaces / u : u < kFewPlaces ? 2 * kFewPlaces / u : 1, L);
  return p;
}

// Their sums, for rows B Lq Hq.
inline size_t few_sums_bytes(int64_t splits, int64_t rows, int D) {
  return splits > 1 ? (size_t)splits * (size_t)rows * (size_t)(D + 2) * 4 : 0;
}

}  // namespace qact
