// How the tiles of keys of all (stream, key head, row tile)s are cut into shares, one for
// each compute unit (shared by the kernel and a host-side check that lays out lists
// and follows every share).
//
// `total` tiles stand in one list, a unit's `len` of them together.  Share w begins at
// place w total / shares, or at a unit's begin near by.  shares <= total, so that none is
// empty: an empty one would leave no sums where a unit's others are joined.  shares total
// is below 2^31.
#pragma once

#include <stdint.h>

namespace qact {

constexpr int share_count(int most, int total) { return most < total ? most : total; }
constexpr int share_place(int w, int total, int shares) {
  return (int)((uint32_t)w * (uint32_t)total / (uint32_t)shares);
}
// A begin so near a unit's that the tiles between take less than a unit's start (7 to 10
// us, a tile 1.0 to 1.3) moves there, but not far beside a share's size.
constexpr int share_slack(int len, int total, int shares) {
  const int near = len / 4 < 8 ? len / 4 : 8, fair = total / shares / 4;
  return near < fair ? near : fair;
}
// place x, in a unit of tiles first ..
constexpr int share_begin(int x, int first, int len, int slack) {
  const int off = x - first;
  return off <= slack ? first : len - off <= slack ? first + len : x;
}
// the share that has the last tile of the unit of tiles first ..
constexpr int share_last(int first, int len, int slack, int total, int shares) {
  return (int)(((uint32_t)(first + len - slack) * (uint32_t)shares + total - 1) / (uint32_t)total) - 1;
}

}  // namespace qact
