// Host-side check of csrc/attn_shares.h: lists of units of all lengths, cut into shares;
// every tile lies in one share, no share is empty, and the sums that a share leaves are
// the ones that are joined.  Prints "ok <lists>".
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "attn_shares.h"

using namespace qact;

static void fail(const char* what, int list, int w) {
  std::printf("%s: list %d share or unit %d\n", what, list, w);
  std::exit(1);
}

int main() {
  std::mt19937 g(7);
  int list = 0;
  for (; list < 4000; ++list) {
    std::vector<int> first, len;
    const int units = 1 + g() % (list % 3 ? 40 : 700), most = 1 + g() % (list % 5 ? 300 : 4000);
    int total = 0, same = 1 + g() % most;
    for (int u = 0; u < units; ++u) {
      first.push_back(total);
      len.push_back(list % 4 == 0 ? same : 1 + (int)(g() % most));
      total += len.back();
    }
    const int shares = share_count(list % 7 ? 256 : 1 + g() % 300, total);
    const auto begin = [&](int w) {
      if (w >= shares) return total;
      const int x = share_place(w, total, shares);
      int u = 0;
      while (u + 1 < units && first[u + 1] <= x) ++u;
      return share_begin(x, first[u], len[u], share_slack(len[u], total, shares));
    };
    if (begin(0) != 0) fail("the first share's begin", list, 0);
    std::vector<int> head(units, -1), end(units, -1);
    int u = 0, longest = 0;
    for (int w = 0; w < shares; ++w) {
      const int at = begin(w), stop = begin(w + 1);
      if (at >= stop) fail("empty", list, w);
      longest = stop - at > longest ? stop - at : longest;
      int later = 0, ahead = 0;                            // sums of units from before, and that go on
      for (int x = at; x < stop;) {
        while (first[u] + len[u] <= x) ++u;
        const int c0 = x - first[u], c1 = len[u] < c0 + stop - x ? len[u] : c0 + stop - x;
        if (c1 <= c0) fail("no tiles", list, w);
        if (c0 == 0) head[u] = w;
        if (c1 == len[u]) end[u] = w;
        if (c1 - c0 < len[u]) ++(c0 == 0 ? ahead : later);
        x += c1 - c0;
      }
      if (later > 1 || ahead > 1) fail("two sums of a kind", list, w);
    }
    for (u = 0; u < units; ++u) {
      if (head[u] < 0 || end[u] < 0) fail("left out", list, u);
      if (head[u] != end[u] &&
          share_last(first[u], len[u], share_slack(len[u], total, shares), total, shares) != end[u])
        fail("the last of a unit's", list, u);
    }
    if (longest > total / shares + 1 + 2 * 8) fail("uneven", list, longest);
  }
  std::printf("ok %d\n", list);
  return 0;
}
