// Attention of a tree of drafted tokens, many rows of a key head: what attn_tile.hip
// does for other queries, with two differences.
//
// Shares.  Streams are of different lengths and few, so equal pieces of each
// leave most compute units waiting for the longest's.  The tiles of keys of all
// (stream, key head, row tile)s stand in one list, which is cut into one share for
// each compute unit, wherever that falls; sums of a part of the keys go to the workspace
// and are joined.  The list follows from the lengths on the device.
//
// Parts.  256 rows: the 8 waves hold 32 each, as there.  Up to 128 rows: 4 times 32 rows
// over the first 32 keys of every staged tile and the same rows over the other 32, so
// that all waves have products to do; two waves' sums meet in shared memory at the
// end.
//
// 16 streams of 32 tokens over 16384 to 32768 keys, 32 query and 8 key heads of 128 (128 rows):
// 288 us, 201 GFLOP at 0.70 PFLOP/s, 7 of them for the join; equal pieces a tenth more; with
// the waves of attn_tile.hip 353.  A tile of keys takes 1.28 us, a unit's start and end 10: MFMA busy
// 0.34 of the cycles, VALU 0.42 (a third of it decoding), shared memory 0.33, a wave
// waiting 0.26 of its time, at 2.4 GHz.  3 streams of 250 tokens over up to 8191 keys, 30 heads of
// 64 (256 rows): 72 to 76 us, a tile 1.1 to 1.4.
#include "attn_rows.h"
#include "attn_shares.h"
#include "attn_stage.h"

namespace qact {

namespace {

constexpr int kTreeWaves = 8, kTreeThreads = 64 * kTreeWaves;
constexpr int tree_rows(int parts) { return 32 * kTreeWaves / parts; }

// Sums of a part of the keys.  Shares of the list: share w's own are of a unit that began
// in an earlier one; behind all shares' stand those of a unit that goes on in the next
// (of unit u at u, or with more units than shares at w).  Equal pieces: one each, unit
// u's are u pieces ..
struct TreeSums {
  float* o;       // [sums][rows of a tile][D]
  float* m;       // [sums][rows] largest logit (log2 units), -inf: nothing seen
  float* l;
  i32x2* cut;     // [units] the share in which a unit begins, and ends (the same: nothing to join)
  int shares;     // of the list; 0: equal pieces
  int pieces;
  int by_unit;    // units <= shares

  static size_t bytes(int64_t sums, int64_t cuts, int rows, int D) {
    return (size_t)(sums * rows * (D + 2) * 4 + cuts * 8);
  }
};

// The list: stream by stream, of one the units (key head, row tile) in order, each `len`
// tiles (one, of no keys, where the stream has none).  A lane holds a stream, 64 at a time;
// all of a wave take part.
__device__ __forceinline__ int tree_len(int n) { return n > 0 ? (n + kTileKeys - 1) / kTileKeys : 1; }
__device__ __forceinline__ int tree_tiles(int nq, int G, int rows) { return (nq * G + rows - 1) / rows; }

struct List {
  int nq, n;                       // of the lane's stream: queries, keys,
  int len, own, behind;            // a unit's tiles, all, the first behind them
  int b0, total, shares;

  // streams b0 .. b0 + 63, `before` tiles in front of them
  __device__ __forceinline__ void scan(const AttnArgs& a, const Kv4TreeSource& src, int rows, int lane, int from,
                                       int before) {
    b0 = from;
    const int b = b0 + lane;
    nq = n = 0;
    if (b < a.B) {
      nq = src.queries(b, a.Lq);
      n = src.keys(b);
    }
    len = tree_len(n);
    behind = own = a.Hkv * tree_tiles(nq, a.Hq / a.Hkv, rows) * len;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(behind, d);
      behind += lane >= d ? y : 0;
    }
    behind += before;
  }
  __device__ __forceinline__ void make(const AttnArgs& a, const Kv4TreeSource& src, int rows, int lane, int parts) {
    total = 0;
    for (int b = 0; b < a.B; b += 64) {
      scan(a, src, rows, lane, b, total);
      total = __builtin_amdgcn_readlane(behind, 63);
    }
    shares = share_count(parts, total);
  }
  // the lane whose stream has tile x (x < total)
  __device__ __forceinline__ int find(const AttnArgs& a, const Kv4TreeSource& src, int rows, int lane, int x) {
    if (a.B > 64) {
      int before = 0;
      for (int b = 0;; b += 64) {
        scan(a, src, rows, lane, b, before);
        before = __builtin_amdgcn_readlane(behind, 63);
        if (x < before) break;
      }
    }
    return __builtin_popcountll(__builtin_amdgcn_ballot_w64(behind <= x));
  }
  __device__ __forceinline__ int first(int l) const { return __builtin_amdgcn_readlane(behind - own, l); }
  __device__ __forceinline__ int begin(const AttnArgs& a, const Kv4TreeSource& src, int rows, int lane, int w) {
    if (w >= shares) return total;
    const int x = share_place(w, total, shares);
    const int l = find(a, src, rows, lane, x), len1 = __builtin_amdgcn_readlane(len, l), from = first(l);
    return share_begin(x, from + (x - from) / len1 * len1, len1, share_slack(len1, total, shares));
  }
  __device__ __forceinline__ int last(int u, int len) const {
    return share_last(u, len, share_slack(len, total, shares), total, shares);
  }
};

// One step a tile (Parts 2): the weights of its half beside the logits of the next
// tile's and the second product of the tile before.  The workgroup meets in the
// middle of a step: from there to the middle of step t, K(t), K(t + 1), V(t - 2) and
// V(t - 1) are read, and K(t + 2) and V(t) written, which replace K(t - 1) and V(t - 3).
// Two steps a tile (Parts 1) as in attn_tile.hip; V is written a tile sooner.
template <int D, int Parts>
__global__ void __launch_bounds__(kTreeThreads, 2)
attn_tree_kernel(AttnArgs a, Kv4TreeSource src, TreeSums sp, int tiles, Gate gate) {
  if (gated_off(gate)) return;
  using T = Tile<Kv4TreeSource, D, kTreeThreads>;
  using R = Rows<true, D>;
  constexpr int kRows = tree_rows(Parts), kGroups = kRows / 32;    // of a tile, of 32
  constexpr int kSooner = Parts == 1 ? 1 : 0;
  constexpr int kBytes = kTileKeys * D * 2, kHalf = kBytes / 2;
  // (values before the first tile: zeros behind the three tiles)
  constexpr int kBefore = Parts == 1 ? 3 * kBytes - kHalf : 3 * kBytes;
  constexpr int kJoin = 32 * (D + 4) * 4;                  // a wave's sums
  constexpr int kLds = 6 * kBytes + kHalf;
  static_assert(kLds >= 4 * kJoin, "the waves' sums");
  __shared__ __align__(16) char lds[kLds];
  __shared__ float ml[2][4][32];
  __shared__ int nan_unit;         // the last unit (from 1) with a NaN among its values' scales
  char* const kt = lds;
  char* const vt = lds + 3 * kBytes;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), group = wave % kGroups, part = wave / kGroups;
  const int G = a.Hq / a.Hkv;
  // (of the two waves of a SIMD one ahead of the other, so that they want its units at
  // different times: 1 per cent, 3 streams of 250 tokens to 32000 keys 2)
  if (wave >= kTreeWaves / 2) __builtin_amdgcn_s_setprio(1);

  if (tid < kHalf / 16) *reinterpret_cast<u32x4*>(vt + 3 * kBytes + 16 * tid) = u32x4{0, 0, 0, 0};
  if (tid == 0) nan_unit = 0;

  int at = 0, stop = 1;
  int64_t b = 0;
  int hk = 0, tile = 0, c0 = 0, nq = 0, n = 0;
  List list;
  if (sp.shares) {
    list.make(a, src, kRows, tid & 63, sp.shares);
    if ((int)blockIdx.x >= list.shares) return;
    stop = list.begin(a, src, kRows, tid & 63, blockIdx.x + 1);
    at = list.begin(a, src, kRows, tid & 63, blockIdx.x);
    if (at >= stop) return;
    const int l = list.find(a, src, kRows, tid & 63, at), rel = at - list.first(l);
    b = list.b0 + l;
    nq = __builtin_amdgcn_readlane(list.nq, l);
    n = __builtin_amdgcn_readlane(list.n, l);
    const int len = tree_len(n), unit = rel / len, own = tree_tiles(nq, G, kRows);
    tile = unit % own;
    hk = unit / own;
    c0 = rel - unit * len;
  } else {
    const int unit = blockIdx.x / sp.pieces, piece = blockIdx.x - unit * sp.pieces;
    tile = unit % tiles;
    hk = unit / tiles % a.Hkv;
    b = unit / tiles / a.Hkv;
    nq = src.queries(b, a.Lq);
    n = src.keys(b);
    if (tile * kRows >= nq * G) return;
    const int len = tree_len(n);
    c0 = at = (int)((int64_t)len * piece / sp.pieces);
    stop = (int)((int64_t)len * (piece + 1) / sp.pieces);
  }
  for (int taken = 1;; ++taken) {
    // (a new value each time: the places that follow from it would be kept in registers
    // beside a unit's, and those of 128 spill)
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));
    const int col = lane & 31, h = lane >> 5;
    const int len = tree_len(n), c1 = min(len, c0 + stop - at);
    const int unit = ((int)b * a.Hkv + hk) * tiles + tile;
    if (sp.shares && c0 == 0 && tid == 0)
      sp.cut[unit] = i32x2{(int)blockIdx.x, c1 == len ? (int)blockIdx.x : list.last(at, len)};
    const int rows = nq * G;
    const int row0 = tile * kRows + group * 32;
    const bool mine = row0 < rows;                           // this wave has rows
    const int all = n - nq;                                  // keys that every row sees
    const int base0 = c0 * kTileKeys, nt = n > 0 ? c1 - c0 : 0;

    const int row = row0 + col, t = row / G;
    const int head = hk * G + row - t * G;
    const uint64_t* const words = src.tree + b * src.stride + (int64_t)min(t, nq - 1) * src.words;
    R r;
    {
      const uint16_t* p = a.q + (b * a.Lq + t) * a.ldq + (int64_t)head * D + 8 * h;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        r.q[i] = u32x4{0, 0, 0, 0};
        if (row < rows) r.q[i] = *reinterpret_cast<const u32x4*>(p + 16 * i);
      }
    }

    // The table's entries of 64 sixteens of keys, one a lane: those of the 16 tiles
    // that hold tile t, of the next 16, and of 16 more on their way; named: bit i, the
    // entry of lane i names a page.
    const auto entries = [&](int block) {
      const int64_t first = (int64_t)(base0 >> 4) + 64 * block + lane;
      const int key = (int)min<int64_t>(16 * first, n - 1);
      return src.c.table[b * src.c.max_pages + (key >> src.c.page_log2)];
    };
    int e0 = 0, e1 = 0, e2 = 0;
    uint64_t named0 = 0, named1 = 0;
    const auto look_at = [&] {
      named0 = __builtin_amdgcn_ballot_w64(src.named(e0));
      named1 = __builtin_amdgcn_ballot_w64(src.named(e1));
    };
    int block = 0;
    // sixteen s of tile i (within the first two blocks): whether it has a page, and
    // which (no branches: they would stand among a step's products)
    const auto has = [&](int i, int s) {
      const int at = 4 * (i - 16 * block) + s;
      return (((at < 64 ? named0 : named1) >> (at & 63)) & 1) != 0;
    };
    const auto page_of = [&](int i, int s) {
      const int at = 4 * (i - 16 * block) + s;
      const int x = __builtin_amdgcn_readlane(e0, at & 63), y = __builtin_amdgcn_readlane(e1, at & 63);
      return at < 64 ? x : y;
    };
    // A thread's units of a tile, 16 elements each: one wave's are consecutive, and from
    // one sixteen of keys.
    struct Unit {
      u32x2 w;
      uint32_t s;                    // the group scales of its lane and three others'
    };
    const auto first_of = [&](int u) { return (u * kTreeThreads + 64 * wave) & (T::kUnits - 1); };
    int to[T::kPer][2];              // the two pieces' places in a staged tile
#pragma unroll
    for (int u = 0; u < T::kPer; ++u)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int y = first_of(u) + lane, key = y / T::kGroups, c = 2 * (y % T::kGroups) + x;
        to[u][x] = T::is_v(u, wave) ? v_piece<D, true>(key, c) : k_piece<D>(key, c);
      }
    const auto load = [&](Unit& r, int u, int i) {
      const bool val = T::is_v(u, wave);
      const int y = first_of(u), s16 = y / T::kGroups >> 4;
      const int p = page_of(i, s16);
      const int64_t first = src.slot(has(i, s16) ? p : 0, hk, base0 + i * kTileKeys + 16 * s16);
      const int64_t slot = first * T::kGroups + y % (16 * T::kGroups);
      r.w = *reinterpret_cast<const u32x2*>((val ? src.c.v_q : src.c.k_q) + slot * 8 + 8 * lane);
      // (a byte's load would be widened, and so waited for, a tile too soon)
      r.s = *reinterpret_cast<const uint32_t*>((val ? src.c.v_s : src.c.k_s) + slot + (lane & ~3));
    };
    // piece x of unit u of tile i into the staged tile `tile` (what has no slot gets a
    // scale of zero: the bytes may be a NaN's).  A NaN's scale may also stand in a drafted
    // token's that some rows do not see, whose weight of zero needs a number: among
    // values it counts as 448 here, and `nans`, a sum of zeros, tells of it.
    float nans = 0.0f;
    const auto store = [&](const Unit& r, int u, int x, int i, char* staged) {
      const int key = first_of(u) / T::kGroups;
      const int left = has(i, key >> 4) ? n - (base0 + i * kTileKeys) - key : 0;
      const uint32_t s = __builtin_amdgcn_ubfe(r.s, 8 * (lane & 3), 8);
      float f = __builtin_amdgcn_cvt_f32_fp8((int)(lane / T::kGroups < left ? s : 0u), 0);
      if (T::is_v(u, wave)) {
        if (x == 0) nans = __builtin_fmaf(f, 0.0f, nans);
        f = fminf(f, 448.0f);
      }
      *reinterpret_cast<u32x4*>(staged + to[u][x]) = codes_f16(r.w[x], f16x2{(_Float16)f, (_Float16)f});
    };
    // group j: K(j + 2) and V(j) (Parts 1: V(j + 1)), loaded two tiles before they are stored
    const auto of_group = [&](int u, int j) { return j + (T::is_v(u, wave) ? kSooner : 2); };
    Unit even[T::kPer], odd[T::kPer];
    if (nt > 0) {
      e0 = entries(0);
      e1 = entries(1);
      e2 = entries(2);
      look_at();
      Unit first[T::kPer], second[T::kPer];
#pragma unroll
      for (int u = 0; u < T::kPer; ++u) {
        if (T::is_v(u, wave) && !kSooner) continue;
        load(first[u], u, 0);
        if (!T::is_v(u, wave)) load(second[u], u, 1);
      }
#pragma unroll
      for (int u = 0; u < T::kPer; ++u) {
        load(even[u], u, of_group(u, 0));
        load(odd[u], u, of_group(u, 1));
      }
#pragma unroll
      for (int u = 0; u < T::kPer; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (T::is_v(u, wave) && !kSooner) continue;
          store(first[u], u, x, 0, T::is_v(u, wave) ? vt : kt);
          if (!T::is_v(u, wave)) store(second[u], u, x, 1, kt + kBytes);
        }
    }

    r.c = query_operand<true>(r.q, a.scale * kLog2e, src.k_scale(), [](float v) { return pair_max(v); });
    r.clear();
    r.set_ones(lane);

    // this lane's places in a staged tile (attn_tile.hip), in its half of the keys
    int ka[D / 16], va[D / 32];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) ka[i] = part * kHalf + k_piece<D>(col, 2 * i + h);
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
      va[d] = kBefore + v_piece<D, true>(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1)) + 8 * (lane & 3);

    f32x16 s0 = {}, s1 = {};
    u32x4 p0[2] = {}, p1[2] = {};
    float sum = 0.0f;
    u32x4 ahead[R::kAhead];
    if (nt > 0) {
      __syncthreads();
      if (mine) {
        r.logits(s0, kt, ka);
        if constexpr (Parts == 2)
#pragma unroll
          for (int d = 0; d < D / 16; ++d) ka[d] += kBytes;
#pragma unroll
        for (int g = 0; g < R::kAhead; ++g)
          ahead[g] = r.template operand<Parts == 1 ? kHalf : 0>(g, kt, ka, vt, va);
      }
    }
    int slot = 0;                                            // t % 3
    // K(t + 2) and V into their tiles, in `turns` turns
    const auto store_turn = [&](int turn, int turns, int i, const Unit(&r)[T::kPer]) {
#pragma unroll
      for (int j = 0; j < T::kParts; ++j)
        if (turn == j * turns / T::kParts) {
          const int u = j / 2;
          const int k = (slot == 0 ? 2 : slot - 1) * kBytes, v = (!kSooner ? slot : slot == 2 ? 0 : slot + 1) * kBytes;
          store(r[u], u, j % 2, of_group(u, i), T::is_v(u, wave) ? vt + v : kt + k);
        }
    };
    // the last turns of tile t: the waves meet, group t + 2 is loaded
    const auto meet_turn = [&](int turn, int i, Unit(&r)[T::kPer]) {
      if (turn == 4) __syncthreads();
#pragma unroll
      for (int u = 0; u < T::kPer; ++u)
        if (turn == 5 + u) load(r[u], u, of_group(u, i + 2));
    };
    const auto turn_over = [&] { slot = slot == 2 ? 0 : slot + 1; };
    // all tiles in pairs (of the last one's, if it has none, no key is seen), 16 to a
    // block of entries
    const auto each = [&](const auto& pair) __attribute__((always_inline)) {
      for (int i = 0; i < nt;) {
        for (const int stop = min(nt, 16 * block + 16); i < stop; i += 2) pair(i);
        ++block;
        e0 = e1;
        e1 = e2;
        e2 = entries(block + 2);
        look_at();
      }
    };
    // what row `row` sees of tile i's keys, all: all rows see all of them
    const auto look_up = [&](int i, bool& whole) {
      const int base = base0 + i * kTileKeys;
      // (bit t of 4: sixteen t of the tile)
      const uint32_t ok = (uint32_t)(named0 >> (4 * (i & 15))) & 15u;
      uint64_t here = ~0ull;
      if (ok != 15u) {
        here = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) here |= (ok >> x) & 1 ? 0xFFFFull << (16 * x) : 0;
      }
      const int left = min(n, base0 + nt * kTileKeys) - base;
      if (left < kTileKeys) here = left <= 0 ? 0 : here & ((1ull << left) - 1);
      whole = here == ~0ull && base + kTileKeys <= all;
      return whole ? here : here & src.row_sees(words, base, all);
    };
    // Tile i.  Parts 2: `s` its logits, `next` the logits of the tile before (whose
    // weights are p); Parts 1: the same of its first half and the half before.
    const auto tile_of = [&](int i, f32x16& s, u32x4(&pn)[2], f32x16& next, u32x4(&p)[2],
                             Unit(&units)[T::kPer]) __attribute__((always_inline)) {
      bool whole;
      const uint64_t here = look_up(i, whole);
      if constexpr (Parts == 2) {
        if (!whole) hide(s, (uint32_t)(here >> (32 * part)), 64, h);
        // on to K(t + 2) and V(t)
        const int ks = slot == 1 ? -2 * kBytes : kBytes;
        const int vs = i == 0 ? part * kHalf - kBefore : slot == 0 ? -2 * kBytes : kBytes;
        r.template step<0, 0>(s, pn, next, p, sum, ahead, kt, ka, vt, va, ks, vs, [&](int turn) {
          if (turn < 4)
            store_turn(turn, 4, i, units);
          else
            meet_turn(turn, i, units);
        });
      } else {
        if (!whole) hide(s, (uint32_t)here, 64, h);
        // on to K(t + 1) and V(t)
        const int ks = slot == 2 ? -2 * kBytes : kBytes;
        const int vs = i == 0 ? -kBefore : slot == 0 ? -2 * kBytes : kBytes;
        r.template step<kHalf, 0>(s, pn, next, p, sum, ahead, kt, ka, vt, va, ks, vs,
                                  [&](int turn) { store_turn(turn - 1, 6, i, units); });
        if (!whole) hide(next, (uint32_t)(here >> 32), 64, h);
        r.template step<0, kHalf>(next, p, s, pn, sum, ahead, kt, ka, vt, va, 0, 0,
                                  [&](int turn) { meet_turn(turn, i, units); });
      }
      turn_over();
    };
    if (mine) {
      each([&](int i) {
        tile_of(i, s0, p0, s1, p1, even);
        if constexpr (Parts == 2)
          tile_of(i + 1, s1, p1, s0, p0, odd);
        else
          tile_of(i + 1, s0, p0, s1, p1, odd);
      });
      if (nt > 0) r.template second<Parts == 1 ? kHalf : 0>(s1, p1, sum, vt, va);
    } else {
      const auto pass = [&](int i, Unit(&units)[T::kPer]) {
#pragma unroll
        for (int turn = 0; turn < 4; ++turn) store_turn(turn, 4, i, units);
#pragma unroll
        for (int turn = 4; turn < 8; ++turn) meet_turn(turn, i, units);
        turn_over();
      };
      each([&](int i) {
        pass(i, even);
        pass(i + 1, odd);
      });
    }

    if (nans != nans) nan_unit = taken;
    __syncthreads();
    // the other half's sums to the common reference
    if constexpr (Parts == 2) {
      float* const join = reinterpret_cast<float*>(lds + group * kJoin) + col * (D + 4);
      if (part == 1) {
        if (h == 0) {
          ml[0][group][col] = r.m;
          ml[1][group][col] = r.l;
        }
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4*>(join + 32 * d + 2 * i + 4 * h) =
                f32x4{r.o[d][i], r.o[d][i + 1], r.o[d][i + 2], r.o[d][i + 3]};
      }
      __syncthreads();
      if (part == 0) {
        const float m1 = ml[0][group][col], top = fmaxf(r.m, m1), ref = top == -INFINITY ? 0.0f : top;
        // (times zero, not left out: a sum that is NaN stays so)
        const float f0 = r.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((r.m - ref) * r.c);
        const float f1 = m1 == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m1 - ref) * r.c);
        r.m = top;
        r.l = __builtin_fmaf(ml[1][group][col], f1, r.l * f0);
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const f32x4 o = *reinterpret_cast<const f32x4*>(join + 32 * d + 2 * i + 4 * h);
#pragma unroll
            for (int j = 0; j < 4; ++j) r.o[d][i + j] = __builtin_fmaf(o[j], f1, r.o[d][i + j] * f0);
          }
      }
      __syncthreads();
    }
    if (part == 0) {
      const bool done = sp.shares ? c1 - c0 == len : sp.pieces == 1;
      uint16_t* const out = a.o + (b * a.Lq + t) * a.ldo + (int64_t)head * D;
      int sum = blockIdx.x;
      if (sp.shares && c0 == 0) sum = sp.shares + (sp.by_unit ? unit : sum);
      const int64_t to = (int64_t)sum * kRows + group * 32 + col;
      if (done) {
        store_rows(r, src.v_scale(), out, h, row < rows);
      } else if (row < rows) {
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4*>(sp.o + to * D + 32 * d + 2 * i + 4 * h) =
                f32x4{r.o[d][i], r.o[d][i + 1], r.o[d][i + 2], r.o[d][i + 3]};
        if (h == 0) {
          sp.m[to] = r.m == -INFINITY ? r.m : r.m * r.c;
          sp.l[to] = r.l;
        }
      }
      // What the products left out: a row that sees a key with a NaN's scale has NaN in
      // that group's elements, over what this wave has just stored there.  (Hardly ever:
      // kv4_append writes no NaN.)
      if (__builtin_expect(nan_unit == taken, 0)) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
          const int base = base0 + i * kTileKeys, key = base + lane;
          const int e = src.c.table[b * src.c.max_pages + (min(key, n - 1) >> src.c.page_log2)];
          const bool there = src.named(e) && key < n;
          const uint8_t* const s = src.c.v_s + src.slot(there ? e : 0, hk, key) * (D / 16);
          const uint64_t sees = src.row_sees(words, base, all);
#pragma unroll 1
          for (int g = 0; g < D / 16; ++g) {
            const uint64_t nan = __builtin_amdgcn_ballot_w64(there && (s[g] & 0x7F) == 0x7F);
            if ((nan & sees) && row < rows) {
              const uint32_t x = done ? 0x7FC07FC0u : 0x7FC00000u;
              u32x4* const p = done ? reinterpret_cast<u32x4*>(out + 16 * g + 8 * h)
                                    : reinterpret_cast<u32x4*>(sp.o + to * D + 16 * g + 8 * h);
              p[0] = u32x4{x, x, x, x};
              if (!done) p[1] = u32x4{x, x, x, x};
            }
          }
        }
      }
    }
    // on to the next unit
    at += c1 - c0;
    if (at >= stop) return;
    c0 = 0;
    if (++tile == tree_tiles(nq, G, kRows)) {
      tile = 0;
      if (++hk == a.Hkv) {
        hk = 0;
        do nq = src.queries(++b, a.Lq);
        while (nq == 0);
        n = src.keys(b);
      }
    }
  }
}

// The rows whose keys were cut: their pieces in order, kTurn of them read at a time; D / 4
// lanes a row.
template <int D, int Parts>
__global__ void __launch_bounds__(256)
join_tree_kernel(AttnArgs a, Kv4TreeSource src, TreeSums sp, int tiles, Gate gate) {
  if (gated_off(gate)) return;
  constexpr int kLanes = D / 4, kPer = 256 / kLanes, kTurn = 4, kRows = tree_rows(Parts);
  const int d = 4 * (threadIdx.x % kLanes);
  const int64_t at = (int64_t)blockIdx.x * kPer + threadIdx.x / kLanes;  // (b Lq + t) Hq + head
  if (at >= a.B * a.Lq * a.Hq) return;
  const uint32_t qrow = (uint32_t)at / a.Hq, b = qrow / (uint32_t)a.Lq;  // (below 2^24)
  const int head = (int)((uint32_t)at - qrow * a.Hq), t = (int)(qrow - b * (uint32_t)a.Lq), G = a.Hq / a.Hkv;
  const int hk = head / G, row = t * G + head - hk * G;
  const int unit = (b * a.Hkv + hk) * tiles + row / kRows;
  int w0 = unit * sp.pieces, w1 = w0 + sp.pieces - 1, from = w0;
  if (sp.shares) {
    const i32x2 cut = sp.cut[unit];                        // (of a row that is there)
    w0 = cut[0];
    w1 = cut[1];
    from = sp.shares + (sp.by_unit ? unit : w0);
  }
  if (t >= src.queries(b, a.Lq) || w0 == w1) return;
  float mt = -INFINITY, l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  for (int s0 = w0; s0 <= w1; s0 += kTurn) {
    float ms[kTurn], ls[kTurn];
    f32x4 os[kTurn];
    float top = mt;
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      ms[j] = -INFINITY;
      ls[j] = 0.0f;
      os[j] = f32x4{0, 0, 0, 0};
      if (s0 + j <= w1) {
        const int64_t i = (int64_t)(s0 + j == w0 ? from : s0 + j) * kRows + row % kRows;
        ms[j] = sp.m[i];
        ls[j] = sp.l[i];
        os[j] = *reinterpret_cast<const f32x4*>(sp.o + i * D + d);
      }
    }
#pragma unroll
    for (int j = 0; j < kTurn; ++j) top = fmaxf(top, ms[j]);
    const float ref = top == -INFINITY ? 0.0f : top;
    const float f = mt == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mt - ref);
    mt = top;
    l *= f;
    o *= f;
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      // (times zero, not left out: a sum that is NaN stays so)
      const float fj = ms[j] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ms[j] - ref);
      l = __builtin_fmaf(ls[j], fj, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(os[j][e], fj, o[e]);
    }
  }
  const float f = l == 0.0f ? 0.0f : src.v_scale() / l;
  *reinterpret_cast<u32x2*>(a.o + qrow * a.ldo + (int64_t)head * D + d) =
      u32x2{bf16_pack(o[0] * f, o[1] * f), bf16_pack(o[2] * f, o[3] * f)};
}

// One workgroup fits a compute unit: this many run at once.
constexpr int kPlaces = 256;
constexpr int kPieces = 16;

// Rows up to which a tile is of two parts.
int parts_of(int64_t Lq, int Hq, int Hkv) { return Lq * (Hq / Hkv) <= tree_rows(2) ? 2 : 1; }
int64_t units_of(int64_t B, int64_t Lq, int Hq, int Hkv) {
  const int rows = tree_rows(parts_of(Lq, Hq, Hkv));
  return B * Hkv * ((Lq * (Hq / Hkv) + rows - 1) / rows);
}

// us: a unit's start and end; a tile of keys; 64 streams of the list; what sums cost, written and
// read again at 4 TB/s, and the launch that joins them.
constexpr double kUnitStart = 10.0, kListTime = 5.0;
double tree_tile_time(int D, int parts) { return D == 64 ? (parts == 2 ? 0.8 : 1.1) : (parts == 2 ? 1.25 : 1.9); }
double tree_join_time(int64_t sums, int rows, int D) { return 4.0 + (double)sums * rows * D * 4 * 1.5 / 4e6; }

// How `units` of `len` tiles are cut: the time of n equal pieces is that of their
// rounds, the shares' that of what each compute unit has.  Streams of one length
// are assumed, and the shares taken up to a tenth more: they stay as good where the
// lengths differ (16 streams of 16384 to 32768 keys, 8 key heads of 128, 128 rows: 1.1 times
// as long in two pieces each as in shares; all of 32000, 4 streams of 16 key heads: 180
// and 180; of 8000: 56 and 59; of 4000: 37 and 40).
struct TreeCut {
  int shares, pieces;
  int64_t sums;
  size_t bytes;
};
TreeCut tree_cut(int64_t B, int64_t units, int rows, int D, int parts, int64_t len, size_t ws_bytes) {
  TreeCut best = {0, 1, 0, 0};
  const double each = tree_tile_time(D, parts);
  double least = (double)((units + kPlaces - 1) / kPlaces) * ((double)len * each + kUnitStart);
  const auto take = [&](int shares, int pieces, int64_t sums) {
    best = {shares, pieces, sums, TreeSums::bytes(sums, shares ? units : 0, rows, D)};
  };
  for (int n = 2; n <= kPieces && n <= len && units * n <= 8 * kPlaces; ++n) {
    if (TreeSums::bytes(units * n, 0, rows, D) > ws_bytes) break;
    const double t = (double)((units * n + kPlaces - 1) / kPlaces) * ((double)((len + n - 1) / n) * each + kUnitStart) +
                     tree_join_time(units * n, rows, D);
    if (t < least) {
      least = t;
      take(0, n, units * n);
    }
  }
  if (units >= 8 * kPlaces || units * len * kPlaces >= (int64_t)1 << 31) return best;
  for (int shares = kPlaces; shares >= kPlaces / 2; shares -= 16) {
    const int64_t sums = shares + (units < shares ? units : shares);
    if (TreeSums::bytes(sums, units, rows, D) > ws_bytes) continue;
    const double per = (double)units / shares;
    const double t = kListTime * (double)((B + 63) / 64) + per * (double)len * each + (1.0 + per) * kUnitStart +
                     tree_join_time(sums, rows, D);
    if (t < 1.1 * least) take(shares, 0, sums);
    break;
  }
  return best;
}

}  // namespace

// (asked for: at most 32 MiB, whatever more would give)
size_t attn_tree_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  const int parts = parts_of(Lq, Hq, Hkv);
  return tree_cut(B, units_of(B, Lq, Hq, Hkv), tree_rows(parts), D, parts, (L + kTileKeys - 1) / kTileKeys,
                  (size_t)32 << 20).bytes;
}

hipError_t launch_attn_tree(const AttnArgs& a, const Kv4TreeSource& src, int64_t L, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  const Gate gt = current_gate();
  const int parts = parts_of(a.Lq, a.Hq, a.Hkv), rows = tree_rows(parts);
  const int64_t units = units_of(a.B, a.Lq, a.Hq, a.Hkv);
  const TreeCut c = tree_cut(a.B, units, rows, a.D, parts, (L + kTileKeys - 1) / kTileKeys, ws_bytes);
  TreeSums sp = {};
  sp.shares = c.shares;
  sp.pieces = c.pieces;
  sp.by_unit = units <= c.shares;
  if (c.bytes) {
    sp.o = static_cast<float*>(ws);
    sp.m = sp.o + c.sums * rows * a.D;
    sp.l = sp.m + c.sums * rows;
    sp.cut = reinterpret_cast<i32x2*>(sp.l + c.sums * rows);
  }
  const dim3 grid((unsigned)(c.shares ? c.shares : units * c.pieces)), block(kTreeThreads);
  const int tiles = (int)(units / (a.B * a.Hkv));
  const int64_t per = 256 / (a.D / 4);
  const dim3 rows_grid((unsigned)((a.B * a.Lq * a.Hq + per - 1) / per));
  const auto go = [&](auto kernel, auto join) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, src, sp, tiles, gt);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !c.bytes) return e;
    hipLaunchKernelGGL(join, rows_grid, dim3(256), 0, stream, a, src, sp, tiles, gt);
    return hipGetLastError();
  };
  if (parts == 2)
    return a.D == 64 ? go(attn_tree_kernel<64, 2>, join_tree_kernel<64, 2>)
                     : go(attn_tree_kernel<128, 2>, join_tree_kernel<128, 2>);
  return a.D == 64 ? go(attn_tree_kernel<64, 1>, join_tree_kernel<64, 1>)
                   : go(attn_tree_kernel<128, 1>, join_tree_kernel<128, 1>);
}

}  // namespace qact
