// Staging of a tile of 64 keys and values in shared memory as 16-bit operands, for
// the kernels of many query rows.
#pragma once

#include "attn_common.h"
#include "attn_rows.h"

namespace qact {

// Staging by T threads: a thread takes kPer units, each of K or of V, the same
// for a whole wave.  A unit is loaded a tile before it is stored; both are
// done piece by piece in the turns of a step, beside the step's MFMAs, and
// without branches, which would keep their scalar work from running there (all
// at once, staging a tile took a third of the time).  So every load has a valid
// place: past the end the last one's, whose keys nobody sees.
template <class Source, int D, int T>
struct Tile;

// NVFP4: a unit is a group of 16 elements, stored as two 16-byte pieces.
template <int D, int T>
struct Tile<Kv4Source, D, T> {
  static constexpr int kGroups = D / 16;
  static constexpr int kUnits = kTileKeys * kGroups;
  static constexpr int kPer = 2 * kUnits / T;
  static constexpr int kParts = 2 * kPer;

  // a unit's fixed places (a wave's lies within one sixteen of keys)
  struct Place {
    const uint8_t *q, *s;          // in the slots of that sixteen
    int key, sixteen;              // key in the tile
    int at[2];                     // each part's place in a staged tile
  };
  struct Regs {
    u32x2 w;
    uint32_t s;                    // group scale
    int left;                      // keys of the tile that have slots, from its start
  };
  static __device__ __forceinline__ bool is_v(int u, int wave) { return u * T + 64 * wave >= kUnits; }
  static __device__ __forceinline__ void place(Place& r, const Kv4Source& s, int64_t, int, int u,
                                               int wave, int lane) {
    const bool val = is_v(u, wave);
    const int y = (u * T + 64 * wave) & (kUnits - 1), key = (y + lane) / kGroups, g = (y + lane) % kGroups;
    const int z = (y + lane) & (16 * kGroups - 1);         // (key % 16, group)
    r.q = (val ? s.c.v_q : s.c.k_q) + 8 * z;
    r.s = (val ? s.c.v_s : s.c.k_s) + z;
    r.key = key;
    r.sixteen = y / kGroups >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      r.at[h] = val ? v_piece<D>(key, 2 * g + h) : k_piece<D>(key, 2 * g + h);
  }
  static __device__ __forceinline__ void load(Regs& r, const Place& pl, const Kv4Source& s,
                                              const Kv4Source::Look& pg, uint64_t, int hk, int base,
                                              int n) {
    const int p = s.entry(pg, pl.sixteen), at = base + 16 * pl.sixteen;
    const bool ok = s.named(p) && at < n;
    const int64_t slot = s.slot(ok ? p : 0, hk, at);
    r.w = *reinterpret_cast<const u32x2*>(pl.q + slot * (D / 2));
    r.s = pl.s[slot * kGroups];
    r.left = ok ? n - base : 0;
  }
  // part h into the staged tile `to`; what has no slot gets a scale of zero (the
  // bytes may be a NaN's)
  static __device__ __forceinline__ void store(const Regs& r, const Place& pl, int h, char* to) {
    const f16x2 sc = scale_f16<0>(pl.key < r.left ? r.s : 0u);
    *reinterpret_cast<u32x4*>(to + pl.at[h]) = codes_f16(r.w[h], sc);
  }
};

template <int D, int T>
struct Tile<Kv4TreeSource, D, T> : Tile<Kv4Source, D, T> {};

// bf16 states: a unit is a 16-byte piece.
template <int D, int T>
struct Tile<CrossSource, D, T> {
  static constexpr int kPieces = D / 8;
  static constexpr int kUnits = kTileKeys * kPieces;
  static constexpr int kPer = 2 * kUnits / T;
  static constexpr int kParts = kPer;

  struct Place {
    const uint16_t* p;             // in state 0 of the sequence
    int64_t ld;
    int key, at;
  };
  struct Regs {
    u32x4 w;
    uint64_t seen;
  };
  static __device__ __forceinline__ bool is_v(int u, int wave) { return u * T + 64 * wave >= kUnits; }
  static __device__ __forceinline__ void place(Place& r, const CrossSource& s, int64_t b, int hk,
                                               int u, int wave, int lane) {
    const bool val = is_v(u, wave);
    const int y = ((u * T + 64 * wave) & (kUnits - 1)) + lane, key = y / kPieces, c = y % kPieces;
    r.ld = val ? s.ldv : s.ldk;
    r.p = (val ? s.v : s.k) + b * s.Lk * r.ld + hk * D + 8 * c;
    r.key = key;
    r.at = val ? v_piece<D>(key, c) : k_piece<D>(key, c);
  }
  static __device__ __forceinline__ void load(Regs& r, const Place& pl, const CrossSource&,
                                              const CrossSource::Look&, uint64_t seen, int,
                                              int base, int n) {
    r.w = *reinterpret_cast<const u32x4*>(pl.p + min(base + pl.key, n - 1) * pl.ld);
    r.seen = seen;
  }
  // (what is not seen may hold NaN: zeros)
  static __device__ __forceinline__ void store(const Regs& r, const Place& pl, int, char* to) {
    const bool on = (r.seen >> pl.key) & 1;
    *reinterpret_cast<u32x4*>(to + pl.at) = u32x4{on ? r.w[0] : 0u, on ? r.w[1] : 0u,
                                                  on ? r.w[2] : 0u, on ? r.w[3] : 0u};
  }
};

}  // namespace qact
