// Attention of many query rows (a frame's tokens, a whole block's): a
// workgroup holds 128 or 256 rows, its waves 32 or 64 each, and takes the
// keys in tiles of 64 that it stages in shared memory as 16-bit operands (an
// NVFP4 tile is expanded once for all rows), one tile ahead of the one that
// the MFMAs read.
//
// What bounds it is the VALU: for heads of 64 the weights of 32 keys take about
// 165 ns of a SIMD, the two products' MFMAs 121.  Both run at once only when ONE
// wave's instructions alternate between them (an MFMA and up to 7 VALU
// instructions: the time of the longer; the same from two waves: nearly the
// sum), so a wave forms the weights of 32 keys while its MFMAs compute the
// logits of the next 32 and the second product of the 32 before.
//
// For the same reason the VALU is left with as little else as possible: no
// maximum is taken of most tiles.  The weights are formed to the reference that
// the row has and summed, which has to be done anyway; only where a sum says
// that a weight may have grown beyond 2^8 times the reference's are the maxima
// taken and the weights formed again (in fp16, too, they stay in range).  A
// lane holds one query row, so that costs one exchange between lanes.
#include "attn_common.h"

namespace qact {

namespace {

constexpr int kTileKeys = 64;
// A weight is p 2^kTileBias relative to the reference, which moves when the
// weights of 32 keys sum to more than kTileMost (2^8 times a weight of 1).
template <bool F16>
constexpr float kTileBias = F16 ? 7.0f : 0.0f;
template <bool F16>
constexpr float kTileMost = F16 ? 32768.0f : 256.0f;

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Position of 16-byte piece c of key `key` in a staged tile (bytes).  K is
// read as 16-byte pieces of 32 keys, V as 32-byte pieces of 8 keys; the
// exchange among a key's pieces spreads either over all banks.
template <int D>
__device__ __forceinline__ int k_piece(int key, int c) {
  return key * (D * 2) + 16 * (c ^ (D == 128 ? key & 15 : (key >> 1) & 7));
}
template <int D>
__device__ __forceinline__ int v_piece(int key, int c) {
  return key * (D * 2) + 32 * ((c >> 1) ^ (D == 128 ? key & 7 : key & 3)) + 16 * (c & 1);
}

// Before a row has seen a key: any logit plus this gives an infinite weight,
// minus infinity (not seen) one of zero.
constexpr float kNoReference = 0x1.fffffep127f;

// How a row tile's keys are cut: n pieces, each `size` parts of `whole` and
// the last one what is left.
struct Pieces {
  int n, size, whole;
};

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

__device__ __forceinline__ float row_max(const f32x16& s) {
  float top = max3(s[0], s[1], s[2]);
#pragma unroll
  for (int i = 3; i < 15; i += 2) top = max3(top, s[i], s[i + 1]);
  return pair_max(fmaxf(top, s[15]));
}

// One wave's rows: 32, a lane's row is its column of S^T (both halves of the
// wave hold it, each half its keys).
template <bool F16, int D>
struct Rows {
  u32x4 q[D / 16];
  f32x16 o[D / 32];
  u32x4 ones;                       // see sums()
  float c, m, l, shift;

  // Sum of a row's weights of 32 keys, on the MFMA: 16x16x32 takes the
  // weights' registers as 16 columns and four groups of k, lanes l and l + 32
  // (l + 16 and l + 48) being the two halves of row l % 16 (of row 16 + l % 16).
  // Rows 0 and 8 of `ones` pick groups 0 and 2, rows 4 and 12 groups 1 and 3,
  // so that every lane's first result is its own row's sum.  (On the VALU the
  // sum costs 30 to 45 ns a step, here 10.)  A weight that is infinite or NaN
  // makes the sums of rows l and l + 16 NaN: settle() sums those itself.
  __device__ __forceinline__ void set_ones(int lane) {
    const int row = lane & 15, g = lane >> 4;
    const uint32_t w = (row & 3) == 0 && ((row >> 2) & 1) == (g & 1) ? (F16 ? 0x3C003C00u : 0x3F803F80u) : 0u;
    ones = u32x4{w, w, w, w};
  }

  // The weights p of 32 keys whose logits are s, formed to the present
  // reference, are about to be used: if one may be too large for some row, move
  // the rows' references to their maxima and form them again.
  __device__ __forceinline__ void settle(const f32x16& s, u32x4 (&p)[2], float sum) {
    if (__builtin_amdgcn_ballot_w64(!(sum <= kTileMost<F16>))) {
      const float mn = fmaxf(m, row_max(s));
      const float ref = mn == -INFINITY ? 0.0f : mn;
      const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - ref) * c);
      m = mn;
      shift = mn == -INFINITY ? kNoReference : kTileBias<F16> - ref * c;
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] *= f;
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i], c, shift));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + 1], c, shift));
        p[i >> 2][i & 3] = pack16<F16>(e0, e1);
        sum += e0 + e1;
      }
      sum = pair_sum(sum);
    }
    l += sum;
  }

  // Step: settle the weights p (formed from `next`, their sum in `sum`); then
  // the logits of 32 keys (K at ka + KV, into `next`) and the second product of
  // p (V at va + KV) alternate with the weights of s, which go to pn and `sum`.
  // `head`: the first operands, read in the step before; this step reads those
  // of the next one (ka, va moved on by ks, vs, at offset NEXT).  side(i): what
  // else is done in turn i of 8.
  static constexpr int kN = 2 * (D / 16);       // products, of the two kinds in turn
  static constexpr int kAhead = 4;              // operands read ahead
  template <int KV>
  __device__ __forceinline__ u32x4 operand(int g, const char* k, const int (&ka)[D / 16],
                                           const char* v, const int (&va)[D / 32]) {
    return g & 1 ? v_operand<KV>(v, va, g / 2 / (D / 32), g / 2 % (D / 32))
                 : *reinterpret_cast<const u32x4*>(k + KV + ka[g / 2]);
  }
  template <int KV, int NEXT, class Side>
  __device__ __forceinline__ void step(const f32x16& s, u32x4 (&pn)[2], f32x16& next,
                                       u32x4 (&p)[2], float& sum, u32x4 (&head)[kAhead],
                                       const char* k, int (&ka)[D / 16], const char* v,
                                       int (&va)[D / 32], int ks, int vs, Side side) {
    u32x4 f[kN + kAhead];
#pragma unroll
    for (int g = 0; g < kAhead; ++g) f[g] = head[g];
    settle(next, p, sum);
    next = f32x16{};
    // the weights of pair i in stages, one a turn, so that no instruction waits
    // for the one before it
    float x[16];
    f32x4 total = {0, 0, 0, 0};
    x[0] = __builtin_fmaf(s[0], c, shift);
    x[1] = __builtin_fmaf(s[1], c, shift);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      side(i);
#pragma unroll
      for (int g = i * kN / 8; g < (i + 1) * kN / 8; ++g) {
        if (g + kAhead < kN) {
          f[g + kAhead] = operand<KV>(g + kAhead, k, ka, v, va);
        } else {
          if (g + kAhead == kN) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) ka[d] += ks;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) va[d] += vs;
          }
          f[g + kAhead] = operand<NEXT>(g + kAhead - kN, k, ka, v, va);
        }
        if (g & 1)
          o[g / 2 % (D / 32)] = mfma32<F16>(f[g], p[g / 2 / (D / 32)], o[g / 2 % (D / 32)]);
        else
          next = mfma32<F16>(f[g], q[g / 2], next);
      }
      if (i == 5) total = mfma16<F16>(ones, pn[0], total);
      if (i > 0) pn[(i - 1) >> 2][(i - 1) & 3] = pack16<F16>(x[2 * i - 2], x[2 * i - 1]);
      x[2 * i] = __builtin_amdgcn_exp2f(x[2 * i]);
      x[2 * i + 1] = __builtin_amdgcn_exp2f(x[2 * i + 1]);
      if (i < 7) {
        x[2 * i + 2] = __builtin_fmaf(s[2 * i + 2], c, shift);
        x[2 * i + 3] = __builtin_fmaf(s[2 * i + 3], c, shift);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    pn[1][3] = pack16<F16>(x[14], x[15]);
    sum = mfma16<F16>(ones, pn[1], total)[0];
#pragma unroll
    for (int g = 0; g < kAhead; ++g) head[g] = f[kN + g];
  }
  // V^T of 16 keys s16 and elements 32 d .. as the second product's operand
  template <int VO>
  static __device__ __forceinline__ u32x4 v_operand(const char* v, const int (&va)[D / 32], int s16,
                                                    int d) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(v + va[d] + VO + (16 * s16 + 8 * j) * (D * 2)));
      const u32x2 pr = __builtin_bit_cast(u32x2, w);
      r[2 * j] = pr[0];
      r[2 * j + 1] = pr[1];
    }
    return r;
  }
  __device__ __forceinline__ void logits(f32x16& next, const char* k, const int (&ka)[D / 16]) {
    next = f32x16{};
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      next = mfma32<F16>(*reinterpret_cast<const u32x4*>(k + ka[i]), q[i], next);
  }
  template <int VO>
  __device__ __forceinline__ void second(const f32x16& s, u32x4 (&p)[2], float sum, const char* v,
                                         const int (&va)[D / 32]) {
    settle(s, p, sum);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      o[i % (D / 32)] = mfma32<F16>(v_operand<VO>(v, va, i / (D / 32), i % (D / 32)),
                                    p[i / (D / 32)], o[i % (D / 32)]);
  }
};

// What is not seen of 32 keys: minus infinity.  `seen` from the first of
// them; left: keys that this lane's row sees from there on.
__device__ __forceinline__ void hide(f32x16& s, uint32_t seen, int left, int h) {
  left -= 4 * h;
  uint32_t bits = seen >> (4 * h);
  bits &= left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1;
#pragma unroll
  for (int i = 0; i < 16; ++i)      // element i is key 8 (i / 4) + 4 h + i % 4
    s[i] = bits & (1u << (8 * (i >> 2) + (i & 3))) ? s[i] : -INFINITY;
}

// Workgroup: (piece of the keys, stream, key head, row tile), the row tile
// running fastest.  W waves of 32 rows each.
//
// Tile t is computed in two steps of 32 keys, each with the logits of the
// step after it and the second product of the step before it.  Shared memory
// holds three tiles of K and of V: between the middles of the second steps of
// tiles t - 1 and t, where the workgroup meets, K(t), V(t - 1), K(t + 1) and
// V(t) are read and K(t + 2) and V(t + 1) written, which replace K(t - 1) and
// V(t - 2), read before.  So operands can be read ahead across the steps.
template <class Source, int D, int W>
__global__ void __launch_bounds__(64 * W, 2)
attn_tile_kernel(AttnArgs a, Source src, AttnSplit sp, int tiles, Pieces pc, Gate gate) {
  if (gated_off(gate)) return;
  using T = Tile<Source, D, 64 * W>;
  constexpr bool kF16 = Source::kF16;
  constexpr int kBytes = kTileKeys * D * 2, kHalf = kBytes / 2;
  __shared__ __align__(16) char kt[3 * kBytes];            // three tiles
  __shared__ __align__(16) char vt[3 * kBytes];

  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = blockIdx.x % tiles;
  const int at = blockIdx.x / tiles, hk = at % a.Hkv;
  const int bs = at / a.Hkv, piece = bs / (int)a.B;
  const int64_t b = bs - piece * (int)a.B;
  const int G = a.Hq / a.Hkv;
  const int nq = src.queries(b, a.Lq), n = src.keys(b);
  const int rows = nq * G;
  if (tile * (32 * W) >= rows) return;
  const int row0 = tile * (32 * W) + wave * 32;           // the wave's first row
  const int wlast = min(row0 + 32, rows) - 1;             // and last (before row0: it has none)

  // keys that every row of the wave sees, that any row of it and of the
  // workgroup sees
  const int all = src.causal ? n - (nq - 1 - row0 / G) : n;
  const int wend = wlast < row0 ? 0 : (src.causal ? n - (nq - 1 - wlast / G) : n);
  const int last = min(tile * (32 * W) + 32 * W, rows) - 1;
  const int end = src.causal ? n - (nq - 1 - last / G) : n;
  const int chunks = (max(end, 0) + kTileKeys - 1) / kTileKeys;
  const int c0 = (int)((int64_t)chunks * (piece * pc.size) / pc.whole);
  const int c1 = (int)((int64_t)chunks * min(piece * pc.size + pc.size, pc.whole) / pc.whole);
  const int base0 = c0 * kTileKeys, nt = c1 - c0;
  // tiles of which this wave's rows see anything
  const int mine = min(nt, max(0, (wend - base0 + kTileKeys - 1) / kTileKeys));

  // seen[j]: the keys of tile t + j; look_v, look_k: what the loads of V(t + 2)
  // and K(t + 3) need.
  typename T::Place place[T::kPer];
  typename T::Regs regs[T::kPer], first[T::kPer], second[T::kPer];
  typename Source::Look look_v = {}, look_k = {};
  uint64_t seen[4] = {0, 0, 0, 0};
  if (nt > 0) {
    const typename Source::Look look0 = src.look(b, base0, n, lane);
    const typename Source::Look look1 = src.look(b, base0 + kTileKeys, n, lane);
    look_v = src.look(b, base0 + 2 * kTileKeys, n, lane);
    look_k = src.look(b, base0 + 3 * kTileKeys, n, lane);
    seen[0] = src.seen(look0, base0, n, lane);
    seen[1] = src.seen(look1, base0 + kTileKeys, n, lane);
    seen[2] = src.seen(look_v, base0 + 2 * kTileKeys, n, lane);
#pragma unroll
    for (int u = 0; u < T::kPer; ++u) {
      const int base1 = base0 + kTileKeys, base2 = base1 + kTileKeys;
      T::place(place[u], src, b, hk, u, wave, lane);
      T::load(first[u], place[u], src, look0, seen[0], hk, base0, n);
      T::load(second[u], place[u], src, look1, seen[1], hk, base1, n);
      if (T::is_v(u, wave))
        regs[u] = second[u];
      else
        T::load(regs[u], place[u], src, look_v, seen[2], hk, base2, n);
    }
  }

  const int row = row0 + col, t = row / G;
  const int upto = src.causal ? n - (nq - 1 - t) : n;
  const int head = hk * G + row - t * G;
  Rows<kF16, D> r;
  {
    const uint16_t* p = a.q + (b * a.Lq + t) * a.ldq + (int64_t)head * D + 8 * h;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      r.q[i] = u32x4{0, 0, 0, 0};
      if (row < rows) r.q[i] = *reinterpret_cast<const u32x4*>(p + 16 * i);
    }
  }
  r.c = query_operand<kF16>(r.q, a.scale * kLog2e, src.k_scale(),
                            [](float v) { return pair_max(v); });
  r.m = -INFINITY;
  r.shift = kNoReference;
  r.l = 0.0f;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) r.o[d] = f32x16{};
  r.set_ones(lane);

  // this lane's places in a staged tile: K of key `col`, piece 2 i + h (keys
  // 32 further on: the same exchange of pieces); V of keys 4 h + lane % 16 / 4
  // (8 and 16 further on: the same), elements 32 d + 16 (lane / 16 % 2) + 4 (lane % 4)
  int ka[D / 16], va[D / 32];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) ka[i] = k_piece<D>(col, 2 * i + h);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
    va[d] = v_piece<D>(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1)) + 8 * (lane & 3);

  f32x16 s0 = {}, s1 = {};
  u32x4 p0[2] = {}, p1[2] = {};
  float sum = 0.0f;
  u32x4 ahead[Rows<kF16, D>::kAhead];
  if (nt > 0) {
#pragma unroll
    for (int j = 0; j < T::kParts; ++j) {
      const int u = j * T::kPer / T::kParts, part = j % (T::kParts / T::kPer);
      T::store(first[u], place[u], part, T::is_v(u, wave) ? vt : kt);
      if (!T::is_v(u, wave)) T::store(second[u], place[u], part, kt + kBytes);
    }
    __syncthreads();
    if (mine > 0) {
      r.logits(s0, kt, ka);
#pragma unroll
      for (int g = 0; g < Rows<kF16, D>::kAhead; ++g)
        ahead[g] = r.template operand<kHalf>(g, kt, ka, vt, va);
    }
  }
  // The tile's turns of staging.  slot: i % 3; the tiles that are stored come
  // after the last one, too (into places that nobody reads any more).
  int slot = 0;
  auto store_turn = [&](int turn) {
#pragma unroll
    for (int j = 0; j < T::kParts; ++j)
      if (turn == 1 + j * 6 / T::kParts) {
        const int u = j * T::kPer / T::kParts, part = j % (T::kParts / T::kPer);
        const int k = (slot == 0 ? 2 : slot - 1) * kBytes, v = (slot == 2 ? 0 : slot + 1) * kBytes;
        T::store(regs[u], place[u], part, T::is_v(u, wave) ? vt + v : kt + k);
      }
  };
  auto load_turn = [&](int turn, int base) {         // base: of tile i
#pragma unroll
    for (int u = 0; u < T::kPer; ++u)
      if (turn == 1 + u * 3 / T::kPer) {
        const bool val = T::is_v(u, wave);
        typename Source::Look look = look_k;
        if (val) look = look_v;
        T::load(regs[u], place[u], src, look, val ? seen[2] : seen[3], hk,
                base + (val ? 2 : 3) * kTileKeys, n);
      }
    if (turn == 0) seen[3] = src.seen(look_k, base + 3 * kTileKeys, n, lane);
    if (turn == 5) {
      look_v = look_k;
      look_k = src.look(b, base + 4 * kTileKeys, n, lane);
      seen[0] = seen[1];
      seen[1] = seen[2];
      seen[2] = seen[3];
      slot = slot == 2 ? 0 : slot + 1;
    }
  };
  int i = 0;
  for (; i < mine; ++i) {
    const int base = base0 + i * kTileKeys;
    const uint64_t here = seen[0];
    const bool whole = here == ~0ull && base + kTileKeys <= all;
    // `va` is at the tile before (in the first there is none: weights of zero
    // on this tile's values), `ka` at this one; on to the next tile of K (after
    // the last: logits that nobody looks at) and to this one of V
    const int ks = slot == 2 ? -2 * kBytes : kBytes;
    const int vs = i == 0 ? 0 : slot == 0 ? -2 * kBytes : kBytes;
    if (!whole) hide(s0, (uint32_t)here, upto - base, h);
    r.template step<kHalf, 0>(s0, p0, s1, p1, sum, ahead, kt, ka, vt, va, ks, vs,
                              [&](int turn) { store_turn(turn); });
    if (!whole) hide(s1, (uint32_t)(here >> 32), upto - base - 32, h);
    r.template step<0, kHalf>(s1, p1, s0, p0, sum, ahead, kt, ka, vt, va, 0, 0, [&](int turn) {
      load_turn(turn, base);
      if (turn == 4) __syncthreads();
    });
  }
  if (mine > 0) r.template second<kHalf>(s1, p1, sum, vt, va);
  // tiles that only other waves' rows see
  for (; i < nt; ++i) {
#pragma unroll
    for (int turn = 0; turn < 8; ++turn) store_turn(turn);
#pragma unroll
    for (int turn = 0; turn < 8; ++turn) load_turn(turn, base0 + i * kTileKeys);
    __syncthreads();
  }

  const float lt = r.l;
  if (pc.n == 1) {
    const float f = lt == 0.0f ? 0.0f : src.v_scale() / lt;
    uint16_t* dst = a.o + (b * a.Lq + t) * a.ldo + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        // elements 8 (i / 4) + 4 h + 0..3 and 8 (i / 4 + 1) + 4 h + 0..3: lanes l and
        // l + 32 exchange halves, so that each holds 8 consecutive ones
        const auto w0 = __builtin_amdgcn_permlane32_swap(
            bf16_pack(r.o[d][i] * f, r.o[d][i + 1] * f),
            bf16_pack(r.o[d][i + 4] * f, r.o[d][i + 5] * f), false, false);
        const auto w1 = __builtin_amdgcn_permlane32_swap(
            bf16_pack(r.o[d][i + 2] * f, r.o[d][i + 3] * f),
            bf16_pack(r.o[d][i + 6] * f, r.o[d][i + 7] * f), false, false);
        if (row < rows)
          *reinterpret_cast<u32x4*>(dst + 32 * d + 2 * i + 8 * h) = u32x4{w0[0], w1[0], w0[1], w1[1]};
      }
  } else if (row < rows) {
    const int64_t to = (int64_t)piece * sp.rows + (b * a.Lq + t) * a.Hq + head;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(sp.o + to * D + 32 * d + 2 * i + 4 * h) =
            f32x4{r.o[d][i], r.o[d][i + 1], r.o[d][i + 2], r.o[d][i + 3]};
    if (h == 0) {
      sp.m[to] = r.m == -INFINITY ? r.m : r.m * r.c;
      sp.l[to] = lt;
    }
  }
}

// rows of a workgroup
constexpr int kTileWaves = 8;
constexpr int kTileRows = 32 * kTileWaves;

// One workgroup fits a CU: this many run at once.  Row tiles that do not fill
// them (or fill them badly) have their keys cut into pieces: S equal ones, or
// as many large ones as fit at once and a small one for the places that are
// left, which takes each of those several times.  The cost in us: the
// time of the slowest place, and for more than one piece the partial sums,
// written and read again, and the launch that joins them.
constexpr int64_t kPlaces = 256;

Pieces pieces_of(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L, size_t ws_bytes) {
  const int64_t rows = B * Lq * Hq;
  const int64_t u = B * Hkv * ((Lq * (Hq / Hkv) + kTileRows - 1) / kTileRows);
  const int64_t chunks = (L + kTileKeys - 1) / kTileKeys;
  const double tau = D == 64 ? 1.1 : 1.9;                      // us a tile of keys
  const int64_t fit = (int64_t)(ws_bytes / AttnSplit::bytes(rows, D));
  Pieces best = {1, 1, 1};
  double least = 0.0;
  for (int n = 1; n <= 16; ++n) {
    if (n > 1 && (n > fit || n > chunks)) break;
    for (int uneven = 0; uneven < 2; ++uneven) {
      Pieces p = {n, 1, n};
      double span;                                              // of the slowest place, of `whole`
      if (!uneven) {
        const int64_t k = u * n;
        span = (double)((k + kPlaces - 1) / kPlaces);
      } else {
        const int64_t left = kPlaces - u * (n - 1);             // places beside the large pieces
        if (n < 2 || left <= 0) continue;
        p.size = (int)((u + left - 1) / left);
        if (p.size < 2) continue;
        p.whole = (n - 1) * p.size + 1;
        span = p.size;
      }
      double cost = span / p.whole * (double)chunks * tau;
      if (n > 1) cost += 4.0 + (double)n * (double)rows * D * 4 * 1.5 / 4e6;
      if (n == 1 || cost < least) {
        least = cost;
        best = p;
      }
    }
  }
  return best;
}

}  // namespace

size_t attn_tile_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  const Pieces p = pieces_of(B, Lq, Hq, Hkv, D, L, (size_t)1 << 40);
  return p.n > 1 ? p.n * AttnSplit::bytes(B * Lq * Hq, D) : 0;
}

template <class Source>
hipError_t launch_attn_tile(const AttnArgs& a, const Source& src, int64_t L, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  const Gate gt = current_gate();
  const int64_t rows = a.B * a.Lq * a.Hq;
  Pieces pc = pieces_of(a.B, a.Lq, a.Hq, a.Hkv, a.D, L, ws_bytes);
#ifdef TS
  if (TS * AttnSplit::bytes(rows, a.D) <= ws_bytes) pc = {TS, TSZ, TWH};
#endif
  const AttnSplit sp = AttnSplit::in(ws, pc.n, rows, a.D);
  const int64_t tiles = (a.Lq * (a.Hq / a.Hkv) + kTileRows - 1) / kTileRows;
  const dim3 grid((unsigned)(a.B * a.Hkv * pc.n * tiles));
  if (a.D == 64)
    hipLaunchKernelGGL((attn_tile_kernel<Source, 64, kTileWaves>), grid, dim3(64 * kTileWaves), 0, stream, a, src,
                       sp, (int)tiles, pc, gt);
  else
    hipLaunchKernelGGL((attn_tile_kernel<Source, 128, kTileWaves>), grid, dim3(64 * kTileWaves), 0, stream, a, src,
                       sp, (int)tiles, pc, gt);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pc.n == 1) return e;
  return launch_attn_join(a, src, sp, pc.n, stream);
}

template hipError_t launch_attn_tile(const AttnArgs&, const Kv4Source&, int64_t, void*, size_t,
                                     hipStream_t);
template hipError_t launch_attn_tile(const AttnArgs&, const CrossSource&, int64_t, void*, size_t,
                                     hipStream_t);

}  // namespace qact
