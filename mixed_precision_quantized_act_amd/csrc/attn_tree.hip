// Attention of a tree of drafted tokens whose rows fill half of a tile's 256 or
// less: the 8 waves of a workgroup are 4 times 32 rows over the first 32 keys of
// every staged tile and the same rows over the other 32, so that all of them have
// products to do (attn_tile.hip gives each wave rows of its own and both halves).
// A wave's two sets of sums meet in shared memory at the end.
#include "attn_cuts.h"
#include "attn_rows.h"
#include "attn_stage.h"

namespace qact {

namespace {

constexpr int kHalfWaves = 8, kHalfRows = 128;
// Workgroup: (piece of the keys, stream, key head, row tile), the row tile running
// fastest.  One step a tile: the weights of its half beside the logits of the next
// tile's and the second product of the tile before.  The workgroup meets in the
// middle of a step: from there to the middle of step t, K(t), K(t + 1), V(t - 2) and
// V(t - 1) are read, and K(t + 2) and V(t) written, which replace K(t - 1) and V(t - 3).
template <int D>
__global__ void __launch_bounds__(64 * kHalfWaves, 2)
attn_tree_kernel(AttnArgs a, Kv4TreeSource src, AttnSplit sp, int tiles, Pieces pc, Gate gate) {
  if (gated_off(gate)) return;
  using T = Tile<Kv4TreeSource, D, 64 * kHalfWaves>;
  using R = Rows<true, D>;
  constexpr int kBytes = kTileKeys * D * 2, kHalf = kBytes / 2;
  constexpr int kZeros = 3 * kBytes;                       // (values before the first tile)
  constexpr int kJoin = 32 * (D + 4) * 4;                  // a wave's sums
  constexpr int kLds = 6 * kBytes + kHalf;
  static_assert(kLds >= 4 * kJoin, "the waves' sums");
  __shared__ __align__(16) char lds[kLds];
  __shared__ float ml[2][4][32];
  char* const kt = lds;
  char* const vt = lds + 3 * kBytes;

  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), part = wave >> 2;   // half of the keys
  const int tile = blockIdx.x % tiles, at = blockIdx.x / tiles, hk = at % a.Hkv;
  const int bs = at / a.Hkv, piece = bs / (int)a.B;
  const int64_t b = bs - piece * (int)a.B;
  const int G = a.Hq / a.Hkv;
  const int nq = src.queries(b, a.Lq), n = src.keys(b);
  const int rows = nq * G;
  if (tile * kHalfRows >= rows) return;
  const int row0 = tile * kHalfRows + (wave & 3) * 32;
  const bool mine = row0 < rows;                           // this wave has rows
  const int all = n - nq;                                  // keys that every row sees
  const int chunks = (n + kTileKeys - 1) / kTileKeys;
  const int c0 = piece_begin(pc, chunks, piece), c1 = piece_end(pc, chunks, piece);
  const int base0 = c0 * kTileKeys, nt = c1 - c0;

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
  // Group j: a thread's units of K(j + 2) and V(j), 16 elements each, loaded two steps
  // before they are stored.
  struct Unit {
    u32x2 w;
    uint32_t s;                    // group scale
  };
  typename T::Place place[T::kPer];
  Unit even[T::kPer], odd[T::kPer];
  const auto load = [&](Unit& r, int u, int j) {
    const int i = j + (T::is_v(u, wave) ? 0 : 2), s16 = place[u].sixteen, key = base0 + i * kTileKeys + 16 * s16;
    const int p = page_of(i, s16);
    const int64_t slot16 = src.slot(has(i, s16) ? p : 0, hk, key);
    r.w = *reinterpret_cast<const u32x2*>(place[u].q + slot16 * (D / 2));
    r.s = place[u].s[slot16 * (D / 16)];
  };
  if (nt > 0) {
    e0 = entries(0);
    e1 = entries(1);
    e2 = entries(2);
    look_at();
    typename T::Regs first[T::kPer], second[T::kPer];
    const Kv4Source::Look look0 = src.look(b, base0, n, lane), look1 = src.look(b, base0 + kTileKeys, n, lane);
#pragma unroll
    for (int u = 0; u < T::kPer; ++u) {
      T::place(place[u], src, b, hk, u, wave, lane);
      if (T::is_v(u, wave)) continue;
      T::load(first[u], place[u], src, look0, 0, hk, base0, n);
      T::load(second[u], place[u], src, look1, 0, hk, base0 + kTileKeys, n);
    }
#pragma unroll
    for (int u = 0; u < T::kPer; ++u) {
      load(even[u], u, 0);
      load(odd[u], u, 1);
    }
#pragma unroll
    for (int j = 0; j < T::kParts; ++j) {
      const int u = j * T::kPer / T::kParts, piece_of = j % (T::kParts / T::kPer);
      if (T::is_v(u, wave)) continue;
      T::store(first[u], place[u], piece_of, kt);
      T::store(second[u], place[u], piece_of, kt + kBytes);
    }
  }

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
  r.c = query_operand<true>(r.q, a.scale * kLog2e, src.k_scale(), [](float v) { return pair_max(v); });
  r.clear();
  r.set_ones(lane);

  // this lane's places in a staged tile (attn_tile.hip), in its half of the keys
  int ka[D / 16], va[D / 32];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) ka[i] = part * kHalf + k_piece<D>(col, 2 * i + h);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
    va[d] = kZeros + v_piece<D>(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1)) + 8 * (lane & 3);
  if (tid < kHalf / 16) *reinterpret_cast<u32x4*>(vt + kZeros + 16 * tid) = u32x4{0, 0, 0, 0};

  f32x16 s0 = {}, s1 = {};
  u32x4 p0[2] = {}, p1[2] = {};
  float sum = 0.0f;
  u32x4 ahead[R::kAhead];
  if (nt > 0) {
    __syncthreads();
    if (mine) {
      r.logits(s0, kt, ka);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) ka[d] += kBytes;
#pragma unroll
      for (int g = 0; g < R::kAhead; ++g) ahead[g] = r.template operand<0>(g, kt, ka, vt, va);
    }
  }
  int slot = 0;                                            // t % 3
  // the first turns of step t: K(t + 2) and V(t) into their tiles
  const auto store_turn = [&](int turn, int i, const Unit(&r)[T::kPer]) {
#pragma unroll
    for (int j = 0; j < T::kParts; ++j)
      if (turn == j * 4 / T::kParts) {
        const int u = j * T::kPer / T::kParts, h2 = j % (T::kParts / T::kPer);
        const bool val = T::is_v(u, wave);
        const int k = (slot == 0 ? 2 : slot - 1) * kBytes, of = i + (val ? 0 : 2);
        // (what has no slot gets a scale of zero: the bytes may be a NaN's)
        const int left = has(of, place[u].sixteen) ? n - (base0 + of * kTileKeys) : 0;
        const f16x2 sc = scale_f16<0>(place[u].key < left ? r[u].s : 0u);
        *reinterpret_cast<u32x4*>((val ? vt + slot * kBytes : kt + k) + place[u].at[h2]) = codes_f16(r[u].w[h2], sc);
      }
  };
  // the others: the waves meet, group t + 2 is loaded
  const auto meet_turn = [&](int turn, int i, Unit(&r)[T::kPer]) {
    if (turn == 4) __syncthreads();
#pragma unroll
    for (int u = 0; u < T::kPer; ++u)
      if (turn == 5 + u) load(r[u], u, i + 2);
  };
  const auto turn_over = [&] { slot = slot == 2 ? 0 : slot + 1; };
  // all tiles in pairs (of the last one's, if it has none, no key is seen), 16 to a
  // block of entries
  const auto each = [&](const auto& pair) {
    for (int i = 0; i < nt;) {
      for (const int stop = min(nt, 16 * block + 16); i < stop; i += 2) pair(i);
      ++block;
      e0 = e1;
      e1 = e2;
      e2 = entries(block + 2);
      look_at();
    }
  };
  // Step t: `s` its logits, `next` the logits of the tile before (whose weights are p)
  const auto step = [&](int i, f32x16& s, u32x4(&pn)[2], f32x16& next, u32x4(&p)[2], Unit(&units)[T::kPer]) {
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
    if (!(here == ~0ull && base + kTileKeys <= all)) {
      here &= src.row_sees(words, base, all);
      hide(s, (uint32_t)(here >> (32 * part)), 64, h);
    }
    // on to K(t + 2) and V(t)
    const int ks = slot == 1 ? -2 * kBytes : kBytes;
    const int vs = i == 0 ? part * kHalf - kZeros : slot == 0 ? -2 * kBytes : kBytes;
    r.template step<0, 0>(s, pn, next, p, sum, ahead, kt, ka, vt, va, ks, vs, [&](int turn) {
      if (turn < 4)
        store_turn(turn, i, units);
      else
        meet_turn(turn, i, units);
    });
    turn_over();
  };
  if (mine) {
    each([&](int i) {
      step(i, s0, p0, s1, p1, even);
      step(i + 1, s1, p1, s0, p0, odd);
    });
    if (nt > 0) r.template second<0>(s1, p1, sum, vt, va);
  } else {
    const auto pass = [&](int i, Unit(&units)[T::kPer]) {
#pragma unroll
      for (int turn = 0; turn < 4; ++turn) store_turn(turn, i, units);
#pragma unroll
      for (int turn = 4; turn < 8; ++turn) meet_turn(turn, i, units);
      turn_over();
    };
    each([&](int i) {
      pass(i, even);
      pass(i + 1, odd);
    });
  }

  // the other half's sums to the common reference
  __syncthreads();
  float* const join = reinterpret_cast<float*>(lds + (wave & 3) * kJoin) + col * (D + 4);
  if (part == 1) {
    if (h == 0) {
      ml[0][wave & 3][col] = r.m;
      ml[1][wave & 3][col] = r.l;
    }
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(join + 32 * d + 2 * i + 4 * h) =
            f32x4{r.o[d][i], r.o[d][i + 1], r.o[d][i + 2], r.o[d][i + 3]};
  }
  __syncthreads();
  if (part == 1) return;
  {
    const float m1 = ml[0][wave & 3][col], top = fmaxf(r.m, m1), ref = top == -INFINITY ? 0.0f : top;
    // (times zero, not left out: a sum that is NaN stays so)
    const float f0 = r.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((r.m - ref) * r.c);
    const float f1 = m1 == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m1 - ref) * r.c);
    r.m = top;
    r.l = __builtin_fmaf(ml[1][wave & 3][col], f1, r.l * f0);
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x4 o = *reinterpret_cast<const f32x4*>(join + 32 * d + 2 * i + 4 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.o[d][i + j] = __builtin_fmaf(o[j], f1, r.o[d][i + j] * f0);
      }
  }
  if (pc.n == 1) {
    store_rows(r, src.v_scale(), a.o + (b * a.Lq + t) * a.ldo + (int64_t)head * D, h, row < rows);
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
      sp.l[to] = r.l;
    }
  }
}

Pieces cut_of(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L, size_t ws_bytes) {
  const int64_t rows = B * Lq * Hq;
  const int64_t u = B * Hkv * ((Lq * (Hq / Hkv) + kHalfRows - 1) / kHalfRows);
  return pieces_of(u, rows, D, (L + kTileKeys - 1) / kTileKeys, (int64_t)(ws_bytes / AttnSplit::bytes(rows, D)));
}

}  // namespace

// (asked for: at most 32 MiB, whatever more pieces would give)
size_t attn_tree_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  const Pieces p = cut_of(B, Lq, Hq, Hkv, D, L, (size_t)32 << 20);
  return p.n > 1 ? p.n * AttnSplit::bytes(B * Lq * Hq, D) : 0;
}

hipError_t launch_attn_tree(const AttnArgs& a, const Kv4TreeSource& src, int64_t L, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  const Gate gt = current_gate();
  const int64_t rows = a.B * a.Lq * a.Hq;
  const Pieces pc = cut_of(a.B, a.Lq, a.Hq, a.Hkv, a.D, L, ws_bytes);
  const AttnSplit sp = AttnSplit::in(ws, pc.n, rows, a.D);
  const int64_t tiles = (a.Lq * (a.Hq / a.Hkv) + kHalfRows - 1) / kHalfRows;
  const dim3 grid((unsigned)(a.B * a.Hkv * pc.n * tiles)), block(64 * kHalfWaves);
  if (a.D == 64)
    hipLaunchKernelGGL(attn_tree_kernel<64>, grid, block, 0, stream, a, src, sp, (int)tiles, pc, gt);
  else
    hipLaunchKernelGGL(attn_tree_kernel<128>, grid, block, 0, stream, a, src, sp, (int)tiles, pc, gt);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pc.n == 1) return e;
  return launch_attn_join(a, src, sp, pc.n, stream);
}

}  // namespace qact
