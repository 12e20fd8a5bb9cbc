// Attention of many query rows (a frame's tokens, a whole block's): a
// workgroup holds 256 rows, its waves 32 each, and takes the keys in tiles of
// 64 that it stages in shared memory as 16-bit operands (an NVFP4 tile is
// expanded once for all rows), ahead of what its MFMAs read.  attn_rows.h says
// what a wave does with them and what bounds it.
//
// 1350 rows to 12376 tokens of a cache, 30 heads of 64: 178 us a call, 128 GFLOP at
// 0.72 PFLOP/s (a large library product: 1.21); in a kernel trace, which slows
// both, 178 for this kernel and 7 for the join.  Heads of 128, 16 of them: 173 us.
// Counters: VALU busy 0.45 of the cycles, MFMA 0.34, a wave waiting for data or the
// others a third of its time, 1.6 of 2 waves on a SIMD.  Why 8 waves: with 4
// a tile is staged for half as many rows (195 us; 3 of them per SIMD spill, 190).
#include "attn_cuts.h"
#include "attn_rows.h"
#include "attn_stage.h"

namespace qact {

namespace {

// Workgroup: (piece of the keys, stream, key head, row tile), the row tile
// running fastest (causal: slowest).  W waves of 32 rows each.
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
  // (and half a tile of zeros: the values before the first tile, read from + kHalf on)
  constexpr int kZeros = 3 * kBytes - kHalf;
  __shared__ __align__(16) char vt[3 * kBytes + kHalf];

  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // causal: the tiles with most keys first, of all heads, so that the short ones
  // fill the end (4096 rows of 32 heads of 64 over themselves: 153 -> 100 us)
  const int others = gridDim.x / tiles;
  const int tile = src.causal ? tiles - 1 - blockIdx.x / others : blockIdx.x % tiles;
  const int at = src.causal ? blockIdx.x % others : blockIdx.x / tiles, hk = at % a.Hkv;
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
  const int c0 = piece_begin(pc, chunks, piece), c1 = piece_end(pc, chunks, piece);
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
  r.clear();
  r.set_ones(lane);

  // this lane's places in a staged tile: K of key `col`, piece 2 i + h (keys
  // 32 further on: the same exchange of pieces); V of keys 4 h + lane % 16 / 4
  // (8 and 16 further on: the same), elements 32 d + 16 (lane / 16 % 2) + 4 (lane % 4)
  int ka[D / 16], va[D / 32];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) ka[i] = k_piece<D>(col, 2 * i + h);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
    va[d] = kZeros + v_piece<D>(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1)) + 8 * (lane & 3);
  if (tid < kHalf / 16) *reinterpret_cast<u32x4*>(vt + kZeros + kHalf + 16 * tid) = u32x4{0, 0, 0, 0};

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
    // `va` is at the tile before (in the first there is none: zeros), `ka` at
    // this one; on to the next tile of K (after the last: logits that nobody
    // looks at) and to this one of V
    const int ks = slot == 2 ? -2 * kBytes : kBytes;
    const int vs = i == 0 ? -kZeros : slot == 0 ? -2 * kBytes : kBytes;
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

// rows of a workgroup
constexpr int kTileWaves = 8;
constexpr int kTileRows = 32 * kTileWaves;

Pieces cut_of(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L, size_t ws_bytes) {
  const int64_t rows = B * Lq * Hq;
  const int64_t u = B * Hkv * ((Lq * (Hq / Hkv) + kTileRows - 1) / kTileRows);
  return pieces_of(u, rows, D, (L + kTileKeys - 1) / kTileKeys,
                   (int64_t)(ws_bytes / AttnSplit::bytes(rows, D)));
}

}  // namespace

// (asked for: at most 32 MiB, whatever more pieces would give)
size_t attn_tile_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  const Pieces p = cut_of(B, Lq, Hq, Hkv, D, L, (size_t)32 << 20);
  return p.n > 1 ? p.n * AttnSplit::bytes(B * Lq * Hq, D) : 0;
}

template <class Source>
hipError_t launch_attn_tile(const AttnArgs& a, const Source& src, int64_t L, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  const Gate gt = current_gate();
  const int64_t rows = a.B * a.Lq * a.Hq;
  const Pieces pc = cut_of(a.B, a.Lq, a.Hq, a.Hkv, a.D, L, ws_bytes);
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
