// Attention of many query rows (a frame's tokens, a whole block's): a
// workgroup holds 128 or 256 rows, its waves 32 or 64 each, and takes the
// keys in tiles of 64 that it stages in shared memory as 16-bit operands (an
// NVFP4 tile is expanded once for all rows), one tile ahead of the one that
// the MFMAs read.
//
// What bounds it is the softmax: for heads of 64 an element of S costs 16
// cycles of a SIMD's MFMA and about 29 of its VALU, 16 of them the
// exponential (a quarter-rate instruction).  So the VALU is left with as
// little else as possible: the running maximum is moved only when a tile
// exceeds it by 2^8 (the weights are at most 2^8 times the 2^kTileBias of the
// reference, in range of fp16), which spares the rescaling of the sums; a
// lane holds one query row, so a maximum needs one exchange between lanes.
#include "attn_common.h"

namespace qact {

namespace {

constexpr int kTileKeys = 64;
constexpr float kTileSlack = 8.0f;
template <bool F16>
constexpr float kTileBias = F16 ? 7.0f : 0.0f;

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
  return key * (D * 2) + 32 * ((c >> 1) ^ (D == 128 ? key & 7 : (key >> 1) & 3)) + 16 * (c & 1);
}

// Staging by T threads: a thread takes units of K or of V, the same side for
// a whole wave.
template <class Source, int D, int T>
struct Tile;

// NVFP4: a unit is a group of 16 elements.
template <int D, int T>
struct Tile<Kv4Source, D, T> {
  static constexpr int kGroups = D / 16;
  static constexpr int kUnits = kTileKeys * kGroups;
  static constexpr int kPer = 2 * kUnits / T;

  struct Regs {
    u32x2 w[kPer];
    uint32_t s[kPer];              // group scale (0: not seen)
    uint64_t seen;
  };
  // (a wave's unit lies within one sixteen of keys: its place is uniform)
  static __device__ __forceinline__ void load(Regs& r, const Kv4Source& s,
                                              const Kv4Source::Pages& pg, int64_t, int hk, int base,
                                              int n, int wave, int lane) {
    r.seen = s.seen(pg, base, n);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int x = u * T + 64 * wave;
      const bool val = x >= kUnits;
      const int y = x & (kUnits - 1), t = y / kGroups >> 4;
      const int p0 = pg.p[0], p1 = pg.p[1], p2 = pg.p[2], p3 = pg.p[3];
      const int p = t < 2 ? (t == 0 ? p0 : p1) : (t == 2 ? p2 : p3);
      const uint32_t z = (uint32_t)(y + lane) & (16 * kGroups - 1);       // (key % 16, group)
      r.w[u] = u32x2{0, 0};
      r.s[u] = 0;
      if (s.named(p) && base + 16 * t + (int)(z / kGroups) < n) {
        const int64_t at = s.slot(p, hk, base + 16 * t);
        r.w[u] = *reinterpret_cast<const u32x2*>((val ? s.c.v_q : s.c.k_q) + at * (D / 2) + 8 * z);
        r.s[u] = ((val ? s.c.v_s : s.c.k_s) + at * kGroups)[z];
      }
    }
  }
  static __device__ __forceinline__ void store(const Regs& r, char* k, char* v, int tid) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int x = u * T + tid;
      const bool val = x >= kUnits;
      const int y = x & (kUnits - 1), key = y / kGroups, g = y % kGroups;
      const f16x2 sc = scale_f16<0>(r.s[u]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4*>(val ? v + v_piece<D>(key, 2 * g + h) : k + k_piece<D>(key, 2 * g + h)) =
            codes_f16(r.w[u][h], sc);
    }
  }
};

// bf16 states: a unit is a 16-byte piece.
template <int D, int T>
struct Tile<CrossSource, D, T> {
  static constexpr int kPieces = D / 8;
  static constexpr int kUnits = kTileKeys * kPieces;
  static constexpr int kPer = 2 * kUnits / T;

  struct Regs {
    u32x4 w[kPer];
    uint64_t seen;
  };
  static __device__ __forceinline__ void load(Regs& r, const CrossSource& s,
                                              const CrossSource::Pages&, int64_t b, int hk,
                                              int base, int n, int wave, int lane) {
    const int64_t row0 = b * s.Lk + base;
    bool on = base + lane < n;
    if (on && s.mask) on = s.mask[row0 + lane] != 0;
    r.seen = __ballot(on);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int x = u * T + 64 * wave;
      const bool val = x >= kUnits;
      const int y = (x & (kUnits - 1)) + lane, key = y / kPieces, c = y % kPieces;
      r.w[u] = u32x4{0, 0, 0, 0};
      if ((r.seen >> key) & 1)           // (what is not seen may hold NaN: zeros)
        r.w[u] = *reinterpret_cast<const u32x4*>(
            (val ? s.v + (row0 + key) * s.ldv : s.k + (row0 + key) * s.ldk) + hk * D + 8 * c);
    }
  }
  static __device__ __forceinline__ void store(const Regs& r, char* k, char* v, int tid) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int x = u * T + tid;
      const bool val = x >= kUnits;
      const int y = x & (kUnits - 1), key = y / kPieces, c = y % kPieces;
      *reinterpret_cast<u32x4*>(val ? v + v_piece<D>(key, c) : k + k_piece<D>(key, c)) = r.w[u];
    }
  }
};

// Workgroup: (stream, key head, split, row tile), the row tile running
// fastest.  W waves of NQ groups of 32 rows each.
template <class Source, int D, int NQ, int W>
__global__ void __launch_bounds__(64 * W, NQ == 1 && D == 64 ? 4 : 2)
attn_tile_kernel(AttnArgs a, Source src, AttnSplit sp, int tiles, int splits, Gate gate) {
  if (gated_off(gate)) return;
  using T = Tile<Source, D, 64 * W>;
  constexpr bool kF16 = Source::kF16;
  constexpr int kBytes = kTileKeys * D * 2;
  __shared__ __align__(16) char lds[2][2][kBytes];

  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = blockIdx.x % tiles;
  const int at = blockIdx.x / tiles, split = at % splits;
  const int hk = at / splits % a.Hkv;
  const int64_t b = at / splits / a.Hkv;
  const int G = a.Hq / a.Hkv;
  const int nq = src.queries(b, a.Lq), n = src.keys(b);
  const int rows = nq * G;
  constexpr int kRows = 32 * NQ * W;
  if (tile * kRows >= rows) return;
  const int row0 = tile * kRows + wave * 32 * NQ;         // the wave's first row
  const int wlast = min(row0 + 32 * NQ, rows) - 1;        // and last (before row0: it has none)

  // keys that every row of the wave sees, that any row of it and of the
  // workgroup sees
  const int all = src.causal ? n - (nq - 1 - row0 / G) : n;
  const int wend = wlast < row0 ? 0 : (src.causal ? n - (nq - 1 - wlast / G) : n);
  const int last = min(tile * kRows + kRows, rows) - 1;
  const int end = src.causal ? n - (nq - 1 - last / G) : n;
  const int chunks = (max(end, 0) + kTileKeys - 1) / kTileKeys;
  const int c0 = (int)((int64_t)chunks * split / splits);
  const int c1 = (int)((int64_t)chunks * (split + 1) / splits);

  u32x4 q[NQ][D / 16];
  float c[NQ], m[NQ], l[NQ];
  int upto[NQ];
  f32x16 o[NQ][D / 32];
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    const int row = row0 + 32 * x + col, t = row / G;
    upto[x] = src.causal ? n - (nq - 1 - t) : n;
    const uint16_t* p = a.q + (b * a.Lq + t) * a.ldq + (int64_t)(hk * G + row - t * G) * D + 8 * h;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      q[x][i] = u32x4{0, 0, 0, 0};
      if (row < rows) q[x][i] = *reinterpret_cast<const u32x4*>(p + 16 * i);
    }
    c[x] = query_operand<kF16>(q[x], a.scale * kLog2e, src.k_scale(),
                               [](float v) { return pair_max(v); });
    m[x] = -INFINITY;
    l[x] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[x][d][i] = 0.0f;
  }

  // this lane's places in a staged tile: K of key `col`, piece 2 i + h (keys
  // 32 further on: the same exchange of pieces); V of keys 4 h + lane % 16 / 4
  // (8 and 16 further on: the same), elements 32 d + 16 (lane / 16 % 2) + 4 (lane % 4)
  int ka[D / 16], va[D / 32];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) ka[i] = k_piece<D>(col, 2 * i + h);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
    va[d] = v_piece<D>(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1)) + 8 * (lane & 3);

  typename T::Regs regs;
  typename Source::Pages pg = {};
  uint64_t seen = 0;
  if (c0 < c1) {
    pg = src.pages(b, c0 * kTileKeys, n);
    T::load(regs, src, pg, b, hk, c0 * kTileKeys, n, wave, lane);
    seen = regs.seen;
    T::store(regs, lds[0][0], lds[0][1], tid);
    pg = src.pages(b, (c0 + 1) * kTileKeys, n);
  }
  for (int ch = c0; ch < c1; ++ch) {
    const char* const kt = lds[(ch - c0) & 1][0];
    const char* const vt = lds[(ch - c0) & 1][1];
    const int base = ch * kTileKeys;
    __syncthreads();         // this tile is staged, and the one before it no longer read
    const bool more = ch + 1 < c1;
    if (more) {
      T::load(regs, src, pg, b, hk, base + kTileKeys, n, wave, lane);
      pg = src.pages(b, base + 2 * kTileKeys, n);
    }
    if (base < wend) {
      const bool whole = seen == ~0ull && base + kTileKeys <= all;
#pragma unroll 1
      for (int k2 = 0; k2 < 2; ++k2) {
        f32x16 s[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) s[x] = f32x16{};
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const u32x4 k = *reinterpret_cast<const u32x4*>(kt + ka[i] + 32 * k2 * (D * 2));
#pragma unroll
          for (int x = 0; x < NQ; ++x) s[x] = mfma32<kF16>(k, q[x][i], s[x]);
        }
        u32x4 p[NQ][2];
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          if (!whole) {            // bit 8 (i / 4) + i % 4: this lane's element i is seen
            const int left = upto[x] - (base + 32 * k2 + 4 * h);
            uint32_t bits = (uint32_t)(seen >> (32 * k2)) >> (4 * h);
            bits &= left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              s[x][i] = bits & (1u << (8 * (i >> 2) + (i & 3))) ? s[x][i] : -INFINITY;
          }
          float top = max3(s[x][0], s[x][1], s[x][2]);
#pragma unroll
          for (int i = 3; i < 15; i += 2) top = max3(top, s[x][i], s[x][i + 1]);
          top = pair_max(fmaxf(top, s[x][15]));
          // (no key seen yet: the difference is infinite; none at all: NaN, not greater)
          if (__builtin_amdgcn_ballot_w64((top - m[x]) * c[x] > kTileSlack)) {
            const float mn = fmaxf(m[x], top);
            const float f = m[x] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m[x] - mn) * c[x]);
            m[x] = mn;
            l[x] *= f;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) o[x][d] *= f;
          }
          const float shift = kTileBias<kF16> - (m[x] == -INFINITY ? 0.0f : m[x] * c[x]);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][i], c[x], shift));
            const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][i + 1], c[x], shift));
            const uint32_t e = pack16<kF16>(e0, e1);
            l[x] = add_pair<kF16>(e, l[x]);
            p[x][i >> 3][(i & 7) >> 1] = e;
          }
        }
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
          for (int d = 0; d < D / 32; ++d) {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(
                  vt + va[d] + (32 * k2 + 16 * s2 + 8 * j) * (D * 2)));
              const u32x2 pr = __builtin_bit_cast(u32x2, w);
              v[2 * j] = pr[0];
              v[2 * j + 1] = pr[1];
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) o[x][d] = mfma32<kF16>(v, p[x][s2], o[x][d]);
          }
      }
    }
    if (more) {
      seen = regs.seen;
      T::store(regs, lds[(ch + 1 - c0) & 1][0], lds[(ch + 1 - c0) & 1][1], tid);
    }
  }

#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    const float lt = pair_sum(l[x]);
    const int row = row0 + 32 * x + col, t = row / G;
    const int head = hk * G + row - t * G;
    // (times zero, not left out: a sum that is NaN stays so)
    if (splits == 1) {
      const float f = lt == 0.0f ? 0.0f : src.v_scale() / lt;
      uint16_t* dst = a.o + (b * a.Lq + t) * a.ldo + (int64_t)head * D;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          // elements 8 (i / 4) + 4 h + 0..3 and 8 (i / 4 + 1) + 4 h + 0..3: lanes l and
          // l + 32 exchange halves, so that each holds 8 consecutive ones
          const auto w0 = __builtin_amdgcn_permlane32_swap(
              bf16_pack(o[x][d][i] * f, o[x][d][i + 1] * f),
              bf16_pack(o[x][d][i + 4] * f, o[x][d][i + 5] * f), false, false);
          const auto w1 = __builtin_amdgcn_permlane32_swap(
              bf16_pack(o[x][d][i + 2] * f, o[x][d][i + 3] * f),
              bf16_pack(o[x][d][i + 6] * f, o[x][d][i + 7] * f), false, false);
          if (row < rows)
            *reinterpret_cast<u32x4*>(dst + 32 * d + 2 * i + 8 * h) = u32x4{w0[0], w1[0], w0[1], w1[1]};
        }
    } else if (row < rows) {
      const int64_t to = (int64_t)split * sp.rows + (b * a.Lq + t) * a.Hq + head;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f32x4*>(sp.o + to * D + 32 * d + 2 * i + 4 * h) =
              f32x4{o[x][d][i], o[x][d][i + 1], o[x][d][i + 2], o[x][d][i + 3]};
      if (h == 0) {
        sp.m[to] = m[x] == -INFINITY ? m[x] : m[x] * c[x];
        sp.l[to] = lt;
      }
    }
  }
}


#ifndef TS
#define TS 1
#endif
// rows of a workgroup
int tile_rows(int D) { return D == 64 ? 256 : 128; }

int64_t splits_of(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) { return TS; }

}  // namespace

size_t attn_tile_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  const int64_t s = splits_of(B, Lq, Hq, Hkv, D, L);
  return s > 1 ? s * AttnSplit::bytes(B * Lq * Hq, D) : 0;
}

template <class Source>
hipError_t launch_attn_tile(const AttnArgs& a, const Source& src, int64_t L, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  const Gate gt = current_gate();
  const int64_t rows = a.B * a.Lq * a.Hq;
  int64_t s = splits_of(a.B, a.Lq, a.Hq, a.Hkv, a.D, L);
  const int64_t fit = (int64_t)(ws_bytes / AttnSplit::bytes(rows, a.D));
  if (s > fit) s = fit > 1 ? fit : 1;
  const AttnSplit sp = AttnSplit::in(ws, s, rows, a.D);
  const int per = tile_rows(a.D);
  const int64_t tiles = (a.Lq * (a.Hq / a.Hkv) + per - 1) / per;
  const dim3 grid((unsigned)(a.B * a.Hkv * s * tiles));
  if (a.D == 64)
    hipLaunchKernelGGL((attn_tile_kernel<Source, 64, 1, 8>), grid, dim3(512), 0, stream, a, src,
                       sp, (int)tiles, (int)s, gt);
  else
    hipLaunchKernelGGL((attn_tile_kernel<Source, 128, 1, 4>), grid, dim3(256), 0, stream, a, src,
                       sp, (int)tiles, (int)s, gt);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || s == 1) return e;
  return launch_attn_join(a, src, sp, (int)s, stream);
}

template hipError_t launch_attn_tile(const AttnArgs&, const Kv4Source&, int64_t, void*, size_t,
                                     hipStream_t);
template hipError_t launch_attn_tile(const AttnArgs&, const CrossSource&, int64_t, void*, size_t,
                                     hipStream_t);

}  // namespace qact
