// Cross attention to few states (a prompt's): many query rows to at most 512
// states (heads of 64; of 128: 256).  All keys and values of a head lie in shared memory, staged once for
// a workgroup's whole share of the query rows, and its waves go through their
// rows, 32 at a time, without meeting again; the next 32 are on their way
// meanwhile.  attn_rows.h says what a wave does with them.
//
// 30 heads of 64, 17550 query tokens, 226 states: 52 us a call (58 in a kernel trace,
// which slows it), 0.50 us of a SIMD for
// 32 rows by 64 keys (the alternating products and weights alone take 0.41 us
// of it) and about 16 us for the rest: launch, staging, each block's first and
// last products and its rows' load and store.  A memory that is read and written
// once would take 27 us.  12 waves instead of 8 spill registers and cost 6 us
// more.
#include "attn_rows.h"

namespace qact {

namespace {

constexpr int kShortWaves = 8;
// Tiles of keys that fit the shared memory.  A kernel of its own for the first
// four spares those the other tiles' places (226 states: 60 and 61.5 us; 512 states,
// 8000 tokens: 45 us, 60 in staged tiles).
template <int D>
constexpr int kShortTiles = D == 64 ? 8 : 4;

// Workgroup: (sequence and key head, share of the row blocks), the share
// running fastest.
template <int D, int kTiles>
__global__ void __launch_bounds__(64 * kShortWaves, 2)
attn_short_kernel(AttnArgs a, CrossSource src, int blocks, int shares, Gate gate) {
  if (gated_off(gate)) return;
  constexpr int W = kShortWaves;
  using R = Rows<false, D>;
  constexpr int kBytes = kTileKeys * D * 2, kHalf = kBytes / 2, kPieces = D / 8;
  // K, V, and half a tile of zeros: the values before the first tile
  constexpr int kZeros = kTiles * kBytes - kHalf;              // (read from + kHalf on)
  constexpr bool kLines = D == 64 && kTiles == 4;
  constexpr int kOut = 2 * kTiles * kBytes + kHalf;
  __shared__ __align__(16) char lds[kOut + (kLines ? W * 32 * 2 * D : 0)];
  char* const kt = lds;
  char* const vt = lds + kTiles * kBytes;

  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int share = blockIdx.x % shares, at = blockIdx.x / shares, hk = at % a.Hkv;
  const int64_t b = at / a.Hkv;
  const int G = a.Hq / a.Hkv;
  const int rows = (int)a.Lq * G;
  const int n = src.keys(b);
  const int nt = (n + kTileKeys - 1) / kTileKeys;
  const int last = (int)((int64_t)blocks * (share + 1) / shares);
  int block = (int)((int64_t)blocks * share / shares) + wave;

  u32x4 next[D / 16];
  auto fetch = [&](int block) {
    const int row = min(32 * block + col, rows - 1), t = G == 1 ? row : row / G;
    const uint16_t* p = a.q + (b * a.Lq + t) * a.ldq + (int64_t)(hk * G + row - t * G) * D + 8 * h;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) next[i] = *reinterpret_cast<const u32x4*>(p + 16 * i);
  };
  if (block < last) fetch(block);
  // Finished rows: where the shared memory has room for them, through it, so that
  // a store writes whole lines, past the caches, whose last dirty lines would be
  // written back after the kernel (60 -> 56 us; whole lines alone: 61).
  R r;
  auto store = [&](int block) {
    if constexpr (kLines) {
      char* const out = lds + kOut + wave * (32 * 2 * D);
      const float f = r.l == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(r.l);
      wave_lds_order();
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 8)
          *reinterpret_cast<u32x4*>(out + k_piece<D>(col, 4 * d + i / 4 + h)) = r.out8(d, i, f);
      wave_lds_order();
#pragma unroll
      for (int j = 0; j < kPieces / 2; ++j) {
        const int line = j * (64 / kPieces) + lane / kPieces, c = lane % kPieces;
        const int row = 32 * block + line, t = G == 1 ? row : row / G;
        const u32x4 w = *reinterpret_cast<const u32x4*>(out + k_piece<D>(line, c));
        if (row < rows)
          __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(
              a.o + (b * a.Lq + t) * a.ldo + (int64_t)(hk * G + row - t * G) * D + 8 * c));
      }
    } else {
      const int row = 32 * block + col, t = G == 1 ? row : row / G;
      store_rows(r, 1.0f, a.o + (b * a.Lq + t) * a.ldo + (int64_t)(hk * G + row - t * G) * D, h,
                 row < rows);
    }
  };
  // a thread's pieces of the keys; what is not seen may hold NaN and is zeroed
  // when that is known
  constexpr int kLoads = kTiles * kTileKeys * kPieces / (64 * W);
  constexpr int kOf = kTileKeys * kPieces / (64 * W);           // of a tile
  u32x4 kr[kLoads], vr[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    if (kTiles > 4 && u / kOf * kTileKeys >= src.Lk) break;
    const int x = u * 64 * W + tid, c = x % kPieces;
    const int64_t row = b * src.Lk + min(x / kPieces, src.Lk - 1);
    kr[u] = *reinterpret_cast<const u32x4*>(src.k + row * src.ldk + hk * D + 8 * c);
    vr[u] = *reinterpret_cast<const u32x4*>(src.v + row * src.ldv + hk * D + 8 * c);
  }

  uint64_t seen[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
    seen[t] = src.seen(src.look(b, t * kTileKeys, n, lane), t * kTileKeys, n, lane);
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    if (kTiles > 4 && u / kOf * kTileKeys >= src.Lk) break;
    const int t = u / kOf, x = u % kOf * 64 * W + tid, key = x / kPieces, c = x % kPieces;
    if (!((seen[t] >> key) & 1)) kr[u] = vr[u] = u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(kt + t * kBytes + k_piece<D>(key, c)) = kr[u];
    *reinterpret_cast<u32x4*>(vt + t * kBytes + v_piece<D>(key, c)) = vr[u];
  }
  if (tid < kHalf / 16) *reinterpret_cast<u32x4*>(vt + kZeros + kHalf + 16 * tid) = u32x4{0, 0, 0, 0};
  __syncthreads();

  int ka[D / 16], va[D / 32];            // as in attn_tile_kernel
#pragma unroll
  for (int i = 0; i < D / 16; ++i) ka[i] = k_piece<D>(col, 2 * i + h);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
    va[d] = kZeros + v_piece<D>(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1)) + 8 * (lane & 3);
  r.set_ones(lane);
  r.c = fmaxf(a.scale * kLog2e, 0x1p-126f);
  for (; block < last; block += W) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) r.q[i] = next[i];
    fetch(min(block + W, last - 1));
    r.clear();
    if (nt > 0) {
      f32x16 s0, s1 = {};
      u32x4 p0[2] = {}, p1[2] = {}, ahead[R::kAhead];
      float sum = 0.0f;
      r.logits(s0, kt, ka);
#pragma unroll
      for (int g = 0; g < R::kAhead; ++g) ahead[g] = r.template operand<kHalf>(g, kt, ka, vt, va);
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        uint64_t here = t < 2 ? (t == 0 ? seen[0] : seen[1]) : (t == 2 ? seen[2] : seen[3]);
        if constexpr (kTiles == 8)
          if (t >= 4) here = t < 6 ? (t == 4 ? seen[4] : seen[5]) : (t == 6 ? seen[6] : seen[7]);
        if ((uint32_t)here != ~0u) hide(s0, (uint32_t)here);
        if (t == 0) r.start(s0);
        r.template step<kHalf, 0>(s0, p0, s1, p1, sum, ahead, kt, ka, vt, va, kBytes,
                                  t == 0 ? -kZeros : kBytes, [](int) {});
        if ((uint32_t)(here >> 32) != ~0u) hide(s1, (uint32_t)(here >> 32));
        r.template step<0, kHalf>(s1, p1, s0, p0, sum, ahead, kt, ka, vt, va, 0, 0, [](int) {});
      }
      r.template second<kHalf>(s1, p1, sum, vt, va);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) ka[i] -= nt * kBytes;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) va[d] += kZeros - (nt - 1) * kBytes;
    }
    // wait for the next rows here, not behind the stores of these
#pragma unroll
    for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(next[i]));
    store(block);
  }
}

// Workgroups that run at once, and the relative times of staging and of one pass
// of a workgroup's waves, of it by tile.
constexpr int64_t kPlaces = 256;
constexpr double kStage = 3.0, kPass = 0.8, kPassTile = 0.6;

}  // namespace

bool attn_short_takes(int64_t Lq, int Hq, int Hkv, int D, int64_t Lk) {
  return Lk >= 1 && Lk <= (D == 64 ? kShortTiles<64> : kShortTiles<128>) * kTileKeys && Lq * (Hq / Hkv) >= 256;
}

template <int D, int kTiles>
static hipError_t launch(const AttnArgs& a, const CrossSource& src, hipStream_t stream) {
  constexpr int W = kShortWaves;
  const int64_t units = a.B * a.Hkv;
  const int blocks = (int)((a.Lq * (a.Hq / a.Hkv) + 31) / 32);
  // shares of a head's rows: the rounds of workgroups times the passes of each
  const double pass = kPass + kPassTile * (double)((src.Lk + kTileKeys - 1) / kTileKeys);
  int shares = 1;
  double least = 0.0;
  for (int s = 1; s <= 64 && (s == 1 || s * W <= blocks); ++s) {
    const int64_t rounds = (units * s + kPlaces - 1) / kPlaces;
    const int64_t passes = (blocks + (int64_t)s * W - 1) / ((int64_t)s * W);
    const double cost = (double)rounds * (kStage + (double)passes * pass);
    if (s == 1 || cost < least) {
      least = cost;
      shares = s;
    }
  }
  hipLaunchKernelGGL((attn_short_kernel<D, kTiles>), dim3((unsigned)(units * shares)), dim3(64 * W), 0,
                     stream, a, src, blocks, shares, current_gate());
  return hipGetLastError();
}

hipError_t launch_attn_short(const AttnArgs& a, const CrossSource& src, hipStream_t stream) {
  if (a.D == 128) return launch<128, kShortTiles<128>>(a, src, stream);
  return src.Lk <= 4 * kTileKeys ? launch<64, 4>(a, src, stream)
                                 : launch<64, kShortTiles<64>>(a, src, stream);
}

}  // namespace qact
