// Cross attention to few states (a prompt's): many query rows to at most 256
// states.  All keys and values of a head lie in shared memory, staged once for
// a workgroup's whole share of the query rows, and its waves go through their
// rows, 32 at a time, without meeting again; the next 32 are on their way
// meanwhile.  attn_rows.h says what a wave does with them.
//
// One pass of 32 rows over 256 states (heads of 64) takes 2.9 us of a SIMD
// that two waves share, against 0.9 us that its bytes take of the memory.
#include "attn_rows.h"

namespace qact {

namespace {

constexpr int kShortWaves = 8;
constexpr int kShortTiles = 4;

// Workgroup: (sequence and key head, share of the row blocks), the share
// running fastest.
template <int D>
__global__ void __launch_bounds__(64 * kShortWaves, 2)
attn_short_kernel(AttnArgs a, CrossSource src, int blocks, int shares, Gate gate) {
  if (gated_off(gate)) return;
  using R = Rows<false, D>;
  constexpr int kBytes = kTileKeys * D * 2, kHalf = kBytes / 2, kPieces = D / 8;
  // K, V, and half a tile of zeros: the values before the first tile
  constexpr int kZeros = kShortTiles * kBytes - kHalf;              // (read from + kHalf on)
  __shared__ __align__(16) char lds[2 * kShortTiles * kBytes + kHalf];
  char* const kt = lds;
  char* const vt = lds + kShortTiles * kBytes;

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
    const int row = min(32 * block + col, rows - 1), t = row / G;
    const uint16_t* p = a.q + (b * a.Lq + t) * a.ldq + (int64_t)(hk * G + row - t * G) * D + 8 * h;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) next[i] = *reinterpret_cast<const u32x4*>(p + 16 * i);
  };
  if (block < last) fetch(block);

  uint64_t seen[kShortTiles];
#pragma unroll
  for (int t = 0; t < kShortTiles; ++t)
    seen[t] = src.seen(src.look(b, t * kTileKeys, n, lane), t * kTileKeys, n, lane);
  // a thread's piece of every eighth (heads of 64) or sixteenth of the keys
#pragma unroll
  for (int t = 0; t < kShortTiles; ++t)
    if (t < nt)
#pragma unroll
      for (int u = 0; u < kTileKeys * kPieces / (64 * kShortWaves); ++u) {
        const int x = u * 64 * kShortWaves + tid, key = x / kPieces, c = x % kPieces;
        u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
        if ((seen[t] >> key) & 1) {      // (what is not seen may hold NaN: zeros)
          const int64_t row = b * src.Lk + t * kTileKeys + key;
          k = *reinterpret_cast<const u32x4*>(src.k + row * src.ldk + hk * D + 8 * c);
          v = *reinterpret_cast<const u32x4*>(src.v + row * src.ldv + hk * D + 8 * c);
        }
        *reinterpret_cast<u32x4*>(kt + t * kBytes + k_piece<D>(key, c)) = k;
        *reinterpret_cast<u32x4*>(vt + t * kBytes + v_piece<D>(key, c)) = v;
      }
  if (tid < kHalf / 16) *reinterpret_cast<u32x4*>(vt + kZeros + kHalf + 16 * tid) = u32x4{0, 0, 0, 0};
  __syncthreads();

  int ka[D / 16], va[D / 32];            // as in attn_tile_kernel
#pragma unroll
  for (int i = 0; i < D / 16; ++i) ka[i] = k_piece<D>(col, 2 * i + h);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
    va[d] = kZeros + v_piece<D>(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1)) + 8 * (lane & 3);
  R r;
  r.set_ones(lane);
  r.c = fmaxf(a.scale * kLog2e, 0x1p-126f);
  for (; block < last; block += kShortWaves) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) r.q[i] = next[i];
    if (block + kShortWaves < last) fetch(block + kShortWaves);
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
        const uint64_t here = t < 2 ? (t == 0 ? seen[0] : seen[1]) : (t == 2 ? seen[2] : seen[3]);
        if ((uint32_t)here != ~0u) hide(s0, (uint32_t)here, 32, h);
        if (t == 0) r.start(s0);
        r.template step<kHalf, 0>(s0, p0, s1, p1, sum, ahead, kt, ka, vt, va, kBytes,
                                  t == 0 ? -kZeros : kBytes, [](int) {});
        if ((uint32_t)(here >> 32) != ~0u) hide(s1, (uint32_t)(here >> 32), 32, h);
        r.template step<0, kHalf>(s1, p1, s0, p0, sum, ahead, kt, ka, vt, va, 0, 0, [](int) {});
      }
      r.template second<kHalf>(s1, p1, sum, vt, va);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) ka[i] -= nt * kBytes;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) va[d] += kZeros - (nt - 1) * kBytes;
    }
    const int row = 32 * block + col, t = row / G;
    store_rows(r, 1.0f, a.o + (b * a.Lq + t) * a.ldo + (int64_t)(hk * G + row - t * G) * D, h,
               row < rows);
  }
}

// Workgroups that run at once, and the time (us) of staging and of one pass of
// the waves of each.
constexpr int64_t kPlaces = 256;
constexpr double kStage = 3.0, kPass64 = 3.2;

}  // namespace

bool attn_short_takes(int64_t B, int64_t Lq, int Hq, int Hkv, int64_t Lk) {
  return Lk <= kShortTiles * kTileKeys && Lq * (Hq / Hkv) >= 32 * kShortWaves;
}

hipError_t launch_attn_short(const AttnArgs& a, const CrossSource& src, hipStream_t stream) {
  const int64_t units = a.B * a.Hkv;
  const int blocks = (int)((a.Lq * (a.Hq / a.Hkv) + 31) / 32);
  // shares of a head's rows: the rounds of workgroups times the passes of each
  int shares = 1;
  double least = 0.0;
  for (int s = 1; s <= 64 && (s == 1 || s * kShortWaves <= blocks); ++s) {
    const int64_t rounds = (units * s + kPlaces - 1) / kPlaces;
    const int64_t passes = (blocks + (int64_t)s * kShortWaves - 1) / ((int64_t)s * kShortWaves);
    const double cost = (double)rounds * (kStage + (double)passes * kPass64);
    if (s == 1 || cost < least) {
      least = cost;
      shares = s;
    }
  }
  const dim3 grid((unsigned)(units * shares)), block(64 * kShortWaves);
  if (a.D == 64)
    hipLaunchKernelGGL((attn_short_kernel<64>), grid, block, 0, stream, a, src, blocks, shares,
                       current_gate());
  else
    hipLaunchKernelGGL((attn_short_kernel<128>), grid, block, 0, stream, a, src, blocks, shares,
                       current_gate());
  return hipGetLastError();
}

}  // namespace qact
