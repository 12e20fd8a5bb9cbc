// Attention of few query rows (single tokens, drafted tokens, short queries):
// the keys and values are read once and that is the time, so the work is
// split over the keys.
//
// A wave takes 64 keys at a time for 16 rows and needs no other wave: K goes
// from memory straight into the MFMA's operand (a lane reads consecutive
// elements of one key, the query operand is laid out to match), V goes
// through a wave-private piece of shared memory from which the transposing
// reads (ds_read_b64_tr_b4 on the 4-bit codes, _tr_b16 on bf16) give V^T.  No
// barrier stands in the loop; the next 64 keys are in flight while these are
// worked on.  The waves of a workgroup and then the workgroups of a row
// are joined at the end with their maxima and sums.
//
// NVFP4 (9/16 byte per element): one conversion (half rate) and one packed
// multiply per two elements, about 0.6 of the VALU's time at 5 TB/s; sixteen
// rows cost no more than one.
//
// 16 streams of 16384 to 32768 tokens, one query token each, 32 query and 8 key
// heads of 128: 92 us and 4.7 for the join in a kernel trace, 463 MB at 5.0 TB/s.  24
// tokens to 300 to 1500 bf16 states, 20 heads of 64: 25 us and 4.8.
#include "attn_common.h"

namespace qact {

namespace {

constexpr int kFewKeys = 64;     // keys of a wave's step
constexpr int kFewRows = 16;     // rows of a tile
constexpr int kFewWaves = 4;

typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Once: no other workgroup reads the same keys (one tile of rows), so they go past
// the caches (16 streams of up to 32768 tokens: 101 -> 94 us; read by two tiles of
// rows: 109 -> 116).  Of bf16 states only the values: a key's line takes two loads
// (24 tokens to 1500 states: values 30 -> 27 us, both 33).
template <bool Once, class T>
__device__ __forceinline__ T fetch(const void* p) {
  if constexpr (Once) return __builtin_nontemporal_load(static_cast<const T*>(p));
  return *static_cast<const T*>(p);
}

template <class Source, int D, bool Once>
struct Few;

// NVFP4: per 64 keys a lane holds for each of four 16-key tiles the codes of
// D/4 elements of key (lane & 15) and their group scales, V's codes as they lie
// and the group scales of V's key `lane`.
template <int D, bool Once>
struct Few<Kv4Source, D, Once> {
  static constexpr int kKWords = D / 32;              // code words per lane and tile
  static constexpr int kVLoads = kFewKeys * D / 2 / 16 / 64;
  static constexpr int kGroups = D / 16;
  static constexpr int kLds = kFewKeys * D / 2 + kGroups * kFewKeys * 2;

  struct Regs {
    uint32_t k[4][kKWords];
    uint32_t ks[4];                                   // kKWords / 2 scale bytes
    u32x4 v[kVLoads];
    uint32_t vs[(kGroups + 3) / 4];
    uint64_t seen;
  };

  static __device__ __forceinline__ void load(Regs& r, const Kv4Source& s,
                                              const Kv4Source::Look& pg, int64_t, int hk, int base,
                                              int n, int lane) {
    const uint32_t key = lane & 15, g = lane >> 4;
    int64_t slot[4];
    r.seen = s.seen(pg, base, n, lane);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      slot[t] = -1;
#pragma unroll
      for (int i = 0; i < kKWords; ++i) r.k[t][i] = 0;
      r.ks[t] = 0;
      const int p = s.entry(pg, t);
      if (base + 16 * t >= n || !s.named(p)) continue;
      slot[t] = s.slot(p, hk, base + 16 * t);
      const uint8_t* kq = s.c.k_q + slot[t] * (D / 2) + (key * (D / 2) + 4 * kKWords * g);
      const uint8_t* ks = s.c.k_s + slot[t] * kGroups + (key * kGroups + kKWords / 2 * g);
      if constexpr (D == 128) {
        const u32x4 w = fetch<Once, u32x4>(kq);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.k[t][i] = w[i];
        r.ks[t] = *reinterpret_cast<const uint16_t*>(ks);
      } else {
        const u32x2 w = fetch<Once, u32x2>(kq);
        r.k[t][0] = w[0];
        r.k[t][1] = w[1];
        r.ks[t] = *ks;
      }
    }
    // V codes: 16-byte vector x of the 64 keys is key x / (D/32)
#pragma unroll
    for (int u = 0; u < kVLoads; ++u) {
      const int x = u * 64 + lane, vk = x / (D / 32);
      r.v[u] = u32x4{0, 0, 0, 0};
      const int64_t lo = slot[(D == 128 ? u : 2 * u) % 4], hi = slot[(D == 128 ? u : 2 * u + 1) % 4];
      const int64_t at = lane < 32 ? lo : hi;
      if (at >= 0)
        r.v[u] = fetch<Once, u32x4>(s.c.v_q + (at + (vk & 15)) * (D / 2) + 16 * (x % (D / 32)));
    }
#pragma unroll
    for (int i = 0; i < (kGroups + 3) / 4; ++i) r.vs[i] = 0;
    const int64_t s0 = slot[0], s1 = slot[1], s2 = slot[2], s3 = slot[3];
    const int64_t at = g < 2 ? (g == 0 ? s0 : s1) : (g == 2 ? s2 : s3);
    if (at >= 0 && base + lane < n) {
      const uint8_t* vs = s.c.v_s + (at + key) * kGroups;
      if constexpr (D == 128) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(vs);
        r.vs[0] = w[0];
        r.vs[1] = w[1];
      } else {
        r.vs[0] = *reinterpret_cast<const uint32_t*>(vs);
      }
    }
  }

  // element of the query operand's piece i, lane group g
  static __device__ __forceinline__ int q_at(int i, int g) { return D / 4 * g + 8 * i; }

  // key tile t, piece i
  static __device__ __forceinline__ void k_tile(const Regs& r, int t, u32x4 (&k)[D / 32]) {
    const f16x2 s0 = scale_f16<0>(r.ks[t]);
    if constexpr (D == 128) {
      const f16x2 s1 = scale_f16<1>(r.ks[t]);
      k[0] = codes_f16(r.k[t][0], s0);
      k[1] = codes_f16(r.k[t][1], s0);
      k[2] = codes_f16(r.k[t][2], s1);
      k[3] = codes_f16(r.k[t][3], s1);
    } else {
      k[0] = codes_f16(r.k[t][0], s0);
      k[1] = codes_f16(r.k[t][1], s0);
    }
  }

  // 16-byte vectors of a key are exchanged among each other by key so that the
  // transposing reads of 64 keys meet few bank conflicts
  static __device__ __forceinline__ int swizzle(int key) {
    return D == 128 ? (key >> 2) & 3 : (key >> 3) & 1;
  }
  static __device__ __forceinline__ void stage_v(const Regs& r, char* lds, int lane) {
#pragma unroll
    for (int u = 0; u < kVLoads; ++u) {
      const int x = u * 64 + lane, vk = x / (D / 32), c = x % (D / 32);
      *reinterpret_cast<u32x4*>(lds + vk * (D / 2) + 16 * (c ^ swizzle(vk))) = r.v[u];
    }
    _Float16* sc = reinterpret_cast<_Float16*>(lds + kFewKeys * D / 2);
    const bool on = (r.seen >> lane) & 1;      // (bytes of slots that are not seen may be NaN codes)
#pragma unroll
    for (int i = 0; i < kGroups / 4; ++i) {
      const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.vs[i], false);
      const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.vs[i], true);
      sc[(4 * i + 0) * kFewKeys + lane] = (_Float16)(on ? a[0] : 0.0f);
      sc[(4 * i + 1) * kFewKeys + lane] = (_Float16)(on ? a[1] : 0.0f);
      sc[(4 * i + 2) * kFewKeys + lane] = (_Float16)(on ? b[0] : 0.0f);
      sc[(4 * i + 3) * kFewKeys + lane] = (_Float16)(on ? b[1] : 0.0f);
    }
  }
  // V^T of elements 16 d .. 16 d + 15: lane (element, g), keys 16 t + 4 g + 0..3,
  // t = 0, 1 in the first operand, 2, 3 in the second
  static __device__ __forceinline__ void v_tile(const char* lds, int d, int lane, u32x4 (&v)[2]) {
    const int i = lane & 15, g = lane >> 4;
    const int key = 16 * (i >> 2) + 4 * g + (i & 3);
    const int c = d >> 1;
    const i32x2 w = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i32x2*)(
        lds + key * (D / 2) + 16 * (c ^ swizzle(key)) + 8 * (d & 1)));
    const char* sc = lds + kFewKeys * D / 2 + (d * kFewKeys + 4 * g) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f16x2 s[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const u32x2 p = *reinterpret_cast<const u32x2*>(sc + 2 * 16 * (2 * h + t));
        s[2 * t] = as_f16x2(p[0]);
        s[2 * t + 1] = as_f16x2(p[1]);
      }
      v[h] = codes_f16((uint32_t)w[h], s);
    }
  }
};

// bf16 states.
template <int D, bool Once>
struct Few<CrossSource, D, Once> {
  static constexpr int kK = D / 32;                    // 16-byte pieces per lane and tile
  static constexpr int kVLoads = kFewKeys * D * 2 / 16 / 64;
  static constexpr int kLds = kFewKeys * D * 2;

  struct Regs {
    u32x4 k[4][kK];
    u32x4 v[kVLoads];
    uint64_t seen;
  };
  static __device__ __forceinline__ void load(Regs& r, const CrossSource& s,
                                              const CrossSource::Look& look, int64_t b, int hk, int base, int n, int lane) {
    const int key = lane & 15, g = lane >> 4;
    const int64_t row0 = b * s.Lk + base;
    r.seen = s.seen(look, base, n, lane);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < kK; ++i) {
        r.k[t][i] = u32x4{0, 0, 0, 0};
        if (base + 16 * t + key < n)
          r.k[t][i] = *reinterpret_cast<const u32x4*>(s.k + (row0 + 16 * t + key) * s.ldk +
                                                      hk * D + 32 * i + 8 * g);
      }
#pragma unroll
    for (int u = 0; u < kVLoads; ++u) {
      const int x = u * 64 + lane, vk = x / (D / 8);
      r.v[u] = u32x4{0, 0, 0, 0};
      if (base + vk < n)
        r.v[u] = fetch<Once, u32x4>(s.v + (row0 + vk) * s.ldv + hk * D + 8 * (x % (D / 8)));
    }
  }
  static __device__ __forceinline__ int q_at(int i, int g) { return 32 * i + 8 * g; }
  static __device__ __forceinline__ void k_tile(const Regs& r, int t, u32x4 (&k)[kK]) {
#pragma unroll
    for (int i = 0; i < kK; ++i) k[i] = r.k[t][i];
  }
  // 32-byte pieces (16 elements) exchanged by key
  static __device__ __forceinline__ int swizzle(int key) {
    return D == 128 ? key & 7 : (key >> 1) & 3;
  }
  static __device__ __forceinline__ void stage_v(const Regs& r, char* lds, int lane) {
#pragma unroll
    for (int u = 0; u < kVLoads; ++u) {
      const int x = u * 64 + lane, vk = x / (D / 8), c = x % (D / 8);
      // a state that is not seen may hold NaN: its weight of zero needs a zero
      const u32x4 w = (r.seen >> vk) & 1 ? r.v[u] : u32x4{0, 0, 0, 0};
      *reinterpret_cast<u32x4*>(lds + vk * (D * 2) + 32 * ((c >> 1) ^ swizzle(vk)) + 16 * (c & 1)) = w;
    }
  }
  static __device__ __forceinline__ void v_tile(const char* lds, int d, int lane, u32x4 (&v)[2]) {
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int key = 16 * t + 4 * g + (i >> 2);
      const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(
          lds + key * (D * 2) + 32 * (d ^ swizzle(key)) + 8 * (i & 3)));
      const u32x2 p = __builtin_bit_cast(u32x2, w);
      v[t >> 1][2 * (t & 1)] = p[0];
      v[t >> 1][2 * (t & 1) + 1] = p[1];
    }
  }
};

// Workgroup: (stream, key head, row tile, split), the split running fastest.
// (Two waves per SIMD keep the compiler from spending more registers than help, 105
// -> 102 us for 16 streams; bf16 of 128 would spill, 54 -> 75 us.)
template <class Source, int D, bool Once>
__global__ void __launch_bounds__(64 * kFewWaves, !Source::kF16 && D == 128 ? 1 : 2)
attn_few_kernel(AttnArgs a, Source src, AttnSplit sp, int tiles, int splits, Gate gate) {
  if (gated_off(gate)) return;
  using F = Few<Source, D, Once>;
  constexpr bool kF16 = Source::kF16;
  constexpr int kJoin = kFewWaves * kFewRows * (D + 4) * 4;       // the waves' sums
  constexpr int kLds = kFewWaves * F::kLds > kJoin ? kFewWaves * F::kLds : kJoin;
  __shared__ __align__(16) char lds[kLds];
  __shared__ float ml[2][kFewWaves][kFewRows];      // each wave's maximum and sum of a row
  __shared__ float fin[2][kFewRows];                // the row's

  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % splits;
  const int at = blockIdx.x / splits, tile = at % tiles;
  const int hk = at / tiles % a.Hkv;
  const int64_t b = at / tiles / a.Hkv;
  const int G = a.Hq / a.Hkv;
  const int nq = src.queries(b, a.Lq), n = src.keys(b);
  const int rows = nq * G;
  const int row0 = tile * kFewRows;
  if (row0 >= rows) return;
  const int row = row0 + col, t = row / G;
  const int64_t qrow = b * a.Lq + t;
  const int head = hk * G + (row - t * G);

  // keys that this lane's row sees, and that every row of the tile sees
  const int upto = src.causal ? n - (nq - 1 - t) : n;
  const int all = src.causal ? n - (nq - 1 - row0 / G) : n;
  const int last = min(row0 + kFewRows, rows) - 1;
  const int end = src.causal ? n - (nq - 1 - last / G) : n;       // that any row sees
  const int chunks = (max(end, 0) + kFewKeys - 1) / kFewKeys;
  const int c0 = (int)((int64_t)chunks * split / splits);
  const int c1 = (int)((int64_t)chunks * (split + 1) / splits);

  u32x4 q[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    q[i] = u32x4{0, 0, 0, 0};
    if (row < rows)
      q[i] = *reinterpret_cast<const u32x4*>(a.q + qrow * a.ldq + (int64_t)head * D + F::q_at(i, g));
  }
  const float c = query_operand<kF16>(q, a.scale * kLog2e, src.k_scale(),
                                      [](float v) { return quad_max(v); });

  char* const vlds = lds + wave * F::kLds;
  f32x4 o[D / 16];
#pragma unroll
  for (int d = 0; d < D / 16; ++d) o[d] = f32x4{0, 0, 0, 0};
  float m = -INFINITY, l = 0.0f;                 // m: largest product, before the scale

  typename F::Regs cur;
  typename Source::Look look = {};
  if (c0 + wave < c1) {
    look = src.look(b, (c0 + wave) * kFewKeys, n, lane);
    F::load(cur, src, look, b, hk, (c0 + wave) * kFewKeys, n, lane);
    look = src.look(b, (c0 + wave + kFewWaves) * kFewKeys, n, lane);
  }
  for (int ch = c0 + wave; ch < c1; ch += kFewWaves) {
    const int base = ch * kFewKeys;
    f32x4 s[4];
#pragma unroll
    for (int t4 = 0; t4 < 4; ++t4) {
      u32x4 k[D / 32];
      F::k_tile(cur, t4, k);
      s[t4] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) s[t4] = mfma16<kF16>(k[i], q[i], s[t4]);
    }
    F::stage_v(cur, vlds, lane);
    const uint64_t seen = cur.seen;
    // the next step's loads, and what those of the one after need
    if (ch + kFewWaves < c1) {
      F::load(cur, src, look, b, hk, base + kFewWaves * kFewKeys, n, lane);
      look = src.look(b, base + 2 * kFewWaves * kFewKeys, n, lane);
    }
    const bool whole = seen == ~0ull && base + kFewKeys <= all;
    if (!whole) {
#pragma unroll
      for (int t4 = 0; t4 < 4; ++t4)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = 16 * t4 + 4 * g + r;
          const bool on = ((seen >> key) & 1) && base + key < upto;
          s[t4][r] = on ? s[t4][r] : -INFINITY;
        }
    }
    float top = m;
#pragma unroll
    for (int t4 = 0; t4 < 4; ++t4)
      top = max3(max3(top, s[t4][0], s[t4][1]), s[t4][2], s[t4][3]);
    top = quad_max(top);
    const float ref = top == -INFINITY ? 0.0f : top;
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - ref) * c);
    const float shift = kPBias<kF16> - ref * c;
    m = top;
    l *= f;
    u32x4 p[2];
#pragma unroll
    for (int t4 = 0; t4 < 4; ++t4) {
      float e[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t4][r], c, shift));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t w = pack16<kF16>(e[2 * r], e[2 * r + 1]);
        l = add_pair<kF16>(w, l);
        p[t4 >> 1][2 * (t4 & 1) + r] = w;
      }
    }
    wave_lds_order();
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      u32x4 v[2];
      F::v_tile(vlds, d, lane, v);
      o[d] *= f;
      o[d] = mfma16<kF16>(v[0], p[0], o[d]);
      o[d] = mfma16<kF16>(v[1], p[1], o[d]);
    }
    wave_lds_order();
  }
  l = quad_sum(l);

  // join the waves: every wave's sums to the common maximum
  __syncthreads();
  if (g == 0) {
    ml[0][wave][col] = m;
    ml[1][wave][col] = l;
  }
  __syncthreads();
  float mt = ml[0][0][col];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) mt = fmaxf(mt, ml[0][w][col]);
  const float ref = mt == -INFINITY ? 0.0f : mt;
  float lt = 0.0f;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) {
    // (times zero, not left out: a sum that is NaN stays so)
    const float mw = ml[0][w][col];
    lt += ml[1][w][col] * (mw == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mw - ref) * c));
  }
  const float fw = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - ref) * c);
  float* const join = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      join[(wave * kFewRows + col) * (D + 4) + 16 * d + 4 * g + r] = o[d][r] * fw;
  if (wave == 0 && g == 0) {
    fin[0][col] = mt == -INFINITY ? mt : mt * c;
    fin[1][col] = lt;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < kFewRows * D / 2; x += 64 * kFewWaves) {
    const int rr = x / (D / 2), d = 2 * (x - rr * (D / 2));
    if (row0 + rr >= rows) break;
    float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      v0 += join[(w * kFewRows + rr) * (D + 4) + d];
      v1 += join[(w * kFewRows + rr) * (D + 4) + d + 1];
    }
    const float mr = fin[0][rr], lr = fin[1][rr];
    const int tr = (row0 + rr) / G, hr = hk * G + (row0 + rr - tr * G);
    if (splits == 1) {
      const float f = lr == 0.0f ? 0.0f : src.v_scale() / lr;
      *reinterpret_cast<uint32_t*>(a.o + (b * a.Lq + tr) * a.ldo + (int64_t)hr * D + d) =
          bf16_pack(v0 * f, v1 * f);
    } else {
      const int64_t to = (int64_t)split * sp.rows + (b * a.Lq + tr) * a.Hq + hr;
      *reinterpret_cast<f32x2_t*>(sp.o + to * D + d) = f32x2_t{v0, v1};
      if (d == 0) {
        sp.m[to] = mr;
        sp.l[to] = lr;
      }
    }
  }
}

// Join the splits of a row, in order, kJoinTurn of them read at a time; D / 4
// lanes per row.  (512 rows of 128 in 8 splits: one split at a time 8.6 us.)
constexpr int kJoinTurn = 4;

template <class Source, int D>
__global__ void __launch_bounds__(256)
attn_join_kernel(AttnArgs a, Source src, AttnSplit sp, int splits, Gate gate) {
  if (gated_off(gate)) return;
  constexpr int kLanes = D / 4, kRows = 256 / kLanes;
  const int d = 4 * (threadIdx.x % kLanes);
  const int64_t at = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;  // (b Lq + t) Hq + head
  if (at >= sp.rows) return;
  const uint32_t qrow = (uint32_t)at / a.Hq, b = qrow / (uint32_t)a.Lq;   // (below 2^24)
  if ((int)(qrow - b * (uint32_t)a.Lq) >= src.queries(b, a.Lq)) return;
  float mt = -INFINITY, l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  for (int s0 = 0; s0 < splits; s0 += kJoinTurn) {
    float ms[kJoinTurn], ls[kJoinTurn];
    f32x4 os[kJoinTurn];
    float top = mt;
#pragma unroll
    for (int j = 0; j < kJoinTurn; ++j) {
      ms[j] = -INFINITY;
      ls[j] = 0.0f;
      os[j] = f32x4{0, 0, 0, 0};
      if (s0 + j < splits) {
        const int64_t i = (s0 + j) * sp.rows + at;
        ms[j] = sp.m[i];
        ls[j] = sp.l[i];
        os[j] = *reinterpret_cast<const f32x4*>(sp.o + i * D + d);
      }
    }
#pragma unroll
    for (int j = 0; j < kJoinTurn; ++j) top = fmaxf(top, ms[j]);
    const float ref = top == -INFINITY ? 0.0f : top;
    const float f = mt == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mt - ref);
    mt = top;
    l *= f;
    o *= f;
#pragma unroll
    for (int j = 0; j < kJoinTurn; ++j) {
      // (times zero, not left out: a sum that is NaN stays so)
      const float fj = ms[j] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ms[j] - ref);
      l = __builtin_fmaf(ls[j], fj, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(os[j][e], fj, o[e]);
    }
  }
  const float f = l == 0.0f ? 0.0f : src.v_scale() / l;
  *reinterpret_cast<u32x2*>(a.o + qrow * a.ldo + (int64_t)((uint32_t)at - qrow * a.Hq) * D + d) =
      u32x2{bf16_pack(o[0] * f, o[1] * f), bf16_pack(o[2] * f, o[3] * f)};
}

// Workgroups to aim for: a few for each of the 256 compute units, so that
// streams of different lengths even out (16 streams of up to 32768 tokens, 8
// heads of 128: 256 143 us, 512 109, 1024 105, 2048 110).  Of bf16 heads of 128
// one workgroup runs at a time on a unit, and each round waits for its first
// keys: one round (16 tokens to 4000 states, 8 heads: 1024 69 us, 512 60, 256 56, 262
// MB at 4.7 TB/s).
constexpr int64_t kFewBlocks = 1024, kFewBlocksWide = 256;

int64_t tiles_of(int64_t B, int64_t Lq, int Hq, int Hkv) {
  return B * Hkv * ((Lq * (Hq / Hkv) + kFewRows - 1) / kFewRows);
}

// Splits wanted for keys up to L.  A step of a workgroup's waves takes about
// 1.8 us of a nearly empty chip and the join 0.22 us a split, so of w steps
// more than sqrt(8 w) splits cost more than they give (one stream of 32768: 32
// splits 21 us, 64 25, 128 37).
int64_t splits_of(int64_t B, int64_t Lq, int Hq, int Hkv, int64_t L, int64_t blocks) {
  const int64_t tiles = tiles_of(B, Lq, Hq, Hkv);
  const int64_t w = (L + kFewKeys * kFewWaves - 1) / (kFewKeys * kFewWaves);
  int64_t s = (blocks + tiles - 1) / tiles;
  s = s < w ? s : w;
  while (s > 1 && s * s > 8 * w) --s;
  if (s <= 1) return 1;
  const int64_t steps = (w + s - 1) / s;
  return (w + steps - 1) / steps;
}

}  // namespace

size_t attn_few_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  const int64_t s = splits_of(B, Lq, Hq, Hkv, L, kFewBlocks);    // (a source may take fewer)
  return s > 1 ? s * AttnSplit::bytes(B * Lq * Hq, D) : 0;
}

template <class Source>
hipError_t launch_attn_few(const AttnArgs& a, const Source& src, int64_t L, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  const int64_t rows = a.B * a.Lq * a.Hq;
  int64_t s = splits_of(a.B, a.Lq, a.Hq, a.Hkv, L, !Source::kF16 && a.D == 128 ? kFewBlocksWide : kFewBlocks);
  const int64_t fit = (int64_t)(ws_bytes / AttnSplit::bytes(rows, a.D));
  if (s > fit) s = fit > 1 ? fit : 1;
  const AttnSplit sp = AttnSplit::in(ws, s, rows, a.D);
  const int64_t tiles = (a.Lq * (a.Hq / a.Hkv) + kFewRows - 1) / kFewRows;
  const dim3 grid((unsigned)(a.B * a.Hkv * tiles * s)), block(64 * kFewWaves);
  const Gate gt = current_gate();
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, src, sp, (int)tiles, (int)s, gt);
  };
  if (tiles == 1)
    a.D == 64 ? go(attn_few_kernel<Source, 64, true>) : go(attn_few_kernel<Source, 128, true>);
  else
    a.D == 64 ? go(attn_few_kernel<Source, 64, false>) : go(attn_few_kernel<Source, 128, false>);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || s == 1) return e;
  return launch_attn_join(a, src, sp, (int)s, stream);
}

template <class Source>
hipError_t launch_attn_join(const AttnArgs& a, const Source& src, const AttnSplit& sp, int splits,
                            hipStream_t stream) {
  const int per = 256 / (a.D / 4);
  const dim3 grid((unsigned)((sp.rows + per - 1) / per));
  if (a.D == 64)
    hipLaunchKernelGGL((attn_join_kernel<Source, 64>), grid, dim3(256), 0, stream, a, src, sp,
                       splits, current_gate());
  else
    hipLaunchKernelGGL((attn_join_kernel<Source, 128>), grid, dim3(256), 0, stream, a, src, sp,
                       splits, current_gate());
  return hipGetLastError();
}

template hipError_t launch_attn_join(const AttnArgs&, const Kv4Source&, const AttnSplit&, int,
                                     hipStream_t);
template hipError_t launch_attn_join(const AttnArgs&, const CrossSource&, const AttnSplit&, int,
                                     hipStream_t);
template hipError_t launch_attn_few(const AttnArgs&, const Kv4Source&, int64_t, void*, size_t,
                                    hipStream_t);
template hipError_t launch_attn_few(const AttnArgs&, const CrossSource&, int64_t, void*, size_t,
                                    hipStream_t);

}  // namespace qact
