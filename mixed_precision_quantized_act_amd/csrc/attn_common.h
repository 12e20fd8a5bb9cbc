// What the attention kernels share: the key/value sources (an NVFP4 cache,
// an encoder's bf16 states), the rows of a key head and the running softmax.
//
// Rows: the query heads that share a key head are rows of one problem; row r
// of stream b and key head hk is query token r / G, head hk G + r % G (G = Hq
// / Hkv), so that keys and values are read once for all of them.
//
// Both kernels compute S^T = K Q^T and then O^T = V^T P^T on MFMA: a lane then
// holds ONE query row (a column of S^T), its maximum and sum need no more
// than two or one exchanges between lane groups, and the rows of S^T that a lane
// holds are, as they lie, its operand of the second product: the order of the
// keys inside one MFMA is free as long as V^T is read in the same order.
#pragma once

#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr float kLog2e = 1.4426950408889634f;

// A 16-byte MFMA operand: 8 fp16 (NVFP4 sources: every element times group
// scale is exact in fp16) or 8 bf16.
template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
template <bool F16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// (by value: __builtin_bit_cast of a vector's element reads its first one)
__device__ __forceinline__ f16x2 as_f16x2(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

__device__ __forceinline__ uint32_t f16_pack(float a, float b) {
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (F16) return f16_pack(a, b);
  return bf16_pack(a, b);
}

// acc + a pair's two elements, in float32
template <bool F16>
__device__ __forceinline__ float add_pair(uint32_t p, float acc) {
  if constexpr (F16)
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, p), f16x2{(_Float16)1.0f, (_Float16)1.0f},
                                  acc, false);
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, p),
                                         bf16x2_t{(__bf16)1.0f, (__bf16)1.0f}, acc, false);
}

// Weights are stored as p 2^kPBias: in fp16 the largest is 2^15, so that
// weights down to 2^-29 of it are normal numbers; in bf16 the range needs none.
template <bool F16>
constexpr float kPBias = F16 ? 15.0f : 0.0f;

// A wave's LDS operations run in the order they are issued, so it reads what
// it wrote without a wait; this keeps the compiler from reordering them (the
// writes and reads use different types).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  return fmaxf(fmaxf(a, b), c);
}

// The same value of lanes l and l ^ 32, and of l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float pair_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float quad_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return pair_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quad_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return pair_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// 8 codes (low nibble first) times a scale pair, 8 fp16, exact.
__device__ __forceinline__ u32x4 codes_f16(uint32_t c, f16x2 s) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * s;
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * s;
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * s;
  const f16x2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * s;
  return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
               __builtin_bit_cast(uint32_t, d), __builtin_bit_cast(uint32_t, e)};
}
// the same with one scale for each element (pairs)
__device__ __forceinline__ u32x4 codes_f16(uint32_t c, const f16x2 (&s)[4]) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * s[0];
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * s[1];
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * s[2];
  const f16x2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * s[3];
  return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
               __builtin_bit_cast(uint32_t, d), __builtin_bit_cast(uint32_t, e)};
}
// E4M3 code in byte I of w -> both halves of an fp16 pair (exact)
template <int I>
__device__ __forceinline__ f16x2 scale_f16(uint32_t w) {
  const _Float16 h = (_Float16)__builtin_amdgcn_cvt_f32_fp8((int)w, I);
  return f16x2{h, h};
}

// ------------------------------------------------------------- sources --

// Keys and values in an NVFP4 cache (fp16 operands).
struct Kv4Source {
  Kv4Cache c;
  const int32_t* lens;
  const int32_t* q_lens;
  int causal;

  static constexpr bool kF16 = true;
  __device__ int queries(int64_t b, int64_t Lq) const {
    if (!q_lens) return (int)Lq;
    const int n = q_lens[b];
    return n < 0 ? 0 : (n < Lq ? n : (int)Lq);
  }
  __device__ int keys(int64_t b) const {
    const int64_t cap = c.pages ? c.max_pages << c.page_log2 : 0;
    const int n = lens[b];
    return n < 0 ? 0 : (n < cap ? n : (int)cap);
  }
  // What the loads of 64 keys need to know first, asked a step ahead: the
  // table's entries for the four sixteens of keys from `base` (base % 16 == 0,
  // n > 0 keys), one in each of four lanes.  A vector load on purpose: a scalar
  // one counts with the shared-memory operations but returns out of their
  // order, so that every wait for one of those would wait for it too (measured: a
  // quarter of the time).
  struct Look {
    int e;
  };
  __device__ __forceinline__ Look look(int64_t b, int base, int n, int lane) const {
    const int at = min(base + 16 * (lane & 3), n - 1);
    return {c.table[b * c.max_pages + ((uint32_t)at >> c.page_log2)]};
  }
  static __device__ __forceinline__ int entry(const Look& k, int t) {
    return __builtin_amdgcn_readlane(k.e, t);
  }
  // whether an entry names a page (pages < 2^31)
  __device__ __forceinline__ bool named(int p) const { return (uint32_t)p < (uint32_t)c.pages; }
  // Bit j: position base + j has a slot and lies before n.
  __device__ __forceinline__ uint64_t seen(const Look& k, int base, int n, int lane) const {
    // (bit t of the ballot: sixteen t's entry)
    const uint32_t ok = (uint32_t)__ballot(named(k.e)) & 15u;
    uint64_t s = ~0ull;
    if (ok != 15u) {
      s = 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) s |= (ok >> t) & 1 ? 0xFFFFull << (16 * t) : 0;
    }
    const int left = n - base;
    return left >= 64 ? s : left <= 0 ? 0 : s & ((1ull << left) - 1);
  }
  // Row of position `at` (its page named) in a [pages][H][page] array.
  __device__ __forceinline__ int64_t slot(int p, int hk, int at) const {
    return (((int64_t)p * c.H + hk) << c.page_log2) + (at & ((1 << c.page_log2) - 1));
  }
  __device__ float k_scale() const { return *c.k_ts; }
  __device__ float v_scale() const { return *c.v_ts; }
};

// Keys and values of an encoder (bf16 operands).
struct CrossSource {
  const uint16_t* k;
  const uint16_t* v;
  int64_t ldk, ldv;
  int Lk;
  const int32_t* k_lens;
  const uint8_t* mask;

  static constexpr bool kF16 = false;
  // The mask's byte for state base + lane.
  struct Look {
    uint32_t on;
  };
  __device__ __forceinline__ Look look(int64_t b, int base, int n, int lane) const {
    if (base + lane >= n) return {0u};
    return {mask ? mask[b * Lk + base + lane] : 1u};
  }
  // Bit j: state base + j is seen (by every row).
  __device__ __forceinline__ uint64_t seen(const Look& k, int, int, int) const {
    return __ballot(k.on != 0);
  }
  static constexpr int causal = 0;
  __device__ int queries(int64_t, int64_t Lq) const { return (int)Lq; }
  __device__ int keys(int64_t b) const {
    if (!k_lens) return Lk;
    const int n = k_lens[b];
    return n < 0 ? 0 : (n < Lk ? n : Lk);
  }
  __device__ float k_scale() const { return 1.0f; }
  __device__ float v_scale() const { return 1.0f; }
};

// ---------------------------------------------------------------- queries --

// A query row's operand pieces.  For fp16 the row is scaled by a power of two
// to a largest value in [1, 2) (an element below 2^-24 of it is lost, one
// below 2^-17 keeps fewer bits: less than the float32 sum's own rounding);
// the exponent returns through `c`, which turns a product into a logit in
// units of log2.  c is a positive number: the sign of the keys' tensor scale goes
// to the row, and where the scale is not finite, or c not a float32, the row is
// NaN, so that rows that see nothing still give zeros.  N pieces of 8 elements per
// lane; `most` combines the lanes that hold one row.
template <bool F16, int N, class Most>
__device__ __forceinline__ float query_operand(u32x4 (&q)[N], float scale_log2e, float k_scale,
                                               Most most) {
  if constexpr (F16) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) top = max(top, fold_max(abs_max8_pk(q[i], u16x2{0, 0})));
    // the exponent field alone; a row of zeros, infinities or NaN stays as it is
    const uint32_t e = __float_as_uint(most(__uint_as_float(top << 16))) >> 23;
    const int ex = e == 0 || e == 255 ? 0 : (int)e - 127;
    const float c = __builtin_ldexpf(scale_log2e, ex) * fabsf(k_scale);
    // (times 1, -1 or NaN, not a branch: 16 heads of 128, 1350 rows, 12376 keys: 175.9
    // -> 173.6 us)
    const bool good = c < INFINITY;
    const float sign = good ? copysignf(1.0f, k_scale) : __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[i][j] = f16_pack(__builtin_ldexpf(bf16_lo(q[i][j]), -ex) * sign,
                           __builtin_ldexpf(bf16_hi(q[i][j]), -ex) * sign);
    return fmaxf(good ? c : 1.0f, 0x1p-126f);
  }
  float c = scale_log2e;
  if (!(c < INFINITY)) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    c = 1.0f;
  }
  // (at least the smallest normal number: a product of minus infinity, what
  // is not seen, with it stays minus infinity)
  return fmaxf(c, 0x1p-126f);
}

// --------------------------------------------------------- split of the keys --

// Partial results of one split: float32 sums of p v (not divided), the
// largest product and the sum of p, for rows [B][Hkv][Lq G] in that order.
struct AttnSplit {
  float* o;       // [splits][rows][D]
  float* m;       // [splits][rows] largest logit (log2 units), -inf: nothing seen
  float* l;       // [splits][rows]
  int64_t rows;

  // `splits` partial results of `rows` rows laid out in a workspace
  static AttnSplit in(void* ws, int64_t splits, int64_t rows, int D) {
    AttnSplit s = {};
    s.rows = rows;
    if (splits > 1) {
      s.o = static_cast<float*>(ws);
      s.m = s.o + splits * rows * D;
      s.l = s.m + splits * rows;
    }
    return s;
  }
  static size_t bytes(int64_t rows, int D) { return (size_t)rows * (D + 2) * 4; }
};

// Few query rows, the keys split over workgroups (attn_few.hip); L: the most
// keys a stream can have.
size_t attn_few_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L);
template <class Source>
hipError_t launch_attn_few(const AttnArgs& a, const Source& src, int64_t L, void* ws,
                           size_t ws_bytes, hipStream_t stream);

// Join `splits` partial results of every row.
template <class Source>
hipError_t launch_attn_join(const AttnArgs& a, const Source& src, const AttnSplit& sp, int splits,
                            hipStream_t stream);

// Many query rows (attn_tile.hip).
size_t attn_tile_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L);
template <class Source>
hipError_t launch_attn_tile(const AttnArgs& a, const Source& src, int64_t L, void* ws,
                            size_t ws_bytes, hipStream_t stream);

// Many query rows to few states (attn_short.hip), where it takes the sizes.
bool attn_short_takes(int64_t Lq, int Hq, int Hkv, int D, int64_t Lk);
hipError_t launch_attn_short(const AttnArgs& a, const CrossSource& src, hipStream_t stream);

}  // namespace qact
