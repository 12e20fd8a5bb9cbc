// Many query rows: what a wave does with 32 of them over tiles of 64 staged
// keys.
//
// VALU and MFMA weigh alike: for heads of 64 the weights of 32 keys take about
// 118 ns of a SIMD (16 exp2 at 4.4, 24 other instructions at 2.0), the two
// products' MFMAs and the sums' 123.  Both run at once only when ONE wave's
// instructions alternate between them (an MFMA and up to 7 VALU instructions: the
// time of the longer; the same from two waves: nearly the sum), so a wave forms
// the weights of 32 keys while its MFMAs compute the logits of the next 32 and the
// second product of the 32 before.  Alternating so, with operands read from shared
// memory, a step takes 206 ns of a SIMD that two waves share.
// Over a whole launch neither unit is busy half of the time (VALU 0.45 and MFMA 0.34
// of the cycles, attn_tile.hip): what is left are the waits around the steps.
//
// For the same reason the VALU is left with as little else as possible: no
// maximum is taken of most tiles.  The weights are formed to the reference that
// the row has and summed, which has to be done anyway; only where a sum says
// that a weight may have grown beyond 2^8 times the reference's are the maxima
// taken and the weights formed again (in fp16, too, they stay in range).  A
// lane holds one query row, so that costs one exchange between lanes.
#pragma once

#include "attn_common.h"

namespace qact {

constexpr int kTileKeys = 64;
// A weight is rounded once, to the operand's type (2^-11 or 2^-8 relative: no
// MFMA takes more), and the sums are of rounded weights.  It is p 2^kTileBias
// relative to the reference, which moves when the
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
// Spread: two pieces of four keys of 128 are read at once, so keys 4 k .. 4 k + 3 differ in
// the exchange's upper bits; by key % 8 they meet.  A tree's 128 rows, waves on half a
// tile each: 291 -> 283 us; the tiles of other queries, all waves on the whole tile: 1350 rows,
// 16 heads, 12376 keys 170.8 -> 172.8, causal 171.6 -> 171.2, to bf16 states no change.
template <int D, bool Spread = false>
__device__ __forceinline__ int v_piece(int key, int c) {
  const int by = D != 128 ? key & 3 : Spread ? 2 * (key & 3) + ((key >> 2) & 1) : key & 7;
  return key * (D * 2) + 32 * ((c >> 1) ^ by) + 16 * (c & 1);
}

// Before a row has seen a key: any logit plus this gives an infinite weight,
// minus infinity (not seen) one of zero.
constexpr float kNoReference = 0x1.fffffep127f;

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

  // Nothing seen yet.
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    shift = kNoReference;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) o[d] = f32x16{};
  }

  // The reference from a row's first logits (what is not seen hidden), which
  // spares the first weights from being formed twice.
  __device__ __forceinline__ void start(const f32x16& s) {
    m = row_max(s);
    shift = m == -INFINITY ? kNoReference : kTileBias<F16> - m * c;
  }

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
        sum = add_pair<F16>(p[i >> 2][i & 3], sum);
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
  // f o as bf16, elements 32 d + 2 i + 8 h .. + 7 of the lane's row (i: 0 or 8):
  // it holds 8 (i / 4) + 4 h + 0..3 and 8 (i / 4 + 1) + 4 h + 0..3 of them, lanes
  // l and l + 32 exchange halves.
  __device__ __forceinline__ u32x4 out8(int d, int i, float f) const {
    const auto w0 = __builtin_amdgcn_permlane32_swap(bf16_pack(o[d][i] * f, o[d][i + 1] * f),
                                                     bf16_pack(o[d][i + 4] * f, o[d][i + 5] * f),
                                                     false, false);
    const auto w1 = __builtin_amdgcn_permlane32_swap(bf16_pack(o[d][i + 2] * f, o[d][i + 3] * f),
                                                     bf16_pack(o[d][i + 6] * f, o[d][i + 7] * f),
                                                     false, false);
    return {w0[0], w1[0], w0[1], w1[1]};
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

// The same where all rows see the same keys (the bits become lane masks on the
// scalar unit: one VALU instruction an element, not three).
__device__ __forceinline__ void hide(f32x16& s, uint32_t seen) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int key = 8 * (i >> 2) + (i & 3);
    const uint64_t lo = (uint32_t)((int32_t)(seen << (31 - key)) >> 31);
    const uint64_t hi = (uint32_t)((int32_t)(seen << (27 - key)) >> 31);
    s[i] = __builtin_amdgcn_inverse_ballot_w64(hi << 32 | lo) ? s[i] : -INFINITY;
  }
}

// A wave's finished rows, rounded to bf16, to `dst` (the lane's row and head).
template <bool F16, int D>
__device__ __forceinline__ void store_rows(const Rows<F16, D>& r, float v_scale, uint16_t* dst, int h,
                                           bool on) {
  // (one last place of float32, before the rounding to bf16; a row's largest
  // weight is near its reference's 1, so the sum is a normal number)
  const float f = r.l == 0.0f ? 0.0f : v_scale * __builtin_amdgcn_rcpf(r.l);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      const u32x4 w = r.out8(d, i, f);
      if (on) *reinterpret_cast<u32x4*>(dst + 32 * d + 2 * i + 8 * h) = w;
    }
}

}  // namespace qact
