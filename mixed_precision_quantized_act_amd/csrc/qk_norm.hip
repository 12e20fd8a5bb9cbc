// qk_norm_rope: the norm of every query and key head and the rotation by the
// token's position, in one pass between the QKV linear and the attention
// (6Bit-Diffusion's transformer blocks project queries and keys with one
// quantized linear).
//
//   layer norm  y = (x - mean) / sqrt(var + eps) * w + b      (over the head)
//   RMS norm    y = x / sqrt(mean x^2 + eps) * w
//   rotation    (u, v) -> (u cos - v sin, v cos + u sin) for the pairs
//               (2i, 2i+1) or (i, i + D/2)
//
// Everything is float32 between one read and one rounding to bf16, so the
// bound is the memory rate: 4 bytes per element and the position's cosines
// and sines.  A head is spread over D/8 lanes (16 bytes each, padded to a
// power of two for the sums); a wave takes several query or several key heads
// of ONE token, so that the token's table row and the norm's weights are read
// once per wave and not once per head.
//
// 17776 tokens, 30 + 30 heads of 64, layer norm, pairs: 55.5 us, 273 MB at 4.9
// TB/s (a copy reaches 5.1).  What is left to do per element is the VALU's
// work; exchanges through shared memory, weights of both kinds per wave, and
// a division of 64 bits took it from 60 to 78 us.
#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

namespace {

// Heads of a token taken one after the other by a lane group (17776 tokens: 2
// 58 us, 4 55.5, 6 59); of few tokens one, so that more waves share them (9 tokens,
// 32 + 8 heads of 128: 4 4.8 us, 1 3.9).
constexpr int kQkHeads = 4;
constexpr int64_t kQkWaves = 2048;

__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                               0xF, 0xF, false));
}

// Sum over the LPH lanes of a head, by lane moves that need no shared memory:
// neighbours, pairs, then mirrors of 8 and 16 lanes (their halves hold equal
// sums).
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
  v += dpp<0xB1>(v);                                             // quad_perm 1 0 3 2
  if constexpr (LPH >= 4) v += dpp<0x4E>(v);                     // quad_perm 2 3 0 1
  if constexpr (LPH >= 8) v += dpp<0x141>(v);                    // row_half_mirror
  if constexpr (LPH >= 16) v += dpp<0x140>(v);                   // row_mirror
  if constexpr (LPH >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// 1 / sqrt(v) to one last place of float32; the hardware's takes a subnormal
// number for zero.
__device__ __forceinline__ float inverse_sqrt(float v) {
  const bool small = v < 0x1p-100f;
  return __builtin_amdgcn_rsqf(small ? v * 0x1p100f : v) * (small ? 0x1p50f : 1.0f);
}

template <int LPH, int U>
__global__ void __launch_bounds__(256)
qk_norm_rope_kernel(QkArgs a, int qchunks, int chunks, Gate gate) {
  if (gated_off(gate)) return;
  const int lane = threadIdx.x & 63;
  const uint32_t item = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= (uint32_t)(a.M * chunks)) return;           // (below 2^26)
  const int64_t tok = item / (uint32_t)chunks;
  const int l = lane & (LPH - 1), chunk = (int)(item % (uint32_t)chunks);
  const int D = a.D;
  const bool in = 8 * l < D;
  // the wave's heads: query heads or key heads
  const bool key = chunk >= qchunks;
  const int H = key ? a.Hk : a.Hq;
  const int head0 = (key ? chunk - qchunks : chunk) * (64 / LPH * U) + lane / LPH;
  const uint16_t* const src = key ? a.k + tok * a.ldk : a.q + tok * a.ldq;
  uint16_t* const dst = key ? a.k_out + tok * a.ldko : a.q_out + tok * a.ldqo;

  u32x4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = head0 + u * (64 / LPH);
    raw[u] = u32x4{0, 0, 0, 0};
    if (in && h < H) raw[u] = *reinterpret_cast<const u32x4*>(src + (int64_t)h * D + 8 * l);
  }

  // the token's cosines and sines for this lane's elements: pairs, 4 of
  // each; halves, 8 of each (both halves of a head share them)
  float cs[8], sn[8];
  bool turn = false;
  if (a.rope != QA_ROPE_NONE) {
    const int64_t pos = a.pos ? (int64_t)a.pos[tok] : tok;
    turn = pos >= 0 && pos < a.P;
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
    if (turn && in) {
      const float* cp = a.cos + pos * (D / 2);
      const float* sp = a.sin + pos * (D / 2);
      if (a.rope == QA_ROPE_PAIRS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = cp[4 * l + i], sn[i] = sp[4 * l + i];
      } else {
        const int at = 8 * l >= D / 2 ? 8 * l - D / 2 : 8 * l;
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = cp[at + i], sn[i] = sp[at + i];
      }
    }
  }

  float w[8], b[8];
  const uint16_t* const wp = key ? a.k_w : a.q_w;
  const uint16_t* const bp = key ? a.k_b : a.q_b;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.0f, b[i] = 0.0f;
  if (wp && in) unpack8(*reinterpret_cast<const u32x4*>(wp + 8 * l), w);
  if (bp && in) unpack8(*reinterpret_cast<const u32x4*>(bp + 8 * l), b);

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = head0 + u * (64 / LPH);
    float x[8];
    unpack8(raw[u], x);
    if (a.norm != QA_NORM_NONE) {
      if (a.norm == QA_NORM_LAYER) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += x[i];
        const float mean = head_sum<LPH>(t) * a.inv_D;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = in ? x[i] - mean : 0.0f;
      }
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = __builtin_fmaf(x[i], x[i], t);
      const float r = inverse_sqrt(head_sum<LPH>(t) * a.inv_D + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __builtin_fmaf(x[i] * r, w[i], b[i]);
    }
    // (a token that is not turned is passed on: times 1 and 0, an infinite
    // element would make its partner NaN)
    if (turn && a.rope == QA_ROPE_PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = x[2 * i], q = x[2 * i + 1];
        x[2 * i] = __builtin_fmaf(p, cs[i], -(q * sn[i]));
        x[2 * i + 1] = __builtin_fmaf(q, cs[i], p * sn[i]);
      }
    } else if (turn && a.rope == QA_ROPE_HALVES) {
      const bool upper = 8 * l >= D / 2;
      const int other = (lane & ~(LPH - 1)) | ((upper ? l - D / 16 : l + D / 16) & (LPH - 1));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl(x[i], other, 64);
        x[i] = __builtin_fmaf(x[i], cs[i], upper ? y * sn[i] : -(y * sn[i]));
      }
    }
    if (in && h < H)
      // (past the caches: left dirty there, the last of them would be written back
      // after the kernel; 60 and 55.5 us)
      __builtin_nontemporal_store(u32x4{bf16_pack(x[0], x[1]), bf16_pack(x[2], x[3]),
                                        bf16_pack(x[4], x[5]), bf16_pack(x[6], x[7])},
                                  reinterpret_cast<u32x4*>(dst + (int64_t)h * D + 8 * l));
  }
}

template <int LPH, int U>
hipError_t launch(const QkArgs& a, hipStream_t stream) {
  const int per = 64 / LPH * U;
  const int qchunks = (a.Hq + per - 1) / per, chunks = qchunks + (a.Hk + per - 1) / per;
  const dim3 grid((unsigned)((a.M * chunks + 3) / 4));
  hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, U>), grid, dim3(256), 0, stream, a, qchunks, chunks,
                     current_gate());
  return hipGetLastError();
}

template <int LPH>
hipError_t launch(const QkArgs& a, hipStream_t stream) {
  const int64_t groups = (int64_t)a.M * (a.Hq + a.Hk);              // of lanes, one head each
  return groups * LPH < kQkWaves * 64 ? launch<LPH, 1>(a, stream) : launch<LPH, kQkHeads>(a, stream);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkArgs& a, hipStream_t stream) {
  const int lanes = a.D / 8;
  if (lanes <= 2) return launch<2>(a, stream);
  if (lanes <= 4) return launch<4>(a, stream);
  if (lanes <= 8) return launch<8>(a, stream);
  if (lanes <= 16) return launch<16>(a, stream);
  return launch<32>(a, stream);
}

}  // namespace qact
