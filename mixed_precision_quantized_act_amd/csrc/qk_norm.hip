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
// power of two for the sums); a wave takes several heads of ONE token, so
// that the token's table row is read once per wave and not once per head.
#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

namespace {

// heads of a token taken one after the other by a lane group
constexpr int kQkHeads = 4;

__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Sum over the LPH lanes of a head.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, LPH);
  return v;
}

template <int LPH, int U>
__global__ void __launch_bounds__(256)
qk_norm_rope_kernel(QkArgs a, int chunks, Gate gate) {
  if (gated_off(gate)) return;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= a.M * chunks) return;
  const int64_t tok = item / chunks;
  const int l = lane & (LPH - 1);
  const int head0 = (int)(item - tok * chunks) * (64 / LPH * U) + lane / LPH;
  const int D = a.D, H = a.Hq + a.Hk;
  const bool in = 8 * l < D;

  u32x4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = head0 + u * (64 / LPH);
    raw[u] = u32x4{0, 0, 0, 0};
    if (in && h < H) {
      const uint16_t* p = h < a.Hq ? a.q + tok * a.ldq + (int64_t)h * D
                                   : a.k + tok * a.ldk + (int64_t)(h - a.Hq) * D;
      raw[u] = *reinterpret_cast<const u32x4*>(p + 8 * l);
    }
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

  float w[2][8], b[2][8];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint16_t* wp = s ? a.k_w : a.q_w;
    const uint16_t* bp = s ? a.k_b : a.q_b;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[s][i] = 1.0f, b[s][i] = 0.0f;
    if (wp && in) unpack8(*reinterpret_cast<const u32x4*>(wp + 8 * l), w[s]);
    if (bp && in) unpack8(*reinterpret_cast<const u32x4*>(bp + 8 * l), b[s]);
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = head0 + u * (64 / LPH);
    const int s = h < a.Hq ? 0 : 1;
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
      const float r = 1.0f / __builtin_sqrtf(head_sum<LPH>(t) * a.inv_D + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = __builtin_fmaf(x[i] * r, s ? w[1][i] : w[0][i], s ? b[1][i] : b[0][i]);
    }
    if (a.rope == QA_ROPE_PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = x[2 * i], q = x[2 * i + 1];
        x[2 * i] = __builtin_fmaf(p, cs[i], -(q * sn[i]));
        x[2 * i + 1] = __builtin_fmaf(q, cs[i], p * sn[i]);
      }
    } else if (a.rope == QA_ROPE_HALVES) {
      const bool upper = 8 * l >= D / 2;
      const int other = (lane & ~(LPH - 1)) | ((upper ? l - D / 16 : l + D / 16) & (LPH - 1));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl(x[i], other, 64);
        x[i] = __builtin_fmaf(x[i], cs[i], upper ? y * sn[i] : -(y * sn[i]));
      }
    }
    if (in && h < H) {
      uint16_t* p = s == 0 ? a.q_out + tok * a.ldqo + (int64_t)h * D
                           : a.k_out + tok * a.ldko + (int64_t)(h - a.Hq) * D;
      *reinterpret_cast<u32x4*>(p + 8 * l) = u32x4{bf16_pack(x[0], x[1]), bf16_pack(x[2], x[3]),
                                                   bf16_pack(x[4], x[5]), bf16_pack(x[6], x[7])};
    }
  }
}

template <int LPH>
hipError_t launch(const QkArgs& a, hipStream_t stream) {
  const int per = 64 / LPH * kQkHeads;
  const int chunks = (a.Hq + a.Hk + per - 1) / per;
  const dim3 grid((unsigned)((a.M * chunks + 3) / 4));
  hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, kQkHeads>), grid, dim3(256), 0, stream, a, chunks,
                     current_gate());
  return hipGetLastError();
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
