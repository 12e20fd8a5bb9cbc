// qk_rope: query and key heads turned by their positions, the angles formed in
// the call (6Bit-Diffusion's transformer blocks project queries and keys with
// one quantized linear; this stands between it and the attention).
//
//   (u, v) -> s (u cos a - v sin a, v cos a + u sin a),  a = pos[m] freq[i]
//
// for the pairs (2 i, 2 i + 1) or (i, i + R/2) of a head's first R elements;
// the others are passed on.  The angle is formed and reduced to a turn's
// fraction in float64 (a position of 2^24 times a frequency of 1 loses 2^-29 of
// a turn there; in float32 it loses everything), its sine and cosine are
// float32, and so are the products up to the one rounding to bf16.
//
// The bound is the memory rate, 4 bytes per element.  A workgroup takes whole
// tokens, forms each token's R/2 sines and cosines once, in shared memory, for
// all its heads, and has the heads' elements on their way meanwhile.
#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

namespace {

constexpr int kRopeMost = 2048;        // sines and cosines of a workgroup's tokens

// A thread's work: 16 elements of a head, two vectors of 8: j < R / 16 the
// vectors j and j + R / 16 of the turned part (the two halves' partners, or 8
// pairs), above them two neighbouring vectors that are passed on.
template <int U>
__global__ void __launch_bounds__(256)
qk_rope_kernel(RopeArgs a, int per, int tokens, Gate gate) {
  if (gated_off(gate)) return;
  __shared__ float2 table[kRopeMost];
  __shared__ int turned[64];
  const int tid = threadIdx.x, half = a.R / 2;
  const int64_t m0 = (int64_t)blockIdx.x * tokens;
  const int here = (int)min<int64_t>(tokens, a.M - m0);
  const int units = a.D / 16, rot = a.R / 16, total = here * per;
  const int begin = blockIdx.y * (256 * U);

  u32x4 w0[U], w1[U];
  uint16_t* dst[U];
  int place[U];                        // table entry of the first pair; -1: passed on, -2: nothing
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = begin + u * 256 + tid;
    place[u] = -2;
    if (i >= total) continue;
    const int t = i / per, x = i - t * per, h = x / units, j = x - h * units;
    const bool key = h >= a.Hq;
    const int64_t m = m0 + t;
    const int first = j < rot ? j : 2 * rot + 2 * (j - rot), second = j < rot ? j + rot : first + 1;
    const int64_t at = (int64_t)(key ? h - a.Hq : h) * a.D + 8 * first;
    const uint16_t* src = (key ? a.k + m * a.ldk : a.q + m * a.ldq) + at;
    dst[u] = (key ? a.k_out + m * a.ldko : a.q_out + m * a.ldqo) + at;
    w0[u] = *reinterpret_cast<const u32x4*>(src);
    w1[u] = *reinterpret_cast<const u32x4*>(src + 8 * (second - first));
    place[u] = j < rot ? t * half + (a.rope == QA_ROPE_PAIRS ? 4 * j : 8 * j) : -1;
  }

  for (int x = tid; x < here * half; x += 256) {
    const int t = x / half, i = x - t * half;
    const int pos = a.pos ? a.pos[m0 + t] : (int)(m0 + t);
    const double turns = (double)pos * a.freq[i] * 0.15915494309189535;      // 1 / (2 pi)
    const float f = (float)(2.0 * (turns - rint(turns)));
    float s, c;
    sincospif(f, &s, &c);
    table[x] = float2{c * a.scale, s * a.scale};
    if (i == 0) turned[t] = pos >= 0;
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (place[u] == -2) continue;
    const int second = place[u] >= 0 ? a.R / 2 : 8;
    if (place[u] >= 0 && turned[place[u] / half]) {
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w0[u][i]);
        x[2 * i + 1] = bf16_hi(w0[u][i]);
        y[2 * i] = bf16_lo(w1[u][i]);
        y[2 * i + 1] = bf16_hi(w1[u][i]);
      }
      const float2* cs = table + place[u];
      if (a.rope == QA_ROPE_PAIRS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = cs[i], q = cs[half / 2 + i];
          const float u0 = x[2 * i], v0 = x[2 * i + 1], u1 = y[2 * i], v1 = y[2 * i + 1];
          x[2 * i] = __builtin_fmaf(u0, p.x, -(v0 * p.y));
          x[2 * i + 1] = __builtin_fmaf(v0, p.x, u0 * p.y);
          y[2 * i] = __builtin_fmaf(u1, q.x, -(v1 * q.y));
          y[2 * i + 1] = __builtin_fmaf(v1, q.x, u1 * q.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 p = cs[i];
          const float u0 = x[i], v0 = y[i];
          x[i] = __builtin_fmaf(u0, p.x, -(v0 * p.y));
          y[i] = __builtin_fmaf(v0, p.x, u0 * p.y);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w0[u][i] = bf16_pack(x[2 * i], x[2 * i + 1]);
        w1[u][i] = bf16_pack(y[2 * i], y[2 * i + 1]);
      }
    }
    *reinterpret_cast<u32x4*>(dst[u]) = w0[u];
    *reinterpret_cast<u32x4*>(dst[u] + second) = w1[u];
  }
}

}  // namespace

hipError_t launch_qk_rope(const RopeArgs& a, hipStream_t stream) {
  const int per = (a.Hq + a.Hk) * (a.D / 16);              // of a token
  int tokens = 1024 / per;
  if (tokens > kRopeMost / (a.R / 2)) tokens = kRopeMost / (a.R / 2);
  if (tokens > 64) tokens = 64;
  if (tokens < 1) tokens = 1;
  const dim3 grid((unsigned)((a.M + tokens - 1) / tokens), (unsigned)((tokens * per + 1023) / 1024));
  hipLaunchKernelGGL(qk_rope_kernel<4>, grid, dim3(256), 0, stream, a, per, tokens, current_gate());
  return hipGetLastError();
}

}  // namespace qact
