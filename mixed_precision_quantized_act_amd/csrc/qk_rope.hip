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
// all its heads, and has the heads' elements on their way meanwhile: one thread two
// vectors, so that many small workgroups hide each other's waits.  17776 tokens of 30 +
// 30 heads of 64 (273 MB): 54.5 us, 5.0 TB/s, where a large copy reaches 5.1.  In a loop over
// three sets of buffers it takes 50, workgroups of 64, 256 and 512 threads 54, 52 and 52, four
// times the vectors a thread 57, stores past the caches 73 (half the head turned) and 54 (all
// of it).  63 tokens of 32 + 8 heads of 128: 4.1 us, a launch.
#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeMost = 8 * kRopeThreads;        // sines and cosines of a workgroup's tokens

// A thread's work: 16 elements of a head, two vectors of 8: j < R / 16 the
// vectors j and j + R / 16 of the turned part (the two halves' partners, or 8
// pairs), above them two neighbouring vectors that are passed on.
__global__ void __launch_bounds__(kRopeThreads)
qk_rope_kernel(RopeArgs a, int per, int tokens, Gate gate) {
  if (gated_off(gate)) return;
  __shared__ float2 table[kRopeMost];
  __shared__ int turned[kRopeThreads];
  const int tid = threadIdx.x, half = a.R / 2;
  const int64_t m0 = (int64_t)blockIdx.x * tokens;
  const int here = (int)min<int64_t>(tokens, a.M - m0);
  const int units = a.D / 16, rot = a.R / 16;

  const int i = blockIdx.y * kRopeThreads + tid, t = i / per, x = i - t * per, h = x / units, j = x - h * units;
  const bool on = t < here, key = h >= a.Hq;
  const int first = j < rot ? j : 2 * rot + 2 * (j - rot), apart = j < rot ? 8 * rot : 8;
  const int64_t m = m0 + t, at = (int64_t)(key ? h - a.Hq : h) * a.D + 8 * first;
  u32x4 w0 = {0, 0, 0, 0}, w1 = w0;
  if (on) {
    const uint16_t* src = (key ? a.k + m * a.ldk : a.q + m * a.ldq) + at;
    w0 = *reinterpret_cast<const u32x4*>(src);
    w1 = *reinterpret_cast<const u32x4*>(src + apart);
  }

  for (int y = tid; y < here * half; y += kRopeThreads) {
    const int n = y / half, f = y - n * half;
    const int pos = a.pos ? a.pos[m0 + n] : (int)(m0 + n);
    const double turns = (double)pos * a.freq[f] * 0.15915494309189535;      // 1 / (2 pi)
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    table[y] = float2{c * a.scale, s * a.scale};
    if (f == 0) turned[n] = pos >= 0;
  }
  __syncthreads();
  if (!on) return;

  if (j < rot && turned[t]) {
    float u[8], v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[2 * k] = bf16_lo(w0[k]);
      u[2 * k + 1] = bf16_hi(w0[k]);
      v[2 * k] = bf16_lo(w1[k]);
      v[2 * k + 1] = bf16_hi(w1[k]);
    }
    const float2* cs = table + t * half;
    const auto turn = [](float& a, float& b, float2 p) {
      const float a0 = a, b0 = b;
      a = __builtin_fmaf(a0, p.x, -(b0 * p.y));
      b = __builtin_fmaf(b0, p.x, a0 * p.y);
    };
    if (a.rope == QA_ROPE_PAIRS) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        turn(u[2 * k], u[2 * k + 1], cs[4 * j + k]);
        turn(v[2 * k], v[2 * k + 1], cs[4 * j + half / 2 + k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(u[k], v[k], cs[8 * j + k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w0[k] = bf16_pack(u[2 * k], u[2 * k + 1]);
      w1[k] = bf16_pack(v[2 * k], v[2 * k + 1]);
    }
  }
  uint16_t* dst = (key ? a.k_out + m * a.ldko : a.q_out + m * a.ldqo) + at;
  *reinterpret_cast<u32x4*>(dst) = w0;
  *reinterpret_cast<u32x4*>(dst + apart) = w1;
}

}  // namespace

hipError_t launch_qk_rope(const RopeArgs& a, hipStream_t stream) {
  const int per = (a.Hq + a.Hk) * (a.D / 16);              // of a token
  const int most = kRopeMost / (a.R / 2), fit = kRopeThreads / per;
  const int tokens = fit < 1 ? 1 : fit < most ? fit : most;
  const dim3 grid((unsigned)((a.M + tokens - 1) / tokens), (unsigned)((tokens * per + kRopeThreads - 1) / kRopeThreads));
  hipLaunchKernelGGL(qk_rope_kernel, grid, dim3(kRopeThreads), 0, stream, a, per, tokens, current_gate());
  return hipGetLastError();
}

}  // namespace qact
