// qlinear_w8a8: the linear of INT8 activations and INT8 weights, a scale for
// each token and each output channel (6Bit-Diffusion, abstract: volatile layers
// keep INT8; here the weights do, too).
//
//   y[m][n] = s_a[m] s_w[n] sum_k a[m][k] w[n][k]  (+ bias[n]) (-> GELU)
//
// The sum is an exact int32 (|a w| <= 2^14, K < 2^17) from
// v_mfma_i32_32x32x32_i8, rounded once to float32.
#include "qgemm_common.h"

namespace qact {

namespace {

struct W8Args {
  const int8_t* a;
  const float* a_s;
  const int8_t* w;
  const float* w_s;
  int64_t M, N, K;
  int nt;
  Gate gate;
};

constexpr uint32_t kSkip = 0x7FFFFFF0u;          // an offset past every buffer range

template <int kEpi>
__global__ void __launch_bounds__(256)
w8a8_simple_kernel(W8Args g, EpiArgs e) {
  if (gated_off(g.gate)) return;
  __shared__ __align__(16) uint8_t stg[4 * 8192];
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)(blockIdx.x / g.nt) * 128 + 32 * wave;
  const int64_t n0 = (int64_t)(blockIdx.x % g.nt) * 128;
  if (m0 >= g.M) return;
  const uint32_t K = (uint32_t)g.K;
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(g.a + m0 * g.K, (uint32_t)(min<int64_t>(g.M - m0, 32) * g.K));
  const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(g.w + n0 * g.K, (uint32_t)(min<int64_t>(g.N - n0, 128) * g.K));
  i32x16 acc[1][4] = {};
  for (uint32_t k = 0; k < K; k += 32) {
    const uint32_t at = k + 16 * lh < K ? k + 16 * lh : kSkip;
    const auto load = [&](__amdgpu_buffer_rsrc_t r, int row) {
      return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                           r, at == kSkip ? (int)kSkip : (int)((uint32_t)row * K + at), 0, 0));
    };
    const i32x4 a = load(ra, lr);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[0][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(load(rw, 32 * j + lr), a, acc[0][j], 0, 0, 0);
  }
  const float rs[1] = {g.a_s[min<int64_t>(m0 + lr, g.M - 1)]};
  float cf[4][16];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      cf[j][r] = g.w_s[min<int64_t>(n0 + 32 * j + 8 * (r >> 2) + 4 * lh + (r & 3), g.N - 1)];
  store_tile<kEpi, 1>([&](int i, int j, int r) { return (float)acc[i][j][r] * cf[j][r]; }, rs, m0, n0,
                      stg + wave * 8192, e, lane);
}

}  // namespace

hipError_t launch_w8a8(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s, int64_t M,
                       int64_t N, int64_t K, const GemmOut& o, void*, size_t, hipStream_t st) {
  const bool vec = (reinterpret_cast<uintptr_t>(o.y) % 16 == 0) && (o.ldy % 4 == 0);
  const EpiArgs e = {o.y, o.ldy, o.out_f32, o.gelu, o.bias, M, N, vec, nullptr, nullptr, nullptr, nullptr};
  const W8Args g = {a_q, a_s, w_q, w_s, M, N, K, (int)((N + 127) / 128), current_gate()};
  const dim3 grid((unsigned)((M + 127) / 128 * g.nt));
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, g, e); };
  if (o.out_f32 || !vec)
    go(w8a8_simple_kernel<kEpiGeneral>);
  else if (o.bias)
    o.gelu ? go(w8a8_simple_kernel<kEpiStagedBiasGelu>) : go(w8a8_simple_kernel<kEpiStagedBias>);
  else
    o.gelu ? go(w8a8_simple_kernel<kEpiStagedGelu>) : go(w8a8_simple_kernel<kEpiPlain>);
  return hipGetLastError();
}

size_t w8a8_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

}  // namespace qact
