// qlinear_bf16: the linear of a few bf16 rows (M <= 32) against an NVFP4
// weight, for the rows that are not worth quantizing: a conditioning vector's
// modulation, one token of each stream (6Bit-Diffusion, Table 2: 4-bit
// weights).
//
//   y[m][n] = s_Tw sum_g s[n][g] sum_{j<16} x[m][16 g + j] c[n][16 g + j]
//
// The weight is read once: 9/16 byte per element, everything else is small,
// so the bound is the memory rate.  The arithmetic per code has to stay below
// it.  An E2M1 code is exact in bf16, so the inner sums run on bf16 MFMA
// (exact products, float32 sums) on the bare codes, half an instruction per
// code; the group's E4M3 scale is then applied in float32 to the sums.  One
// 16x16x32 MFMA holds two scale groups of 16 weight rows: its 16 activation
// rows are the same 8 rows twice, rows 0-7 with x in the first group's half
// of k and zeros in the second's, rows 8-15 the other way round.  The result
// holds each group's sum apart, and four FMAs scale 512 codes.  (A scale
// multiplied into each weight and rounded into bf16 would take twice the
// VALU time.)
//
// Layout: a lane reads 16 bytes of one weight row: the four lane groups of 16
// hold groups (0, 1), (2, 3), (4, 5), (6, 7) of 128 elements.  Swapping the
// odd lane groups' first register with the even ones' second puts both halves
// of a group side by side, as the MFMA wants them.
#include "qact_device.h"
#include "qact_internal.h"
#include "qgemm_common.h"

namespace qact {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kGvRows = 16;        // weight rows of a tile
constexpr int kGvStep = 128;       // elements of a row per step
constexpr int kGvWaves = 8;        // waves of a workgroup, at most: they split K

struct GemvArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* wq;
  const uint8_t* ws;
  const float* wts;
  int M;
  int64_t N, K;
  const uint16_t* bias;
  void* y;
  int64_t ldy;
  int out_f32, gelu;
};

// 8 codes -> 8 bf16 (exact)
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t c) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2);
  const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// One step's operands of a lane.
struct GemvStep {
  u32x4 code;
  uint32_t scale;
};

// CT: tiles of 8 activation rows.
template <int CT>
__global__ void __launch_bounds__(64 * kGvWaves)
qgemv_kernel(GemvArgs a, Gate gate) {
  if (gated_off(gate)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kGvRows;
  const int64_t n = min(n0 + c, a.N - 1);
  const uint8_t* const wrow = a.wq + n * (a.K / 2);
  const uint8_t* const srow = a.ws + n * (a.K / 16);
  const int nsteps = (int)((a.K + kGvStep - 1) / kGvStep);

  auto load = [&](int s) {
    GemvStep r;
    const int64_t k = (int64_t)s * kGvStep;
    if (k + kGvStep <= a.K) {
      r.code = *reinterpret_cast<const u32x4*>(wrow + k / 2 + 16 * g);
      __builtin_memcpy(&r.scale, srow + k / 16 + 4 * (g >> 1), 4);
    } else {                       // the row's last, partial step: 16 elements at a time
      r.code = u32x4{0, 0, 0, 0};
      r.scale = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (k + 32 * g + 16 * h < a.K) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(wrow + k / 2 + 16 * g + 8 * h);
          r.code[2 * h] = v[0];
          r.code[2 * h + 1] = v[1];
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t grp = k / 16 + 4 * (g >> 1) + j;
        if (grp < a.K / 16) r.scale |= (uint32_t)srow[grp] << (8 * j);
      }
    }
    return r;
  };

  f32x4 acc[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) acc[t] = f32x4{0, 0, 0, 0};

  // this lane's activation row of each tile; rows 0-7 of the MFMA take the
  // lower lane groups' k, rows 8-15 the upper ones'
  const bool mine = (c >> 3) == (g >> 1);
  const uint16_t* xrow[CT];
  bool on[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int m = 8 * t + (c & 7);
    on[t] = mine && m < a.M;
    xrow[t] = a.x + (int64_t)(m < a.M ? m : 0) * a.ldx;
  }

  GemvStep cur;
  if (wave < nsteps) cur = load(wave);
  for (int s = wave; s < nsteps; s += waves) {
    GemvStep next = cur;
    if (s + waves < nsteps) next = load(s + waves);
    const int64_t k = (int64_t)s * kGvStep;
    // both halves of groups (0 | 4), (2 | 6), (1 | 5), (3 | 7) side by side
    const auto p = __builtin_amdgcn_permlane16_swap(cur.code[0], cur.code[1], false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(cur.code[2], cur.code[3], false, false);
    const uint32_t codes[4] = {p[0], p[1], q[0], q[1]};
    constexpr int kGrp[4] = {0, 2, 1, 3};
    const f32x2_t slo = __builtin_amdgcn_cvt_pk_f32_fp8((int)cur.scale, false);
    const f32x2_t shi = __builtin_amdgcn_cvt_pk_f32_fp8((int)cur.scale, true);
    const float sc[4] = {slo[0], shi[0], slo[1], shi[1]};        // groups 0, 2, 1, 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8 w = codes_bf16(codes[i]);
      const int64_t kx = k + 16 * (kGrp[i] + 4 * (g >> 1)) + 8 * (g & 1);
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        u32x4 xv = {0, 0, 0, 0};
        if (on[t] && kx < a.K) xv = *reinterpret_cast<const u32x4*>(xrow[t] + kx);
        const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, xv), w, f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(d[r], sc[i], acc[t][r]);
      }
    }
    cur = next;
  }

  // rows 8-15 hold the same activation rows' other groups; then the waves'
  // sums in wave order
  __shared__ float red[kGvWaves][8 * CT][kGvRows];
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v = acc[t][r] + __shfl_xor(acc[t][r], 32, 64);
      if (g < 2) red[wave][8 * t + 4 * g + r][c] = v;
    }
  __syncthreads();
  const float ts = *a.wts;
  for (int i = threadIdx.x; i < a.M * kGvRows; i += blockDim.x) {
    const int m = i / kGvRows, col = i % kGvRows;
    const int64_t nn = n0 + col;
    if (nn >= a.N) continue;
    float v = red[0][m][col];
    for (int w = 1; w < waves; ++w) v += red[w][m][col];
    v *= ts;
    if (a.bias) v += __uint_as_float((uint32_t)a.bias[nn] << 16);
    if (a.gelu) v = gelu_tanh(v);
    if (a.out_f32)
      static_cast<float*>(a.y)[m * a.ldy + nn] = v;
    else
      static_cast<uint16_t*>(a.y)[m * a.ldy + nn] = (uint16_t)bf16_pack(v, v);
  }
}

}  // namespace

hipError_t launch_qgemv(const uint16_t* x, int64_t ldx, const uint8_t* w_q, const uint8_t* w_s,
                        const float* w_ts, int64_t M, int64_t N, int64_t K, const GemmOut& o,
                        hipStream_t stream) {
  const GemvArgs a = {x, ldx, w_q, w_s, w_ts, (int)M, N, K, o.bias, o.y, o.ldy, o.out_f32, o.gelu};
  const int64_t nsteps = (K + kGvStep - 1) / kGvStep;
  const int waves = (int)(nsteps < kGvWaves ? nsteps : kGvWaves);
  const dim3 grid((unsigned)((N + kGvRows - 1) / kGvRows)), block(64 * waves);
  const Gate gt = current_gate();
  if (M <= 8)
    hipLaunchKernelGGL(qgemv_kernel<1>, grid, block, 0, stream, a, gt);
  else if (M <= 16)
    hipLaunchKernelGGL(qgemv_kernel<2>, grid, block, 0, stream, a, gt);
  else
    hipLaunchKernelGGL(qgemv_kernel<4>, grid, block, 0, stream, a, gt);
  return hipGetLastError();
}

}  // namespace qact
