// qlinear_bf16: the linear of a few bf16 rows (M <= 32) against an NVFP4
// weight, for the rows that are not worth quantizing: a conditioning vector's
// modulation, one token of each stream (6Bit-Diffusion, Table 2: 4-bit
// weights).
//
//   y[m][n] = s_Tw sum_g s[n][g] sum_{j<16} x[m][16 g + j] c[n][16 g + j]
//
// The weight is read once, 9/16 byte per element, and everything else is
// small, so the bound is the memory rate, and the arithmetic per code has to
// stay below it.  The inner sums run on bf16 MFMA (exact products, float32
// sums) in two ways.
//
// At most 8 rows: on the bare codes, which are exact in bf16 (half an
// instruction per code); the group's E4M3 scale is applied in float32 to the
// sums.  One 16x16x32 MFMA holds two scale groups of 16 weight rows: its 16
// activation rows are the same 8 rows twice, rows 0-7 with x in the first
// group's half of k and zeros in the second's, rows 8-15 the other way round.
// The result holds each group's sum apart, and one FMA (at most 2 rows) to
// four scale 512 codes.
//
// More rows: on code times scale, which is exact in bf16 too; that takes 2
// VALU instructions per code and lane, whatever the rows, but the MFMA's 16
// rows are 16 rows of x, so that these are read once and not twice.
//
// A workgroup has 16, 32 or 64 weight rows, and its waves split K, 256
// elements at a time: a line of codes.  More weight rows read the activations
// less often (32 rows of 8192 against 16384 weight rows: 83, 51 and 35 us;
// 1 row: 26.7, 22.5 and 20.8 us) but leave fewer workgroups (16 rows of 7680
// against 1920: 12.8, 15.8 and 23.8 us) or full rounds of them (2 rows of 4096
// against 12288: 14.8, 14.5 and 13.2 us, against 24576: 23.4, 19.6 and 24.4).
//
// Against few weight rows the activations are what a compute unit reads most
// of, so their rows are then shared out as well, 8 or 16 to a workgroup (16 rows
// of 7680 against 1920: 12.9 us whole, 10.5 in eights; 32 rows of 4096 against
// 1024: 13.2 and 7.3), as long as all workgroups run at once (16 rows of 4096
// against 4096: 9.0 and 12.4 us).
//
// 1 row, 8192 to 16384: 20.8 us, 3.6 TB/s of the 5.1 that a copy reaches, with
// the launch.
#include "qact_device.h"
#include "qact_internal.h"
#include "qgemm_common.h"

namespace qact {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kGvRows = 16;        // weight rows of an MFMA
constexpr int kGvStep = 256;       // elements of a row per step: a line of codes
constexpr int kGvWaves = 8;        // waves of a workgroup, at most
constexpr int64_t kGvPlaces = 256; // compute units

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

// The same times their group's scale: exact, too (2 and 4 significant bits,
// powers 2^-10 to 2^11).
__device__ __forceinline__ bf16x8 scaled_bf16(uint32_t c, float s) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
  const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
  const f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
  return __builtin_bit_cast(bf16x8, u32x4{bf16_pack(a[0] * s, a[1] * s), bf16_pack(b[0] * s, b[1] * s),
                                          bf16_pack(d[0] * s, d[1] * s), bf16_pack(e[0] * s, e[1] * s)});
}

// What lanes without a share of the activations read.
__device__ const u32x4 kGvZeros[kGvStep / 8] = {};

// The waves' sums of `rows` activation rows by `cols` weight rows, joined in
// wave order, and the epilogue.
template <int ROWS, int COLS>
__device__ __forceinline__ void finish(const GemvArgs& a, const float (*red)[ROWS][COLS], int waves,
                                       int64_t n0) {
  __syncthreads();
  const float ts = *a.wts;
  for (int i = threadIdx.x; i < a.M * COLS; i += blockDim.x) {
    const int m = i / COLS, col = i % COLS;
    const int64_t n = n0 + col;
    if (n >= a.N) continue;
    float v = red[0][m][col];
    for (int w = 1; w < waves; ++w) v += red[w][m][col];
    v *= ts;
    if (a.bias) v += __uint_as_float((uint32_t)a.bias[n] << 16);
    if (a.gelu) v = gelu_tanh(v);
    if (a.out_f32)
      static_cast<float*>(a.y)[m * a.ldy + n] = v;
    else
      static_cast<uint16_t*>(a.y)[m * a.ldy + n] = (uint16_t)bf16_pack(v, v);
  }
}

// The workgroup's rows of the call's: `most` from blockIdx.y.
__device__ __forceinline__ void own_rows(GemvArgs& a, int most) {
  const int64_t first = most * (int64_t)blockIdx.y;
  a.x += first * a.ldx;
  a.y = static_cast<char*>(a.y) + first * a.ldy * (a.out_f32 ? 4 : 2);
  a.M = min(most, a.M - (int)first);
}

// At most 8 activation rows.  A lane reads pieces of 16 bytes (two groups) of a
// weight row, lane groups 0 and 1 the even and odd ones of the step's first
// half, 2 and 3 of its second.  Swapping the odd lane groups' first register
// with the even ones' second puts both halves of a group side by side, as the
// MFMA wants them.  NR: results that a lane uses of each MFMA (row m
// is row 4 (m % 2) + m / 2 of the MFMA, so that two rows need one result of each
// lane); RT: tiles of 16 weight rows; W: waves, at most, which split K.
template <int NR, int RT, int W>
__global__ void __launch_bounds__(64 * W)
qgemv_kernel(GemvArgs a, Gate gate) {
  if (gated_off(gate)) return;
  own_rows(a, 8);
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4, up = g >> 1;
  const int64_t n0 = (int64_t)blockIdx.x * (kGvRows * RT);
  const int nsteps = (int)((a.K + kGvStep - 1) / kGvStep), whole = (int)(a.K / kGvStep);

  const uint8_t *code[RT], *scale[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t n = min(n0 + kGvRows * t + c, a.N - 1);
    code[t] = a.wq + n * (a.K / 2) + 16 * (g & 1) + 64 * up;
    scale[t] = a.ws + n * (a.K / 16) + 8 * up;
  }
  // this lane's activation row; rows 0-7 of the MFMA take the lower lane
  // groups' k, rows 8-15 the upper ones'
  const int m = min(2 * (c & 3) + ((c >> 2) & 1), a.M - 1);
  const bool mine = (c >> 3) == up;
  const uint16_t* const x = a.x + (int64_t)m * a.ldx + 128 * up + 8 * (g & 1);

  struct Weights {
    u32x4 code[RT][2];
    u32x2 scale[RT];
  };
  auto weights = [&](int s) {
    Weights r;
    const int64_t k = (int64_t)s * kGvStep;
    if (s < whole) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        r.code[t][0] = *reinterpret_cast<const u32x4*>(code[t] + k / 2);
        r.code[t][1] = *reinterpret_cast<const u32x4*>(code[t] + k / 2 + 32);
        __builtin_memcpy(&r.scale[t], scale[t] + k / 16, 8);
      }
    } else {                       // the row's last, partial step: 16 elements at a time
      const int64_t left = a.K - k - 128 * up;       // of this lane's 128
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          r.code[t][u] = u32x4{0, 0, 0, 0};
          r.scale[t][u] = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (64 * u + 32 * (g & 1) + 16 * h < left) {
              const u32x2 v = *reinterpret_cast<const u32x2*>(code[t] + k / 2 + 32 * u + 8 * h);
              r.code[t][u][2 * h] = v[0];
              r.code[t][u][2 * h + 1] = v[1];
            }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (16 * (4 * u + j) < left)
              r.scale[t][u] |= (uint32_t)scale[t][k / 16 + 4 * u + j] << (8 * j);
        }
    }
    return r;
  };
  // Result i of 8 holds the lane's groups 4 (i / 4) + kGrp[i % 4]; four results'
  // activations are read while those of the four before are used.
  constexpr int kGrp[4] = {0, 2, 1, 3};
  struct Acts {
    u32x4 v[4];
  };
  auto acts = [&](int s, int u) {
    Acts r;
    const int64_t k = (int64_t)s * kGvStep;
    const uint16_t* p = mine ? x + k : reinterpret_cast<const uint16_t*>(kGvZeros);
    const int64_t left = a.K - k - 128 * up;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 64 * u + 16 * kGrp[i];
      if (s < whole) {
        r.v[i] = *reinterpret_cast<const u32x4*>(p + at);
      } else {
        r.v[i] = u32x4{0, 0, 0, 0};
        if (at < left) r.v[i] = *reinterpret_cast<const u32x4*>(p + at);
      }
    }
    return r;
  };

  float acc[RT][NR] = {};
  int s = wave;                    // (there are no more waves than steps)
  Weights cur = weights(s);
  Acts xs = acts(s, 0);
  for (; s < nsteps; s += waves) {
    const int to = s + waves < nsteps ? s + waves : s;
    const Weights next = weights(to);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Acts xn = u == 0 ? acts(s, 1) : acts(to, 0);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        // both halves of a group side by side
        const u32x4 w = cur.code[t][u];
        const auto p = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
        const auto q = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
        const uint32_t codes[4] = {p[0], p[1], q[0], q[1]};
        const f32x2_t slo = __builtin_amdgcn_cvt_pk_f32_fp8((int)cur.scale[t][u], false);
        const f32x2_t shi = __builtin_amdgcn_cvt_pk_f32_fp8((int)cur.scale[t][u], true);
        const float sc[4] = {slo[0], shi[0], slo[1], shi[1]};      // in the order of kGrp
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, xs.v[i]), codes_bf16(codes[i]), f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[t][r] = __builtin_fmaf(d[r], sc[i], acc[t][r]);
        }
      }
      xs = xn;
    }
    cur = next;
  }

  // rows 8-15 hold the same activation rows' other groups
  __shared__ float red[W][8][kGvRows * RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float v = acc[t][r] + __shfl_xor(acc[t][r], 32, 64);
      if (g < 2) red[wave][2 * r + g][kGvRows * t + c] = v;
    }
  finish<8, kGvRows * RT>(a, red, waves, n0);
}

// More rows: MT tiles of 16 activation rows, RT of 16 weight rows.
template <int MT, int RT, int W>
__global__ void __launch_bounds__(64 * W)
qgemv_wide_kernel(GemvArgs a, Gate gate) {
  if (gated_off(gate)) return;
  own_rows(a, 16 * MT);
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (kGvRows * RT);
  const int nsteps = (int)((a.K + kGvStep - 1) / kGvStep), whole = (int)(a.K / kGvStep);

  // A lane loads pieces g and g + 4 (32 elements each) of a step's 8; lane
  // groups then exchange, so that MFMA p holds piece p, group g its elements
  // 8 g .. + 7.  (The activations are then read 64 bytes of a row at a time; with
  // a lane's own pieces, 16 bytes of each of 64 lines, that took most of the time.)
  const uint8_t *code[RT], *scale[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t n = min(n0 + kGvRows * t + c, a.N - 1);
    code[t] = a.wq + n * (a.K / 2) + 16 * g;
    scale[t] = a.ws + n * (a.K / 16);
  }
  const uint16_t* x[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
    x[j] = a.x + (int64_t)min(16 * j + c, a.M - 1) * a.ldx + 8 * g;

  struct Weights {
    u32x4 code[RT][2], scale[RT];
  };
  auto weights = [&](int s) {
    Weights r;
    const int64_t k = (int64_t)s * kGvStep;
    if (s < whole) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        r.code[t][0] = *reinterpret_cast<const u32x4*>(code[t] + k / 2);
        r.code[t][1] = *reinterpret_cast<const u32x4*>(code[t] + k / 2 + 64);
        __builtin_memcpy(&r.scale[t], scale[t] + k / 16, 16);
      }
    } else {                       // the row's last, partial step: 16 elements at a time
      const int64_t left = a.K - k;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        r.code[t][0] = r.code[t][1] = r.scale[t] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (128 * (h / 2) + 32 * g + 16 * (h % 2) < left) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(code[t] + k / 2 + 64 * (h / 2) + 8 * (h % 2));
            r.code[t][h / 2][2 * (h % 2)] = v[0];
            r.code[t][h / 2][2 * (h % 2) + 1] = v[1];
          }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (16 * j < left) r.scale[t][j / 4] |= (uint32_t)scale[t][k / 16 + j] << (8 * (j % 4));
      }
    }
    return r;
  };
  struct Acts {
    u32x4 v[4][MT];
  };
  auto acts = [&](int s, int u) {
    Acts r;
    const int64_t k = (int64_t)s * kGvStep, left = a.K - k - 8 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int at = 128 * u + 32 * i;
        if (s < whole) {
          r.v[i][j] = *reinterpret_cast<const u32x4*>(x[j] + k + at);
        } else {
          r.v[i][j] = u32x4{0, 0, 0, 0};
          if (at < left) r.v[i][j] = *reinterpret_cast<const u32x4*>(x[j] + k + at);
        }
      }
    return r;
  };

  f32x4 acc[RT][MT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[t][j] = f32x4{0, 0, 0, 0};
  int s = wave;                    // (there are no more waves than steps)
  Weights cur = weights(s);
  Acts xs = acts(s, 0);
  for (; s < nsteps; s += waves) {
    const int to = s + waves < nsteps ? s + waves : s;
    const Weights next = weights(to);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Acts xn = u == 0 ? acts(s, 1) : acts(to, 0);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const u32x4 w = cur.code[t][u];
        const auto e0 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto e1 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        const auto p0 = __builtin_amdgcn_permlane16_swap(e0[0], e1[0], false, false);
        const auto p1 = __builtin_amdgcn_permlane16_swap(e0[1], e1[1], false, false);
        const uint32_t codes[4] = {p0[0], p0[1], p1[0], p1[1]};
        // group 2 p + g / 2 of piece p
        const uint32_t s0 = cur.scale[t][2 * u] >> (8 * (g >> 1));
        const uint32_t s1 = cur.scale[t][2 * u + 1] >> (8 * (g >> 1));
        const float sc[4] = {__builtin_amdgcn_cvt_f32_fp8((int)s0, 0), __builtin_amdgcn_cvt_f32_fp8((int)s0, 2),
                             __builtin_amdgcn_cvt_f32_fp8((int)s1, 0), __builtin_amdgcn_cvt_f32_fp8((int)s1, 2)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 wv = scaled_bf16(codes[i], sc[i]);
#pragma unroll
          for (int j = 0; j < MT; ++j)
            acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, xs.v[i][j]), wv, acc[t][j], 0, 0, 0);
        }
      }
      xs = xn;
    }
    cur = next;
  }

  __shared__ float red[W][16 * MT][kGvRows * RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[wave][16 * j + 4 * g + r][kGvRows * t + c] = acc[t][j][r];
  finish<16 * MT, kGvRows * RT>(a, red, waves, n0);
}

template <int RT>
hipError_t launch(const GemvArgs& a, hipStream_t stream) {
  constexpr int W = kGvWaves;
  const int64_t nsteps = (a.K + kGvStep - 1) / kGvStep;
  const int64_t tiles = (a.N + kGvRows * RT - 1) / (kGvRows * RT);
  // activation rows of a workgroup: 8, 16 or 32, the fewest that leave one
  // workgroup for each compute unit or make all of them one
  int most = 8;
  while (most < a.M && tiles * ((a.M + most - 1) / most) > kGvPlaces) most *= 2;
  const dim3 grid((unsigned)tiles, (unsigned)((a.M + most - 1) / most));
  const dim3 block((unsigned)(64 * (nsteps < W ? nsteps : W)));
  const Gate gt = current_gate();
  if (a.M <= 2)
    hipLaunchKernelGGL((qgemv_kernel<1, RT, W>), grid, block, 0, stream, a, gt);
  else if (a.M <= 4)
    hipLaunchKernelGGL((qgemv_kernel<2, RT, W>), grid, block, 0, stream, a, gt);
  else if (most == 8)
    hipLaunchKernelGGL((qgemv_kernel<4, RT, W>), grid, block, 0, stream, a, gt);
  else if (most == 16)
    hipLaunchKernelGGL((qgemv_wide_kernel<1, RT, W>), grid, block, 0, stream, a, gt);
  else
    hipLaunchKernelGGL((qgemv_wide_kernel<2, RT, W>), grid, block, 0, stream, a, gt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_qgemv(const uint16_t* x, int64_t ldx, const uint8_t* w_q, const uint8_t* w_s,
                        const float* w_ts, int64_t M, int64_t N, int64_t K, const GemmOut& o,
                        hipStream_t stream) {
  const GemvArgs a = {x, ldx, w_q, w_s, w_ts, (int)M, N, K, o.bias, o.y, o.ldy, o.out_f32, o.gelu};
  // The time of the fullest compute unit in tiles of 16 weight rows: the rounds
  // of workgroups (8 waves a unit) by what a tile costs among 1, 2 or 4.
  const int64_t nsteps = (K + kGvStep - 1) / kGvStep;
  const int64_t places = kGvPlaces * kGvWaves / (nsteps < kGvWaves ? nsteps : kGvWaves);
  const auto load = [&](int64_t rt, double each) {
    const int64_t groups = (N + kGvRows * rt - 1) / (kGvRows * rt);
    return (double)((groups + places - 1) / places * rt) * each;
  };
  const double one = load(1, M <= 8 ? 1.4 : 1.5), two = load(2, M <= 8 ? 1.05 : 1.1), four = load(4, 1.0);
  if (four <= two && four <= one) return launch<4>(a, stream);
  if (two <= one) return launch<2>(a, stream);
  return launch<1>(a, stream);
}

}  // namespace qact
