// qlinear_w8a8 of few rows, or of few outputs: a workgroup has 16 MT rows and 16 NT
// columns, and its W waves share out K, 128 elements (a line of each row) at a
// time.  Each wave moves its own lines into its own ring of S slots and reads
// them as operands (v_mfma_i32_16x16x64_i8), so no barrier stands in the loop; the
// waves' sums meet in shared memory.
//
// Few rows are bound by the weight's bytes: 1 row of 8192 against 16384 takes 26.6 us,
// 134 MB at 5.05 TB/s (a copy reaches 5.11).  With more of them the bound is what a
// compute unit can move into its shared memory, about 75 B/ns in lines of 128 bytes
// (64 rows of 1920 against 7680: 8.0 us, of 7680 against 1920: 9.3).  Straight from
// memory into the operands' registers, 16 rows x 64 bytes an instruction, it moves
// about half of that and keeps fewer bytes on their way: 64 rows of 1920 against 7680
// 9.1 us, of 7680 against 1920 13.7.  Few outputs of a long K leave compute units
// idle: K is then cut among workgroups as well and the cuts are joined.
#include "w8a8.h"

namespace qact {

namespace {

template <int MT, int NT, int W, int S>
struct Split {
  static constexpr int kRows = 16 * (MT + NT), kSlot = kRows * kSplitK, kLoads = kRows / 8;
  static constexpr int kSums = W * MT * NT * 1024;
  static constexpr int kSmem = W * S * kSlot > kSums ? W * S * kSlot : kSums;
  static_assert(kSmem <= 160 * 1024, "LDS");
};

// Four neighbouring outputs of row m from column n on, from their sums.
template <bool F32, bool GELU>
__device__ __forceinline__ void finish(i32x4 v, int m, int n, const W8Args& g, const EpiArgs& e) {
  const float rs = g.a_s[m];
  float f[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int nc = min(n + c, (int)e.N - 1);
    f[c] = __builtin_fmaf((float)v[c] * g.w_s[nc], rs,
                          e.bias ? __uint_as_float((uint32_t)e.bias[nc] << 16) : 0.0f);
    if constexpr (GELU) f[c] = gelu_tanh(f[c]);
  }
  // (four columns at any address that their type allows)
  const int64_t to = (int64_t)m * e.ldy + n;
  const bool whole = n + 4 <= (int)e.N;
  if constexpr (F32) {
    typedef __attribute__((ext_vector_type(4), aligned(4))) float Group;
    float* const y = static_cast<float*>(e.y) + to;
    if (whole) {
      *reinterpret_cast<Group*>(y) = f32x4{f[0], f[1], f[2], f[3]};
    } else {
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (n + c < (int)e.N) y[c] = f[c];
    }
  } else {
    typedef __attribute__((ext_vector_type(2), aligned(2))) uint32_t Group;
    uint16_t* const y = static_cast<uint16_t*>(e.y) + to;
    const u32x2 w = {bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3])};
    if (whole) {
      *reinterpret_cast<Group*>(y) = w;
    } else {
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (n + c < (int)e.N) y[c] = (uint16_t)(w[c / 2] >> (16 * (c & 1)));
    }
  }
}

template <int MT, int NT, int W, int S, bool F32, bool GELU>
__global__ void __launch_bounds__(64 * W)
w8a8_split_kernel(W8Args g, EpiArgs e) {
  if (gated_off(g.gate)) return;
  using P = Split<MT, NT, W, S>;
  __shared__ __align__(16) uint8_t smem[P::kSmem];
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Each of the 8 chips of compute units (workgroups are dealt to them in turn) takes
  // neighbouring tiles, rows fastest, so that those of the same weight rows read
  // them through one cache (256 rows of 7680 against 1920: 15.3 -> 13 us), and each
  // begins an eighth of its tiles further on than the one before, so that they do not
  // all read places a power of two apart (1 row of 8192 against 16384: 31.8 -> 26.6).
  const int tiles = g.mt * g.nt, per = (tiles + 7) / 8, chip = blockIdx.x & 7;
  const int tile = chip * per + ((int)(blockIdx.x >> 3) + chip * (per / 8)) % per;
  if (tile >= tiles) return;
  const int m0 = tile % g.mt * (16 * MT), n0 = tile / g.mt * (16 * NT);
  const uint32_t K = (uint32_t)g.K;
  const __amdgpu_buffer_rsrc_t ra = operand(g.a, m0, e.M, 16 * MT, g.K);
  const __amdgpu_buffer_rsrc_t rw = operand(g.w, n0, e.N, 16 * NT, g.K);
  uint8_t* const ring = smem + wave * S * P::kSlot;
  // this workgroup's lines of K
  const int first = (int)blockIdx.y * g.split_chunks;
  const int last = min(first + g.split_chunks, (int)((K + kSplitK - 1) / kSplitK));
  // 16-byte chunk c (of 8) of row r lies at slot c ^ (r / 2) % 8, so that the 16 rows
  // of an operand spread over the banks; an instruction moves 8 rows
  const int r8 = lane >> 3;
  const auto load = [&](int i, int c) {           // (lines from `last` on: zeros)
    uint8_t* const to = ring + i * P::kSlot;
#pragma unroll
    for (int d = 0; d < P::kLoads; ++d) {
      const int row = 8 * d + r8;
      const uint32_t k = (uint32_t)c * kSplitK + 16u * (uint32_t)((lane & 7) ^ ((row >> 1) & 7));
      const bool weight = d >= 2 * MT;
      const uint32_t at = c < last && k < K ? (uint32_t)(weight ? row - 16 * MT : row) * K + k : kSkip;
      if (weight)
        dma16(rw, to + d * 1024, at);
      else
        dma16(ra, to + d * 1024, at);
    }
  };
#pragma unroll
  for (int i = 0; i < S; ++i) load(i, first + wave + W * i);
  i32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  int slot = 0;
  for (int c = first + wave; c < last; c += W) {
    wait_vm<(S - 1) * P::kLoads>();
    const uint8_t* const from = ring + slot * P::kSlot;
    i32x4 a[2][MT], w[2][NT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int off = col * kSplitK + 16 * ((4 * h + quad) ^ ((col >> 1) & 7));
#pragma unroll
      for (int j = 0; j < NT; ++j) w[h][j] = *reinterpret_cast<const i32x4*>(from + (MT + j) * 16 * kSplitK + off);
#pragma unroll
      for (int i = 0; i < MT; ++i) a[h][i] = *reinterpret_cast<const i32x4*>(from + i * 16 * kSplitK + off);
    }
    // the operands are in their registers before their slot is filled again
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(w[h][j]));
#pragma unroll
      for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(a[h][i]));
    }
    load(slot, c + W * S);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][j], a[h][i], acc[i][j], 0, 0, 0);
    slot = slot == S - 1 ? 0 : slot + 1;
  }
  wait_vm<0>();           // (what was moved in behind the last line, too)
  __syncthreads();
  i32x4* const sums = reinterpret_cast<i32x4*>(smem);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[(wave * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // four neighbouring columns of a row per thread
  for (int x = threadIdx.x; x < MT * NT * 64; x += 64 * W) {
    const int t = x >> 6, l = x & 63, i = t / NT, j = t % NT;
    const int m = m0 + 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m >= (int)e.M || n >= (int)e.N) continue;
    i32x4 v = sums[x];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[w * MT * NT * 64 + x];
    if (g.splits == 1) {
      finish<F32, GELU>(v, m, n, g, e);
    } else {
      const int64_t wide = (e.N + 3) / 4;
      reinterpret_cast<i32x4*>(g.part)[((int64_t)blockIdx.y * e.M + m) * wide + n / 4] = v;
    }
  }
}

// The sums of the cuts of K, joined (whole numbers: in any order the same).
template <bool F32, bool GELU>
__global__ void __launch_bounds__(256)
w8a8_join_kernel(W8Args g, EpiArgs e) {
  if (gated_off(g.gate)) return;
  const uint32_t wide = (uint32_t)((e.N + 3) / 4), at = blockIdx.x * 256 + threadIdx.x;    // (below 2^31)
  if (at >= (uint32_t)e.M * wide) return;
  const int m = (int)(at / wide), n = 4 * (int)(at % wide);
  const i32x4* const part = reinterpret_cast<const i32x4*>(g.part) + at;
  i32x4 v = part[0];
  for (int s = 1; s < g.splits; ++s) v += part[(int64_t)s * e.M * wide];
  finish<F32, GELU>(v, m, n, g, e);
}

template <bool F32, bool GELU>
hipError_t launch_one(int shape, const dim3& grid, const W8Args& g, const EpiArgs& e, hipStream_t st) {
  int i = 0;
#define QACT_W8_LAUNCH(MT, NT, W, S) \
  if (shape == i++) hipLaunchKernelGGL((w8a8_split_kernel<MT, NT, W, S, F32, GELU>), grid, dim3(64 * W), 0, st, g, e);
  QACT_W8_SPLITS(QACT_W8_LAUNCH)
#undef QACT_W8_LAUNCH
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || g.splits == 1) return err;
  const int64_t n = e.M * ((e.N + 3) / 4);
  hipLaunchKernelGGL((w8a8_join_kernel<F32, GELU>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, g, e);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w8a8_split(int shape, int splits, const W8Args& g0, const EpiArgs& e, hipStream_t st) {
  W8Args g = g0;
  const SplitShape& s = kSplitShapes[shape];
  g.mt = (int)((e.M + 16 * s.mt - 1) / (16 * s.mt));
  g.nt = (int)((e.N + 16 * s.nt - 1) / (16 * s.nt));
  const int chunks = (int)((g.K + kSplitK - 1) / kSplitK);
  g.split_chunks = (chunks + splits - 1) / splits;
  g.splits = (chunks + g.split_chunks - 1) / g.split_chunks;
  const dim3 grid((unsigned)(8 * ((g.mt * g.nt + 7) / 8)), (unsigned)g.splits);
  if (e.out_f32)
    return e.gelu ? launch_one<true, true>(shape, grid, g, e, st) : launch_one<true, false>(shape, grid, g, e, st);
  return e.gelu ? launch_one<false, true>(shape, grid, g, e, st) : launch_one<false, false>(shape, grid, g, e, st);
}

}  // namespace qact
