// The NVFP4 key/value cache: kv4_append encodes new tokens into its pages,
// kv4_read decodes tokens back to bf16.  The format is act_quant's NVFP4 with
// a given tensor scale (6Bit-Diffusion, abstract: E2M1 elements, one E4M3
// scale per 16), the groups along a head's elements, so that a token never
// touches another token's bytes.
//
// Both stream: 2 + 9/16 bytes per element.  A lane holds a group of 16 elements
// (32 bytes of a token), so that its scale needs no other lane and finding the
// slot (a chain of a table entry and three divisions) is paid for once per group.
//
// 1350 tokens, 30 heads of 64, keys and values: 5.9 us to append and as much to read
// back with their launches, 13 MB each; of single tokens the launch is the time.
#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

namespace {

// The slot of stream b's token at position `pos`: its row in a
// [pages][H][page] array for this head, or -1 when the table names no page.
__device__ __forceinline__ int64_t kv4_slot(const Kv4Cache& c, int64_t b, int64_t pos, int head) {
  if (pos < 0 || pos >= c.max_pages << c.page_log2) return -1;
  const int64_t p = c.table[b * c.max_pages + (pos >> c.page_log2)];
  if (p < 0 || p >= c.pages) return -1;
  return ((p * c.H + head) << c.page_log2) + (pos & ((1 << c.page_log2) - 1));
}

struct Kv4Group {
  int64_t row;      // b * T + t
  uint32_t b, t;
  int head, group;  // head and group of 16 elements within it
};

// Group i of the call's (below 2^30): all its groups, token by token.
__device__ __forceinline__ Kv4Group kv4_group(const Kv4Cache& c, uint32_t T, uint32_t i) {
  const uint32_t per = c.D / 16, row = i / (c.H * per), j = i - row * (c.H * per);
  Kv4Group r;
  r.row = row;
  r.head = (int)(j / per);
  r.group = (int)(j - r.head * per);
  r.b = row / T;
  r.t = row - r.b * T;
  return r;
}

// blockIdx.y: keys, values
__global__ void __launch_bounds__(256)
kv4_append_kernel(Kv4Cache c, const uint16_t* __restrict__ k, int64_t ldk,
                  const uint16_t* __restrict__ v, int64_t ldv, uint32_t T, uint32_t groups,
                  const int32_t* __restrict__ start, const int32_t* __restrict__ count, Gate gate) {
  if (gated_off(gate)) return;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= groups) return;
  const bool val = blockIdx.y != 0;
  const Kv4Group g = kv4_group(c, T, i);
  if (count && (int)g.t >= count[g.b]) return;
  // (the values on their way while the table is asked for the slot)
  const uint16_t* src = (val ? v + g.row * ldv : k + g.row * ldk) + (int64_t)g.head * c.D + 16 * g.group;
  const u32x4 w0 = reinterpret_cast<const u32x4*>(src)[0], w1 = reinterpret_cast<const u32x4*>(src)[1];
  const float s_t = val ? *c.v_ts : *c.k_ts;
  const int64_t slot = kv4_slot(c, g.b, (int64_t)start[g.b] + g.t, g.head);
  if (slot < 0) return;
  const uint32_t most = fold_max(abs_max8_pk(w1, abs_max8_pk(w0, u16x2{0, 0})));
  const uint32_t enc = e4m3_encode(__uint_as_float(most << 16) * recip0(6.0f * s_t));
  const float inv = recip0(e4m3_decode(enc) * s_t);
  *reinterpret_cast<u32x2*>((val ? c.v_q : c.k_q) + slot * (c.D / 2) + 8 * g.group) =
      u32x2{e2m1_pack8(w0, inv), e2m1_pack8(w1, inv)};
  (val ? c.v_s : c.k_s)[slot * (c.D / 16) + g.group] = (uint8_t)enc;
}

__global__ void __launch_bounds__(256)
kv4_read_kernel(Kv4Cache c, uint16_t* __restrict__ k, int64_t ldk, uint16_t* __restrict__ v,
                int64_t ldv, uint32_t T, uint32_t groups, const int32_t* __restrict__ start,
                const int32_t* __restrict__ count, Gate gate) {
  if (gated_off(gate)) return;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= groups) return;
  const bool val = blockIdx.y != 0;
  const Kv4Group g = kv4_group(c, T, i);
  if (count && (int)g.t >= count[g.b]) return;
  const int64_t slot = kv4_slot(c, g.b, (int64_t)start[g.b] + g.t, g.head);
  if (slot < 0) return;
  const u32x2 codes = *reinterpret_cast<const u32x2*>((val ? c.v_q : c.k_q) + slot * (c.D / 2) +
                                                      8 * g.group);
  const uint32_t sb = (val ? c.v_s : c.k_s)[slot * (c.D / 16) + g.group];
  // element x group scale is exact in float32; one rounding by the tensor
  // scale, one to bf16
  const float s = __builtin_amdgcn_cvt_f32_fp8((int)sb, 0);
  const float ts = val ? *c.v_ts : *c.k_ts;
  uint16_t* dst = (val ? v + g.row * ldv : k + g.row * ldk) + (int64_t)g.head * c.D + 16 * g.group;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2_t e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[h], 1.0f, 0);
    const f32x2_t e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[h], 1.0f, 1);
    const f32x2_t e2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[h], 1.0f, 2);
    const f32x2_t e3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[h], 1.0f, 3);
    reinterpret_cast<u32x4*>(dst)[h] =
        u32x4{bf16_pack(e0[0] * s * ts, e0[1] * s * ts), bf16_pack(e1[0] * s * ts, e1[1] * s * ts),
              bf16_pack(e2[0] * s * ts, e2[1] * s * ts), bf16_pack(e3[0] * s * ts, e3[1] * s * ts)};
  }
}

// The kept tokens of a stream: a workgroup takes one key head's keys or values,
// `cols` groups of 16 elements of every token, a group per lane and turn, and
// holds them all in registers before it writes the first, so that sources and
// places may be the same slots in any order.
constexpr int kKeepTurns = 8;

__global__ void __launch_bounds__(256)
kv4_keep_kernel(Kv4Cache c, int T, int cols, const int32_t* __restrict__ start,
                const int32_t* __restrict__ path, const int32_t* __restrict__ count, Gate gate) {
  if (gated_off(gate)) return;
  const int64_t b = blockIdx.x / (uint32_t)c.H;
  const int head = (int)(blockIdx.x - (uint32_t)b * c.H);
  const bool val = blockIdx.z != 0;
  uint8_t* const q = val ? c.v_q : c.k_q;
  uint8_t* const s = val ? c.v_s : c.k_s;
  const int n = count ? min(count[b], T) : T;
  const int64_t first = start[b];
  const int col0 = blockIdx.y * cols, width = min(cols, c.D / 16 - col0);
  u32x2 w[kKeepTurns];
  uint32_t sc[kKeepTurns];
  int64_t to[kKeepTurns];
#pragma unroll
  for (int u = 0; u < kKeepTurns; ++u) {
    const int x = u * 256 + threadIdx.x, i = x / width, col = col0 + (x - i * width);
    w[u] = u32x2{0, 0};
    sc[u] = 0;
    to[u] = -1;
    if (i >= n) continue;
    const int64_t src = kv4_slot(c, b, first + path[b * T + i], head);
    const int64_t dst = kv4_slot(c, b, first + i, head);
    if (src < 0 || dst < 0 || src == dst) continue;
    w[u] = *reinterpret_cast<const u32x2*>(q + src * (c.D / 2) + 8 * col);
    sc[u] = s[src * (c.D / 16) + col];
    to[u] = dst;
  }
  // (in their registers before any wave of the workgroup stores)
#pragma unroll
  for (int u = 0; u < kKeepTurns; ++u) asm volatile("" : "+v"(w[u]), "+v"(sc[u]));
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kKeepTurns; ++u) {
    if (to[u] < 0) continue;
    const int x = u * 256 + threadIdx.x, col = col0 + x % width;
    *reinterpret_cast<u32x2*>(q + to[u] * (c.D / 2) + 8 * col) = w[u];
    s[to[u] * (c.D / 16) + col] = (uint8_t)sc[u];
  }
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Cache& c, const uint16_t* k, int64_t ldk, const uint16_t* v,
                             int64_t ldv, int64_t B, int64_t T, const int32_t* start,
                             const int32_t* count, hipStream_t stream) {
  const uint32_t groups = (uint32_t)(B * T * c.H * (c.D / 16));       // (below 2^30)
  const dim3 grid((groups + 255) / 256, 2);
  hipLaunchKernelGGL(kv4_append_kernel, grid, dim3(256), 0, stream, c, k, ldk, v, ldv,
                     (uint32_t)T, groups,
                     start, count, current_gate());
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Cache& c, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv,
                           int64_t B, int64_t T, const int32_t* start, const int32_t* count,
                           hipStream_t stream) {
  const uint32_t groups = (uint32_t)(B * T * c.H * (c.D / 16));       // (below 2^30)
  const dim3 grid((groups + 255) / 256, 2);
  hipLaunchKernelGGL(kv4_read_kernel, grid, dim3(256), 0, stream, c, k, ldk, v, ldv,
                     (uint32_t)T, groups,
                     start, count, current_gate());
  return hipGetLastError();
}

hipError_t launch_kv4_keep(const Kv4Cache& c, int64_t B, int64_t T, const int32_t* start,
                           const int32_t* path, const int32_t* count, hipStream_t stream) {
  const int groups = c.D / 16, fit = (int)(256 * kKeepTurns / T), cols = fit < groups ? fit : groups;
  const dim3 grid((unsigned)(B * c.H), (unsigned)((groups + cols - 1) / cols), 2);
  hipLaunchKernelGGL(kv4_keep_kernel, grid, dim3(256), 0, stream, c, (int)T, cols, start, path, count,
                     current_gate());
  return hipGetLastError();
}

}  // namespace qact
