// The NVFP4 key/value cache: kv4_append encodes new tokens into its pages,
// kv4_read decodes tokens back to bf16.  The format is act_quant's NVFP4 with
// a given tensor scale (6Bit-Diffusion, abstract: E2M1 elements, one E4M3
// scale per 16), the groups along a head's elements, so that a token never
// touches another token's bytes.
//
// Both stream: 2 + 9/16 bytes per element.  A lane holds 8 elements (one
// 16-byte vector); the two halves of a group sit in neighbouring lanes.  The
// page table is one cached load per lane.
#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

namespace {

// The slot of stream b's token at position `pos`: its row in a
// [pages][H][page] array for head 0, or -1 when the table names no page.
__device__ __forceinline__ int64_t kv4_slot(const Kv4Cache& c, int64_t b, int64_t pos) {
  if (pos < 0 || pos >= c.max_pages << c.page_log2) return -1;
  const int64_t p = c.table[b * c.max_pages + (pos >> c.page_log2)];
  if (p < 0 || p >= c.pages) return -1;
  return ((p * c.H) << c.page_log2) + (pos & ((1 << c.page_log2) - 1));
}

struct Kv4Token {
  int64_t row;      // b * T + t
  int64_t slot;     // cache row of this head, -1: none
  int head, vec;    // head and 8-element vector within it
};

__device__ __forceinline__ Kv4Token kv4_token(const Kv4Cache& c, int64_t T, const int32_t* start,
                                              const int32_t* count, int64_t i) {
  const int vpr = c.H * (c.D / 8);
  Kv4Token r;
  r.row = i / vpr;
  const int j = (int)(i - r.row * vpr);
  r.head = j / (c.D / 8);
  r.vec = j - r.head * (c.D / 8);
  const int64_t b = r.row / T, t = r.row - b * T;
  r.slot = -1;
  if (!count || t < count[b]) {
    r.slot = kv4_slot(c, b, (int64_t)start[b] + t);
    if (r.slot >= 0) r.slot += (int64_t)r.head << c.page_log2;
  }
  return r;
}

// blockIdx.y: keys, values
__global__ void __launch_bounds__(256)
kv4_append_kernel(Kv4Cache c, const uint16_t* __restrict__ k, int64_t ldk,
                  const uint16_t* __restrict__ v, int64_t ldv, int64_t T, int64_t nvec,
                  const int32_t* __restrict__ start, const int32_t* __restrict__ count, Gate gate) {
  if (gated_off(gate)) return;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool val = blockIdx.y != 0;
  Kv4Token tk;
  tk.slot = -1;
  u32x4 w = {0, 0, 0, 0};
  if (i < nvec) {
    tk = kv4_token(c, T, start, count, i);
    if (tk.slot >= 0) {
      const uint16_t* src = (val ? v + tk.row * ldv : k + tk.row * ldk) + tk.head * c.D + 8 * tk.vec;
      w = *reinterpret_cast<const u32x4*>(src);
    }
  }
  const float s_t = val ? *c.v_ts : *c.k_ts;
  const float g = recip0(6.0f * s_t);
  const uint32_t own = fold_max(abs_max8_pk(w, u16x2{0, 0}));
  // the other half of the group: quad_perm [1, 0, 3, 2] swaps lanes 2j, 2j+1
  const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)own, 0xB1, 0xF, 0xF, false);
  const uint32_t enc = e4m3_encode(__uint_as_float(max(own, other) << 16) * g);
  const uint32_t codes = e2m1_pack8(w, recip0(e4m3_decode(enc) * s_t));
  if (tk.slot >= 0) {
    uint8_t* q = (val ? c.v_q : c.k_q) + tk.slot * (c.D / 2) + 4 * tk.vec;
    *reinterpret_cast<uint32_t*>(q) = codes;
    if ((tk.vec & 1) == 0) (val ? c.v_s : c.k_s)[tk.slot * (c.D / 16) + tk.vec / 2] = (uint8_t)enc;
  }
}

__global__ void __launch_bounds__(256)
kv4_read_kernel(Kv4Cache c, uint16_t* __restrict__ k, int64_t ldk, uint16_t* __restrict__ v,
                int64_t ldv, int64_t T, int64_t nvec, const int32_t* __restrict__ start,
                const int32_t* __restrict__ count, Gate gate) {
  if (gated_off(gate)) return;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= nvec) return;
  const bool val = blockIdx.y != 0;
  const Kv4Token tk = kv4_token(c, T, start, count, i);
  if (tk.slot < 0) return;
  const uint32_t codes = *reinterpret_cast<const uint32_t*>((val ? c.v_q : c.k_q) +
                                                            tk.slot * (c.D / 2) + 4 * tk.vec);
  const uint32_t sb = (val ? c.v_s : c.k_s)[tk.slot * (c.D / 16) + tk.vec / 2];
  // element x group scale is exact in float32; one rounding by the tensor
  // scale, one to bf16
  const float s = __builtin_amdgcn_cvt_f32_fp8((int)sb, 0);
  const float ts = val ? *c.v_ts : *c.k_ts;
  u32x4 o;
#define QACT_KV4_PAIR(i)                                                               \
  {                                                                                    \
    const f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, i);        \
    o[i] = bf16_pack(e[0] * s * ts, e[1] * s * ts);                                    \
  }
  QACT_KV4_PAIR(0)
  QACT_KV4_PAIR(1)
  QACT_KV4_PAIR(2)
  QACT_KV4_PAIR(3)
#undef QACT_KV4_PAIR
  uint16_t* dst = (val ? v + tk.row * ldv : k + tk.row * ldk) + tk.head * c.D + 8 * tk.vec;
  *reinterpret_cast<u32x4*>(dst) = o;
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Cache& c, const uint16_t* k, int64_t ldk, const uint16_t* v,
                             int64_t ldv, int64_t B, int64_t T, const int32_t* start,
                             const int32_t* count, hipStream_t stream) {
  const int64_t nvec = B * T * c.H * (c.D / 8);
  const dim3 grid((unsigned)((nvec + 255) / 256), 2);
  hipLaunchKernelGGL(kv4_append_kernel, grid, dim3(256), 0, stream, c, k, ldk, v, ldv, T, nvec,
                     start, count, current_gate());
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Cache& c, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv,
                           int64_t B, int64_t T, const int32_t* start, const int32_t* count,
                           hipStream_t stream) {
  const int64_t nvec = B * T * c.H * (c.D / 8);
  const dim3 grid((unsigned)((nvec + 255) / 256), 2);
  hipLaunchKernelGGL(kv4_read_kernel, grid, dim3(256), 0, stream, c, k, ldk, v, ldv, T, nvec,
                     start, count, current_gate());
  return hipGetLastError();
}

}  // namespace qact
