// Attention of bf16 queries over an NVFP4 cache (attn_kv4) and over an
// encoder's bf16 states (attn_cross):
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale (q . k_j) - max)
//
// over the keys j that the row sees; a row that sees none gives zeros.
//
// One wave per (query row, head): the lanes hold D / 64 elements each and
// take the keys one after the other with a running maximum and sum.
#include "qact_device.h"
#include "qact_internal.h"

namespace qact {

namespace {

// Keys and values in an NVFP4 cache.
struct Kv4Source {
  Kv4Cache c;
  const int32_t* lens;
  const int32_t* q_lens;
  int causal;

  __device__ int64_t rows(int64_t b, int64_t Lq) const {
    return q_lens ? min((int64_t)q_lens[b], Lq) : Lq;
  }
  __device__ int64_t upto(int64_t b, int64_t t, int64_t nq) const {
    const int64_t n = min((int64_t)lens[b], c.max_pages << c.page_log2);
    return causal ? n - (nq - 1 - t) : n;
  }
  __device__ bool seen(int64_t b, int64_t j, int64_t& slot, int h) const {
    const int64_t p = c.table[b * c.max_pages + (j >> c.page_log2)];
    if (p < 0 || p >= c.pages) return false;
    slot = ((p * c.H + h) << c.page_log2) + (j & ((1 << c.page_log2) - 1));
    return true;
  }
  static __device__ float element(const uint8_t* q, const uint8_t* s, int64_t slot, int D, int d) {
    const uint32_t code = (q[slot * (D / 2) + d / 2] >> (4 * (d & 1))) & 15u;
    return 0.5f * (float)e2m1_twice(code) * e4m3_decode(s[slot * (D / 16) + d / 16]);
  }
  __device__ float key(int64_t, int64_t, int, int64_t slot, int d) const {
    return element(c.k_q, c.k_s, slot, c.D, d);
  }
  __device__ float value(int64_t, int64_t, int, int64_t slot, int d) const {
    return element(c.v_q, c.v_s, slot, c.D, d);
  }
  __device__ float k_scale() const { return *c.k_ts; }
  __device__ float v_scale() const { return *c.v_ts; }
};

// Keys and values of an encoder, bf16.
struct CrossSource {
  const uint16_t* k;
  const uint16_t* v;
  int64_t ldk, ldv, Lk;
  int D;
  const int32_t* k_lens;
  const uint8_t* mask;

  __device__ int64_t rows(int64_t, int64_t Lq) const { return Lq; }
  __device__ int64_t upto(int64_t b, int64_t, int64_t) const {
    return k_lens ? min((int64_t)k_lens[b], Lk) : Lk;
  }
  __device__ bool seen(int64_t b, int64_t j, int64_t&, int) const {
    return !mask || mask[b * Lk + j];
  }
  __device__ float key(int64_t b, int64_t j, int h, int64_t, int d) const {
    return __uint_as_float((uint32_t)k[(b * Lk + j) * ldk + h * D + d] << 16);
  }
  __device__ float value(int64_t b, int64_t j, int h, int64_t, int d) const {
    return __uint_as_float((uint32_t)v[(b * Lk + j) * ldv + h * D + d] << 16);
  }
  __device__ float k_scale() const { return 1.0f; }
  __device__ float v_scale() const { return 1.0f; }
};

template <class Source, int D>
__global__ void __launch_bounds__(256)
attn_rows_kernel(AttnArgs a, Source src, Gate gate) {
  if (gated_off(gate)) return;
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= a.B * a.Lq * a.Hq) return;
  const int h = (int)(item % a.Hq);
  const int64_t row = item / a.Hq, b = row / a.Lq, t = row - b * a.Lq;
  const int64_t nq = src.rows(b, a.Lq);
  if (t >= nq) return;
  const int hk = h / (a.Hq / a.Hkv);
  const float c = a.scale * 1.4426950408889634f * src.k_scale();
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)a.q[row * a.ldq + h * D + lane + 64 * e] << 16);
    o[e] = 0.0f;
  }
  const int64_t upto = src.upto(b, t, nq);
  for (int64_t j = 0; j < upto; ++j) {
    int64_t slot = 0;
    if (!src.seen(b, j, slot, hk)) continue;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      s = __builtin_fmaf(q[e], src.key(b, j, hk, slot, lane + 64 * e), s);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) s += __shfl_xor(s, x, 64);
    s *= c;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - mn);
    const float p = s == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s - mn);
    m = mn;
    l = __builtin_fmaf(l, f, p);
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = __builtin_fmaf(o[e], f, p * src.value(b, j, hk, slot, lane + 64 * e));
  }
  const float r = l == 0.0f ? 0.0f : src.v_scale() / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.o[row * a.ldo + h * D + lane + 64 * e] = (uint16_t)bf16_pack(o[e] * r, 0.0f);
}

template <class Source>
hipError_t launch(const AttnArgs& a, const Source& src, hipStream_t stream) {
  const dim3 grid((unsigned)((a.B * a.Lq * a.Hq + 3) / 4));
  if (a.D == 64)
    hipLaunchKernelGGL((attn_rows_kernel<Source, 64>), grid, dim3(256), 0, stream, a, src,
                       current_gate());
  else
    hipLaunchKernelGGL((attn_rows_kernel<Source, 128>), grid, dim3(256), 0, stream, a, src,
                       current_gate());
  return hipGetLastError();
}

}  // namespace

size_t attn_ws_bytes(int64_t, int64_t, int, int, int, int64_t) { return 0; }

hipError_t launch_attn_kv4(const AttnArgs& a, const Kv4Cache& c, const int32_t* lens,
                           const int32_t* q_lens, bool causal, void*, size_t, hipStream_t stream) {
  return launch(a, Kv4Source{c, lens, q_lens, causal ? 1 : 0}, stream);
}

hipError_t launch_attn_cross(const AttnArgs& a, const uint16_t* k, int64_t ldk, const uint16_t* v,
                             int64_t ldv, int64_t Lk, const int32_t* k_lens, const uint8_t* mask,
                             void*, size_t, hipStream_t stream) {
  return launch(a, CrossSource{k, v, ldk, ldv, Lk, a.D, k_lens, mask}, stream);
}

}  // namespace qact
