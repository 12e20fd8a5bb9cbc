// Attention of bf16 queries over an NVFP4 cache (attn_kv4; attn_kv4_tree: of a
// tree of drafted tokens) and over an encoder's bf16 states (attn_cross):
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale (q . k_j) - max)
//
// over the keys j that the row sees; a row that sees none gives zeros.
#include "attn_common.h"

namespace qact {

namespace {

// Rows of a key head from which the tiles of many rows are used (4 streams of 8
// key heads of 128, 4000 tokens: 64 rows 22.8 us, by the few rows' kernel 27.7;
// one stream of 8 heads of 64, 8000 tokens: 48 rows 17.3 and 14.2).
constexpr int64_t kManyRows = 64;

bool many(int64_t Lq, int Hq, int Hkv) { return Lq * (Hq / Hkv) >= kManyRows; }

template <class Source>
hipError_t launch(const AttnArgs& a, const Source& src, int64_t L, void* ws, size_t ws_bytes,
                  hipStream_t stream) {
  if (many(a.Lq, a.Hq, a.Hkv)) return launch_attn_tile(a, src, L, ws, ws_bytes, stream);
  return launch_attn_few(a, src, L, ws, ws_bytes, stream);
}

}  // namespace

size_t attn_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  if (many(Lq, Hq, Hkv)) return attn_tile_ws_bytes(B, Lq, Hq, Hkv, D, L);
  return attn_few_ws_bytes(B, Lq, Hq, Hkv, D, L);
}

size_t attn_cross_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t Lk) {
  return attn_short_takes(Lq, Hq, Hkv, D, Lk) ? 0 : attn_ws_bytes(B, Lq, Hq, Hkv, D, Lk);
}

hipError_t launch_attn_kv4(const AttnArgs& a, const Kv4Cache& c, const int32_t* lens,
                           const int32_t* q_lens, bool causal, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  return launch(a, Kv4Source{c, lens, q_lens, causal ? 1 : 0}, c.max_pages << c.page_log2, ws,
                ws_bytes, stream);
}

namespace {

// Rows of a key head up to which a tree's are taken in halves of 128.
bool halves(int64_t Lq, int Hq, int Hkv) { return Lq * (Hq / Hkv) <= 128; }

}  // namespace

size_t attn_kv4_tree_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  if (many(Lq, Hq, Hkv) && halves(Lq, Hq, Hkv)) return attn_tree_ws_bytes(B, Lq, Hq, Hkv, D, L);
  return attn_ws_bytes(B, Lq, Hq, Hkv, D, L);
}

hipError_t launch_attn_kv4_tree(const AttnArgs& a, const Kv4Cache& c, const int32_t* lens,
                                const int32_t* q_lens, const uint64_t* tree, int64_t stride, void* ws,
                                size_t ws_bytes, hipStream_t stream) {
  const Kv4TreeSource src = {{c, lens, q_lens, 0}, tree, stride, (int)((a.Lq + 63) / 64)};
  const int64_t L = c.max_pages << c.page_log2;
  if (many(a.Lq, a.Hq, a.Hkv) && halves(a.Lq, a.Hq, a.Hkv)) return launch_attn_tree(a, src, L, ws, ws_bytes, stream);
  return launch(a, src, L, ws, ws_bytes, stream);
}

hipError_t launch_attn_cross(const AttnArgs& a, const uint16_t* k, int64_t ldk, const uint16_t* v,
                             int64_t ldv, int64_t Lk, const int32_t* k_lens, const uint8_t* mask,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  const CrossSource src = {k, v, ldk, ldv, (int)Lk, k_lens, mask};
  if (attn_short_takes(a.Lq, a.Hq, a.Hkv, a.D, Lk)) return launch_attn_short(a, src, stream);
  return launch(a, src, Lk, ws, ws_bytes, stream);
}

}  // namespace qact
