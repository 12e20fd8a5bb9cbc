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
  return attn_few_ws_bytes(false, B, Lq, Hq, Hkv, D, L);
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

// Which kernel takes a tree.  The few rows' (16 or 32 a wave, by itself) up to 48
// rows of a key head, and where a SIMD has at most 6 of its steps of 16 rows and 64 keys
// (the start of the tiles of many rows takes as long: 64 rows, 8 key heads of
// 128, 4000 keys: 14.3 us, by the tiles 19.0; 128 rows, 32 key heads, 1000 keys: 22.5 and
// 24.7; 4000 keys: 37.8 and 31.6).  Above, tiles of 128 or 256 rows, but up to 64 rows,
// half a tile, only below 64 steps a SIMD (128 key heads, 4000 keys: 49.7 us and
// 53.7 by the few rows'; 32768 keys: 285 and 212).
bool tree_few(int64_t B, int64_t Lq, int Hq, int Hkv, int64_t L) {
  const int64_t rows = Lq * (Hq / Hkv), steps = B * Hkv * ((rows + 15) / 16) * ((L + 63) / 64);
  return rows <= 48 || steps <= 6 * 1024 || (rows <= 64 && steps >= 64 * 1024);
}

}  // namespace

size_t attn_kv4_tree_ws_bytes(int64_t B, int64_t Lq, int Hq, int Hkv, int D, int64_t L) {
  return tree_few(B, Lq, Hq, Hkv, L) ? attn_few_ws_bytes(true, B, Lq, Hq, Hkv, D, L)
                                     : attn_tree_ws_bytes(B, Lq, Hq, Hkv, D, L);
}

hipError_t launch_attn_kv4_tree(const AttnArgs& a, const Kv4Cache& c, const int32_t* lens,
                                const int32_t* q_lens, const uint64_t* tree, int64_t stride, void* ws,
                                size_t ws_bytes, hipStream_t stream) {
  const Kv4TreeSource src = {{c, lens, q_lens, 0}, tree, stride, (int)((a.Lq + 63) / 64)};
  const int64_t L = c.max_pages << c.page_log2;
  if (tree_few(a.B, a.Lq, a.Hq, a.Hkv, L)) return launch_attn_few(a, src, L, ws, ws_bytes, stream);
  return launch_attn_tree(a, src, L, ws, ws_bytes, stream);
}

hipError_t launch_attn_cross(const AttnArgs& a, const uint16_t* k, int64_t ldk, const uint16_t* v,
                             int64_t ldv, int64_t Lk, const int32_t* k_lens, const uint8_t* mask,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  const CrossSource src = {k, v, ldk, ldv, (int)Lk, k_lens, mask};
  if (attn_short_takes(a.Lq, a.Hq, a.Hkv, a.D, Lk)) return launch_attn_short(a, src, stream);
  return launch(a, src, Lk, ws, ws_bytes, stream);
}

}  // namespace qact
