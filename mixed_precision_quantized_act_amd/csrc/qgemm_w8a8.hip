// qlinear_w8a8: the linear of INT8 activations and INT8 weights, a scale for
// each token and each output channel (6Bit-Diffusion, abstract: volatile layers
// keep INT8; here the weights do, too).  This file: many rows; w8a8_split.hip: few.
//
// A workgroup of 4 waves computes a tile on v_mfma_i32_32x32x32_i8.  K runs in units
// of 64: the unit's rows are moved (buffer_load ... lds) into a ring of 4 slots three
// units ahead, each wave reads its operands one unit ahead, and both kinds of memory
// instruction stand among the unit's products.  Of the 256 x 256 tile a wave owns
// 128 x 128 (16 accumulators of 32 x 32, all 256 accumulation registers), so that a
// unit's 1024 cycles of products read 64 KB of shared memory and move 32 KB; tiles
// half as large need half as much again and were 15 % slower (two of them on a
// compute unit, to hide each other's ends: 17776 rows of 7680 against 1920 320 us).
//
// What bounds it is power: 17776 rows of 1920 against 5760 take 200 us (1.97 POP/s, a
// library's product 235 to 254), of 7680 against 1920 255 us (2.05 POP/s; 254 to 257), both
// with a bias.  The clock goes down to 1.63 GHz with the matrix units busy 0.63 of the cycles; with zeros as
// operands the same launches take 186 and 211 us.
#include "w8a8.h"

namespace qact {

namespace {

constexpr int kUnitK = 64;                       // K per unit (two k-steps of 32)

// Position of 16-byte chunk c (of 4) of row r of a unit in shared memory: exchanged
// by bit 2 of the row, so that the 32 rows of an operand spread over the banks.
__device__ __forceinline__ constexpr int chunk_slot(int r, int c) { return c ^ ((r >> 2) & 3); }

// A workgroup's tile: 4 waves, WM of them along the rows, 32 FM rows and 128
// columns each.
template <int FM_, int WM_, int SLOTS>
struct Shape {
  static constexpr int FM = FM_, WM = WM_, WN = 4 / WM_, kSlots = SLOTS;
  static constexpr int TM = 32 * FM * WM, TN = 128 * WN;
  static constexpr int kWOff = TM * kUnitK, kSlot = (TM + TN) * kUnitK;
  static constexpr int kRing = kSlots * kSlot > 32768 ? kSlots * kSlot : 32768;
  static constexpr int kColF = kRing, kBias = kColF + TN * 4, kRowS = kBias + TN * 4, kSmem = kRowS + TM * 4;
  static constexpr int kLoads = (TM + TN) / 64;  // DMA instructions per wave and unit
  static constexpr int kReads = 2 * (FM + 4);    // operand reads
  static constexpr int kMfmas = 8 * FM;
  static constexpr int kSegs = kMfmas / 4;
  static_assert(kSmem <= 160 * 1024, "LDS");
};

template <class S>
struct Frag {
  i32x4 a[2][S::FM];
  i32x4 w[2][4];
};

template <class S>
__device__ __forceinline__ void pin_frag(Frag<S>& f) {
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
    for (int i = 0; i < S::FM; ++i) asm volatile("" : "+v"(f.a[ks][i]));
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(f.w[ks][j]));
  }
}

__device__ __forceinline__ void ring_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The outputs of a wave's 32 FM rows x 128 columns.  Half a block of 32 rows (64
// columns) at a time goes as it lies in the accumulators, whole numbers, through 8
// KB of shared memory, from which a lane takes 8 neighbouring columns of a row: so
// its columns' scales and bias are the same for all rows, every store is 16 bytes
// (bf16) of a row's 128, and a value costs a conversion, two multiplications (the
// second with the bias added, one rounding) and half a packing.  The next half
// is on its way through shared memory while this one is worked on.
// rows: the wave's row scales, cols, bias: its columns', all in shared memory.
template <int FM, bool F32, bool GELU, bool LINES>
__device__ __forceinline__ void store_sums(const i32x16 (&acc)[FM][4], const float* rows, const float* cols,
                                           const float* bias, int row0, int col0, uint8_t* stg, const EpiArgs& e,
                                           int lane) {
  asm volatile("" : "+v"(lane));       // (places are formed here, not kept through the loop before)
  const int lr = lane & 31, lh = lane >> 5, k = lane & 7, r8 = lane >> 3;
  f32x4 cf[2][2], bs[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      cf[h][c] = *reinterpret_cast<const f32x4*>(cols + 64 * h + 8 * k + 4 * c);
      bs[h][c] = *reinterpret_cast<const f32x4*>(bias + 64 * h + 8 * k + 4 * c);
    }
  i32x4 v[2][8];
  // half block x (of 2 FM) through shared memory: 16-byte chunk c of row r (16 of
  // 4 columns) at slot c ^ (r & 15)
  auto turn = [&](int x) {
    const int i = x >> 1, h = x & 1;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<i32x4*>(stg + lr * 256 + 16 * ((8 * j + 2 * q + lh) ^ (lr & 15))) =
            i32x4{acc[i][2 * h + j][4 * q], acc[i][2 * h + j][4 * q + 1], acc[i][2 * h + j][4 * q + 2],
                  acc[i][2 * h + j][4 * q + 3]};
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * it + r8;
        v[x & 1][2 * it + c] = *reinterpret_cast<const i32x4*>(stg + r * 256 + 16 * ((2 * k + c) ^ (r & 15)));
      }
  };
  // groups of 8 columns at any address that their type allows
  constexpr int kBytes = F32 ? 4 : 2;
  typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t By2;
  typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t By4;
  using Group = std::conditional_t<F32, By4, By2>;
  const int left = min((int)e.M - row0, 32 * FM);
  const int64_t pitch = e.ldy * kBytes;
  char* const base = static_cast<char*>(e.y) + ((int64_t)row0 * e.ldy + col0) * kBytes;
  turn(0);
#pragma unroll
  for (int x = 0; x < 2 * FM; ++x) {
    if (x + 1 < 2 * FM) turn(x + 1);
    const int h = x & 1, col = 64 * h + 8 * k, cols = (int)e.N - col0 - col;       // columns from this one on
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int r = 32 * (x >> 1) + 8 * it + r8;
      const float rs = rows[r];
      float f[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        f[c] = __builtin_fmaf((float)v[h][2 * it + c / 4][c % 4] * cf[h][c / 4][c % 4], rs, bs[h][c / 4][c % 4]);
        if constexpr (GELU) f[c] = gelu_tanh(f[c]);
      }
      u32x4 w[F32 ? 2 : 1];
      if constexpr (F32) {
        w[0] = __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]});
        w[1] = __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]});
      } else {
        w[0] = u32x4{bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7])};
      }
      if (r >= left) continue;
      char* const y = base + r * pitch + col * kBytes;
      if (cols >= 8) {
        if constexpr (LINES) {
          __builtin_nontemporal_store((Group)w[0], reinterpret_cast<Group*>(y));
          if constexpr (F32) __builtin_nontemporal_store((Group)w[1], reinterpret_cast<Group*>(y + 16));
        } else {
          *reinterpret_cast<Group*>(y) = w[0];
          if constexpr (F32) *reinterpret_cast<Group*>(y + 16) = w[1];
        }
      } else if (cols > 0) {
#pragma unroll
        for (int c = 0; c < 7; ++c)
          if (c < cols) {
            if constexpr (F32)
              reinterpret_cast<float*>(y)[c] = f[c];
            else
              reinterpret_cast<uint16_t*>(y)[c] = (uint16_t)(w[0][c / 2] >> (16 * (c & 1)));
          }
      }
    }
  }
}

// A thread's share of a tile's scales and bias, on its way to shared memory.
template <class S>
struct Factors {
  float col, bias, row;
  __device__ __forceinline__ void load(const W8Args& g, const EpiArgs& e, int m0, int n0) {
    const int c = min(n0 + (int)threadIdx.x % S::TN, (int)e.N - 1);
    col = g.w_s[c];
    bias = e.bias ? __uint_as_float((uint32_t)e.bias[c] << 16) : 0.0f;
    row = g.a_s[min(m0 + (int)threadIdx.x % S::TM, (int)e.M - 1)];
  }
  __device__ __forceinline__ void put(uint8_t* smem) const {
    const int tid = threadIdx.x;
    if (tid < S::TN) {
      reinterpret_cast<float*>(smem + S::kColF)[tid] = col;
      reinterpret_cast<float*>(smem + S::kBias)[tid] = bias;
    }
    if (tid < S::TM) reinterpret_cast<float*>(smem + S::kRowS)[tid] = row;
  }
};

// What a tile's workgroup does, for tiles one by one and in a stream.
template <class S>
struct Work {
  i32x16 acc[S::FM][4];
  Frag<S> f0, f1;
  int lane, wave, wm, wn;

  __device__ __forceinline__ void begin() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave % S::WM;
    wn = wave / S::WM;
  }
  // DMA instruction idx of unit u into the ring slot at s: 16 rows of 64 bytes, the
  // 1 KB blocks wave, wave + 4, ... of the activations, then of the weights.  Rows
  // past the operand lie outside its buffer, chunks past K are skipped: zeros.
  __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t ra, __amdgpu_buffer_rsrc_t rw, uint8_t* s, int u,
                                        int idx, uint32_t K) const {
    constexpr int kA = S::TM / 64;
    const int blk = wave + 4 * (idx < kA ? idx : idx - kA);
    const int row = 16 * blk + (lane >> 2);
    const uint32_t kb = (uint32_t)u * kUnitK + 16u * (uint32_t)chunk_slot(row, lane & 3);
    const uint32_t off = kb < K ? (uint32_t)row * K + kb : kSkip;
    if (idx < kA)
      dma16(ra, s + blk * 1024, off);
    else
      dma16(rw, s + S::kWOff + blk * 1024, off);
  }
  // operand read idx of the unit at s
  __device__ __forceinline__ void read(const uint8_t* s, int idx, Frag<S>& f) const {
    const int ks = idx / (S::FM + 4), r = idx % (S::FM + 4), lr = lane & 31;
    const int off = 16 * chunk_slot(lr, 2 * ks + (lane >> 5));
    if (r < 4)
      f.w[ks][r] = *reinterpret_cast<const i32x4*>(s + S::kWOff + (128 * wn + 32 * r + lr) * 64 + off);
    else
      f.a[ks][r - 4] = *reinterpret_cast<const i32x4*>(s + (32 * S::FM * wm + 32 * (r - 4) + lr) * 64 + off);
  }
  // The unit in `cur`, with DMA instructions (dma(idx)) and the reads of the next
  // unit (next(idx)) among its products: those in all segments, these in the first
  // ones, so that they are there when it begins.  First: the sums begin.
  template <bool First, bool Dma, bool Read, class D, class R>
  __device__ __forceinline__ void compute(Frag<S>& cur, Frag<S>& nxt, const D& dma, const R& next) {
    pin_frag<S>(cur);
    constexpr int kReadSegs = S::kSegs > 2 ? S::kSegs - 2 : S::kSegs;
    const i32x16 zero = {};
#pragma unroll
    for (int seg = 0; seg < S::kSegs; ++seg) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int x = seg * 4 + m, ks = x / (4 * S::FM), i = x / 4 % S::FM, j = x % 4;
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(cur.w[ks][j], cur.a[ks][i],
                                                          First && ks == 0 ? zero : acc[i][j], 0, 0, 0);
      }
      if constexpr (Dma) {
#pragma unroll
        for (int d = seg * S::kLoads / S::kSegs; d < (seg + 1) * S::kLoads / S::kSegs; ++d) dma(d);
      }
      if constexpr (Read) {
        if (seg < kReadSegs) {
#pragma unroll
          for (int r = seg * S::kReads / kReadSegs; r < (seg + 1) * S::kReads / kReadSegs; ++r) next(r);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (Read) pin_frag<S>(nxt);
  }
  // the outputs of the tile at (m0, n0), through the idle 32 KB at stg
  template <bool F32, bool GELU>
  __device__ __forceinline__ void store(const uint8_t* smem, uint8_t* stg, int m0, int n0, const EpiArgs& e) const {
    const int r = 32 * S::FM * wm, c = 128 * wn;
    const auto go = [&](auto lines) {
      store_sums<S::FM, F32, GELU, decltype(lines)::value>(
          acc, reinterpret_cast<const float*>(smem + S::kRowS) + r, reinterpret_cast<const float*>(smem + S::kColF) + c,
          reinterpret_cast<const float*>(smem + S::kBias) + c, m0 + r, n0 + c, stg + wave * 8192, e, lane);
    };
    e.vec_ok ? go(std::true_type()) : go(std::false_type());
  }
  // Before unit u: this wave's DMA of unit u + 1 has landed (Vm; later ones may be
  // in flight) and its reads of unit u are done; behind the barrier that holds for
  // every wave, and nobody reads unit u's slot any more.
  template <bool Vm>
  static __device__ __forceinline__ void sync() {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (Vm) wait_vm<(S::kSlots - 2) * S::kLoads>();
    wait_lds();
    ring_barrier();
  }
};

// One tile at (m0, n0).
template <class S, bool F32, bool GELU>
__device__ __forceinline__ void tile_body(const W8Args& g, const EpiArgs& e, uint8_t* smem, int m0, int n0) {
  Work<S> t;
  t.begin();
  const int units = g.units;
  const uint32_t K = (uint32_t)g.K;
  Factors<S> fac;
  fac.load(g, e, m0, n0);
  const __amdgpu_buffer_rsrc_t ra = operand(g.a, m0, e.M, S::TM, g.K);
  const __amdgpu_buffer_rsrc_t rw = operand(g.w, n0, e.N, S::TN, g.K);
  const auto slot = [&](int u) { return smem + (u % S::kSlots) * S::kSlot; };
  const auto issue = [&](int u, int d) { t.issue(ra, rw, slot(u), u, d, K); };
#pragma unroll
  for (int u = 0; u < S::kSlots; ++u)
#pragma unroll
    for (int d = 0; d < S::kLoads; ++d) issue(u, d);
  wait_vm<(S::kSlots - 1) * S::kLoads>();
  ring_barrier();
#pragma unroll
  for (int r = 0; r < S::kReads; ++r) t.read(slot(0), r, t.f0);
  fac.put(smem);
  const auto one = [&](auto first, int u, Frag<S>& cur, Frag<S>& nxt) {
    Work<S>::template sync<true>();
    t.template compute<decltype(first)::value, true, true>(
        cur, nxt, [&](int d) { issue(u + S::kSlots, d); }, [&](int r) { t.read(slot(u + 1), r, nxt); });
  };
  one(std::true_type(), 0, t.f0, t.f1);
  one(std::false_type(), 1, t.f1, t.f0);
  for (int u = 2; u < units; u += 2) {
    one(std::false_type(), u, t.f0, t.f1);
    one(std::false_type(), u + 1, t.f1, t.f0);
  }
  wait_vm<0>();       // no DMA into shared memory outlives the workgroup
  wait_lds();
  __syncthreads();
  t.template store<F32, GELU>(smem, smem, m0, n0, e);
}

// Tiles blockIdx.x, blockIdx.x + kW8Places, ... of the first g.main_tiles: the units of
// all of them are one stream through the ring, so that the next tile's first
// units are there when this one's outputs are on their way.  The last unit of a
// tile moves nothing in, which leaves its slot to the outputs; before these, all
// that was moved in has landed, so that a tile's first two units wait for nothing
// (no count assumes an order among loads and stores).
template <class S, bool F32, bool GELU>
__device__ __forceinline__ void stream_body(const W8Args& g, const EpiArgs& e, uint8_t* smem) {
  static_assert(S::kSlots == 4 && S::kSlot >= 32768 && S::TM == 256 && S::TN == 256, "ring");
  struct Tile {
    int m0, n0;
    const int8_t *a, *w;
    uint32_t a_bytes, w_bytes;
    bool ok;
  };
  const auto tile_k = [&](int k) {
    Tile r = {};
    TileWork tw;
    const int bid = (int)blockIdx.x + k * (int)kW8Places;
    r.ok = bid < 8 * ((g.main_tiles + 7) / 8) && tile_work(kWhole, bid, g.main_tiles, 1, g.units, g.units, tw);
    int tm = 0, tn = 0;
    if (r.ok) tile_coords(tw.logical, g.mt, g.nt, 8, tm, tn);
    r.m0 = tm * S::TM;
    r.n0 = tn * S::TN;
    r.a = g.a + r.m0 * g.K;
    r.w = g.w + r.n0 * g.K;
    r.a_bytes = r.ok ? (uint32_t)min((int)e.M - r.m0, S::TM) * (uint32_t)g.K : 0u;
    r.w_bytes = r.ok ? (uint32_t)min((int)e.N - r.n0, S::TN) * (uint32_t)g.K : 0u;
    return r;
  };
  Work<S> t;
  t.begin();
  const int units = (g.units + 1) & ~1;
  const uint32_t K = (uint32_t)g.K;
  Tile cur = tile_k(0), nxt = tile_k(1);
  if (!cur.ok) return;
  int sbase = 0;
  const auto slot = [&](int u) { return smem + ((sbase + u) & 3) * S::kSlot; };
  const auto issue = [&](int u, int d) {             // (u >= units: of the next tile)
    const bool in_next = u >= units;
    const Tile& x = in_next ? nxt : cur;
    t.issue(buffer_rsrc(x.a, x.a_bytes), buffer_rsrc(x.w, x.w_bytes), slot(u), in_next ? u - units : u, d, K);
  };
  const auto one = [&](auto first, auto vm, auto dma, int u, Frag<S>& c, Frag<S>& n) {
    Work<S>::template sync<decltype(vm)::value>();
    t.template compute<decltype(first)::value, decltype(dma)::value, true>(
        c, n, [&](int d) { issue(u + S::kSlots, d); }, [&](int r) { t.read(slot(u + 1), r, n); });
  };
  using T = std::true_type;
  using F = std::false_type;
  Factors<S> fac;
  fac.load(g, e, cur.m0, cur.n0);
#pragma unroll
  for (int u = 0; u < S::kSlots; ++u)
#pragma unroll
    for (int d = 0; d < S::kLoads; ++d) issue(u, d);
  wait_vm<0>();
  ring_barrier();
#pragma unroll
  for (int r = 0; r < S::kReads; ++r) t.read(slot(0), r, t.f0);
  for (int k = 0;; ++k) {
    fac.put(smem);
    fac.load(g, e, nxt.m0, nxt.n0);
    one(T(), F(), T(), 0, t.f0, t.f1);
    one(F(), F(), T(), 1, t.f1, t.f0);
    for (int u = 2; u < units - 2; u += 2) {
      one(F(), T(), T(), u, t.f0, t.f1);
      one(F(), T(), T(), u + 1, t.f1, t.f0);
    }
    one(F(), T(), T(), units - 2, t.f0, t.f1);
    one(F(), T(), F(), units - 1, t.f1, t.f0);
    wait_vm<0>();
    t.template store<F32, GELU>(smem, slot(units - 1), cur.m0, cur.n0, e);
    // every wave is past the slot and the factors
    wait_lds();
    ring_barrier();
    if (!nxt.ok) break;
#pragma unroll
    for (int d = 0; d < S::kLoads; ++d) issue(units + S::kSlots - 1, d);
    cur = nxt;
    sbase = (sbase + units) & 3;
    nxt = tile_k(k + 2);
  }
  wait_vm<0>();
}

using Large = Shape<4, 2, 4>;

// The first g.main_tiles large tiles in a stream, a workgroup for each compute unit,
// and the others in tiles of shape S.
template <class S, bool F32, bool GELU>
__global__ void __launch_bounds__(256, 1)
w8a8_stream_kernel(W8Args g, EpiArgs e) {
  if (gated_off(g.gate)) return;
  __shared__ __align__(16) uint8_t smem[Large::kSmem > S::kSmem ? Large::kSmem : S::kSmem];
  if ((int)blockIdx.x < g.main_blocks) {
    stream_body<Large, F32, GELU>(g, e, smem);
    return;
  }
  if constexpr (S::TM < Large::TM || S::TN < Large::TN) {
    constexpr int kM = Large::TM / S::TM, kN = Large::TN / S::TN;
    const int n = g.mt * g.nt - g.main_tiles, bid = (int)blockIdx.x - g.main_blocks;
    TileWork tw;
    if (!tile_work(kWhole, bid, n * kM * kN, 1, g.units, g.units, tw)) return;
    int tm, tn;
    tile_coords(g.main_tiles + tw.logical / (kM * kN), g.mt, g.nt, 8, tm, tn);
    const int sub = tw.logical % (kM * kN);
    const int m0 = tm * Large::TM + sub % kM * S::TM, n0 = tn * Large::TN + sub / kM * S::TN;
    if (m0 >= e.M || n0 >= e.N) return;
    tile_body<S, F32, GELU>(g, e, smem, m0, n0);
  }
}

// All in tiles of shape S, one by one.
template <class S, bool F32, bool GELU>
__global__ void __launch_bounds__(256, 1)
w8a8_tile_kernel(W8Args g, EpiArgs e) {
  if (gated_off(g.gate)) return;
  __shared__ __align__(16) uint8_t smem[S::kSmem];
  TileWork tw;
  if (!tile_work(kWhole, (int)blockIdx.x, g.mt * g.nt, 1, g.units, g.units, tw)) return;
  int tm, tn;
  tile_coords(tw.logical, g.mt, g.nt, 8, tm, tn);
  tile_body<S, F32, GELU>(g, e, smem, tm * S::TM, tn * S::TN);
}

template <class S>
hipError_t launch(const W8Args& g0, int64_t streamed, const EpiArgs& e, hipStream_t st) {
  W8Args g = g0;
  const auto go = [&](auto stream_kernel, auto tile_kernel, int rows, int cols) {
    g.mt = (int)w8_up(e.M, rows);
    g.nt = (int)w8_up(e.N, cols);
    g.main_tiles = (int)streamed;
    g.main_blocks = streamed ? (int)kW8Places : 0;
    const int rest = (g.mt * g.nt - g.main_tiles) * (rows / S::TM) * (cols / S::TN);
    const dim3 grid((unsigned)(g.main_blocks + 8 * ((rest + 7) / 8)));
    if (streamed)
      hipLaunchKernelGGL(stream_kernel, grid, dim3(256), 0, st, g, e);
    else
      hipLaunchKernelGGL(tile_kernel, grid, dim3(256), 0, st, g, e);
    return hipGetLastError();
  };
  const auto pick = [&](auto f32, auto gelu) {
    constexpr bool F = decltype(f32)::value, G = decltype(gelu)::value;
    if constexpr (Large::TM % S::TM == 0) {
      if (streamed) return go(w8a8_stream_kernel<S, F, G>, w8a8_tile_kernel<S, F, G>, Large::TM, Large::TN);
    }
    return go(w8a8_tile_kernel<S, F, G>, w8a8_tile_kernel<S, F, G>, S::TM, S::TN);
  };
  using T = std::true_type;
  using N = std::false_type;
  if (e.out_f32) return e.gelu ? pick(T(), T()) : pick(T(), N());
  return e.gelu ? pick(N(), T()) : pick(N(), N());
}

}  // namespace

hipError_t launch_w8a8(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s, int64_t M,
                       int64_t N, int64_t K, const GemmOut& o, void* ws, size_t ws_bytes, hipStream_t st) {
  // Whole lines go past the caches, as the outputs of all compute units come at once
  // (17776 rows of 1920 against 5760: 218.8 -> 214 us); of rows that begin anywhere the
  // caches put the pieces of a line together (1350 rows of 2000 against 7777, float32:
  // 52.1 -> 42.5).
  const int64_t item = o.out_f32 ? 4 : 2;
  const bool lines = reinterpret_cast<uintptr_t>(o.y) % 128 == 0 && o.ldy * item % 128 == 0;
  const EpiArgs e = {o.y, o.ldy, o.out_f32, o.gelu, o.bias, M, N, lines, nullptr, nullptr, nullptr, nullptr};
  W8Args g = {};
  g.a = a_q;
  g.a_s = a_s;
  g.w = w_q;
  g.w_s = w_s;
  g.K = K;
  g.units = (int)w8_up(K, kUnitK);
  g.part = static_cast<int32_t*>(ws);
  g.gate = current_gate();
  const W8Plan p = w8_plan(M, N, K, ws_bytes);
  if (p.split) return launch_w8a8_split(p.shape, p.cuts, g, e, st);
  switch (p.shape) {
    case kTile128: return launch<Shape<1, 4, 4>>(g, p.streamed, e, st);
    case kTile256x128: return launch<Shape<2, 4, 4>>(g, p.streamed, e, st);
    case kTile192x256: return launch<Shape<3, 2, 4>>(g, p.streamed, e, st);
    default: return launch<Large>(g, p.streamed, e, st);
  }
}

size_t w8a8_ws_bytes(int64_t M, int64_t N, int64_t K) {
  return w8_part_bytes(M, N, w8_plan(M, N, K, (size_t)64 << 20).cuts);
}

}  // namespace qact
