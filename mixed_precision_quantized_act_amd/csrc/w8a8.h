// What the kernels of qlinear_w8a8 share.
//
//   y[m][n] = s_a[m] s_w[n] sum_k a[m][k] w[n][k]  (+ bias[n]) (-> GELU)
//
// The sum is an exact int32 (|a w| <= 2^14, K < 2^17), rounded once to float32, so
// the kernels, tiles and splits below give the same bits.
#pragma once

#include "qgemm_common.h"
#include "w8a8_plan.h"

namespace qact {

constexpr uint32_t kSkip = 0x7FFFFFF0u;          // an offset past every buffer range

struct W8Args {
  const int8_t* a;
  const float* a_s;
  const int8_t* w;
  const float* w_s;
  int64_t K;
  int units, mt, nt;               // K in units of 64, tiles
  int main_tiles, main_blocks;     // tiles taken in a stream, and its workgroups
  int splits, split_chunks;        // cuts of K, in lines of 128
  int32_t* part;                   // their sums [splits][M][N rounded up to 4]
  Gate gate;
};

// A tile's operands: rows past the end lie outside the buffers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t operand(const int8_t* p, int row0, int64_t rows, int most,
                                                          int64_t K) {
  const int n = max(0, min((int)rows - row0, most));
  return buffer_rsrc(p + row0 * K, (uint32_t)n * (uint32_t)K);
}

// few rows, or few outputs (w8a8_split.hip)
hipError_t launch_w8a8_split(int shape, int splits, const W8Args& g, const EpiArgs& e, hipStream_t st);

}  // namespace qact
