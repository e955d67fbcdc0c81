// split_sum.cuh — sums over the splits of a weight gradient's partials, in order.
#pragma once

#include <stdint.h>

namespace feql {

// A block takes kSumOut neighbouring outputs of all planes.  The order of the sums
// makes a chain of as many additions as there are splits, but not of loads: the
// block brings kSumLines lines (one plane of one split each, 32 loads a thread in
// flight) to shared memory and a thread adds its column from there.  188 splits of
// 51 x 35 x 4 values: 9 us; a thread that walks its column in memory, eight splits
// in flight, took 46.
constexpr int kSumOut = 32;
constexpr int kSumThreads = 256;
constexpr int kSumLines = 256;

// Blocks over the D C outputs of dW and the D of db (channels are at most 2^16).
inline unsigned split_sum_blocks(int C, int D) {
  return static_cast<unsigned>((static_cast<int64_t>(C) * D + kSumOut - 1) / kSumOut +
                               (D + kSumOut - 1) / kSumOut);
}

// ws [splits][K][n]: afterwards buf[k][lane] is the sum over the splits of output e
// (the lane's) of plane k.  The whole block calls.
template <int K>
__device__ __forceinline__ void split_sums(const float *__restrict__ ws, int64_t n, int64_t e,
                                           int splits, float (&buf)[kSumLines][kSumOut]) {
  constexpr int kWarps = kSumThreads / kSumOut, kRows = kSumLines / K;
  constexpr int kCols = (K + kWarps - 1) / kWarps;  // planes a thread sums
  const int lane = threadIdx.x % kSumOut, w = threadIdx.x / kSumOut;
  float sum[kCols] = {};
  for (int s0 = 0; s0 < splits; s0 += kRows) {
    const int rows = splits - s0 < kRows ? splits - s0 : kRows, lines = rows * K;
    const float *p = ws + static_cast<int64_t>(s0) * K * n + e;
    float v[kSumLines / kWarps];
#pragma unroll
    for (int i = 0; i < kSumLines / kWarps; ++i) {
      const int l = w + i * kWarps;
      v[i] = l < lines && e < n ? __ldg(p + l * n) : 0.f;
    }
    __syncthreads();  // the lines before have been added
#pragma unroll
    for (int i = 0; i < kSumLines / kWarps; ++i) buf[w + i * kWarps][lane] = v[i];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const int k = w + c * kWarps;
      if (k < K) {
#pragma unroll 8
        for (int r = 0; r < rows; ++r) sum[c] += buf[r * K + k][lane];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    if (w + c * kWarps < K) buf[w + c * kWarps][lane] = sum[c];
  __syncthreads();
}

}  // namespace feql
