// split_sum.cuh — sums over the splits of a weight gradient's partials, in order.
#pragma once

#include <stdint.h>

#include "host.cuh"

namespace feql {

// Two forms, both in the order of the splits (the same bits).  One thread an output walks
// its splits in memory; that is enough where the outputs fill the GPU or the splits are
// few (kWide).  Else the walk's latency would be all there is, and a block takes kSumOut neighbouring outputs of all planes.  The order of the sums
// makes a chain of as many additions as there are splits, but not of loads: the
// block brings kSumLines lines (one plane of one split each, 32 loads a thread in
// flight) to shared memory and a thread adds its column from there.  188 splits of
// 51 x 35 x 4 values: 9 us; a thread that walks its column in memory, eight splits
// in flight, took 46.
// Threads against blocks, us for both kernels of a weight gradient: order 4, 768 x 768 of
// 64 tokens 29 against 107, 512 x 512 (5 splits) 266 and 302, 35 x 51 (188) 63 and 23;
// order 3, 160 x 160 (11) 18 and 20; order 16, 96 x 96 (32) 49 and 43; order 8, 64 x 64 47
// and 30.
constexpr int kSumOut = 32;
constexpr int kSumThreads = 256;
constexpr int kSumLines = 256;
constexpr int kSumFew = 12;  // splits that a thread walks

inline bool split_sum_wide(int C, int D, int splits, int sms) {
  return splits <= kSumFew || static_cast<int64_t>(C) * D + D >= 256ll * sms;
}

// Blocks over the D C outputs of dW and the D of db (channels are at most 2^16).
inline unsigned split_sum_blocks(int C, int D, bool wide, int sms) {
  if (wide) return static_cast<unsigned>(grid_for(static_cast<int64_t>(C) * D + D, kSumThreads, sms));
  return static_cast<unsigned>((static_cast<int64_t>(C) * D + kSumOut - 1) / kSumOut +
                               (D + kSumOut - 1) / kSumOut);
}

// The sums of output e's K planes by one thread.
template <int K>
__device__ __forceinline__ void split_walk(const float *__restrict__ ws, int64_t n, int64_t e,
                                           int splits, float (&sum)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) sum[k] = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float *p = ws + static_cast<int64_t>(s) * K * n + e;
#pragma unroll
    for (int k = 0; k < K; ++k) sum[k] += p[k * n];
  }
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
