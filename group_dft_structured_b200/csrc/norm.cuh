// norm.cuh — layer norm of equivariant features, forward and backward.
//
// A token's features x[c,t] (c < C channels, t < T group elements, group index
// innermost) are normalised over all F = C T of them, and the affine parameters
// are per channel, so the layer commutes with the group's action on the t axis:
//   mu = mean(x), var = mean((x - mu)^2), r = (var + eps)^-1/2, xh = (x - mu) r
//   y[c,t] = xh[c,t] gamma[c] + beta[c]
//   g = dy gamma,  dx = r (g - mean(g) - xh mean(g xh))
//   dgamma[c] = sum_{n,t} dy xh,  dbeta[c] = sum_{n,t} dy
//
// HBM-bound (a few operations per value): every row is read once into
// registers, its moments come from shuffles over the G threads that hold it,
// and it is written once.  G is the smallest power of two for which K packs of
// 16 bytes per thread hold the row: a part of a warp for short rows (several
// rows per warp and load instruction), a warp, or a whole block.  The variance
// is the mean of squared deviations, a second pass over registers: no
// cancellation for rows whose mean is large.
//
// The parameter gradients are sums down the rows.  A thread keeps its columns
// for all the rows it visits, so it accumulates them in registers (fp32), the
// block adds its row groups in a fixed order and writes one partial row, and a
// second kernel adds the blocks' partials: no atomics, bit-identical runs.
//
// Measured on 401408 x 24 x 4, fp16: forward 30 us (157 MB, 5.2 TB/s), backward 42
// (234 MB, 5.6 TB/s) and its reduction 8.  The instructions issue on 72 % of the
// cycles (22 a value forward: the row's two sums and the converts), which bounds
// it as much as DRAM does.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "vec.cuh"

namespace feql {

constexpr int kNormThreads = 256;      // block of the part-warp and warp row groups
constexpr int kNormMaxThreads = 512;   // largest row group

// Sum over the G threads of a row group (G a power of two, or the whole block
// when G > 32), the same bits in every thread of the group.
__device__ __forceinline__ float norm_group_sum(float v, int G, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < G) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (G > 32) {
    const int w = threadIdx.x >> 5, nw = G >> 5;
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < nw; ++i) v += red[i];
    __syncthreads();
  }
  return v;
}

struct NormShape {
  int64_t N;
  int C, T, F;
  int G;          // threads of a row group
  int nchunk;     // packs in a row: F / V
};

// Per-thread affine parameters: one value for each A neighbouring columns (A
// divides both the pack and T, so they share a channel).
template <typename Ty, int V, int K, int A>
__device__ __forceinline__ void norm_params(const Ty *__restrict__ p, float dflt, int lane,
                                            const NormShape &s, Ty (&out)[K][V / A]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int q = lane + k * s.G;
#pragma unroll
    for (int a = 0; a < V / A; ++a)
      out[k][a] = (p != nullptr && q < s.nchunk) ? p[(q * V + a * A) / s.T] : narrow<Ty>(dflt);
  }
}

// Blocks of kNormMaxThreads per SM that the registers are shared out for: two (64
// registers) where the packs in flight and the sums leave room for unpacking.
constexpr int norm_blocks_fwd(int bytes_per_thread, int params) {
  return bytes_per_thread / 4 + params < 40 ? 2 : 1;
}
constexpr int norm_blocks_bwd(int bytes_per_thread, int sums) {
  return bytes_per_thread / 4 + sums <= 40 ? 2 : 1;
}

template <typename Ty, int V, int K, int A>
__global__ void __launch_bounds__(kNormMaxThreads,
                                  norm_blocks_fwd(K * V * sizeof(Ty), 2 * K * V / A))
norm_fwd_kernel(const Ty *__restrict__ x, const Ty *__restrict__ gamma,
                const Ty *__restrict__ beta, Ty *__restrict__ y, float2 *__restrict__ stats,
                const NormShape s, float eps) {
  __shared__ float red[32];
  const int lane = threadIdx.x & (s.G - 1);
  const int per_block = blockDim.x / s.G, sub = threadIdx.x / s.G;
  Ty gm[K][V / A], bt[K][V / A];
  norm_params<Ty, V, K, A>(gamma, 1.f, lane, s, gm);
  norm_params<Ty, V, K, A>(beta, 0.f, lane, s, bt);
  const float inv = 1.f / static_cast<float>(s.F);
  // the bound is the same for a whole block, so the shuffles below are full
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * per_block; row0 < s.N;
       row0 += static_cast<int64_t>(gridDim.x) * per_block) {
    const int64_t row = row0 + sub;
    const bool live = row < s.N;
    const Ty *xr = x + row * s.F;
    Pack<Ty, V> v[K];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int q = lane + k * s.G;
      if (live && q < s.nchunk) v[k].load(xr + q * V);
      else v[k].zero();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float f[V];
      v[k].unpack(f);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += f[j];
    }
    const float mu = norm_group_sum(sum, s.G, red) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k].renew();
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (lane + k * s.G < s.nchunk) {
        float f[V];
        v[k].unpack(f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = f[j] - mu;
          sq = fmaf(d, d, sq);
        }
      }
    const float var = norm_group_sum(sq, s.G, red) * inv;
    const float r = 1.f / sqrtf(var + eps);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k].renew();
    if (!live) continue;
    if (stats != nullptr && lane == 0) stats[row] = make_float2(mu, r);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int q = lane + k * s.G;
      if (q < s.nchunk) {
        float f[V];
        v[k].unpack(f);
#pragma unroll
        for (int j = 0; j < V; ++j)
          f[j] = fmaf((f[j] - mu) * r, widen(gm[k][j / A]), widen(bt[k][j / A]));
        Pack<Ty, V> o;
        o.pack(f);
        o.store(y + row * s.F + q * V);
      }
    }
  }
}

// part[block][2][F / A]: this block's sums of dy xh and dy over its rows and
// over each A columns.
template <typename Ty, int V, int K, int A>
__global__ void __launch_bounds__(kNormMaxThreads,
                                  norm_blocks_bwd(2 * K * V * sizeof(Ty), 2 * K * V / A))
norm_bwd_kernel(const Ty *__restrict__ x, const Ty *__restrict__ dy, const Ty *__restrict__ gamma,
                const float2 *__restrict__ stats, Ty *__restrict__ dx, float *__restrict__ part,
                const NormShape s) {
  __shared__ float red[32];
  __shared__ float fold[kNormThreads / 32][32][V / A][2];
  const int lane = threadIdx.x & (s.G - 1);
  const int per_block = blockDim.x / s.G, sub = threadIdx.x / s.G;
  Ty gm[K][V / A];
  norm_params<Ty, V, K, A>(gamma, 1.f, lane, s, gm);
  float ag[K][V / A], ab[K][V / A];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int a = 0; a < V / A; ++a) ag[k][a] = ab[k][a] = 0.f;
  const float inv = 1.f / static_cast<float>(s.F);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * per_block; row0 < s.N;
       row0 += static_cast<int64_t>(gridDim.x) * per_block) {
    const int64_t row = row0 + sub;
    const bool live = row < s.N;
    Pack<Ty, V> v[K], w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int q = lane + k * s.G;
      const bool in = live && q < s.nchunk;
      v[k].zero();
      w[k].zero();
      if (in) {
        v[k].load(x + row * s.F + q * V);
        w[k].load(dy + row * s.F + q * V);
      }
    }
    const float2 st = live ? stats[row] : make_float2(0.f, 0.f);
    float s1 = 0.f, s2 = 0.f;  // sums of g and g xh (dy = 0 outside the row)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float f[V], d[V];
      v[k].unpack(f);
      w[k].unpack(d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (f[j] - st.x) * st.y, g = d[j] * widen(gm[k][j / A]);
        s1 += g;
        s2 = fmaf(g, xh, s2);
        ab[k][j / A] += d[j];
        ag[k][j / A] = fmaf(d[j], xh, ag[k][j / A]);
      }
    }
    const float m1 = norm_group_sum(s1, s.G, red) * inv;
    const float m2 = norm_group_sum(s2, s.G, red) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k].renew();
      w[k].renew();
    }
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int q = lane + k * s.G;
      if (q < s.nchunk) {
        float f[V], d[V];
        v[k].unpack(f);
        w[k].unpack(d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (f[j] - st.x) * st.y, g = d[j] * widen(gm[k][j / A]);
          f[j] = st.y * (g - m1 - xh * m2);
        }
        Pack<Ty, V> o;
        o.pack(f);
        o.store(dx + row * s.F + q * V);
      }
    }
  }
  // the block's row groups, added in a fixed order: within a warp by shuffles
  // over the lanes that hold the same columns, then warp by warp
  const int nv = s.F / A;
  float *pg = part + static_cast<int64_t>(blockIdx.x) * 2 * nv, *pb = pg + nv;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (s.G <= 32) {
      const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
#pragma unroll
      for (int a = 0; a < V / A; ++a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (o >= s.G) {
            ag[k][a] += __shfl_xor_sync(0xffffffffu, ag[k][a], o);
            ab[k][a] += __shfl_xor_sync(0xffffffffu, ab[k][a], o);
          }
        fold[w][l][a][0] = ag[k][a];
        fold[w][l][a][1] = ab[k][a];
      }
      __syncthreads();
      if (w == 0 && l < s.G) {
#pragma unroll
        for (int a = 0; a < V / A; ++a) {
          float g = 0.f, b = 0.f;
          for (int i = 0; i < kNormThreads / 32; ++i) {
            g += fold[i][l][a][0];
            b += fold[i][l][a][1];
          }
          const int q = l + k * s.G;
          if (q < s.nchunk) {
            pg[q * (V / A) + a] = g;
            pb[q * (V / A) + a] = b;
          }
        }
      }
      __syncthreads();
    } else {
      const int q = lane + k * s.G;
      if (q < s.nchunk) {
#pragma unroll
        for (int a = 0; a < V / A; ++a) {
          pg[q * (V / A) + a] = ag[k][a];
          pb[q * (V / A) + a] = ab[k][a];
        }
      }
    }
  }
}

// dgamma[c], dbeta[c] from the partials, in a fixed order: 32 partial columns
// (m = T / A neighbours belong to a channel) by 32 row lanes per block.  Launched
// as the programmatic dependent of the kernel that writes the partials.
constexpr int kNormRedLanes = 32;
template <typename Ty>
__global__ void __launch_bounds__(32 * kNormRedLanes)
norm_reduce_kernel(const float *__restrict__ part, Ty *__restrict__ dgamma,
                   Ty *__restrict__ dbeta, int C, int m, int blocks) {
  __shared__ float sum[2][kNormRedLanes][33];
  const int col = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int per = 32 / m;  // channels per block
  const int c0 = blockIdx.x * per;
  const int64_t nv = static_cast<int64_t>(C) * m;
  const int64_t at = static_cast<int64_t>(c0) * m + col;
  float g = 0.f, b = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (col < per * m && at < nv) {
#pragma unroll 4
    for (int i = r; i < blocks; i += kNormRedLanes) {
      g += part[2 * i * nv + at];
      b += part[(2 * i + 1) * nv + at];
    }
  }
  sum[0][r][col] = g;
  sum[1][r][col] = b;
  __syncthreads();
  if (r < 2) {  // warp 0: dgamma's columns, warp 1: dbeta's
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kNormRedLanes; ++i) v += sum[r][i][col];
    float t = v;
    for (int j = 1; j < m; ++j) t += __shfl_down_sync(0xffffffffu, v, j);
    const int c = c0 + col / m;
    Ty *to = r == 0 ? dgamma : dbeta;
    if (to != nullptr && col % m == 0 && col < per * m && c < C) to[c] = narrow<Ty>(t);
  }
}

// Rows longer than a block's registers hold (rare: tens of thousands of
// features): one block per row, the row read again from the caches for each
// pass; the parameter gradients by a column pass over row splits.
constexpr int kNormLongThreads = 1024;

__device__ __forceinline__ float norm_block_sum(float v, float *red) {
  return norm_group_sum(v, kNormLongThreads, red);
}

template <typename Ty>
__global__ void __launch_bounds__(kNormLongThreads)
norm_fwd_long_kernel(const Ty *__restrict__ x, const Ty *__restrict__ gamma,
                     const Ty *__restrict__ beta, Ty *__restrict__ y, float2 *__restrict__ stats,
                     const NormShape s, float eps) {
  __shared__ float red[32];
  const float inv = 1.f / static_cast<float>(s.F);
  for (int64_t row = blockIdx.x; row < s.N; row += gridDim.x) {
    const Ty *xr = x + row * s.F;
    float v = 0.f;
    for (int f = threadIdx.x; f < s.F; f += kNormLongThreads) v += widen(xr[f]);
    const float mu = norm_block_sum(v, red) * inv;
    v = 0.f;
    for (int f = threadIdx.x; f < s.F; f += kNormLongThreads) {
      const float d = widen(xr[f]) - mu;
      v = fmaf(d, d, v);
    }
    const float r = 1.f / sqrtf(norm_block_sum(v, red) * inv + eps);
    if (stats != nullptr && threadIdx.x == 0) stats[row] = make_float2(mu, r);
    for (int f = threadIdx.x; f < s.F; f += kNormLongThreads) {
      const int c = f / s.T;
      const float gm = gamma != nullptr ? widen(gamma[c]) : 1.f;
      const float bt = beta != nullptr ? widen(beta[c]) : 0.f;
      y[row * s.F + f] = narrow<Ty>(fmaf((widen(xr[f]) - mu) * r, gm, bt));
    }
  }
}

template <typename Ty>
__global__ void __launch_bounds__(kNormLongThreads)
norm_dx_long_kernel(const Ty *__restrict__ x, const Ty *__restrict__ dy,
                    const Ty *__restrict__ gamma, const float2 *__restrict__ stats,
                    Ty *__restrict__ dx, const NormShape s) {
  __shared__ float red[32];
  const float inv = 1.f / static_cast<float>(s.F);
  for (int64_t row = blockIdx.x; row < s.N; row += gridDim.x) {
    const float2 st = stats[row];
    float s1 = 0.f, s2 = 0.f;
    for (int f = threadIdx.x; f < s.F; f += kNormLongThreads) {
      const float gm = gamma != nullptr ? widen(gamma[f / s.T]) : 1.f;
      const float g = widen(dy[row * s.F + f]) * gm;
      s1 += g;
      s2 = fmaf(g, (widen(x[row * s.F + f]) - st.x) * st.y, s2);
    }
    const float m1 = norm_block_sum(s1, red) * inv, m2 = norm_block_sum(s2, red) * inv;
    for (int f = threadIdx.x; f < s.F; f += kNormLongThreads) {
      const float gm = gamma != nullptr ? widen(gamma[f / s.T]) : 1.f;
      const float g = widen(dy[row * s.F + f]) * gm;
      const float xh = (widen(x[row * s.F + f]) - st.x) * st.y;
      dx[row * s.F + f] = narrow<Ty>(st.y * (g - m1 - xh * m2));
    }
  }
}

// part[split][2][F] of columns blockIdx.x * blockDim.x .., rows split by split.
template <typename Ty>
__global__ void __launch_bounds__(kNormThreads)
norm_cols_long_kernel(const Ty *__restrict__ x, const Ty *__restrict__ dy,
                      const float2 *__restrict__ stats, float *__restrict__ part,
                      const NormShape s, int64_t split_len) {
  const int f = blockIdx.x * kNormThreads + threadIdx.x;
  if (f >= s.F) return;
  const int64_t r0 = blockIdx.y * split_len;
  const int64_t r1 = r0 + split_len < s.N ? r0 + split_len : s.N;
  float g = 0.f, b = 0.f;
  for (int64_t row = r0; row < r1; ++row) {
    const float2 st = stats[row];
    const float d = widen(dy[row * s.F + f]);
    b += d;
    g = fmaf(d, (widen(x[row * s.F + f]) - st.x) * st.y, g);
  }
  float *p = part + static_cast<int64_t>(blockIdx.y) * 2 * s.F;
  p[f] = g;
  p[s.F + f] = b;
}

}  // namespace feql
