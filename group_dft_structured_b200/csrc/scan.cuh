// scan.cuh — gated linear recurrence over the tokens of a sequence, forward,
// backward and one token at a time.
//
// Per sequence and feature f = (c, t), with gate logits g per channel (shared
// over the group axis) or per (c, t):
//   a_l = sigma(g_l),  h_l = a_l h_{l-1} + (1 - a_l) u_l,  h_{-1} = h0
// Pointwise in the group index, so it commutes with the group's action; convex,
// so |h| <= max(|h0|, |u|) and fp16 outputs stay in range.  Backward:
//   delta_l = dh_l + c_l,  c_{l-1} = a_l delta_l  (c of the last row: dhN),
//   du = (1 - a) delta,  dg = delta (h_{l-1} - u) a (1 - a),  dh0 = c_{-1}
//
// HBM-bound (some ten operations per value), but serial along the sequence.
// An affine step (a, b): h -> a h + b composes associatively, so a block takes a
// tile of rows x 32 features at once: a thread scans R rows of V neighbouring
// features in registers (local states and prefix products), the row groups of
// a warp join by shuffles, the warps through shared memory, and a cluster of K
// blocks, which splits a long sequence's rows when there are too few sequences
// and features to fill the GPU, through distributed shared memory; the block
// then walks to the next tile with the state in registers.  Every value is read
// once and written once.  States, products and sums are fp32.
//
// The backward pass needs h_{l-1}.  The forward saves the fp32 state that
// enters every tile of the backward kernel (1/Q of the rows), and the backward
// kernel scans its tile again from there: cheaper than reading h back, and the
// gradient sees unrounded states.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "vec.cuh"

namespace feql {

constexpr int kScanMaxCluster = 8;
constexpr int kScanLanes = 32;  // features per tile at most (TX * V)

struct ScanShape {
  const int *offsets;  // [B + 1] row offsets of packed sequences, or nullptr (dense)
  int64_t N;           // rows of all sequences
  int64_t L;           // rows per sequence (dense)
  int B, F, C, T;
  int FG;              // gates per row: F, or C when shared over the group axis
  int m;               // shared gates: lanes per channel (T / V)
  int FT;              // features per tile
  int ntiles;
  int K;               // blocks per cluster (split of the sequence's rows)
  int Q;               // rows between saved states
};

// Sequence b's rows [s, e), forced into the buffers whatever the offsets hold.
__device__ __forceinline__ void scan_rows(const ScanShape &p, int b, int64_t &s, int64_t &e) {
  if (p.offsets == nullptr) {
    s = b * p.L;
    e = s + p.L;
    return;
  }
  s = p.offsets[b];
  e = p.offsets[b + 1];
  if (s < 0) s = 0;
  if (s > p.N) s = p.N;
  if (e > p.N) e = p.N;
  if (e < s) e = s;
}

// fp32 states of V neighbouring features (F and f are multiples of V).
template <int V>
__device__ __forceinline__ void load_state(const float *p, float (&v)[V]) {
  Pack<float, V> k;
  k.load(p);
  k.unpack(v);
}
template <int V>
__device__ __forceinline__ void store_state(float *p, const float (&v)[V]) {
  Pack<float, V> k;
  k.pack(v);
  k.store(p);
}

// Saved states: sequence b's k-th is row s / Q + b + k of [N / Q + B][F].  The
// ranges of two sequences cannot meet: ceil(len / Q) <= e / Q - s / Q + 1.
__device__ __forceinline__ int64_t scan_save_row(const ScanShape &p, int b, int64_t s, int64_t l) {
  return s / p.Q + b + l / p.Q;
}

// a = sigma(g) and na = 1 - a = sigma(-g), each to full relative precision (a
// subtraction would lose the small one).  fp16 gates: the hardware's exponential
// and division, about 2^-21, far below the rounding of the outputs.
template <typename Ty>
__device__ __forceinline__ void scan_gate(float g, float &a, float &na) {
  const float e = sizeof(Ty) == 2 ? __expf(-fabsf(g)) : expf(-fabsf(g));
  const float big = sizeof(Ty) == 2 ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e);
  const float small = e * big;
  a = g >= 0.f ? big : small;
  na = g >= 0.f ? small : big;
}

__device__ __forceinline__ uint32_t cluster_rank_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Block-wide join of the threads' affine maps, thread (tx, ty) holding rows
// ty R .. of features tx V ..: from the state `carry` that enters the cluster's
// rows, `in` = the state that enters this thread's rows, and carry becomes the
// state after the cluster's last row.  kRev: rows run from high to low (the
// last warp, row group and block come first).  GV: values of A per thread (1
// when the V features share a gate).
template <int V, int NW, int GV>
struct ScanJoin {
  static constexpr int TX = kScanLanes / V;  // lanes along features; V row groups per warp
  // [parity][warp][A | B][feature] and, for clusters, [parity][rank][A | B][feature]
  float warp_tot[2][NW][2][kScanLanes];
  float rank_tot[2][kScanMaxCluster][2][kScanLanes];
};

template <int V, int NW, int GV, bool kRev>
__device__ __forceinline__ void scan_join(ScanJoin<V, NW, GV> &sm, int parity, int K, int rank,
                                          const float (&A)[GV], const float (&Bv)[V],
                                          float (&carry)[V], float (&in)[V]) {
  constexpr int TX = ScanJoin<V, NW, GV>::TX;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tx = lane % TX, ty = lane / TX;  // row group within the warp
  const int pos = kRev ? V - 1 - ty : ty;    // its place in scan order
  // inclusive scan over the warp's row groups
  float ia[GV], ib[V];
#pragma unroll
  for (int j = 0; j < GV; ++j) ia[j] = A[j];
#pragma unroll
  for (int j = 0; j < V; ++j) ib[j] = Bv[j];
#pragma unroll
  for (int o = 1; o < V; o <<= 1) {
    float pa[GV], pb[V];
#pragma unroll
    for (int j = 0; j < GV; ++j)
      pa[j] = kRev ? __shfl_down_sync(0xffffffffu, ia[j], o * TX)
                   : __shfl_up_sync(0xffffffffu, ia[j], o * TX);
#pragma unroll
    for (int j = 0; j < V; ++j)
      pb[j] = kRev ? __shfl_down_sync(0xffffffffu, ib[j], o * TX)
                   : __shfl_up_sync(0xffffffffu, ib[j], o * TX);
    if (pos >= o) {
#pragma unroll
      for (int j = 0; j < V; ++j) ib[j] = fmaf(ia[GV == 1 ? 0 : j], pb[j], ib[j]);
#pragma unroll
      for (int j = 0; j < GV; ++j) ia[j] *= pa[j];
    }
  }
  // exclusive maps within the warp
  float ea[GV], eb[V];
#pragma unroll
  for (int j = 0; j < GV; ++j) {
    ea[j] = 1.f;
    if constexpr (V > 1) {
      const float q = kRev ? __shfl_down_sync(0xffffffffu, ia[j], TX)
                           : __shfl_up_sync(0xffffffffu, ia[j], TX);
      if (pos > 0) ea[j] = q;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    eb[j] = 0.f;
    if constexpr (V > 1) {
      const float q = kRev ? __shfl_down_sync(0xffffffffu, ib[j], TX)
                           : __shfl_up_sync(0xffffffffu, ib[j], TX);
      if (pos > 0) eb[j] = q;
    }
  }
  if (NW == 1 && K == 1) {
    // the warp is the block: its total comes from the last row group's lanes
    const int src = (kRev ? 0 : V - 1) * TX + tx;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      in[j] = fmaf(ea[GV == 1 ? 0 : j], carry[j], eb[j]);
      const float a = ia[GV == 1 ? 0 : j];
      const float ta = V > 1 ? __shfl_sync(0xffffffffu, a, src) : a;
      const float tb = V > 1 ? __shfl_sync(0xffffffffu, ib[j], src) : ib[j];
      carry[j] = fmaf(ta, carry[j], tb);
    }
    return;
  }
  if (pos == V - 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sm.warp_tot[parity][warp][0][tx * V + j] = ia[GV == 1 ? 0 : j];
      sm.warp_tot[parity][warp][1][tx * V + j] = ib[j];
    }
  }
  __syncthreads();
  float c[V];
#pragma unroll
  for (int j = 0; j < V; ++j) c[j] = carry[j];
  if (K > 1) {
    if (threadIdx.x < kScanLanes) {
      float ta = 1.f, tb = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const int w = kRev ? NW - 1 - i : i;
        const float a = sm.warp_tot[parity][w][0][threadIdx.x];
        tb = fmaf(a, tb, sm.warp_tot[parity][w][1][threadIdx.x]);
        ta *= a;
      }
      const uint32_t at = static_cast<uint32_t>(
          __cvta_generic_to_shared(&sm.rank_tot[parity][rank][0][threadIdx.x]));
      for (int r = 0; r < K; ++r) {
        const uint32_t to = cluster_rank_addr(at, r);
        cluster_store(to, ta);
        cluster_store(to + kScanLanes * 4, tb);
      }
    }
    // One barrier per tile: the other parity's buffer takes the next tile's
    // totals, and this one is written again only after the next barrier, which
    // every block reaches with its reads of this tile done.
    cluster_sync();
    for (int i = 0; i < K; ++i) {
      const int r = kRev ? K - 1 - i : i;
      if (r == rank) {
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] = carry[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
        carry[j] = fmaf(sm.rank_tot[parity][r][0][tx * V + j], carry[j],
                        sm.rank_tot[parity][r][1][tx * V + j]);
    }
  }
  float mine[V];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int w = kRev ? NW - 1 - i : i;
    if (w == warp) {
#pragma unroll
      for (int j = 0; j < V; ++j) mine[j] = c[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      c[j] = fmaf(sm.warp_tot[parity][w][0][tx * V + j], c[j],
                  sm.warp_tot[parity][w][1][tx * V + j]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    in[j] = fmaf(ea[GV == 1 ? 0 : j], mine[j], eb[j]);
    if (K == 1) carry[j] = c[j];
  }
}

// Rows that belong to no sequence (before the first offset, behind the last)
// are zeroed in the outputs, so that what consumes them sees numbers: by the
// blocks of the first and of the last sequence, each for its features.
template <typename Ty, int V, int TY>
__device__ __forceinline__ void scan_zero_rest(const ScanShape &p, int b, int rank, int ty,
                                               int64_t s, int64_t e, Ty *out, int width, int col,
                                               bool live) {
  if (p.offsets == nullptr || !live) return;
  Pack<Ty, V> z;
  z.zero();
  const int64_t step = static_cast<int64_t>(p.K) * TY;
  if (b == 0)
    for (int64_t r = static_cast<int64_t>(rank) * TY + ty; r < s; r += step)
      z.store(out + r * width + col);
  if (b == p.B - 1)
    for (int64_t r = e + static_cast<int64_t>(rank) * TY + ty; r < p.N; r += step)
      z.store(out + r * width + col);
}

template <typename Ty, int V, int R, int NW, bool kShared>
__global__ void __launch_bounds__(NW * 32)
scan_fwd_kernel(const Ty *__restrict__ u, const Ty *__restrict__ g, const float *__restrict__ h0,
                Ty *__restrict__ h, float *__restrict__ hN, float *__restrict__ save,
                const ScanShape p) {
  constexpr int GV = kShared ? 1 : V;
  constexpr int TX = kScanLanes / V, TY = NW * V, RT = TY * R;
  __shared__ ScanJoin<V, NW, GV> sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tx = lane % TX, ty = warp * V + lane / TX;
  const int rank = blockIdx.x % p.K, unit = blockIdx.x / p.K;
  const int tile = unit % p.ntiles, b = unit / p.ntiles;
  const int f = tile * p.FT + tx * V;
  const bool live = tx * V < p.FT && f < p.F;
  const int gf = kShared ? f / p.T : f;
  int64_t s, e;
  scan_rows(p, b, s, e);
  const int64_t len = e - s;
  float carry[V] = {};
  if (live && h0 != nullptr) load_state<V>(h0 + static_cast<int64_t>(b) * p.F + f, carry);
  int parity = 0;
  for (int64_t base = 0; base < len; base += static_cast<int64_t>(p.K) * RT, parity ^= 1) {
    const int64_t l0 = base + rank * RT + ty * R;
    Pack<Ty, V> ru[R];
    Pack<Ty, GV> rg[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (live && l0 + r < len) {
        ru[r].load(u + (s + l0 + r) * p.F + f);
        rg[r].load(g + (s + l0 + r) * p.FG + gf);
      }
    // local states from a zero state, and prefix products
    float P[R][GV], hl[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float a[GV], na[GV], uv[V];
      if (live && l0 + r < len) {
        float gv[GV];
        rg[r].unpack(gv);
        ru[r].unpack(uv);
#pragma unroll
        for (int j = 0; j < GV; ++j) scan_gate<Ty>(gv[j], a[j], na[j]);
      } else {
#pragma unroll
        for (int j = 0; j < GV; ++j) { a[j] = 1.f; na[j] = 0.f; }
#pragma unroll
        for (int j = 0; j < V; ++j) uv[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < GV; ++j) P[r][j] = r == 0 ? a[j] : a[j] * P[r == 0 ? 0 : r - 1][j];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int q = GV == 1 ? 0 : j;
        hl[r][j] = r == 0 ? na[q] * uv[j] : fmaf(a[q], hl[r == 0 ? 0 : r - 1][j], na[q] * uv[j]);
      }
    }
    float in[V];
    scan_join<V, NW, GV, false>(sm, parity, p.K, rank, P[R - 1], hl[R - 1], carry, in);
    if (live && l0 < len) {
      if (save != nullptr && l0 % p.Q == 0)
        store_state<V>(save + scan_save_row(p, b, s, l0) * p.F + f, in);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (l0 + r < len) {
          float o[V];
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = fmaf(P[r][GV == 1 ? 0 : j], in[j], hl[r][j]);
          Pack<Ty, V> k;
          k.pack(o);
          k.store(h + (s + l0 + r) * p.F + f);
        }
    }
  }
  scan_zero_rest<Ty, V, TY>(p, b, rank, ty, s, e, h, p.F, f, live);
  if (hN != nullptr && live && rank == 0 && ty == 0)
    store_state<V>(hN + static_cast<int64_t>(b) * p.F + f, carry);
}

template <typename Ty, int V, int R, int NW, bool kShared>
__global__ void __launch_bounds__(NW * 32)
scan_bwd_kernel(const Ty *__restrict__ dh, const Ty *__restrict__ u, const Ty *__restrict__ g,
                const float *__restrict__ save, const float *__restrict__ dhN,
                Ty *__restrict__ du, Ty *__restrict__ dg, float *__restrict__ dh0,
                const ScanShape p) {
  constexpr int GV = kShared ? 1 : V;
  constexpr int TX = kScanLanes / V, TY = NW * V, RT = TY * R;
  __shared__ ScanJoin<V, NW, GV> sf, sr;  // the states (forward) and the gradient (reverse)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tx = lane % TX, ty = warp * V + lane / TX;
  const int rank = blockIdx.x % p.K, unit = blockIdx.x / p.K;
  const int tile = unit % p.ntiles, b = unit / p.ntiles;
  const int f = tile * p.FT + tx * V;
  const bool live = tx * V < p.FT && f < p.F;
  const int gf = kShared ? f / p.T : f;
  int64_t s, e;
  scan_rows(p, b, s, e);
  const int64_t len = e - s;
  float carry[V] = {};
  if (live && dhN != nullptr) load_state<V>(dhN + static_cast<int64_t>(b) * p.F + f, carry);
  const int64_t step = static_cast<int64_t>(p.K) * RT;
  int parity = 0;
  for (int64_t base = len > 0 ? (len - 1) / step * step : -1; base >= 0;
       base -= step, parity ^= 1) {
    const int64_t t0 = base + rank * RT;  // the block's first row (a multiple of Q = RT)
    const int64_t l0 = t0 + ty * R;
    Pack<Ty, V> ru[R], rd[R];
    Pack<Ty, GV> rg[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (live && l0 + r < len) {
        ru[r].load(u + (s + l0 + r) * p.F + f);
        rd[r].load(dh + (s + l0 + r) * p.F + f);
        rg[r].load(g + (s + l0 + r) * p.FG + gf);
      }
    float state[V] = {};  // the state that enters the block's rows
    if (live && t0 < len) load_state<V>(save + scan_save_row(p, b, s, t0) * p.F + f, state);
    float a[R][GV], na[R][GV], P[R][GV], hl[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float uv[V];
      if (live && l0 + r < len) {
        float gv[GV];
        rg[r].unpack(gv);
        ru[r].unpack(uv);
#pragma unroll
        for (int j = 0; j < GV; ++j) scan_gate<Ty>(gv[j], a[r][j], na[r][j]);
      } else {
#pragma unroll
        for (int j = 0; j < GV; ++j) { a[r][j] = 1.f; na[r][j] = 0.f; }
#pragma unroll
        for (int j = 0; j < V; ++j) uv[j] = 0.f;
        rd[r].zero();
      }
#pragma unroll
      for (int j = 0; j < GV; ++j)
        P[r][j] = r == 0 ? a[r][j] : a[r][j] * P[r == 0 ? 0 : r - 1][j];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int q = GV == 1 ? 0 : j;
        hl[r][j] = r == 0 ? na[r][q] * uv[j]
                          : fmaf(a[r][q], hl[r == 0 ? 0 : r - 1][j], na[r][q] * uv[j]);
      }
    }
    float Bc[V], in[V], cin[V];
#pragma unroll
    for (int j = 0; j < V; ++j) Bc[j] = 0.f;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float d[V];
      rd[r].unpack(d);
#pragma unroll
      for (int j = 0; j < V; ++j) Bc[j] = a[r][GV == 1 ? 0 : j] * (d[j] + Bc[j]);
    }
    scan_join<V, NW, GV, false>(sf, parity, 1, 0, P[R - 1], hl[R - 1], state, in);
    scan_join<V, NW, GV, true>(sr, parity, p.K, rank, P[R - 1], Bc, carry, cin);
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float d[V], uv[V], o[V], gsum = 0.f, og[GV];
      rd[r].unpack(d);
      const bool row = live && l0 + r < len;
      if (row) {
        ru[r].unpack(uv);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) uv[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int q = GV == 1 ? 0 : j;
        const int b4 = r == 0 ? 0 : r - 1;
        const float before = r == 0 ? in[j] : fmaf(P[b4][q], in[j], hl[b4][j]);
        const float delta = d[j] + cin[j];
        o[j] = na[r][q] * delta;
        cin[j] = a[r][q] * delta;
        const float gg = cin[j] * na[r][q] * (before - uv[j]);
        if (kShared) gsum += gg;
        else og[q] = gg;
      }
      if constexpr (kShared) {
        // a channel's T features sit in m neighbouring lanes
        float sum = gsum;
        for (int k = 1; k < p.m; ++k) sum += __shfl_down_sync(0xffffffffu, gsum, k);
        og[0] = sum;
      }
      if (row) {
        Pack<Ty, V> k;
        k.pack(o);
        k.store(du + (s + l0 + r) * p.F + f);
        Pack<Ty, GV> kg;
        kg.pack(og);
        if (!kShared || tx % p.m == 0) kg.store(dg + (s + l0 + r) * p.FG + gf);
      }
    }
  }
  scan_zero_rest<Ty, V, TY>(p, b, rank, ty, s, e, du, p.F, f, live);
  scan_zero_rest<Ty, GV, TY>(p, b, rank, ty, s, e, dg, p.FG, gf,
                             live && (!kShared || tx % p.m == 0));
  if (dh0 != nullptr && live && rank == 0 && ty == 0)
    store_state<V>(dh0 + static_cast<int64_t>(b) * p.F + f, carry);
}

// One token of each of B sequences: h = a h + (1 - a) u on the fp32 states in
// place, and the new state rounded to the data type.  Latency-bound: one value
// per thread, one launch.
template <typename Ty>
__global__ void __launch_bounds__(256)
scan_step_kernel(const Ty *__restrict__ u, const Ty *__restrict__ g, float *__restrict__ state,
                 Ty *__restrict__ h, int64_t n, int T) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
    float a, na;
    scan_gate<Ty>(widen(g[i / T]), a, na);  // T = 1 for a gate per (c, t)
    const float v = fmaf(a, state[i], na * widen(u[i]));
    state[i] = v;
    h[i] = narrow<Ty>(v);
  }
}

}  // namespace feql
