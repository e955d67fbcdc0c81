// feql_ops.cu — C ABI of the operators that stand around the layer: layer norm
// (feql_norm_*) and the gated linear recurrence (feql_scan_*), declared in
// include/feql.h.  Host side only: argument checks, plans and launches.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/feql.h"
#include "host.cuh"
#include "norm.cuh"
#include "scan.cuh"

using namespace feql;

namespace {

constexpr int kMaxOrder = 16;  // group orders T of the feature layout

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool ok_ptr(const void *p, bool needed) { return p == nullptr ? !needed : aligned16(p); }

// ------------------------------------------------------------------- norm
struct NormPlan {
  int V, A, K, threads;
  bool in_regs;  // a row fits the registers of one row group
  NormShape s;
};

// The variants of 16-byte packs per thread that keep out of local memory: eight
// in the forward, four of fp16 in the backward, only where channels' parameters
// and sums are shared by four values.
constexpr bool norm_has(int V, int K, int A, bool half, bool bwd) {
  const bool wide = V == (half ? 8 : 4);
  if (!wide) return K == 2 || (K == 8 && !(bwd && V == 4 && A == 1));
  if (K == 8) return !bwd && A == 4;
  if (K == 4) return !(bwd && half && A == 1);
  return K >= 1 && K <= 3;
}

// Packs: the widest of 16 bytes or less that divides a row, so that every row
// starts on a pack.  Row groups: the (K, G) with the fewest idle slots; on
// ties, four packs per thread (fewer shuffles per value, 64 bytes in flight).
// Narrow packs serve odd row lengths; they get fewer variants.
NormPlan norm_plan(int64_t N, int C, int T, bool half, bool bwd) {
  NormPlan q;
  const int F = C * T;
  q.V = half ? 8 : 4;
  const int wide = q.V;
  while (F % q.V != 0) q.V /= 2;
  // neighbours that share a channel's parameters and sums
  q.A = T % 4 == 0 && q.V % 4 == 0 ? 4 : (T % 2 == 0 && q.V % 2 == 0 ? 2 : 1);
  q.s = {N, C, T, F, 0, F / q.V};
  static const int wide_ks[] = {4, 2, 3, 1, 8}, narrow_ks[] = {8, 2};
  const int *ks = q.V == wide ? wide_ks : narrow_ks;
  const int nk = q.V == wide ? 5 : 2;
  q.in_regs = false;
  int best = 0;
  for (int i = 0; i < nk; ++i) {
    if (!norm_has(q.V, ks[i], q.A, half, bwd)) continue;
    int G = 1;
    while (G * ks[i] < q.s.nchunk && G <= kNormMaxThreads) G *= 2;
    if (G > kNormMaxThreads) continue;
    const int cost = G * ks[i] * (G > 32 ? 5 : 4);  // a group of several warps meets at barriers
    if (!q.in_regs || cost < best) {
      q.in_regs = true;
      best = cost;
      q.K = ks[i];
      q.s.G = G;
    }
  }
  if (!q.in_regs) q.s.G = kNormLongThreads;
  q.threads = q.in_regs ? (q.s.G > 32 ? q.s.G : kNormThreads) : kNormLongThreads;
  return q;
}

// Blocks of the row loop: what the SMs hold at 64 registers a thread.
int norm_blocks(const NormPlan &q, int sms) {
  const int64_t want = q.in_regs ? ceil_div(q.s.N, q.threads / q.s.G) : q.s.N;
  const int64_t cap = static_cast<int64_t>(sms) * (1024 / q.threads);
  return static_cast<int>(want < cap ? want : cap);
}

constexpr int64_t kNormLongRows = 64;  // rows of a split of the long rows' column pass
int64_t norm_long_splits(int64_t N) {
  const int64_t n = ceil_div(N, kNormLongRows);
  return n < 32 ? n : 32;
}

#define FEQL_NORM_WIDE(X, Ty, V, A) \
  X(Ty, V, 1, A) X(Ty, V, 2, A) X(Ty, V, 3, A) X(Ty, V, 4, A) X(Ty, V, 8, A)
#define FEQL_NORM_NARROW(X, Ty, V, A) X(Ty, V, 2, A) X(Ty, V, 8, A)
#define FEQL_NORM_HALF(X)                                                                \
  FEQL_NORM_WIDE(X, __half, 8, 1) FEQL_NORM_WIDE(X, __half, 8, 2)                        \
  FEQL_NORM_WIDE(X, __half, 8, 4)                                                        \
  FEQL_NORM_NARROW(X, __half, 4, 1) FEQL_NORM_NARROW(X, __half, 4, 2)                    \
  FEQL_NORM_NARROW(X, __half, 4, 4)                                                      \
  FEQL_NORM_NARROW(X, __half, 2, 1) FEQL_NORM_NARROW(X, __half, 2, 2)                    \
  FEQL_NORM_NARROW(X, __half, 1, 1)
#define FEQL_NORM_FLOAT(X)                                                               \
  FEQL_NORM_WIDE(X, float, 4, 1) FEQL_NORM_WIDE(X, float, 4, 2)                          \
  FEQL_NORM_WIDE(X, float, 4, 4)                                                         \
  FEQL_NORM_NARROW(X, float, 2, 1) FEQL_NORM_NARROW(X, float, 2, 2)                      \
  FEQL_NORM_NARROW(X, float, 1, 1)

int norm_fwd_launch(const NormPlan &q, bool half, const void *x, const void *gamma,
                    const void *beta, void *y, float2 *stats, float eps, int grid,
                    cudaStream_t st) {
#define FEQL_CASE(Ty, VV, KK, AA)                                                             \
  if constexpr (norm_has(VV, KK, AA, sizeof(Ty) == 2, false))                                 \
  if (q.V == VV && q.K == KK && q.A == AA) {                                                  \
    norm_fwd_kernel<Ty, VV, KK, AA><<<grid, q.threads, 0, st>>>(                              \
        static_cast<const Ty *>(x), static_cast<const Ty *>(gamma),                           \
        static_cast<const Ty *>(beta), static_cast<Ty *>(y), stats, q.s, eps);                \
    return launch_status();                                                                   \
  }
  if (half) {
    FEQL_NORM_HALF(FEQL_CASE)
  } else {
    FEQL_NORM_FLOAT(FEQL_CASE)
  }
#undef FEQL_CASE
  return FEQL_ERR_UNSUPPORTED;
}

int norm_bwd_launch(const NormPlan &q, bool half, const void *x, const void *dy,
                    const void *gamma, const float2 *stats, void *dx, float *part, int grid,
                    cudaStream_t st) {
#define FEQL_CASE(Ty, VV, KK, AA)                                                             \
  if constexpr (norm_has(VV, KK, AA, sizeof(Ty) == 2, true))                                  \
  if (q.V == VV && q.K == KK && q.A == AA) {                                                  \
    norm_bwd_kernel<Ty, VV, KK, AA><<<grid, q.threads, 0, st>>>(                              \
        static_cast<const Ty *>(x), static_cast<const Ty *>(dy),                              \
        static_cast<const Ty *>(gamma), stats, static_cast<Ty *>(dx), part, q.s);             \
    return launch_status();                                                                   \
  }
  if (half) {
    FEQL_NORM_HALF(FEQL_CASE)
  } else {
    FEQL_NORM_FLOAT(FEQL_CASE)
  }
#undef FEQL_CASE
  return FEQL_ERR_UNSUPPORTED;
}

template <typename Ty>
int norm_bwd_long(const NormPlan &q, const void *x, const void *dy, const void *gamma,
                  const float2 *stats, void *dx, float *part, int grid, cudaStream_t st) {
  const Ty *xt = static_cast<const Ty *>(x), *dt = static_cast<const Ty *>(dy);
  norm_dx_long_kernel<Ty><<<grid, kNormLongThreads, 0, st>>>(
      xt, dt, static_cast<const Ty *>(gamma), stats, static_cast<Ty *>(dx), q.s);
  const int64_t splits = norm_long_splits(q.s.N);
  dim3 cols(static_cast<unsigned>(ceil_div(q.s.F, kNormThreads)), static_cast<unsigned>(splits));
  norm_cols_long_kernel<Ty><<<cols, kNormThreads, 0, st>>>(xt, dt, stats, part, q.s,
                                                          ceil_div(q.s.N, splits));
  return launch_status();
}

template <typename Ty>
int norm_reduce(const float *part, void *dgamma, void *dbeta, int C, int m, int blocks,
                cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(C, 32 / m)));
  cfg.blockDim = dim3(32 * kNormRedLanes);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, norm_reduce_kernel<Ty>, part, static_cast<Ty *>(dgamma),
                            static_cast<Ty *>(dbeta), C, m, blocks) == cudaSuccess
             ? FEQL_OK
             : FEQL_ERR_CUDA;
}

int norm_check(int64_t N, int C, int T, int dtype) {
  if (!valid_dtype(dtype) || N < 0 || N > kMaxTokens || check_shape(C, 1) != FEQL_OK)
    return FEQL_ERR_INVALID_ARG;
  if (T < 1 || T > kMaxOrder) return FEQL_ERR_UNSUPPORTED;
  return FEQL_OK;
}

// ------------------------------------------------------------------- scan
struct ScanPlan {
  int V, TX, NW;
  ScanShape s;
};

// Rows per thread: what keeps the values in use within 128 registers, so that
// two blocks of 256 threads share an SM.
constexpr int scan_rows_fwd(bool half, int V) { return V == 4 && !half ? 4 : 8; }
constexpr int scan_rows_bwd(bool half, int V) { return half ? (V == 4 ? 4 : 8) : 8 / V; }

// A thread's features are V neighbours: 4, or fewer where a row (or, for
// shared gates, a channel) is not a multiple of 4.  One warp per block walks
// a sequence by itself when there are enough (sequence, tile) units to fill
// the GPU with warps or the sequences are short; else eight warps share a
// tile of rows.  (Six warps and 96 registers, for three blocks per SM, were
// measured: no faster.)  Then
// sequences are cut into segments where whole ones would leave SMs idle: dense
// sequences when not every SM gets a unit, packed ones (whose longest the host
// does not know) always, in segments of an even share for two blocks (16 of one
// warp) per SM, two (16) tiles at least.
ScanPlan scan_plan(int B, int64_t N, int C, int T, bool shared, bool packed, bool half, bool bwd,
                   int sms) {
  ScanPlan q;
  const int F = C * T;
  const bool sh = shared && T > 1;
  const int unit = sh ? T : F;
  q.V = unit % 4 == 0 ? 4 : (unit % 2 == 0 ? 2 : 1);
  q.s.offsets = nullptr;
  q.s.N = N;
  q.s.L = B > 0 ? N / B : 0;
  q.s.B = B;
  q.s.F = F;
  q.s.C = C;
  q.s.T = T;
  q.s.FG = shared ? C : F;
  q.s.m = sh ? T / q.V : 1;
  // lanes along features: 32 features to a tile, or 64 where hardly a lane stays
  // idle (rows of 128 bytes: half the cache lines per byte, fewer groups to join)
  q.TX = 32 / q.V;
  if (q.V == 4 && ceil_div(F, 64) * 64 * 8 <= 9 * F && (!sh || 64 % T == 0)) q.TX = 16;
  const int most = q.TX * q.V;
  q.s.FT = sh ? most / T * T : most;
  q.s.ntiles = static_cast<int>(ceil_div(F, q.s.FT));
  const int64_t units = static_cast<int64_t>(B) * q.s.ntiles;
  const int64_t avg = B > 0 ? ceil_div(N, B) : 0;
  const int warp_rows = 32 / q.TX * (bwd ? scan_rows_bwd(half, q.V) : scan_rows_fwd(half, q.V));
  q.NW = (units >= 16ll * sms || avg <= 64) ? 1 : 8;
  const int tile = q.NW * warp_rows;
  q.s.seg_rows = 0;
  if (packed || (q.NW == 8 && units < sms)) {
    const int64_t blocks = static_cast<int64_t>(sms) * (q.NW == 8 ? 2 : 16);
    const int64_t share = ceil_div(ceil_div(N * q.s.ntiles, blocks), tile) * tile;
    const int64_t least = q.NW == 8 ? 2 * tile : 16 * tile;
    const int64_t rows = share > least ? share : least;
    if (rows < (packed ? N : q.s.L)) q.s.seg_rows = rows;
  }
  q.s.whole = 0;
  q.s.per = 1;
  // Dense sequences that fill the GPU once or twice and then less than half of it:
  // those of the last round are cut.  128 x 3136 x 24 x 4 backward, 384 units of which
  // 296 run at a time: 85 us, 92 with whole ones; 50 x 3000 x 96 x 4 fp32 forward 136 and
  // 215.  Where the rest is near half a round it can cost a little: 128 x 3136 x 24 x 4
  // forward with a gate per value 71 and 66.
  const int64_t cap = static_cast<int64_t>(sms) * scan_blocks(8, !bwd && sh && q.V > 1);
  if (!packed && q.NW == 8 && units > cap && units < 3 * cap) {
    const int64_t whole = units / cap * cap / q.s.ntiles, rest = (B - whole) * q.s.ntiles;
    if (rest > 0 && 2 * rest <= cap) {
      const int64_t part = ceil_div(ceil_div(q.s.L, cap / rest), tile) * tile;
      const int64_t rows = part > 2 * tile ? part : 2 * tile;
      if (rows < q.s.L) {
        q.s.seg_rows = rows;
        q.s.whole = static_cast<int>(whole);
      }
    }
  }
  if (!packed && q.s.seg_rows != 0) q.s.per = static_cast<int>(ceil_div(q.s.L, q.s.seg_rows));
  q.s.slots = q.s.seg_rows == 0 ? B
              : packed          ? N / q.s.seg_rows + B
                                : q.s.whole + static_cast<int64_t>(B - q.s.whole) * q.s.per;
  q.s.maps = nullptr;
  return q;
}

size_t scan_maps_bytes(const ScanPlan &q) {
  if (q.s.seg_rows == 0) return 0;
  return static_cast<size_t>(q.s.slots) * q.s.ntiles * 2 * q.TX * q.V * 4;
}

// The main kernel, as the programmatic dependent of the maps' kernel where
// there is one: its first loads need nothing of it.
template <typename... Args>
int scan_launch(void (*kernel)(Args...), const ScanPlan &q, int smem, cudaStream_t st,
                Args... args) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return FEQL_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = q.s.seg_rows != 0 ? 1 : 0;
  cfg.gridDim = dim3(static_cast<unsigned>(q.s.slots * q.s.ntiles));
  cfg.blockDim = dim3(static_cast<unsigned>(q.NW * 32));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FEQL_OK : FEQL_ERR_CUDA;
}

template <typename Ty, int V, int TX, bool kShared, bool kRev>
int scan_maps(const ScanPlan &q, const Ty *x, const Ty *g, cudaStream_t st) {
  if (q.s.seg_rows == 0) return FEQL_OK;
  const unsigned grid = static_cast<unsigned>((q.s.slots - q.s.whole) * q.s.ntiles);
  scan_maps_kernel<Ty, V, TX, 8, kShared, kRev><<<grid, 256, 0, st>>>(x, g, q.s);
  return launch_status();
}

#define FEQL_SCAN_CASES(X, Ty) \
  X(Ty, 4, 16, 8, true) X(Ty, 4, 16, 8, false) X(Ty, 4, 16, 1, true) X(Ty, 4, 16, 1, false) \
  X(Ty, 4, 8, 8, true) X(Ty, 4, 8, 8, false) X(Ty, 4, 8, 1, true) X(Ty, 4, 8, 1, false) \
  X(Ty, 2, 16, 8, true) X(Ty, 2, 16, 8, false) X(Ty, 2, 16, 1, true) X(Ty, 2, 16, 1, false) \
  X(Ty, 1, 32, 8, true) X(Ty, 1, 32, 8, false) X(Ty, 1, 32, 1, true) X(Ty, 1, 32, 1, false)

template <typename Ty, int V, int TX, int NW, bool kShared>
int scan_fwd_run(const ScanPlan &q, const Ty *u, const Ty *g, const float *h0, Ty *h, float *hN,
                 float *diff, cudaStream_t st) {
  constexpr int R = scan_rows_fwd(sizeof(Ty) == 2, V);
  const int bad = scan_maps<Ty, V, TX, kShared, false>(q, u, g, st);
  if (bad != FEQL_OK) return bad;
  auto kernel = scan_fwd_kernel<Ty, V, TX, R, NW, kShared, false>;
  if constexpr (sizeof(Ty) == 2)
    if (diff != nullptr) kernel = scan_fwd_kernel<Ty, V, TX, R, NW, kShared, true>;
  return scan_launch(kernel, q, scan_feed_bytes<Ty, V, R, NW, kShared>(1, false), st, u, g, h0, h,
                     hN, diff, q.s);
}

template <typename Ty, int V, int TX, int NW, bool kShared>
int scan_bwd_run(const ScanPlan &q, const Ty *dh, const Ty *u, const Ty *g, const Ty *h,
                 const float *h0, const float *diff, const float *dhN, Ty *du, Ty *dg, float *dh0,
                 cudaStream_t st) {
  constexpr int R = scan_rows_bwd(sizeof(Ty) == 2, V);
  constexpr bool kDiff = sizeof(Ty) == 2;
  const int bad = scan_maps<Ty, V, TX, kShared, true>(q, dh, g, st);
  if (bad != FEQL_OK) return bad;
  return scan_launch(scan_bwd_kernel<Ty, V, TX, R, NW, kShared, kDiff>, q,
                     scan_feed_bytes<Ty, V, R, NW, kShared>(kDiff ? 1 : 3, kDiff), st, dh, u, g, h,
                     h0, diff, dhN, du, dg, dh0, q.s);
}

template <typename Ty>
int scan_fwd(const ScanPlan &q, const void *u, const void *g, const float *h0, void *h, float *hN,
             float *diff, cudaStream_t st) {
  const bool sh = q.s.FG != q.s.F;
#define FEQL_CASE(T_, VV, XX, NWW, SH)                                               \
  if (q.V == VV && q.TX == XX && q.NW == NWW && sh == SH)                            \
    return scan_fwd_run<T_, VV, XX, NWW, SH>(q, static_cast<const T_ *>(u),          \
                                             static_cast<const T_ *>(g), h0,         \
                                             static_cast<T_ *>(h), hN, diff, st);
  FEQL_SCAN_CASES(FEQL_CASE, Ty)
#undef FEQL_CASE
  return FEQL_ERR_UNSUPPORTED;
}

template <typename Ty>
int scan_bwd(const ScanPlan &q, const void *dh, const void *u, const void *g, const void *h,
             const float *h0, const float *diff, const float *dhN, void *du, void *dg, float *dh0,
             cudaStream_t st) {
  const bool sh = q.s.FG != q.s.F;
#define FEQL_CASE(T_, VV, XX, NWW, SH)                                                          \
  if (q.V == VV && q.TX == XX && q.NW == NWW && sh == SH)                                       \
    return scan_bwd_run<T_, VV, XX, NWW, SH>(                                                   \
        q, static_cast<const T_ *>(dh), static_cast<const T_ *>(u), static_cast<const T_ *>(g), \
        static_cast<const T_ *>(h), h0, diff, dhN, static_cast<T_ *>(du),                       \
        static_cast<T_ *>(dg), dh0, st);
  FEQL_SCAN_CASES(FEQL_CASE, Ty)
#undef FEQL_CASE
  return FEQL_ERR_UNSUPPORTED;
}

int scan_check(int64_t B, int64_t N, int C, int T, int dtype, bool packed) {
  if (!valid_dtype(dtype) || B < 0 || B > kMaxTokens || N < 0 || N > kMaxTokens ||
      check_shape(C, 1) != FEQL_OK)
    return FEQL_ERR_INVALID_ARG;
  if (B == 0 ? N != 0 : (!packed && N % B != 0)) return FEQL_ERR_INVALID_ARG;
  if (T < 1 || T > kMaxOrder) return FEQL_ERR_UNSUPPORTED;
  return FEQL_OK;
}

}  // namespace

extern "C" {

int feql_norm_forward(const void *x, const void *gamma, const void *beta, void *y, float *stats,
                      int64_t N, int C, int T, float eps, int dtype, feql_stream stream) {
  const int bad = norm_check(N, C, T, dtype);
  if (bad != FEQL_OK) return bad;
  if (!(eps > 0.f) || isinf(eps)) return FEQL_ERR_INVALID_ARG;
  if (!ok_ptr(x, N > 0) || !ok_ptr(y, N > 0) || !ok_ptr(gamma, false) || !ok_ptr(beta, false) ||
      !ok_ptr(stats, false))
    return FEQL_ERR_INVALID_ARG;
  if (N == 0) return FEQL_OK;
  DeviceInfo dev;
  const int st = device_info(&dev);
  if (st != FEQL_OK) return st;
  const bool half = is_half(dtype);
  const NormPlan q = norm_plan(N, C, T, half, false);
  const int grid = norm_blocks(q, dev.sms);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float2 *sp = reinterpret_cast<float2 *>(stats);
  if (q.in_regs) return norm_fwd_launch(q, half, x, gamma, beta, y, sp, eps, grid, s);
  if (half)
    norm_fwd_long_kernel<__half><<<grid, kNormLongThreads, 0, s>>>(
        static_cast<const __half *>(x), static_cast<const __half *>(gamma),
        static_cast<const __half *>(beta), static_cast<__half *>(y), sp, q.s, eps);
  else
    norm_fwd_long_kernel<float><<<grid, kNormLongThreads, 0, s>>>(
        static_cast<const float *>(x), static_cast<const float *>(gamma),
        static_cast<const float *>(beta), static_cast<float *>(y), sp, q.s, eps);
  return launch_status();
}

size_t feql_norm_backward_workspace_bytes(int64_t N, int C, int T, int dtype) {
  if (norm_check(N, C, T, dtype) != FEQL_OK) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != FEQL_OK) return 0;
  const NormPlan q = norm_plan(N, C, T, is_half(dtype), true);
  const int64_t rows = q.in_regs ? norm_blocks(q, dev.sms) : norm_long_splits(N);
  const size_t bytes = static_cast<size_t>(rows) * 2 * (q.s.F / (q.in_regs ? q.A : 1)) * 4;
  return bytes > 16 ? bytes : 16;
}

int feql_norm_backward(const void *x, const void *dy, const float *stats, const void *gamma,
                       void *dx, void *dgamma, void *dbeta, void *ws, size_t ws_bytes, int64_t N,
                       int C, int T, int dtype, feql_stream stream) {
  const int bad = norm_check(N, C, T, dtype);
  if (bad != FEQL_OK) return bad;
  if (!ok_ptr(x, N > 0) || !ok_ptr(dy, N > 0) || !ok_ptr(stats, N > 0) || !ok_ptr(dx, N > 0) ||
      !ok_ptr(gamma, false) || !ok_ptr(dgamma, false) || !ok_ptr(dbeta, false) || !ok_ptr(ws, true))
    return FEQL_ERR_INVALID_ARG;
  if (ws_bytes < feql_norm_backward_workspace_bytes(N, C, T, dtype)) return FEQL_ERR_INVALID_ARG;
  DeviceInfo dev;
  int st = device_info(&dev);
  if (st != FEQL_OK) return st;
  const bool half = is_half(dtype);
  const NormPlan q = norm_plan(N, C, T, half, true);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const float2 *sp = reinterpret_cast<const float2 *>(stats);
  float *part = static_cast<float *>(ws);
  int rows = 0;  // partial rows to add
  if (N > 0) {
    const int grid = norm_blocks(q, dev.sms);
    rows = q.in_regs ? grid : static_cast<int>(norm_long_splits(N));
    if (q.in_regs)
      st = norm_bwd_launch(q, half, x, dy, gamma, sp, dx, part, grid, s);
    else
      st = half ? norm_bwd_long<__half>(q, x, dy, gamma, sp, dx, part, grid, s)
                : norm_bwd_long<float>(q, x, dy, gamma, sp, dx, part, grid, s);
    if (st != FEQL_OK) return st;
  }
  if (dgamma == nullptr && dbeta == nullptr) return FEQL_OK;
  const int m = q.in_regs ? T / q.A : T;
  return half ? norm_reduce<__half>(part, dgamma, dbeta, C, m, rows, s)
              : norm_reduce<float>(part, dgamma, dbeta, C, m, rows, s);
}

size_t feql_scan_workspace_bytes(int64_t B, int64_t N, int C, int T, int shared, int packed_rows,
                                 int dtype) {
  const bool packed = packed_rows != 0;
  if (scan_check(B, N, C, T, dtype, true) != FEQL_OK) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != FEQL_OK) return 0;
  size_t most = 16;
  for (bool bwd : {false, true}) {
    const size_t bytes = scan_maps_bytes(
        scan_plan(static_cast<int>(B), N, C, T, shared != 0, packed, is_half(dtype), bwd, dev.sms));
    if (bytes > most) most = bytes;
  }
  return most;
}

// The checked plan of a call: FEQL_OK and the plan, or what to return.
static int scan_prepare(int64_t B, int64_t N, int C, int T, int shared, int dtype,
                        const int32_t *offsets, bool bwd, void *ws, size_t ws_bytes, ScanPlan *q) {
  DeviceInfo dev;
  const int st = device_info(&dev);
  if (st != FEQL_OK) return st;
  const bool packed = offsets != nullptr;
  *q = scan_plan(static_cast<int>(B), N, C, T, shared != 0, packed, is_half(dtype), bwd, dev.sms);
  if (q->s.slots * q->s.ntiles > INT32_MAX) return FEQL_ERR_UNSUPPORTED;
  if (q->s.seg_rows != 0 && (ws == nullptr || ws_bytes < scan_maps_bytes(*q)))
    return FEQL_ERR_INVALID_ARG;
  q->s.offsets = offsets;
  q->s.maps = static_cast<float *>(ws);
  return FEQL_OK;
}

static int scan_forward(const void *u, const void *g, const float *h0, const int32_t *offsets,
                        void *h, float *hN, float *diff, void *ws, size_t ws_bytes, int64_t B,
                        int64_t N, int C, int T, int shared, int dtype, feql_stream stream) {
  const int bad = scan_check(B, N, C, T, dtype, offsets != nullptr);
  if (bad != FEQL_OK) return bad;
  if (!ok_ptr(u, N > 0) || !ok_ptr(g, N > 0) || !ok_ptr(h, N > 0) || !ok_ptr(h0, false) ||
      !ok_ptr(hN, false) || !ok_ptr(offsets, false) || !ok_ptr(ws, false))
    return FEQL_ERR_INVALID_ARG;
  if (B == 0) return FEQL_OK;
  ScanPlan q;
  const int st = scan_prepare(B, N, C, T, shared, dtype, offsets, false, ws, ws_bytes, &q);
  if (st != FEQL_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return is_half(dtype) ? scan_fwd<__half>(q, u, g, h0, h, hN, diff, s)
                        : scan_fwd<float>(q, u, g, h0, h, hN, nullptr, s);
}

int feql_scan_forward(const void *u, const void *g, const float *h0, const int32_t *offsets,
                      void *h, float *hN, void *ws, size_t ws_bytes, int64_t B, int64_t N, int C,
                      int T, int shared, int dtype, feql_stream stream) {
  return scan_forward(u, g, h0, offsets, h, hN, nullptr, ws, ws_bytes, B, N, C, T, shared, dtype,
                      stream);
}

int feql_scan_forward_diff(const void *u, const void *g, const float *h0, const int32_t *offsets,
                           void *h, float *hN, float *diff, void *ws, size_t ws_bytes, int64_t B,
                           int64_t N, int C, int T, int shared, int dtype, feql_stream stream) {
  if (!valid_dtype(dtype) || !ok_ptr(diff, N > 0)) return FEQL_ERR_INVALID_ARG;
  if (!is_half(dtype)) return FEQL_ERR_UNSUPPORTED;
  return scan_forward(u, g, h0, offsets, h, hN, diff, ws, ws_bytes, B, N, C, T, shared, dtype,
                      stream);
}

int feql_scan_backward(const void *dh, const void *u, const void *g, const void *h,
                       const float *h0, const float *dhN, const int32_t *offsets, void *du,
                       void *dg, float *dh0, void *ws, size_t ws_bytes, int64_t B, int64_t N,
                       int C, int T, int shared, int dtype, feql_stream stream) {
  const int bad = scan_check(B, N, C, T, dtype, offsets != nullptr);
  if (bad != FEQL_OK) return bad;
  if (!ok_ptr(dh, N > 0) || !ok_ptr(u, N > 0) || !ok_ptr(g, N > 0) || !ok_ptr(h, N > 0) ||
      !ok_ptr(du, N > 0) || !ok_ptr(dg, N > 0) || !ok_ptr(h0, false) || !ok_ptr(dhN, false) ||
      !ok_ptr(dh0, false) || !ok_ptr(offsets, false) || !ok_ptr(ws, false))
    return FEQL_ERR_INVALID_ARG;
  if (is_half(dtype)) return FEQL_ERR_UNSUPPORTED;
  if (B == 0) return FEQL_OK;
  ScanPlan q;
  const int st = scan_prepare(B, N, C, T, shared, dtype, offsets, true, ws, ws_bytes, &q);
  if (st != FEQL_OK) return st;
  return scan_bwd<float>(q, dh, u, g, h, h0, nullptr, dhN, du, dg, dh0,
                         reinterpret_cast<cudaStream_t>(stream));
}

int feql_scan_backward_diff(const void *dh, const void *g, const float *diff, const float *dhN,
                            const int32_t *offsets, void *du, void *dg, float *dh0, void *ws,
                            size_t ws_bytes, int64_t B, int64_t N, int C, int T, int shared,
                            int dtype, feql_stream stream) {
  const int bad = scan_check(B, N, C, T, dtype, offsets != nullptr);
  if (bad != FEQL_OK) return bad;
  if (!ok_ptr(dh, N > 0) || !ok_ptr(g, N > 0) || !ok_ptr(diff, N > 0) || !ok_ptr(du, N > 0) ||
      !ok_ptr(dg, N > 0) || !ok_ptr(dhN, false) || !ok_ptr(dh0, false) ||
      !ok_ptr(offsets, false) || !ok_ptr(ws, false))
    return FEQL_ERR_INVALID_ARG;
  if (!is_half(dtype)) return FEQL_ERR_UNSUPPORTED;
  if (B == 0) return FEQL_OK;
  ScanPlan q;
  const int st = scan_prepare(B, N, C, T, shared, dtype, offsets, true, ws, ws_bytes, &q);
  if (st != FEQL_OK) return st;
  return scan_bwd<__half>(q, dh, nullptr, g, nullptr, nullptr, diff, dhN, du, dg, dh0,
                          reinterpret_cast<cudaStream_t>(stream));
}

int feql_scan_step(const void *u, const void *g, float *state, void *h, int64_t B, int C, int T,
                   int shared, int dtype, feql_stream stream) {
  const int bad = scan_check(B, B, C, T, dtype, true);
  if (bad != FEQL_OK) return bad;
  if (!ok_ptr(u, B > 0) || !ok_ptr(g, B > 0) || !ok_ptr(state, B > 0) || !ok_ptr(h, B > 0))
    return FEQL_ERR_INVALID_ARG;
  if (B == 0) return FEQL_OK;
  DeviceInfo dev;
  const int st = device_info(&dev);
  if (st != FEQL_OK) return st;
  const int64_t n = B * static_cast<int64_t>(C) * T;
  const int64_t want = ceil_div(n, 256), cap = 8ll * dev.sms;
  const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
  const int per = shared ? T : 1;  // values per gate
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (is_half(dtype))
    scan_step_kernel<__half><<<grid, 256, 0, s>>>(static_cast<const __half *>(u),
                                                  static_cast<const __half *>(g), state,
                                                  static_cast<__half *>(h), n, per);
  else
    scan_step_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float *>(u),
                                                 static_cast<const float *>(g), state,
                                                 static_cast<float *>(h), n, per);
  return launch_status();
}

}  // extern "C"
