// feql_ops.cu — C ABI of the operators that stand around the layer: layer norm
// (feql_norm_*) and the gated linear recurrence (feql_scan_*), declared in
// include/feql.h.  Host side only: argument checks, plans and launches.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

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
  q.A = (T % 4 == 0 && q.V % 4 == 0) ? 4 : 1;
  q.s = {N, C, T, F, 0, F / q.V};
  static const int wide_fwd[] = {4, 2, 3, 1, 8}, wide_bwd[] = {4, 2, 3, 1}, narrow_k[] = {2, 8};
  const int *ks = q.V == wide ? (bwd ? wide_bwd : wide_fwd) : narrow_k;
  const int nk = q.V == wide ? (bwd ? 4 : 5) : 2;
  q.in_regs = false;
  int best = 0;
  for (int i = 0; i < nk; ++i) {
    int G = 1;
    while (G * ks[i] < q.s.nchunk && G <= kNormMaxThreads) G *= 2;
    if (G > kNormMaxThreads) continue;
    if (!q.in_regs || G * ks[i] < best) {
      q.in_regs = true;
      best = G * ks[i];
      q.K = ks[i];
      q.s.G = G;
    }
  }
  if (!q.in_regs) q.s.G = kNormLongThreads;
  q.threads = q.in_regs ? (q.s.G > 32 ? q.s.G : kNormThreads) : kNormLongThreads;
  return q;
}

// Blocks of the row loop: enough to fill the GPU; the backward's partial sums
// are one row per block, so it takes half as many.
int norm_blocks(const NormPlan &q, int sms, bool bwd) {
  const int64_t want = q.in_regs ? ceil_div(q.s.N, q.threads / q.s.G) : q.s.N;
  const int64_t cap = static_cast<int64_t>(sms) * ((bwd ? 1024 : 2048) / q.threads);
  return static_cast<int>(want < cap ? want : cap);
}

constexpr int64_t kNormLongRows = 64;  // rows of a split of the long rows' column pass
int64_t norm_long_splits(int64_t N) {
  const int64_t n = ceil_div(N, kNormLongRows);
  return n < 32 ? n : 32;
}

#define FEQL_NORM_WIDE(X, Ty, V, A) X(Ty, V, 1, A) X(Ty, V, 2, A) X(Ty, V, 3, A) X(Ty, V, 4, A)
#define FEQL_NORM_NARROW(X, Ty, V, A) X(Ty, V, 2, A) X(Ty, V, 8, A)
#define FEQL_NORM_HALF(X)                                                                \
  FEQL_NORM_WIDE(X, __half, 8, 1) FEQL_NORM_WIDE(X, __half, 8, 4)                        \
  FEQL_NORM_NARROW(X, __half, 4, 1) FEQL_NORM_NARROW(X, __half, 4, 4)                    \
  FEQL_NORM_NARROW(X, __half, 2, 1) FEQL_NORM_NARROW(X, __half, 1, 1)
#define FEQL_NORM_FLOAT(X)                                                               \
  FEQL_NORM_WIDE(X, float, 4, 1) FEQL_NORM_WIDE(X, float, 4, 4)                          \
  FEQL_NORM_NARROW(X, float, 2, 1) FEQL_NORM_NARROW(X, float, 1, 1)

int norm_fwd_launch(const NormPlan &q, bool half, const void *x, const void *gamma,
                    const void *beta, void *y, float2 *stats, float eps, int grid,
                    cudaStream_t st) {
#define FEQL_CASE(Ty, VV, KK, AA)                                                             \
  if (q.V == VV && q.K == KK && q.A == AA) {                                                  \
    norm_fwd_kernel<Ty, VV, KK, AA><<<grid, q.threads, 0, st>>>(                              \
        static_cast<const Ty *>(x), static_cast<const Ty *>(gamma),                           \
        static_cast<const Ty *>(beta), static_cast<Ty *>(y), stats, q.s, eps);                \
    return launch_status();                                                                   \
  }
  if (half) {
    FEQL_NORM_HALF(FEQL_CASE)
    FEQL_CASE(__half, 8, 8, 1)
    FEQL_CASE(__half, 8, 8, 4)
  } else {
    FEQL_NORM_FLOAT(FEQL_CASE)
    FEQL_CASE(float, 4, 8, 1)
    FEQL_CASE(float, 4, 8, 4)
  }
#undef FEQL_CASE
  return FEQL_ERR_UNSUPPORTED;
}

int norm_bwd_launch(const NormPlan &q, bool half, const void *x, const void *dy,
                    const void *gamma, const float2 *stats, void *dx, float *part, int grid,
                    cudaStream_t st) {
#define FEQL_CASE(Ty, VV, KK, AA)                                                             \
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
  norm_reduce_kernel<Ty><<<static_cast<unsigned>(ceil_div(C, kNormRedCh)), kNormRedCh * 32, 0,
                           st>>>(part, static_cast<Ty *>(dgamma), static_cast<Ty *>(dbeta), C, m,
                                 blocks);
  return launch_status();
}

int norm_check(int64_t N, int C, int T, int dtype) {
  if (!valid_dtype(dtype) || N < 0 || N > kMaxTokens || check_shape(C, 1) != FEQL_OK)
    return FEQL_ERR_INVALID_ARG;
  if (T < 1 || T > kMaxOrder) return FEQL_ERR_UNSUPPORTED;
  return FEQL_OK;
}

// ------------------------------------------------------------------- scan
struct ScanPlan {
  int V, NW;
  ScanShape s;
};

// Rows per thread.  Forward: what keeps the local states and products (two
// fp32 per value, one more for fp32 data in flight) within 128 registers, so
// that two blocks of 256 threads share an SM; the backward holds twice as much
// per value.
constexpr int scan_rows_fwd(bool half, int V) { return V == 4 && !half ? 4 : 8; }
constexpr int scan_rows_bwd(int V) { return V == 4 ? 4 : 8; }

// A thread's features are V neighbours: 4, or fewer where a row (or, for
// shared gates, a channel) is not a multiple of 4.  One warp per block walks
// a sequence by itself when there are enough (sequence, tile) units to fill
// the GPU with warps or the sequences are short; else eight warps share a
// tile of rows, and clusters of blocks split the rows while the units do not
// give every SM two blocks and the sequences are long enough.
ScanPlan scan_plan(int B, int64_t N, int C, int T, bool shared, bool half, int sms) {
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
  q.s.FT = sh ? kScanLanes / T * T : kScanLanes;
  q.s.ntiles = static_cast<int>(ceil_div(F, q.s.FT));
  const int64_t units = static_cast<int64_t>(B) * q.s.ntiles;
  const int64_t avg = B > 0 ? ceil_div(N, B) : 0;
  const int warp_rows = q.V * scan_rows_fwd(half, q.V);
  q.NW = (units >= 16ll * sms || avg <= 2 * warp_rows) ? 1 : 8;
  q.s.K = 1;
  if (q.NW == 8)
    while (q.s.K < kScanMaxCluster && units * q.s.K < 2 * sms && 8ll * warp_rows * q.s.K < avg)
      q.s.K *= 2;
  q.s.Q = q.NW * q.V * scan_rows_bwd(q.V);
  return q;
}

int64_t scan_save_floats(const ScanPlan &q) {
  return (q.s.N / q.s.Q + q.s.B) * static_cast<int64_t>(q.s.F);
}

template <typename... Args>
int scan_launch(void (*kernel)(Args...), const ScanPlan &q, cudaStream_t st, Args... args) {
  const int64_t grid = static_cast<int64_t>(q.s.B) * q.s.ntiles * q.s.K;
  if (grid > INT32_MAX) return FEQL_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(q.s.K);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = q.s.K > 1 ? 1 : 0;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(q.NW * 32));
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FEQL_OK : FEQL_ERR_CUDA;
}

#define FEQL_SCAN_CASES(X, Ty) \
  X(Ty, 4, 8, true) X(Ty, 4, 8, false) X(Ty, 4, 1, true) X(Ty, 4, 1, false) \
  X(Ty, 2, 8, true) X(Ty, 2, 8, false) X(Ty, 2, 1, true) X(Ty, 2, 1, false) \
  X(Ty, 1, 8, true) X(Ty, 1, 8, false) X(Ty, 1, 1, true) X(Ty, 1, 1, false)

template <typename Ty>
int scan_fwd(const ScanPlan &q, const void *u, const void *g, const float *h0, void *h, float *hN,
             float *save, cudaStream_t st) {
  const bool sh = q.s.FG != q.s.F;
#define FEQL_CASE(T_, VV, NWW, SH)                                                             \
  if (q.V == VV && q.NW == NWW && sh == SH)                                                    \
    return scan_launch(scan_fwd_kernel<T_, VV, scan_rows_fwd(sizeof(T_) == 2, VV), NWW, SH>, q, \
                       st, static_cast<const T_ *>(u), static_cast<const T_ *>(g), h0,         \
                       static_cast<T_ *>(h), hN, save, q.s);
  FEQL_SCAN_CASES(FEQL_CASE, Ty)
#undef FEQL_CASE
  return FEQL_ERR_UNSUPPORTED;
}

template <typename Ty>
int scan_bwd(const ScanPlan &q, const void *dh, const void *u, const void *g, const float *save,
             const float *dhN, void *du, void *dg, float *dh0, cudaStream_t st) {
  const bool sh = q.s.FG != q.s.F;
#define FEQL_CASE(T_, VV, NWW, SH)                                                            \
  if (q.V == VV && q.NW == NWW && sh == SH)                                                   \
    return scan_launch(scan_bwd_kernel<T_, VV, scan_rows_bwd(VV), NWW, SH>, q, st,            \
                       static_cast<const T_ *>(dh), static_cast<const T_ *>(u),               \
                       static_cast<const T_ *>(g), save, dhN, static_cast<T_ *>(du),          \
                       static_cast<T_ *>(dg), dh0, q.s);
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
  const int grid = norm_blocks(q, dev.sms, false);
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
  const int64_t rows = q.in_regs ? norm_blocks(q, dev.sms, true) : norm_long_splits(N);
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
    const int grid = norm_blocks(q, dev.sms, true);
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

size_t feql_scan_save_bytes(int64_t B, int64_t N, int C, int T, int shared, int dtype) {
  if (scan_check(B, N, C, T, dtype, true) != FEQL_OK) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != FEQL_OK) return 0;
  const ScanPlan q =
      scan_plan(static_cast<int>(B), N, C, T, shared != 0, is_half(dtype), dev.sms);
  const size_t bytes = static_cast<size_t>(scan_save_floats(q)) * 4;
  return bytes > 16 ? bytes : 16;
}

int feql_scan_forward(const void *u, const void *g, const float *h0, const int32_t *offsets,
                      void *h, float *hN, void *save, int64_t B, int64_t N, int C, int T,
                      int shared, int dtype, feql_stream stream) {
  const int bad = scan_check(B, N, C, T, dtype, offsets != nullptr);
  if (bad != FEQL_OK) return bad;
  if (!ok_ptr(u, N > 0) || !ok_ptr(g, N > 0) || !ok_ptr(h, N > 0) || !ok_ptr(h0, false) ||
      !ok_ptr(hN, false) || !ok_ptr(save, false) || !ok_ptr(offsets, false))
    return FEQL_ERR_INVALID_ARG;
  if (B == 0) return FEQL_OK;
  DeviceInfo dev;
  const int st = device_info(&dev);
  if (st != FEQL_OK) return st;
  ScanPlan q = scan_plan(static_cast<int>(B), N, C, T, shared != 0, is_half(dtype), dev.sms);
  q.s.offsets = offsets;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float *sv = static_cast<float *>(save);
  return is_half(dtype) ? scan_fwd<__half>(q, u, g, h0, h, hN, sv, s)
                        : scan_fwd<float>(q, u, g, h0, h, hN, sv, s);
}

int feql_scan_backward(const void *dh, const void *u, const void *g, const void *save,
                       const float *dhN, const int32_t *offsets, void *du, void *dg, float *dh0,
                       int64_t B, int64_t N, int C, int T, int shared, int dtype,
                       feql_stream stream) {
  const int bad = scan_check(B, N, C, T, dtype, offsets != nullptr);
  if (bad != FEQL_OK) return bad;
  if (!ok_ptr(dh, N > 0) || !ok_ptr(u, N > 0) || !ok_ptr(g, N > 0) || !ok_ptr(save, N > 0) ||
      !ok_ptr(du, N > 0) || !ok_ptr(dg, N > 0) || !ok_ptr(dhN, false) || !ok_ptr(dh0, false) ||
      !ok_ptr(offsets, false))
    return FEQL_ERR_INVALID_ARG;
  if (B == 0) return FEQL_OK;
  DeviceInfo dev;
  const int st = device_info(&dev);
  if (st != FEQL_OK) return st;
  ScanPlan q = scan_plan(static_cast<int>(B), N, C, T, shared != 0, is_half(dtype), dev.sms);
  q.s.offsets = offsets;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const float *sv = static_cast<const float *>(save);
  return is_half(dtype) ? scan_bwd<__half>(q, dh, u, g, sv, dhN, du, dg, dh0, s)
                        : scan_bwd<float>(q, dh, u, g, sv, dhN, du, dg, dh0, s);
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
