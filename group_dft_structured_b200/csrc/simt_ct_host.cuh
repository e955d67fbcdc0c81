// simt_ct_host.cuh — host interface of the CUDA-core kernels of the cyclic groups C_T.
// Ty is the data type, float or __half; T an order other than 4 in 2..16.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "act.cuh"
#include "plan.cuh"

namespace feql {

constexpr int kCtMaxT = 16;
constexpr int kCtTile = 32;     // tokens x outputs (or d x c for dW) per block
constexpr int kCtK = 8;         // channels (or tokens, for dW) per shared-memory chunk

struct CtDwPlan {
  int tiles_d, tiles_c, splits;
  int64_t split_len;
};

// Token splits: about two blocks per SM over all (d, c) tiles, at most 64 (the
// reduce adds them in order, by split_sum.cuh).
inline CtDwPlan make_ct_dw_plan(int64_t N, int C, int D, int sms) {
  CtDwPlan p;
  p.tiles_d = static_cast<int>(cdiv(D, kCtTile));
  p.tiles_c = static_cast<int>(cdiv(C, kCtTile));
  int64_t s = 2 * static_cast<int64_t>(sms) / (p.tiles_d * p.tiles_c);
  if (s < 1) s = 1;
  if (s > 64) s = 64;
  const int64_t chunks = cdiv(N, kCtK);
  if (s > chunks) s = chunks;
  p.split_len = N > 0 ? align_up(cdiv(N, s), kCtK) : kCtK;
  p.splits = N > 0 ? static_cast<int>(cdiv(N, p.split_len)) : 0;
  return p;
}

inline int64_t ct_dw_ws_floats(const CtDwPlan &p, int T, int C, int D) {
  return static_cast<int64_t>(p.splits) * (static_cast<int64_t>(T) * D * C + D);
}

template <typename Ty>
int ct_simt_wfft(int T, const void *W, void *What, int C, int D, cudaStream_t s, int sms);

// Forward or dX pass; ep: activation, residual and saved slope, or nullptr; twice: of
// fp16 data, without ep, twice the result.
template <typename Ty>
int ct_simt_pass(int T, const void *in, const float *Wp, const void *bias, void *out, int64_t N,
                 int Ci, int Do, cudaStream_t s, const Epilogue *ep, bool twice);

template <typename Ty>
int ct_simt_dw(int T, const void *x, const void *dy, void *dW, void *db, float *ws, size_t ws_bytes,
               int64_t N, int C, int D, cudaStream_t s, int sms, float scale);

}  // namespace feql
