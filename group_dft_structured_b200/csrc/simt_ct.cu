// simt_ct.cu — launches of the CUDA-core kernels of the cyclic groups C_T
// (simt_ct.cuh), one instance per order and data type: a translation unit of its
// own, so that they compile beside the tensor-core kernels.
#include "simt_ct_host.cuh"

#include "host.cuh"
#include "simt_ct.cuh"

namespace feql {

namespace {

#define FEQL_CT_ORDERS(X) X(2) X(3) X(5) X(6) X(7) X(8) X(9) X(10) X(11) X(12) X(13) X(14) X(15) X(16)

template <int T, typename Ty>
int ct_simt_wfft_launch(const void *W, void *What, int C, int D, cudaStream_t s, int sms) {
  ct_simt_wfft_kernel<T, Ty><<<grid_for(static_cast<int64_t>(C) * D, 256, sms), 256, 0, s>>>(
      static_cast<const Ty *>(W), static_cast<float *>(What), C, D);
  return launch_status();
}

template <int T, typename Ty>
int ct_simt_pass_launch(const void *in, const float *Wp, const void *bias, void *out, int64_t N,
                        int Ci, int Do, cudaStream_t s, const Epilogue *ep, bool twice) {
  const int64_t gx = cdiv(N, kCtTile);
  if (gx > INT32_MAX) return FEQL_ERR_UNSUPPORTED;
  dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(cdiv(Do, kCtTile)));
  if (grid.y > 65535) return FEQL_ERR_UNSUPPORTED;
  auto kernel = ep == nullptr ? ct_simt_fwd_kernel<T, Ty>
                : ep_is_max(epilogue_kind(*ep)) ? ct_simt_fwd_kernel<T, Ty, kEpMax>
                                                : ct_simt_fwd_kernel<T, Ty, kEpSigmoid>;
  if constexpr (sizeof(Ty) == 2)
    if (twice) kernel = ct_simt_fwd_kernel<T, Ty, kEpNone, 2>;
  kernel<<<grid, kCtThreads, 0, s>>>(static_cast<const Ty *>(in), Wp,
                                     static_cast<const Ty *>(bias), static_cast<Ty *>(out), N, Ci,
                                     Do, ep != nullptr ? *ep : Epilogue{});
  return launch_status();
}

template <int T, typename Ty>
int ct_simt_dw_launch(const void *x, const void *dy, void *dW, void *db, float *ws, size_t ws_bytes,
                      int64_t N, int C, int D, cudaStream_t s, int sms, float scale) {
  const CtDwPlan p = make_ct_dw_plan(N, C, D, sms);
  if (ws_bytes < static_cast<size_t>(ct_dw_ws_floats(p, T, C, D)) * 4) return FEQL_ERR_INVALID_ARG;
  float *ws_db = ws + static_cast<int64_t>(p.splits) * T * D * C;
  if (p.splits > 0) {
    const int64_t grid = static_cast<int64_t>(p.splits) * p.tiles_d * p.tiles_c;
    if (grid > INT32_MAX) return FEQL_ERR_UNSUPPORTED;
    ct_simt_dw_kernel<T, Ty><<<static_cast<unsigned>(grid), kCtThreads, 0, s>>>(
        static_cast<const Ty *>(x), static_cast<const Ty *>(dy), ws, ws_db, N, C, D, p.split_len,
        p.tiles_d, p.tiles_c);
  }
  const bool wide = split_sum_wide(C, D, p.splits, sms);
  auto reduce = wide ? ct_simt_dw_reduce_kernel<T, Ty, true> : ct_simt_dw_reduce_kernel<T, Ty, false>;
  reduce<<<split_sum_blocks(C, D, wide, sms), kSumThreads, 0, s>>>(
      ws, ws_db, static_cast<Ty *>(dW), static_cast<Ty *>(db), p.splits, C, D, scale);
  return launch_status();
}

}  // namespace

template <typename Ty>
int ct_simt_wfft(int T, const void *W, void *What, int C, int D, cudaStream_t s, int sms) {
  switch (T) {
#define FEQL_CASE(t) case t: return ct_simt_wfft_launch<t, Ty>(W, What, C, D, s, sms);
    FEQL_CT_ORDERS(FEQL_CASE)
#undef FEQL_CASE
    default: return FEQL_ERR_UNSUPPORTED;
  }
}

template <typename Ty>
int ct_simt_pass(int T, const void *in, const float *Wp, const void *bias, void *out, int64_t N,
                 int Ci, int Do, cudaStream_t s, const Epilogue *ep, bool twice) {
  switch (T) {
#define FEQL_CASE(t) \
  case t: return ct_simt_pass_launch<t, Ty>(in, Wp, bias, out, N, Ci, Do, s, ep, twice);
    FEQL_CT_ORDERS(FEQL_CASE)
#undef FEQL_CASE
    default: return FEQL_ERR_UNSUPPORTED;
  }
}

template <typename Ty>
int ct_simt_dw(int T, const void *x, const void *dy, void *dW, void *db, float *ws, size_t ws_bytes,
               int64_t N, int C, int D, cudaStream_t s, int sms, float scale) {
  switch (T) {
#define FEQL_CASE(t) \
  case t: return ct_simt_dw_launch<t, Ty>(x, dy, dW, db, ws, ws_bytes, N, C, D, s, sms, scale);
    FEQL_CT_ORDERS(FEQL_CASE)
#undef FEQL_CASE
    default: return FEQL_ERR_UNSUPPORTED;
  }
}

template int ct_simt_wfft<float>(int, const void *, void *, int, int, cudaStream_t, int);
template int ct_simt_pass<float>(int, const void *, const float *, const void *, void *, int64_t, int,
                              int, cudaStream_t, const Epilogue *, bool);
template int ct_simt_dw<float>(int, const void *, const void *, void *, void *, float *, size_t, int64_t,
                            int, int, cudaStream_t, int, float);
template int ct_simt_wfft<__half>(int, const void *, void *, int, int, cudaStream_t, int);
template int ct_simt_pass<__half>(int, const void *, const float *, const void *, void *, int64_t, int,
                               int, cudaStream_t, const Epilogue *, bool);
template int ct_simt_dw<__half>(int, const void *, const void *, void *, void *, float *, size_t, int64_t,
                             int, int, cudaStream_t, int, float);

}  // namespace feql
