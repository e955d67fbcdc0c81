// act.cuh — activation and residual in the epilogue of the layer's products,
//   y = res + act(z),  z = EqLinear(x) + b,
// and the elementwise gradient dz = dy act'(z).
//
// Pointwise on every group value, so the layer stays equivariant.  GELU (its
// tanh form, as in the MLP block) and SiLU are one family: z sigma(v) with
// v = z (ka + kb z^2), because (1 + tanh(w)) / 2 = sigma(2 w); one exponential
// and one division per value, without tanh's cancellation for negative z.
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "../../include/feql.h"
#include "vec.cuh"

namespace feql {

struct Epilogue {
  const void *res;  // [N][Do][T] or nullptr
  void *z;          // [N][Do][T] pre-activation for the backward pass, or nullptr
  int act;          // feql_activation
  float ka, kb;     // v = z (ka + kb z^2) of GELU and SiLU
  float nka, nkb;   // the same times -log2(e): exp(-v) = 2^(z (nka + nkb z^2))
  float lo;         // max(z, lo): 0 for ReLU, -inf for no activation
  float least;      // ReLU: the smallest positive z that is saved
};

inline Epilogue make_epilogue(int act, const void *res, void *z) {
  Epilogue e;
  e.res = res;
  e.z = z;
  e.act = act;
  const float k0 = 0.7978845608028654f;  // sqrt(2 / pi)
  e.ka = act == FEQL_ACT_GELU ? 2.f * k0 : 1.f;
  e.kb = act == FEQL_ACT_GELU ? 2.f * k0 * 0.044715f : 0.f;
  e.nka = -1.4426950408889634f * e.ka;
  e.nkb = -1.4426950408889634f * e.kb;
  e.lo = act == FEQL_ACT_RELU ? 0.f : -INFINITY;
  e.least = act == FEQL_ACT_RELU ? 5.9604645e-8f : 0.f;
  return e;
}

// Variants of an epilogue: none (the layer alone); max(z, lo), which is ReLU or,
// with lo = -inf, no activation; the sigmoid family.
enum EpKind { kEpNone = 0, kEpMax = 1, kEpSigmoid = 2 };

inline int epilogue_kind(const Epilogue &e) {
  return e.act == FEQL_ACT_GELU || e.act == FEQL_ACT_SILU ? kEpSigmoid : kEpMax;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// res + act(z).  In the sigmoid family exp(-v) overflows to inf for v below -88,
// where z / inf = -0 stands for a value under 1e-36.
template <int kKind, bool kFast>
__device__ __forceinline__ float act_apply(const Epilogue &e, float z, float res) {
  if constexpr (kKind == kEpMax) return max_nan(z, e.lo) + res;
  if constexpr (kFast)
    return fmaf(z, rcp_fast(1.f + ex2_fast(z * fmaf(e.nkb * z, z, e.nka))), res);
  return z / (1.f + expf(-z * fmaf(e.kb * z, z, e.ka))) + res;
}

template <bool kFast>
__device__ __forceinline__ float act_slope(const Epilogue &e, float z) {
  if (e.act == FEQL_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  const float z2 = z * z;
  float p, q;
  sigmoid_pair<kFast>(z * fmaf(e.kb, z2, e.ka), p, q);
  // where sigma(-v) or sigma(v) has underflowed the second term is 0, whatever
  // its other factor
  const float pq = p * q;
  return pq > 0.f ? fmaf(z * pq, fmaf(3.f * e.kb, z2, e.ka), p) : p;
}

// The saved z keeps the side of ReLU's corner it was computed on: a positive
// value below half the least fp16 subnormal is saved as that subnormal, not 0.
template <int kKind>
__device__ __forceinline__ float act_saved(const Epilogue &e, float z) {
  return kKind == kEpMax && z > 0.f ? fmaxf(z, e.least) : z;
}

// Two values of an fp16 epilogue: their packed z in zw, and z0, z1 become the
// results; rw: their residual (zeros where there is none).
template <int kKind>
__device__ __forceinline__ void act_pair(const Epilogue &e, float &z0, float &z1, uint32_t rw,
                                         uint32_t &zw) {
  const __half2 h = __floats2half2_rn(act_saved<kKind>(e, z0), act_saved<kKind>(e, z1));
  zw = *reinterpret_cast<const uint32_t *>(&h);
  const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&rw));
  z0 = act_apply<kKind, true>(e, z0, r.x);
  z1 = act_apply<kKind, true>(e, z1, r.y);
}

// dz = dy act'(z) on n values, V per access; HBM-bound (three streams).  The
// z of fp16 data was rounded once: act' is off by at most 2^-11 |z act''(z)| <
// 2^-12 from it, half a step of dz.
template <typename Ty, int V>
__global__ void __launch_bounds__(256)
act_bwd_kernel(const Ty *__restrict__ dy, const Ty *__restrict__ z, Ty *__restrict__ dz, int64_t n,
               const Epilogue e) {
  constexpr bool kFast = sizeof(Ty) == 2;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t i = i0; i < n / V; i += step) {
    Pack<Ty, V> a, b;
    a.load(dy + i * V);
    b.load(z + i * V);
    float d[V], w[V];
    a.unpack(d);
    b.unpack(w);
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] *= act_slope<kFast>(e, w[j]);
    a.pack(d);
    a.store(dz + i * V);
  }
  const int64_t at = n / V * V + i0;
  if (i0 < n % V) dz[at] = narrow<Ty>(widen(dy[at]) * act_slope<kFast>(e, widen(z[at])));
}

}  // namespace feql
