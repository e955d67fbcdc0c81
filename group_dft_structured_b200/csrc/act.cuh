// act.cuh — activation and residual in the epilogue of the layer's products,
//   y = res + act(z),  z = EqLinear(x) + b,
// and the elementwise gradient dz = dy act'(z).
//
// Pointwise on every group value, so the layer stays equivariant.  GELU (its
// tanh form, as in the MLP block) and SiLU are one family: z p, p = sigma(v),
// v = z (ka + kb z^2), because (1 + tanh(w)) / 2 = sigma(2 w); one exponential
// and one division per value, without tanh's cancellation for negative z.
//
// For the backward pass the forward saves the slope act'(z) = p (1 + z (1 - p) v'(z)),
// not z: it has p at hand, so the slope costs five products, and the backward
// pass multiplies.  Rounding it moves dz by half a step, as rounding z would.
// (Saving z and computing the slope in the backward was tried: with two more
// hardware functions and some 16 instructions per value the fused backward of
// 401408 x 24 -> 96 took 235 us, its separate kernels 226.)
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "../../include/feql.h"
#include "vec.cuh"

namespace feql {

struct Epilogue {
  const void *res;  // [N][Do][T] or nullptr
  void *slope;      // [N][Do][T] act'(z) for the backward pass, or nullptr
  int act;          // feql_activation
  float ka, kb;     // v = z (ka + kb z^2) of GELU and SiLU
  float nka, nkb;   // the same times -log2(e): exp(-v) = 2^(z (nka + nkb z^2))
  float lo;         // max(z, lo): 0 for ReLU, -inf for no activation
};

inline Epilogue make_epilogue(int act, const void *res, void *slope) {
  Epilogue e;
  e.res = res;
  e.slope = slope;
  e.act = act;
  const float k0 = 0.7978845608028654f;  // sqrt(2 / pi)
  e.ka = act == FEQL_ACT_GELU ? 2.f * k0 : 1.f;
  e.kb = act == FEQL_ACT_GELU ? 2.f * k0 * 0.044715f : 0.f;
  e.nka = -1.4426950408889634f * e.ka;
  e.nkb = -1.4426950408889634f * e.kb;
  e.lo = act == FEQL_ACT_RELU ? 0.f : -INFINITY;
  return e;
}

// Variants of an epilogue: none (the layer alone); max(z, lo), which is ReLU or,
// with lo = -inf, no activation; the sigmoid family; each without and with its
// slope on the tensor cores' fp16 path (elsewhere the slope is always at hand).
enum EpKind { kEpNone = 0, kEpMax = 1, kEpSigmoid = 2, kEpMaxSlope = 3, kEpSigmoidSlope = 4 };

__host__ __device__ constexpr bool ep_is_max(int kind) {
  return kind == kEpMax || kind == kEpMaxSlope;
}
__host__ __device__ constexpr bool ep_has_slope(int kind) { return kind >= kEpMaxSlope; }

inline int epilogue_kind(const Epilogue &e) {
  const bool sig = e.act == FEQL_ACT_GELU || e.act == FEQL_ACT_SILU;
  if (e.slope == nullptr) return sig ? kEpSigmoid : kEpMax;
  return sig ? kEpSigmoidSlope : kEpMaxSlope;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A z that is no number must show in y and in the slope (an overflowed x, a diverged
// W: a loss scaler looks for it), and so must z = -inf, as 0 times infinity does.

// z^2 up to 1e8: from |z| = 1e4 on p is 0 or 1 and the slope's cubic factor must
// stay finite beside a 1 - p or p of zero.  (A NaN comes back in the product with z.)
__device__ __forceinline__ float act_square(float z) { return fminf(z * z, 1e8f); }

// y = res + act(z) and slope = act'(z) of one value.  In the sigmoid family exp(-v)
// overflows to inf for v below -88, where p = 0 stands for a value under 1e-36.
// kFast (fp16 outputs): the hardware's exponential and reciprocal, off by 2^-20 or
// so, far below the outputs' rounding.
template <int kKind, bool kFast>
__device__ __forceinline__ float act_value(const Epilogue &e, float z, float res, float &slope) {
  if constexpr (ep_is_max(kKind)) {
    slope = z <= e.lo ? 0.f : 1.f;
    return max_nan(z, e.lo) + res;
  }
  const float z2 = act_square(z);
  float p, q;  // sigma(v), sigma(-v)
  if constexpr (kFast) {
    p = rcp_fast(1.f + ex2_fast(z * fmaf(e.nkb, z2, e.nka)));
    q = 1.f - p;
  } else {
    sigmoid_pair<false>(z * fmaf(e.kb, z2, e.ka), p, q);
  }
  // (|z| beyond 1e31 would overflow beside a p or q of zero: those cases are set;
  // z - z is 0, or NaN for a z of -inf)
  const float t = z * fmaf(3.f * e.kb, z2, e.ka) * q;
  slope = p <= 0.f ? z - z : fmaf(p, t, p);
  if (!kFast && !(q > 0.f)) slope = p;
  return fmaf(z, p, res);
}

// act(z) and the slopes of two values in fp16's accuracy (the slopes only of
// kinds that have them).
template <int kKind>
__device__ __forceinline__ void act_pair(const Epilogue &e, const float (&z)[2], float (&y)[2],
                                         float (&s)[2]) {
  if constexpr (ep_is_max(kKind)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (ep_has_slope(kKind)) s[j] = z[j] <= e.lo ? 0.f : 1.f;
      y[j] = max_nan(z[j], e.lo);
    }
  } else {
    const float one[2] = {1.f, 1.f}, ka[2] = {e.nka, e.nka}, kb[2] = {e.nkb, e.nkb};
    const float ca[2] = {e.ka, e.ka}, cb[2] = {3.f * e.kb, 3.f * e.kb};
    // below -1e4 act and slope are 0, and the slope's cubic factor stays finite
    // beside a p of zero; above, z is beyond fp16 before the factor overflows
    const float c[2] = {max_nan(z[0], -1e4f), max_nan(z[1], -1e4f)};
    float z2[2], v[2], p[2];
    vec_mul(z2, c, c);
    vec_fma(v, kb, z2, ka);
    vec_mul(v, v, c);
#pragma unroll
    for (int j = 0; j < 2; ++j) p[j] = rcp_fast(1.f + ex2_fast(v[j]));
    // (not contracted with the residual's sum: the same y with and without slopes; z is
    // read no more, y may be its place.  z and not c: -inf times 0 is no number)
#pragma unroll
    for (int j = 0; j < 2; ++j) y[j] = __fmul_rn(z[j], p[j]);
    if constexpr (ep_has_slope(kKind)) {
      // p + z p (1 - p) v'(z), and z p is y
      float q[2], t[2];
      vec_sub(q, one, p);
      vec_fma(t, cb, z2, ca);
      vec_mul(t, t, y);
      vec_fma(s, t, q, p);
    }
  }
}

// GELU's and SiLU's slopes reach 1.13, so dz = dy slope of a finite fp16 dy can leave
// fp16's range.  It is held divided by a power of two, as the layer's operand planes
// are, so that the layer's backward takes every finite dy with an activation too.

// dz / 4 on a packed fp16 pair, rounded once (dy / 4 is exact above the subnormals).
__device__ __forceinline__ uint32_t act_grad_q(uint32_t dy, uint32_t slope) {
  const __half2 q = __hmul2(*reinterpret_cast<const __half2 *>(&dy), __float2half2_rn(0.25f));
  const __half2 h = __hmul2(q, *reinterpret_cast<const __half2 *>(&slope));
  return *reinterpret_cast<const uint32_t *>(&h);
}

// What the passes that read dz from memory multiply their results by.
template <typename Ty>
constexpr int act_dz_scale() { return sizeof(Ty) == 2 ? 2 : 1; }

// dz = dy slope (fp16: dz / 2) on n values, 16 bytes per access; HBM-bound (three
// streams), 144 us on 401408 x 96 x 4 fp16 (6.4 TB/s).
template <typename Ty>
__global__ void __launch_bounds__(256)
act_bwd_kernel(const Ty *__restrict__ dy, const Ty *__restrict__ slope, Ty *__restrict__ dz,
               int64_t n) {
  constexpr int V = 16 / sizeof(Ty);
  constexpr float k = 1.f / act_dz_scale<Ty>();
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t i = i0; i < n / V; i += step) {
    Pack<Ty, V> a, b;
    a.load(dy + i * V);
    b.load(slope + i * V);
    float d[V], w[V];
    a.unpack(d);
    b.unpack(w);
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] *= k * w[j];
    a.pack(d);
    a.store(dz + i * V);
  }
  const int64_t at = n / V * V + i0;
  if (i0 < n % V) dz[at] = narrow<Ty>(widen(dy[at]) * (k * widen(slope[at])));
}

}  // namespace feql
