// vec.cuh — packs of neighbouring values moved by one load or store, and the
// conversions between the data types and fp32.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace feql {

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }

template <typename Ty>
__device__ __forceinline__ Ty narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

template <int Bytes>
struct Word;
template <>
struct Word<2> { using type = unsigned short; };
template <>
struct Word<4> { using type = unsigned int; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };

// V neighbouring values (2, 4, 8 or 16 bytes), kept as the bits that memory holds.
template <typename Ty, int V>
struct Pack {
  typename Word<V * sizeof(Ty)>::type w;

  __device__ __forceinline__ void unpack(float (&f)[V]) const {
    if constexpr (sizeof(Ty) == 4) {
      const float *p = reinterpret_cast<const float *>(&w);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = p[j];
    } else if constexpr (V == 1) {
      f[0] = __half2float(__ushort_as_half(w));
    } else {
      const __half2 *p = reinterpret_cast<const __half2 *>(&w);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 q = __half22float2(p[j]);
        f[2 * j] = q.x;
        f[2 * j + 1] = q.y;
      }
    }
  }

  __device__ __forceinline__ void pack(const float (&f)[V]) {
    if constexpr (sizeof(Ty) == 4) {
      float *p = reinterpret_cast<float *>(&w);
#pragma unroll
      for (int j = 0; j < V; ++j) p[j] = f[j];
    } else if constexpr (V == 1) {
      w = __half_as_ushort(__float2half_rn(f[0]));
    } else {
      __half2 *p = reinterpret_cast<__half2 *>(&w);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) p[j] = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
    }
  }

  __device__ __forceinline__ void load(const Ty *p) {
    w = *reinterpret_cast<const decltype(w) *>(p);
  }
  __device__ __forceinline__ void store(Ty *p) const {
    *reinterpret_cast<typename Word<V * sizeof(Ty)>::type *>(p) = w;
  }
  __device__ __forceinline__ void zero() { w = decltype(w){}; }

  // Keeps the compiler from holding unpacked values (twice the registers for
  // fp16) from here on: the next unpack() is a new one.
  __device__ __forceinline__ void renew() {
    if constexpr (sizeof(w) >= 4) {
      uint32_t *p = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(w) / 4); ++i) asm volatile("" : "+r"(p[i]));
    }
  }
};

// fp32 vectors of V values.  (The paired fp32 instructions were measured: fewer issue
// slots, no time won, 104 against 99 us in the recurrence's backward and 351 against
// 328 us in the layer's training step through GELU.)
template <int V>
__device__ __forceinline__ void vec_fma(float (&d)[V], const float (&a)[V], const float (&b)[V],
                                        const float (&c)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = fmaf(a[j], b[j], c[j]);
}
template <int V>
__device__ __forceinline__ void vec_mul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = a[j] * b[j];
}
template <int V>
__device__ __forceinline__ void vec_add(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = a[j] + b[j];
}
template <int V>
__device__ __forceinline__ void vec_sub(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = a[j] - b[j];
}
// Gate values of a row spread over its V features: themselves, or the one.
template <int V, int GV>
__device__ __forceinline__ void spread(float (&d)[V], const float (&g)[GV]) {
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = g[GV == 1 ? 0 : j];
}

__device__ __forceinline__ float ex2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// sigma(v) and sigma(-v), each to full relative precision.  kFast (fp16
// outputs): the hardware's exponential and reciprocal, off by 2^-21 or so, far
// below the outputs' rounding, subnormals flushed.
template <bool kFast>
__device__ __forceinline__ void sigmoid_pair(float v, float &p, float &q) {
  const float e = kFast ? ex2_fast(-kLog2e * fabsf(v)) : expf(-fabsf(v));
  const float big = kFast ? rcp_fast(1.f + e) : 1.f / (1.f + e);
  const float small = e * big;
  p = v >= 0.f ? big : small;
  q = v >= 0.f ? small : big;
}

}  // namespace feql
