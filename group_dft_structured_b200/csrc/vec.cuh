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
};

}  // namespace feql
