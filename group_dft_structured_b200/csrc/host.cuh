// host.cuh — host-side helpers shared by the library's translation units:
// device properties (cached per device) and argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/feql.h"

namespace feql {

constexpr int kMaxDevices = 64;
constexpr int kMaxChannels = 1 << 16;            // per group element
constexpr int64_t kMaxTokens = (1ll << 31) - 1;  // TMA coordinates are int32

struct DeviceInfo {
  int sms = 0;
  int smem_optin = 0;
  int cc_major = 0, cc_minor = 0;
};

// Properties of the current device.
inline int device_info(DeviceInfo *out) {
  static std::mutex mu;
  static DeviceInfo known[kMaxDevices];
  static bool ok[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FEQL_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  if (!ok[dev]) {
    DeviceInfo d;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return FEQL_ERR_CUDA;
    known[dev] = d;
    ok[dev] = true;
  }
  *out = known[dev];
  return FEQL_OK;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_dtype(int dt) { return dt >= FEQL_FP16 && dt <= FEQL_FP16_SIMT; }

inline bool is_half(int dt) { return dt == FEQL_FP16 || dt == FEQL_FP16_SIMT; }

inline int check_shape(int C, int D) {
  if (C <= 0 || D <= 0 || C > kMaxChannels || D > kMaxChannels) return FEQL_ERR_INVALID_ARG;
  return FEQL_OK;
}

inline int launch_status() {
  return cudaGetLastError() == cudaSuccess ? FEQL_OK : FEQL_ERR_CUDA;
}

// Blocks of a grid-stride loop over `work` items.
inline int grid_for(int64_t work, int threads, int sms) {
  int64_t g = (work + threads - 1) / threads;
  const int64_t cap = static_cast<int64_t>(sms) * 8;
  if (g > cap) g = cap;
  if (g < 1) g = 1;
  return static_cast<int>(g);
}

}  // namespace feql
