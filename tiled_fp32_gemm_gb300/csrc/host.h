// Host helpers shared by the C entry points (api.cu, layers_api.cu): the
// current device, the per-device scratch pool, and argument checks.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "kernels.h"
#include "mt_sgemm.h"

namespace mt {
namespace host {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  int sms = 0;
  int smem_optin = 0;  // max dynamic shared memory per block with opt-in
  bool valid = false;
};

// The current device and its properties (looked up once per device).
mt_status current_device(int* dev, DeviceInfo* info);

// The device's stream-ordered scratch pool (created on first use).
mt_status pool_for(int dev, cudaMemPool_t* pool);

// The record the current device's kernels write to: nullptr in normal
// builds (and if the lookup fails).
BoundsRecord* bounds_record();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool overlaps(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  if (a_bytes <= 0 || b_bytes <= 0 || !a || !b) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(b_bytes) && b0 < a0 + static_cast<uintptr_t>(a_bytes);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bytes from the first to one past the last element of a rows x cols view
// with row stride ld and elements of `elem` bytes.
inline int64_t extent_bytes(int64_t rows, int64_t cols, int64_t ld, int elem = 4) {
  return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * elem : 0;
}

}  // namespace host
}  // namespace mt
