// Argument checks and scratch shared by the C entry points of the row-wise
// operators and the fused products (layers_api.cu, model_api.cu).
#pragma once

#include <atomic>
#include <climits>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "host.h"

namespace mt {
namespace host {

// Largest row, column or contraction count of a product: tile coordinates
// past the edge stay inside 32 bits.
constexpr int64_t kMaxSize = INT32_MAX - 255;
// Longest row of a norm: the row-wise kernels step a 32-bit column by up to
// 512, and round the columns up to whole strips of 32.
constexpr int64_t kMaxRow = INT32_MAX - 511;

// A rows x cols view of `elem`-byte values with row pitch ld, for the checks.
struct View {
  const void* p;
  int64_t rows, cols, ld;
  int elem;

  int64_t bytes() const { return extent_bytes(rows, cols, ld, elem); }
  bool empty() const { return rows == 0 || cols == 0; }
  // The pitch holds a row, the span fits 64-bit offsets, and the pointer is
  // there and aligned to its element unless there is nothing to address.
  bool valid() const {
    if (ld < (cols > 1 ? cols : 1) || ld > INT64_MAX / 64) return false;
    if (rows > 0 && ld > INT64_MAX / 64 / rows) return false;
    if (empty()) return true;
    return p && (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(elem - 1)) == 0;
  }
  bool same(const View& o) const { return p == o.p && ld == o.ld && elem == o.elem; }
  // Whether the views share a byte.  Columns of one wider buffer (the same
  // pitch) may lie side by side in spans that overlap; other pitches are
  // judged by their spans.
  bool hits(const View& o) const {
    if (!overlaps(p, bytes(), o.p, o.bytes())) return false;
    const int64_t pitch = ld * elem;
    if (rows < 2 || o.rows < 2 || o.ld * o.elem != pitch) return true;
    const int64_t apart = static_cast<const char*>(o.p) - static_cast<const char*>(p);
    const int64_t first = (apart % pitch + pitch) % pitch;  // o's column 0 in a row of this
    return first < cols * elem || first + o.cols * o.elem > pitch;
  }
};

// Scratch from the device's pool for one call; freed on the call's stream.
struct Scratch {
  void* p = nullptr;
  cudaStream_t stream;

  explicit Scratch(cudaStream_t s) : stream(s) {}
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
  ~Scratch() {
    if (p) cudaFreeAsync(p, stream);
  }
  mt_status get(int dev, int64_t bytes) {
    if (bytes <= 0) return MT_OK;
    cudaMemPool_t pool = nullptr;
    const mt_status st = pool_for(dev, &pool);
    if (st != MT_OK) return st;
    if (cudaMallocFromPoolAsync(&p, static_cast<size_t>(bytes), pool, stream) != cudaSuccess) {
      cudaGetLastError();
      p = nullptr;
      return MT_ERR_CUDA;
    }
    return MT_OK;
  }
};

inline bool half_type(int t) { return t == MT_DTYPE_F16 || t == MT_DTYPE_BF16; }

// What a group of kernels needs before its first launch on a device (their
// shared-memory limits).
struct OncePerDevice {
  std::mutex mutex;
  std::atomic<uint8_t> ready[kMaxDevices];

  mt_status run(int dev, cudaError_t (*prepare)()) {
    if (ready[dev].load(std::memory_order_acquire)) return MT_OK;
    std::lock_guard<std::mutex> lock(mutex);
    if (prepare() != cudaSuccess) {
      cudaGetLastError();
      return MT_ERR_LAUNCH;
    }
    ready[dev].store(1, std::memory_order_release);
    return MT_OK;
  }
};

// The fused products' kernels made ready.
mt_status prepare_linear(int dev);

}  // namespace host
}  // namespace mt
