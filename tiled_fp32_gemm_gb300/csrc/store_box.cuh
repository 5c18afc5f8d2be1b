// Stores of a drain warp's 32 rows through shared memory: boxes of 32 rows x 128
// bytes in the 128-byte-swizzled layout, which tensor copies take to memory as
// whole lines.  Stored from registers, a row a lane, 16 bytes of each of 32 rows
// leave at a time; a column a lane, 64 bytes an instruction of 2-byte values.
#pragma once

#include <cstdint>

#include "row_util.cuh"
#include "tcgen05.cuh"

namespace mt {
namespace f16tc {

constexpr int STORE_ROWS = 32, STORE_ROW_BYTES = 128;
constexpr int STORE_BOX_BYTES = STORE_ROWS * STORE_ROW_BYTES;

// The warp's box is free: the copy that read it last has done so (lane 0 has
// issued them all).
__device__ __forceinline__ void store_begin(int lane) {
  if (lane == 0) tc::bulk_wait_read();
  __syncwarp();
}

// Values at, at + 1, .. of row `lane` of the box.  Eight lanes' 16-byte pieces
// fall on all banks: piece j of row r lies at j ^ (r % 8).
template <class T, int N>
__device__ __forceinline__ void store_fill(uint8_t* box, int lane, int at, const float (&v)[N]) {
  constexpr int PER = 16 / static_cast<int>(sizeof(T));
  const int first = at / PER;
#pragma unroll
  for (int j = 0; j < N / PER; ++j) {
    uint4 u;
    if constexpr (sizeof(T) == 2) {
      float part[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) part[i] = v[j * PER + i];
      row::Pack8<T> o;
      o.set(part);
      u = o.u;
    } else {
      u = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                     __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
    }
    *reinterpret_cast<uint4*>(box + lane * STORE_ROW_BYTES + (((first + j) ^ (lane & 7)) << 4)) = u;
  }
}

// Sends the box to (x, y) of the map's matrix, or adds it to what is there.
__device__ __forceinline__ void store_end(const void* map, const uint8_t* box, int lane, int x,
                                          int y, bool any, bool add) {
  tc::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0 && any) {
    if (add) tc::tma_add_2d(map, smem_u32(box), x, y);
    else tc::tma_store_2d(map, smem_u32(box), x, y);
    tc::bulk_commit();
  }
}

}  // namespace f16tc
}  // namespace mt
