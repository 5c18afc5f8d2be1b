// The fused linear layer on one CTA tile per cluster: 128 columns x BT rows
// of Y, K cut into one slice per CTA of the cluster.
//
// The weight's columns are the MMA's M side (128 lanes of tensor memory), the
// tokens its N side, so a few tokens cost a narrow MMA and the weight, which
// is all there is to read then, streams through a ring of BT-dependent depth
// with two CTAs on an SM.  Per CTA (192 threads):
//   warp 0, one thread: TMA loads of the slice's K tiles (128 bytes of K);
//   warp 1, one thread: 4 tcgen05.mma 128 x BT per K tile, commit -> empty;
//   warps 2-5: the sums, from tensor memory.  With one CTA they are finished
//     and stored from registers.  With more, every CTA leaves its sums in its
//     shared memory (the ring, idle by then), and after a cluster barrier CTA
//     r adds rows r * q .. of all of them, in slice order, so the result does
//     not depend on timing.
// Every wait is bounded, as in the other tcgen05 kernels; a CTA that gave up
// leaves its flag where its cluster sees it, and none of them stores.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "gemm_f16.cuh"
#include "layers.h"
#include "linear.cuh"

namespace mt {
namespace linear {

using namespace f16tc;

constexpr int PREFETCH_STAGES = 1;  // rings of the weight's tiles prefetched to L2
constexpr int BC = LINEAR_BC;  // columns of Y per tile

template <int BT_>
struct SplitGeometry {
  static constexpr int BT = BT_;
  static constexpr int W_BYTES = BC * ROW_BYTES;
  static constexpr int X_BYTES = BT * ROW_BYTES;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  // Two CTAs share an SM's 227 KB.
  static constexpr int STAGES = 108 * 1024 / STAGE_BYTES;
  static constexpr uint32_t TMEM_COLS = BT < 32 ? 32 : BT;
  static constexpr int SUM_BYTES = BT * BC * 4;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 /*alignment*/ + 256;
  static_assert(SUM_BYTES <= STAGES * STAGE_BYTES, "the sums fit the ring");
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs on an SM");
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// FINISH_ROWS columns of this thread's TMEM lane; zeros for an empty slice of
// K, whose tensor memory holds nothing.  (Warp w may access TMEM lanes
// 32*(w%4) .. +31.)
__device__ __forceinline__ void load_sums(uint32_t addr, bool any, Rows& v) {
  if (any) {
    tmem_ld16(addr, v);
  } else {
#pragma unroll
    for (int i = 0; i < FINISH_ROWS; ++i) v[i] = 0.0f;
  }
}

template <class E, int BT, bool W_MN, bool X_MN>
__global__ void __launch_bounds__(THREADS, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmap_w,
                        const __grid_constant__ CUtensorMap tmap_x, uint32_t idesc,
                        const LinearEpilogue ep, int Kt, int tiles_t, int split, int fault_inject) {
  static_assert(E::BYTES == 2 || (!W_MN && !X_MN), "8-bit operands are K-major");
  using G = SplitGeometry<BT>;
  constexpr int STAGES = G::STAGES;
  constexpr int BK_ELEMS = ROW_BYTES / E::BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * G::STAGE_BYTES);
  constexpr int FULL = 0, EMPTY = STAGES, ACC_FULL = 2 * STAGES, NBARS = 2 * STAGES + 1;
  static_assert(NBARS * 8 + 8 <= 256, "barriers, TMEM slot and abort flag fit 256 bytes");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const WaitCtx wc{abort_flag, &g_status};
  auto bar = [&](int i) { return smem_u32(bars + i); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / split;
  // Tiles of one weight panel follow each other, so the panel is read from
  // memory once and found in L2 by the rest.
  const int c0 = tile / tiles_t * BC, t0 = tile % tiles_t * BT;
  const int kt0 = static_cast<int>(static_cast<int64_t>(Kt) * rank / split);
  const int kt1 = static_cast<int>(static_cast<int64_t>(Kt) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    if (Kt > 0) {  // without a product the maps hold nothing
      prefetch_tmap(&tmap_w);
      prefetch_tmap(&tmap_x);
    }
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar(FULL + s), 1);   // producer arrival + tx bytes
      mbar_init(bar(EMPTY + s), 1);  // MMA commit
    }
    mbar_init(bar(ACC_FULL), 1);  // MMA commit
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), G::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_launch_dependents();
  // While the kernel before this one ends, the first of the weight's tiles
  // travel to L2 (a hint: nothing is read before grid_wait).
  if (warp == 0 && lane == 0)
    for (int kt = kt0; kt < min(kt1, kt0 + PREFETCH_STAGES * STAGES); ++kt)
      prefetch_operand<BC, W_MN>(&tmap_w, c0, kt * BK_ELEMS);
  grid_wait();

  float* const sums = reinterpret_cast<float*>(smem);  // [row][column], over the ring
  int issued = 0;  // producer: K tiles issued
  bool ready = true;
  if (warp == 0) {
    if (lane == 0 && !fault_inject) {
      for (int kt = kt0; kt < kt1; ++kt, ++issued) {
        const int s = issued % STAGES, round = issued / STAGES;
        if (issued >= STAGES && !wait_phase(bar(EMPTY + s), (round + 1) & 1u, wc)) break;
        const uint32_t st = smem_u32(smem + s * G::STAGE_BYTES);
        mbar_arrive_expect_tx(bar(FULL + s), G::STAGE_BYTES);
        load_operand<BC, W_MN>(st, &tmap_w, c0, kt * BK_ELEMS, bar(FULL + s));
        load_operand<BT, X_MN>(st + G::W_BYTES, &tmap_x, t0, kt * BK_ELEMS, bar(FULL + s));
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool stop = false;
      for (int g = 0; g < kt1 - kt0; ++g) {
        const int s = g % STAGES, round = g / STAGES;
        if (!wait_phase(bar(FULL + s), round & 1u, wc)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t w_base = smem_u32(smem + s * G::STAGE_BYTES);
        const uint32_t x_base = w_base + G::W_BYTES;
#pragma unroll
        for (int j = 0; j < ROW_BYTES / 32; ++j)
          E::mma(tmem, operand_desc<W_MN>(w_base, j), operand_desc<X_MN>(x_base, j), idesc,
                 g > 0 || j > 0);
        mma_commit(bar(EMPTY + s));
      }
      // Every MMA issued has retired once ACC_FULL completes, also after a
      // wait that ran out.
      mma_commit(bar(ACC_FULL));
      if (stop) wait_phase(bar(ACC_FULL), 0, wc, false);
    }
  } else {
    const int q = warp & 3;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int rows = min(BT, ep.T - t0);  // >= 1
    ready = wait_phase(bar(ACC_FULL), 0, wc, true,
                       TIMEOUT_NS + 20000ull * static_cast<uint64_t>(kt1 - kt0));
    ready = __all_sync(0xffffffffu, ready && !*abort_flag);
    tc_fence_after();
    __syncwarp();
    if (ready && split > 1) {
#pragma unroll 1
      for (int t = 0; t < rows; t += FINISH_ROWS) {
        Rows v;
        load_sums(t_row + t, kt1 > kt0, v);
#pragma unroll
        for (int i = 0; i < FINISH_ROWS; ++i)
          if (t + i < rows) sums[(t + i) * BC + q * 32 + lane] = v[i];
      }
    }
  }

  if (split > 1) {
    __syncwarp();
    cluster_sync();  // every CTA's sums (or its abort flag) are in place
    if (warp >= 2)
      for (int s = 0; s < split; ++s)
        ready = ready && !ld_cluster_s32(map_to_cta(smem_u32(const_cast<int*>(abort_flag)), s));
  }
  if (warp >= 2 && ready) {
    const int q = warp & 3, c = q * 32 + lane;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int rows = min(BT, ep.T - t0), per = (rows + split - 1) / split;
    const int first = rank * per, last = min(rows, first + per);
    finish(ep, c0 + c, t0 + first, t0 + last, [&](int row, Rows& v) {
      const int t = row - t0;
      if (split == 1) {
        load_sums(t_row + t, kt1 > kt0, v);
        return;
      }
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) v[i] = 0.0f;
#pragma unroll 1
      for (int s = 0; s < split; ++s) {
        const uint32_t from = map_to_cta(smem_u32(sums + t * BC + c), s);
#pragma unroll
        for (int i = 0; i < FINISH_ROWS; ++i)
          if (t + i < last) v[i] += ld_cluster_f32(from + i * BC * 4);
      }
    });
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();  // no CTA leaves while its sums are being read
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // Let the copies the producer issued land before the CTA exits.
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
      wait_phase(bar(FULL + i % STAGES), (i / STAGES) & 1u, wc, false);
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, G::TMEM_COLS);
  }
}

template <class E, int BT, bool W_MN, bool X_MN>
LinearKernel entry() {
  return LinearKernel{reinterpret_cast<const void*>(linear_split_kernel<E, BT, W_MN, X_MN>),
                      SplitGeometry<BT>::SMEM_BYTES, SplitGeometry<BT>::STAGES};
}

template <bool W_MN>
LinearKernel entry_16(int bt) {
  switch (bt) {
    case 16: return entry<Half, 16, W_MN, false>();
    case 32: return entry<Half, 32, W_MN, false>();
    case 64: return entry<Half, 64, W_MN, false>();
    case 128: return entry<Half, 128, W_MN, false>();
  }
  return LinearKernel{};
}

}  // namespace linear

using namespace linear;

LinearKernel linear_split_kernel_for(int dtype, int bt, bool w_mn, bool x_mn) {
  if (dtype == DT_E4M3) {
    if (w_mn || x_mn) return LinearKernel{};
    switch (bt) {
      case 16: return entry<E4m3, 16, false, false>();
      case 32: return entry<E4m3, 32, false, false>();
      case 64: return entry<E4m3, 64, false, false>();
      case 128: return entry<E4m3, 128, false, false>();
    }
    return LinearKernel{};
  }
  if (!x_mn) return w_mn ? entry_16<true>(bt) : entry_16<false>(bt);
  // Transposed X comes with transposed W only (the weight gradient), and its
  // boxes are 64 rows.
  if (!w_mn) return LinearKernel{};
  if (bt == 64) return entry<Half, 64, true, true>();
  return bt == 128 ? entry<Half, 128, true, true>() : LinearKernel{};
}

cudaError_t linear_split_read_and_clear_status(unsigned int* status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, f16tc::g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(f16tc::g_status, &zero, sizeof(unsigned int));
}

}  // namespace mt
