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
// One launch takes one product or two that do not depend on one another (the
// layer's two gradients), of the same type and tile; each either splits its
// tiles over the launch's clusters or takes a tile per CTA.
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

template <class E, int BT>
__global__ void __launch_bounds__(THREADS, 2)
    linear_split_kernel(const __grid_constant__ SplitProblems problems, int fault_inject) {
  using G = SplitGeometry<BT>;
  constexpr int STAGES = G::STAGES;
  constexpr int BK_ELEMS = ROW_BYTES / E::BYTES;
  // Transposed operands: 16-bit only, and their boxes are 64 rows.
  constexpr bool CAN_W_MN = E::BYTES == 2, CAN_X_MN = CAN_W_MN && BT >= MN_BOX;
  const SplitProblem& P =
      problems.p[static_cast<int>(blockIdx.x) >= problems.p[1].first_cta ? 1 : 0];
  const LinearEpilogue& ep = P.ep;
  const int Kt = P.ktiles;
  const bool w_mn = CAN_W_MN && P.w_mn, x_mn = CAN_X_MN && P.x_mn;
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
  const int split = P.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = (static_cast<int>(blockIdx.x) - P.first_cta) / split;
  if (tile >= P.tiles) return;  // fills up an unsplit product's last cluster
  // Tiles of one weight panel follow each other, so the panel is read from
  // memory once and found in L2 by the rest.
  const int c0 = tile / P.tiles_t * BC, t0 = tile % P.tiles_t * BT;
  const int kt0 = static_cast<int>(static_cast<int64_t>(Kt) * rank / split);
  const int kt1 = static_cast<int>(static_cast<int64_t>(Kt) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    if (Kt > 0) {  // without a product the maps hold nothing
      prefetch_tmap(&P.map_w);
      prefetch_tmap(&P.map_x);
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
    for (int kt = kt0; kt < min(kt1, kt0 + STAGES); ++kt) {
      if (w_mn) prefetch_operand<BC, true>(&P.map_w, c0, kt * BK_ELEMS);
      else prefetch_operand<BC, false>(&P.map_w, c0, kt * BK_ELEMS);
    }
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
        if (w_mn) load_operand<BC, true>(st, &P.map_w, c0, kt * BK_ELEMS, bar(FULL + s));
        else load_operand<BC, false>(st, &P.map_w, c0, kt * BK_ELEMS, bar(FULL + s));
        if (x_mn) load_operand<BT, true>(st + G::W_BYTES, &P.map_x, t0, kt * BK_ELEMS, bar(FULL + s));
        else load_operand<BT, false>(st + G::W_BYTES, &P.map_x, t0, kt * BK_ELEMS, bar(FULL + s));
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
          E::mma(tmem, w_mn ? operand_desc<true>(w_base, j) : operand_desc<false>(w_base, j),
                 x_mn ? operand_desc<true>(x_base, j) : operand_desc<false>(x_base, j), P.idesc,
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
#pragma unroll 4
      for (int s = 0; s < split; ++s) {
        const uint32_t from = map_to_cta(smem_u32(sums + t * BC + c), s);
#pragma unroll
        for (int i = 0; i < FINISH_ROWS; ++i)
          if (t + i < last) v[i] += ld_cluster_f32(from + i * BC * 4);
      }
    });
  }
  if (split > 1) {
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

template <class E, int BT>
LinearKernel entry() {
  return LinearKernel{reinterpret_cast<const void*>(linear_split_kernel<E, BT>),
                      SplitGeometry<BT>::SMEM_BYTES, SplitGeometry<BT>::STAGES};
}

template <class E>
LinearKernel entry_for(int bt) {
  switch (bt) {
    case 16: return entry<E, 16>();
    case 32: return entry<E, 32>();
    case 64: return entry<E, 64>();
    default: return entry<E, 128>();
  }
}

}  // namespace linear

using namespace linear;

LinearKernel linear_split_kernel_for(int dtype, int bt) {
  return dtype == DT_E4M3 ? entry_for<E4m3>(bt) : entry_for<Half>(bt);
}

cudaError_t linear_split_read_and_clear_status(unsigned int* status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, f16tc::g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(f16tc::g_status, &zero, sizeof(unsigned int));
}

}  // namespace mt
